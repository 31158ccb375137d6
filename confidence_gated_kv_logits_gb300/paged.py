"""Binding of the paged-cache and beam operators (``include/confkv_paged.h``).

``PagedKV`` wraps the caller's page pools; ``PagedBatch`` (from
``PagedKV.batch``) is one step's ragged batch, checked once and used by every
layer's ``append`` and ``attend``; ``BeamSelect`` keeps the scratch of the beam
selection.  Tensors are checked (device, type, layout) and passed on; nothing
is copied, converted or computed here.  As everywhere in CUDA, a tensor that
is used on another stream than its own must stay alive until that work is
done (``Tensor.record_stream``).

The per-call checks live in ``_paged_ops.so`` (csrc/paged_py.cpp): for a single
token they and the launch are the call's whole cost.
"""
import ctypes

FP16, BF16, FP32 = 0, 1, 2
ZEROED = 16384                      # CONFKV_PAGED_ZEROED
torch = None                        # imported with the first handle
_ops = None


def _load():
    """The library; torch and the argument checks, on first use (importing the
    package needs neither)."""
    global torch, _ops
    from . import load_library
    L = load_library()
    if _ops is None:
        import torch as t
        try:
            from . import _paged_ops
        except ImportError as e:
            raise ImportError(f"_paged_ops.so cannot be loaded ({e}): build it with "
                              "confidence_gated_kv_logits_gb300.build.build()") from e
        torch, _ops = t, _paged_ops
    return L


class BatchStruct(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_words", ctypes.c_int32)]


class PrefixStruct(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("group_start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("partial", ctypes.c_void_p), ("partial_bytes", ctypes.c_size_t)]


class NormStruct(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("norm_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("axis", ctypes.c_void_p), ("axes", ctypes.c_int32)]


def declare(L):
    """Argument types of the functions in include/confkv_paged.h."""
    vp, ci, cl, cf, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                          ctypes.c_size_t)
    L.confkv_paged_create.restype = ci
    L.confkv_paged_create.argtypes = [ci] * 8 + [vp, vp, vp, sz, ctypes.POINTER(vp)]
    L.confkv_paged_scratch.restype = sz
    L.confkv_paged_scratch.argtypes = [ci, ci]
    L.confkv_paged_free.restype = None
    L.confkv_paged_free.argtypes = [vp]
    L.confkv_paged_last_error.restype = ctypes.c_char_p
    L.confkv_paged_last_error.argtypes = [vp]
    L.confkv_paged_status.restype = ci
    L.confkv_paged_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
    L.confkv_paged_append.restype = ci
    L.confkv_paged_append.argtypes = [vp, vp, ci, ci, vp, cl, vp, cl, vp, cl, vp, cl, vp, vp, ci,
                                      ci, vp]
    L.confkv_paged_attend.restype = ci
    L.confkv_paged_attend.argtypes = [vp, vp, ci, ci, vp, cl, vp, vp, cf, vp]
    L.confkv_paged_append_normed.restype = ci
    L.confkv_paged_append_normed.argtypes = [vp, vp, ci, ci, vp, cl, vp, cl, vp, cl, vp, cl, vp, vp, ci, ci, vp, vp]
    L.confkv_paged_partial.restype = sz
    L.confkv_paged_partial.argtypes = [ci, ci, ci]
    L.confkv_paged_attend_shared.restype = ci
    L.confkv_paged_attend_shared.argtypes = [vp, vp, vp, ci, ci, vp, cl, vp, vp, cf, vp]
    L.confkv_paged_weigh.restype = ci
    L.confkv_paged_weigh.argtypes = [vp, vp, ci, ci, vp, cl, vp, vp, vp, vp, ci, vp, cf, cf, cf, vp]
    L.confkv_paged_evict.restype = ci
    L.confkv_paged_evict.argtypes = [vp, ci, ci, vp, vp, ci, vp, vp, ci, vp, vp, ci, vp, vp, vp, vp]
    L.confkv_paged_commit.restype = ci
    L.confkv_paged_commit.argtypes = [vp, ci, ci, vp, vp, vp, ci, vp, vp, vp]
    L.confkv_paged_fork.restype = ci
    L.confkv_paged_fork.argtypes = [vp, ci, ci, ci] + [vp] * 7
    L.confkv_beam_workspace.restype = sz
    L.confkv_beam_workspace.argtypes = [ci] * 5
    L.confkv_beam_select.restype = ci
    L.confkv_beam_select.argtypes = [vp, ci, cl, ci, ci, ci, ci, vp, vp, ci, vp, vp, vp, vp, vp,
                                     sz, ci, vp]


def _dtype_code(dtype):
    return {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32}.get(dtype)


class _Device:
    """An object on one device with scratch of its own."""

    _ob = None
    _parked = []                        # scratch of handles that ended inside a capture

    def _dense(self, t, shape, name):
        """Address of a contiguous int32 tensor."""
        if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name}: want contiguous int32 {tuple(shape)} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
        return t.data_ptr()

    def _scratch(self, n, zeroed):
        """Device scratch, its first `zeroed` bytes zero whichever stream comes first."""
        while self._parked:
            torch.cuda.synchronize(self._parked[-1].device)
            self._parked.pop()
        self._mem = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._mem[:zeroed].zero_()
        home = torch.cuda.current_stream(self.device)
        home.synchronize()
        self._home = home.cuda_stream
        return self._mem.data_ptr()

    def _leave(self):
        # the scratch goes back to its own stream's allocator: work of others has to be done
        # (waiting for it would break a capture that runs: kept until the next handle is made)
        ob, self._ob = self._ob, None
        if ob is not None and _ops.release(ob):
            if torch.cuda.is_current_stream_capturing():
                self._parked.append(self._mem)
            else:
                torch.cuda.synchronize(self.device)


class PagedBatch:
    """One step's ragged batch (``PagedKV.batch``).  It holds the tensors that
    it was made from; their contents are read by each call on the GPU."""

    def __init__(self, struct, tensors, batch, mask_rows, index):
        self._struct = struct
        self._index = index                 # of its tensors' device
        self._ref = ctypes.addressof(struct)
        self._tensors = tensors
        self.size = batch
        self.mask_rows = mask_rows


class SharedPrefix:
    """Prefixes that groups of neighbouring sequences share (``PagedKV.prefix``),
    and the attention's scratch for them: calls with one object must be ordered, and
    it is kept until their work is done."""

    def __init__(self, struct, tensors, rows, index):
        self._struct = struct
        self._index = index
        self._ref = ctypes.addressof(struct)
        self._tensors = tensors
        self.rows = rows


class PagedKV(_Device):
    """Operators on a paged cache [layers, pages, kv_heads, page_size, head_dim]
    (fp16 or bf16) that the caller owns; ``heads`` query heads.  Keeps the
    attention's scratch: attend calls on one object must be ordered."""

    def __init__(self, k_pages, v_pages, heads):
        from . import ConfKVError, ERR_INVALID_ARG
        self._h = None
        self._L = _load()
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.dim() != 5 or not t.is_cuda or not t.is_contiguous() or _dtype_code(t.dtype) not in (FP16, BF16):
                raise ValueError(f"{name}: want a contiguous fp16 or bf16 CUDA tensor [layers, pages, "
                                 f"kv_heads, page_size, head_dim], got {t.dtype} {tuple(t.shape)}")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages differ in shape, type or device")
        self.device, self.dtype = k_pages.device, k_pages.dtype
        self._index = k_pages.get_device()
        self.k_pages, self.v_pages = k_pages, v_pages
        self.layers, self.pages, self.kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.heads = heads
        n = self._L.confkv_paged_scratch(self.head_dim, self._index)
        if not n:
            raise ConfKVError(ERR_INVALID_ARG, f"head_dim {self.head_dim} is not supported")
        h = ctypes.c_void_p()
        rc = self._L.confkv_paged_create(self.layers, heads, self.kv_heads, self.head_dim, self.pages,
                                         self.page_size, _dtype_code(self.dtype), self._index,
                                         k_pages.data_ptr(), v_pages.data_ptr(),
                                         self._scratch(n, ZEROED), n, ctypes.byref(h))
        if rc:
            raise ConfKVError(rc, "confkv_paged_create failed")
        self._h = h.value
        self._ob = _ops.make(self._h, 0, 0, self._home, heads, self.kv_heads, self.head_dim, 0, self._index,
                             _dtype_code(self.dtype))

    def close(self):
        if getattr(self, "_h", None):
            self._leave()
            self._L.confkv_paged_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc):
        from . import ConfKVError
        if rc:
            raise ConfKVError(rc, self._L.confkv_paged_last_error(self._h).decode())

    def status(self, check=True):
        """The FLAG_* bits that the GPU has latched since the last call
        (synchronises); raises if there are any unless ``check`` is false."""
        if not self._h:
            raise ValueError("the handle is closed")
        f = ctypes.c_int32()
        rc = self._L.confkv_paged_status(self._h, ctypes.byref(f))
        if check:
            self._check(rc)
        return f.value

    def batch(self, page_table, ctx_len, q_start, mask=None):
        """A ragged batch: page_table int32 [B, blocks], ctx_len int32 [B],
        q_start int32 [B + 1], mask int32 [rows, words] (ancestor bits) or None."""
        if page_table.dim() != 2:
            raise ValueError("page_table: want [batch, blocks]")
        B, blocks = page_table.shape
        s = BatchStruct(B, blocks, self._dense(page_table, (B, blocks), "page_table"),
                        self._dense(ctx_len, (B,), "ctx_len"),
                        self._dense(q_start, (B + 1,), "q_start"), None, 0)
        rows = -1
        if mask is not None:
            if mask.dim() != 2 or mask.shape[1] < 1:
                raise ValueError("mask: want int32 [rows, words], a word per row at least")
            rows = mask.shape[0]
            s.mask = self._dense(mask, mask.shape, "mask")
            s.mask_words = mask.shape[1]
        return PagedBatch(s, (page_table, ctx_len, q_start, mask), B, rows, self._index)

    def prefix(self, group_start, prefix_len, rows):
        """Shared prefixes: sequences group_start[g] .. group_start[g + 1] - 1 (int32
        [groups + 1]) have their first prefix_len[g] (int32 [groups]) cached tokens in
        common, for ``attend`` of up to `rows` rows.  Their contents are read by each call."""
        from . import ConfKVError, ERR_INVALID_ARG
        if prefix_len.dim() != 1 or prefix_len.shape[0] < 1:
            raise ValueError("prefix_len: want [groups], one at least")
        groups = prefix_len.shape[0]
        n = self._L.confkv_paged_partial(rows, self.heads, self.head_dim)
        if not n:
            raise ConfKVError(ERR_INVALID_ARG, f"{rows} rows are not supported")
        scratch = torch.empty(n, dtype=torch.uint8, device=self.device)
        s = PrefixStruct(groups, self._dense(group_start, (groups + 1,), "group_start"),
                         self._dense(prefix_len, (groups,), "prefix_len"), scratch.data_ptr(), n)
        return SharedPrefix(s, (group_start, prefix_len, scratch), rows, self._index)

    def append(self, layer, batch, k, v, *, q=None, q_out=None, positions=None, inv_freq=None,
               interleaved=False, q_norm=None, k_norm=None, eps=1e-6, axis=None, stream=None):
        """Stores k, v [rows, kv_heads, head_dim] of the batch's new tokens in
        layer `layer`, k rotated by `positions` (int32 [rows]; None: places in
        the sequence) x `inv_freq` (fp32 [rotary / 2]; None: not rotated), and
        rotates q [rows, heads, head_dim] into q_out (q itself allowed).  q_norm, k_norm
        [head_dim] (fp32 or the cache's type): each head of q, of k is divided by its
        root mean square (eps beside the mean) and multiplied by them before.  axis int32
        [rotary / 2]: positions are [rows, axes], pair i turns by the axis[i]-th."""
        if batch._index != self._index:
            raise ValueError("the batch's tensors are on another device")
        if q_norm is not None or k_norm is not None or axis is not None:
            rc = _ops.append_normed(self._ob, batch._ref, layer, k, v, q, q_out, positions, inv_freq, interleaved,
                                    q_norm, k_norm, eps, axis, stream)
            if rc:
                self._check(rc)
            return
        rc = _ops.append(self._ob, batch._ref, layer, k, v, q, q_out, positions, inv_freq, interleaved, stream)
        if rc:
            self._check(rc)

    def attend(self, layer, batch, q, out, *, lse=None, scale=0.0, prefix=None, stream=None):
        """Attention of q [rows, heads, head_dim] over layer `layer` into out
        (contiguous, same shape and type); lse fp32 [rows, heads] or None;
        scale 0: 1 / sqrt(head_dim).  prefix (``prefix``): what groups of the batch's
        sequences share is read once for the group (for few rows faster from some 130 MB of
        prefix K and V on, counted for every sequence)."""
        if batch._index != self._index:
            raise ValueError("the batch's tensors are on another device")
        if prefix is not None:
            if prefix._index != self._index:
                raise ValueError("the prefix's tensors are on another device")
            rc = _ops.attend_shared(self._ob, batch._ref, prefix._ref, batch.mask_rows, layer, q, out, lse, scale, stream)
            if rc:
                self._check(rc)
            return
        rc = _ops.attend(self._ob, batch._ref, batch.mask_rows, layer, q, out, lse, scale, stream)
        if rc:
            self._check(rc)

    def weigh(self, layer, batch, q, lse, mass, mass_out, pos=None, *, positions=None, decay=1.0, gain=1.0, scale=0.0,
              stream=None):
        """Adds the attention weights of q's rows (lse as ``attend`` gave it) to each
        token's accumulated weight: mass_out = decay mass + gain sum, fp32 [batch,
        kv_heads, cap] (mass_out may be mass).  New tokens start from 0; pos int32
        likewise receives their positions (int32 [rows]; None: their places).  Sequences
        without new rows are not written, in a mass_out of its own either.  A drafted
        tree is weighed behind ``commit``, by its accepted rows alone."""
        if batch._index != self._index:
            raise ValueError("the batch's tensors are on another device")
        rc = _ops.weigh(self._ob, batch._ref, batch.size, batch.mask_rows, layer, q, lse, mass, mass_out, pos, positions,
                        decay, gain, scale, stream)
        if rc:
            self._check(rc)

    def evict(self, page_table, length, mass, pos, keep, mass_out, pos_out, new_len, *, protect=0, first=None, stream=None):
        """Keeps the keep[b] tokens of the largest mass of every layer and KV head (before
        them places below first[b] and the `protect` newest positions) and moves those behind
        into evicted ones' places; mass, pos [layers, batch, kv_heads, cap] and their
        outputs (both may be the inputs); length, keep, new_len int32 [batch] or
        [layers, batch].  Places from first[b] on lie in pages that no other sequence
        names: what several share is below it, and never changes."""
        rc = _ops.evict(self._ob, self.layers, page_table, length, mass, pos, keep, mass_out, pos_out, new_len, protect,
                        first, stream)
        if rc:
            self._check(rc)

    def commit(self, page_table, ctx_len, path, path_len, new_len, stream=None):
        """Moves the accepted drafted tokens path [B, cap] (path_len [B] of them)
        behind the cached ones in every layer; new_len [B] receives ctx_len + path_len.
        Masses do not move (``weigh``)."""
        rc = _ops.commit(self._ob, page_table, ctx_len, path, path_len, new_len, stream)
        if rc:
            self._check(rc)

    def fork(self, parent, beams, table_in, len_in, tail_pages, table_out, len_out, stream=None):
        """Reorders beams: row r of [batch x beams] takes over its parent's pages,
        the part-filled last one as a copy in tail_pages[r].  parent: int32
        [rows] or [batch, beams].  Masses and positions are gathered by the caller."""
        rc = _ops.fork(self._ob, parent, beams, table_in, len_in, tail_pages, table_out, len_out, stream)
        if rc:
            self._check(rc)


class BeamSelect(_Device):
    """The `keep` best continuations of `batch` sequences of `beams` beams over
    `vocab` tokens.  Keeps the scratch: calls on one object must be ordered."""

    def __init__(self, batch, beams, vocab, keep, dtype=None, device=None):
        from . import ConfKVError, ERR_INVALID_ARG
        self._L = _load()
        self.logits_dtype = torch.float32 if dtype is None else dtype
        self._code = _dtype_code(self.logits_dtype)
        if self._code is None:
            raise ValueError("dtype: want float16, bfloat16 or float32")
        self.sizes = (batch, beams, vocab, keep)
        n = self._L.confkv_beam_workspace(batch, beams, vocab, keep, self._code)
        if not n:
            raise ConfKVError(ERR_INVALID_ARG, f"beam sizes {self.sizes} are not supported")
        if device is not None and not isinstance(device, int):
            device = torch.device(device)
            if device.type != "cuda":
                raise ValueError(f"device: want a CUDA device, got {device}")
            device = device.index                # ("cuda" alone: the current one)
        self._index = torch.cuda.current_device() if device is None else device
        self.device = torch.device("cuda", self._index)
        ws = self._scratch(n, n)
        self._ob = _ops.make(1, ws, n, self._home, batch, beams, vocab, keep, self._index, self._code)

    def __del__(self):
        try:
            self._leave()
        except Exception:
            pass

    def select(self, logits, scores, score_out, parent_out, token_out, *, finished=None, pad_token=0,
               flags_out=None, stream=None):
        """logits [batch, beams, vocab] (rows may be strided), scores fp32
        [batch, beams]; score_out fp32, parent_out and token_out int32 [batch,
        keep]; finished bool [batch, beams]; flags_out int32 [batch, beams]."""
        rc = _ops.select(self._ob, logits, scores, finished, pad_token, score_out, parent_out, token_out,
                         flags_out, stream)
        if rc:
            from . import ConfKVError
            raise ConfKVError(rc, "confkv_beam_select refused its arguments" if rc == -1 else "confkv_beam_select")
