"""Binding of the paged-cache and beam operators (``include/confkv_paged.h``).

``PagedKV`` wraps the caller's page pools; ``PagedBatch`` (from
``PagedKV.batch``) is one step's ragged batch, checked once and used by every
layer's ``append`` and ``attend``; ``BeamSelect`` keeps the scratch of the beam
selection.  Tensors are checked (device, type, layout) and passed on; nothing
is copied, converted or computed here.  As everywhere in CUDA, a tensor that
is used on another stream than its own must stay alive until that work is
done (``Tensor.record_stream``).

The checks are written for few attribute reads per tensor: for a single token
they and the launch are the call's whole cost.
"""
import ctypes

FP16, BF16, FP32 = 0, 1, 2
ZEROED = 16384                      # CONFKV_PAGED_ZEROED
torch = None                        # imported with the first handle
_raw_stream = None
_F32 = _I32 = None


def _load():
    """The library; torch, on first use (importing the package needs none)."""
    global torch, _raw_stream, _F32, _I32
    from . import load_library
    if torch is None:
        import torch as t
        torch, _raw_stream = t, t._C._cuda_getCurrentRawStream
        _F32, _I32 = t.float32, t.int32
    return load_library()


class BatchStruct(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_words", ctypes.c_int32)]


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
    """Checks of tensor arguments against one device."""

    def _dense(self, t, dtype, shape, name):
        """Address of a contiguous tensor."""
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name}: want contiguous {dtype} {tuple(shape)} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
        return t.data_ptr()

    def _rows(self, t, shape, name):
        """Address and row stride of a [rows, heads, head_dim] tensor whose rows are dense."""
        if t.dtype is self.dtype and t.shape == shape and t.get_device() == self._index:
            rows, heads, d = shape
            step, head, one = t.stride()
            if one == 1 and (head == d or heads == 1):
                return t.data_ptr(), step if rows > 1 else heads * d
        raise ValueError(f"{name}: want {self.dtype} {tuple(shape)} on {self.device} with dense rows, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")

    def _scratch(self, n, zeroed):
        """Device scratch, its first `zeroed` bytes zero whichever stream comes first."""
        self._mem = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._mem[:zeroed].zero_()
        home = torch.cuda.current_stream(self.device)
        home.synchronize()
        self._home, self._away = home.cuda_stream, False
        return self._mem.data_ptr()

    def _stream(self, stream):
        s = _raw_stream(self._index) if stream is None else stream.cuda_stream
        if s != self._home:
            self._away = True
        return s

    def _leave(self):
        # the scratch goes back to its own stream's allocator: work of others has to be done
        if self._away:
            torch.cuda.synchronize(self.device)


class PagedBatch:
    """One step's ragged batch (``PagedKV.batch``).  It holds the tensors that
    it was made from; their contents are read by each call on the GPU."""

    def __init__(self, struct, tensors, batch, mask_rows):
        self._struct = struct
        self._ref = ctypes.addressof(struct)
        self._tensors = tensors
        self.size = batch
        self.mask_rows = mask_rows


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
        s = BatchStruct(B, blocks, self._dense(page_table, _I32, (B, blocks), "page_table"),
                        self._dense(ctx_len, _I32, (B,), "ctx_len"),
                        self._dense(q_start, _I32, (B + 1,), "q_start"), None, 0)
        rows = None
        if mask is not None:
            if mask.dim() != 2 or mask.shape[1] < 1:
                raise ValueError("mask: want int32 [rows, words], a word per row at least")
            rows = mask.shape[0]
            s.mask = self._dense(mask, _I32, mask.shape, "mask")
            s.mask_words = mask.shape[1]
        return PagedBatch(s, (page_table, ctx_len, q_start, mask), B, rows)

    def append(self, layer, batch, k, v, *, q=None, q_out=None, positions=None, inv_freq=None,
               interleaved=False, stream=None):
        """Stores k, v [rows, kv_heads, head_dim] of the batch's new tokens in
        layer `layer`, k rotated by `positions` (int32 [rows]; None: places in
        the sequence) x `inv_freq` (fp32 [rotary / 2]; None: not rotated), and
        rotates q [rows, heads, head_dim] into q_out (q itself allowed)."""
        rows = k.shape[0]
        shape = (rows, self.kv_heads, self.head_dim)
        kp, ks = self._rows(k, shape, "k")
        vp, vs = self._rows(v, shape, "v")
        qp = op = fp = pp = None
        qs = os_ = rotary = 0
        if q is not None or q_out is not None:
            if q is None or q_out is None:
                raise ValueError("q and q_out go together")
            shape = (rows, self.heads, self.head_dim)
            qp, qs = self._rows(q, shape, "q")
            op, os_ = self._rows(q_out, shape, "q_out")
        if inv_freq is not None:
            if inv_freq.dim() != 1:
                raise ValueError("inv_freq: want [rotary / 2]")
            rotary = 2 * inv_freq.shape[0]
            fp = self._dense(inv_freq, _F32, inv_freq.shape, "inv_freq")
        if positions is not None:
            pp = self._dense(positions, _I32, (rows,), "positions")
        rc = self._L.confkv_paged_append(self._h, batch._ref, layer, rows, kp, ks, vp, vs, qp, qs, op,
                                         os_, pp, fp, rotary, 1 if interleaved else 0,
                                         self._stream(stream))
        if rc:
            self._check(rc)

    def attend(self, layer, batch, q, out, *, lse=None, scale=0.0, stream=None):
        """Attention of q [rows, heads, head_dim] over layer `layer` into out
        (contiguous, same shape and type); lse fp32 [rows, heads] or None;
        scale 0: 1 / sqrt(head_dim)."""
        rows = q.shape[0]
        if batch.mask_rows is not None and batch.mask_rows < rows:
            raise ValueError(f"the batch's mask has {batch.mask_rows} rows, q has {rows}")
        shape = (rows, self.heads, self.head_dim)
        qp, qs = self._rows(q, shape, "q")
        op = self._dense(out, self.dtype, shape, "out")
        lp = None if lse is None else self._dense(lse, _F32, (rows, self.heads), "lse")
        rc = self._L.confkv_paged_attend(self._h, batch._ref, layer, rows, qp, qs, op, lp, scale,
                                         self._stream(stream))
        if rc:
            self._check(rc)

    def commit(self, page_table, ctx_len, path, path_len, new_len, stream=None):
        """Moves the accepted drafted tokens path [B, cap] (path_len [B] of them)
        behind the cached ones in every layer; new_len [B] receives ctx_len + path_len."""
        if page_table.dim() != 2 or path.dim() != 2:
            raise ValueError("page_table and path: want [batch, blocks] and [batch, cap]")
        B, blocks = page_table.shape
        cap = path.shape[1]
        one = (B,)
        rc = self._L.confkv_paged_commit(
            self._h, B, blocks, self._dense(page_table, _I32, (B, blocks), "page_table"),
            self._dense(ctx_len, _I32, one, "ctx_len"), self._dense(path, _I32, (B, cap), "path"), cap,
            self._dense(path_len, _I32, one, "path_len"), self._dense(new_len, _I32, one, "new_len"),
            self._stream(stream))
        if rc:
            self._check(rc)

    def fork(self, parent, beams, table_in, len_in, tail_pages, table_out, len_out, stream=None):
        """Reorders beams: row r of [batch x beams] takes over its parent's pages,
        the part-filled last one as a copy in tail_pages[r].  parent: int32
        [rows] or [batch, beams]."""
        if table_in.dim() != 2:
            raise ValueError("table_in: want [rows, blocks]")
        n, blocks = table_in.shape
        one = (n,)
        if parent.dim() == 2 and parent.shape[1] == beams and parent.numel() == n:
            pp = self._dense(parent, _I32, parent.shape, "parent")
        else:
            pp = self._dense(parent, _I32, one, "parent")
        rc = self._L.confkv_paged_fork(
            self._h, n, beams, blocks, pp, self._dense(table_in, _I32, (n, blocks), "table_in"),
            self._dense(len_in, _I32, one, "len_in"), self._dense(tail_pages, _I32, one, "tail_pages"),
            self._dense(table_out, _I32, (n, blocks), "table_out"), self._dense(len_out, _I32, one, "len_out"),
            self._stream(stream))
        if rc:
            self._check(rc)


class BeamSelect(_Device):
    """The `keep` best continuations of `batch` sequences of `beams` beams over
    `vocab` tokens.  Keeps the scratch: calls on one object must be ordered."""

    def __init__(self, batch, beams, vocab, keep, dtype=None, device=None):
        from . import ConfKVError, ERR_INVALID_ARG
        self._L = _load()
        self.logits_dtype = _F32 if dtype is None else dtype
        self._code = _dtype_code(self.logits_dtype)
        if self._code is None:
            raise ValueError("dtype: want float16, bfloat16 or float32")
        self.sizes = (batch, beams, vocab, keep)
        n = self._L.confkv_beam_workspace(batch, beams, vocab, keep, self._code)
        if not n:
            raise ConfKVError(ERR_INVALID_ARG, f"beam sizes {self.sizes} are not supported")
        if device is None:
            device = torch.cuda.current_device()
        self._index = device if isinstance(device, int) else torch.device(device).index or 0
        self.device = torch.device("cuda", self._index)
        self._bytes = n
        self._ws = self._scratch(n, n)

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
        B, W, V, K = self.sizes
        stride = V
        if logits.dtype is not self.logits_dtype or logits.get_device() != self._index \
                or logits.shape != (B, W, V):
            raise ValueError(f"logits: want {self.logits_dtype} {(B, W, V)} on {self.device}, got "
                             f"{logits.dtype} {tuple(logits.shape)} on {logits.device}")
        if not logits.is_contiguous():
            s = logits.stride()
            stride = s[1] if W > 1 else s[0]
            if s[2] != 1 or (B > 1 and s[0] != W * stride) or stride < V:
                raise ValueError(f"logits: want evenly spaced dense rows, got strides {s}")
        at, out = (B, W), (B, K)
        fp = gp = None
        if finished is not None:
            fp = self._dense(finished, torch.uint8 if finished.dtype is torch.uint8 else torch.bool, at, "finished")
        if flags_out is not None:
            gp = self._dense(flags_out, _I32, at, "flags_out")
        rc = self._L.confkv_beam_select(
            logits.data_ptr(), self._code, stride, B, W, V, K, self._dense(scores, _F32, at, "scores"), fp,
            pad_token, self._dense(score_out, _F32, out, "score_out"),
            self._dense(parent_out, _I32, out, "parent_out"), self._dense(token_out, _I32, out, "token_out"),
            gp, self._ws, self._bytes, self._index, self._stream(stream))
        if rc:
            from . import ConfKVError
            raise ConfKVError(rc, "confkv_beam_select refused its arguments" if rc == -1 else "confkv_beam_select")
