"""Binding of the paged-cache and beam operators (``include/confkv_paged.h``).

``PagedKV`` wraps the caller's page pools; ``PagedBatch`` (from
``PagedKV.batch``) is one step's ragged batch, checked once and used by every
layer's ``append`` and ``attend``; ``BeamSelect`` keeps the scratch of the beam
selection.  Tensors are checked (device, type, layout) and passed on; nothing
is copied, converted or computed here.  As everywhere in CUDA, a tensor that
is used on another stream than its own must stay alive until that work is
done (``Tensor.record_stream``).
"""
import ctypes

FP16, BF16, FP32 = 0, 1, 2


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
    L.confkv_paged_create.argtypes = [ci] * 8 + [vp, vp, ctypes.POINTER(vp)]
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
                                     sz, vp]


def _dtype_code(dtype):
    import torch
    return {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32}.get(dtype)


class _Device:
    """Checks of tensor arguments against one device."""

    def _ints(self, t, shape, name):
        import torch
        if t.dtype is not torch.int32 or t.get_device() != self._index or not t.is_contiguous() \
                or tuple(t.shape) != shape:
            raise ValueError(f"{name}: want contiguous int32 {shape} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _rows(self, t, rows, heads, name):
        """Address and row stride of a [rows, heads, head_dim] tensor whose rows are dense."""
        s = t.stride()
        if t.dtype is not self.dtype or t.get_device() != self._index \
                or t.shape != (rows, heads, self.head_dim) \
                or s[2] != 1 or (s[1] != self.head_dim and heads > 1):
            raise ValueError(f"{name}: want {self.dtype} {(rows, heads, self.head_dim)} on "
                             f"{self.device} with dense rows, got {t.dtype} {tuple(t.shape)} "
                             f"strides {s} on {t.device}")
        return t.data_ptr(), (s[0] if rows > 1 else max(s[0], heads * self.head_dim))

    def _stream(self, stream):
        if stream is None:
            import torch
            stream = torch.cuda.current_stream(self.device)
        return stream.cuda_stream


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
    (fp16 or bf16) that the caller owns; ``heads`` query heads."""

    def __init__(self, k_pages, v_pages, heads):
        from . import ConfKVError, load_library
        self._h = None
        self._L = load_library()
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
        h = ctypes.c_void_p()
        rc = self._L.confkv_paged_create(self.layers, heads, self.kv_heads, self.head_dim, self.pages,
                                         self.page_size, _dtype_code(self.dtype), self._index,
                                         k_pages.data_ptr(), v_pages.data_ptr(), ctypes.byref(h))
        if rc:
            raise ConfKVError(rc, "confkv_paged_create failed")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            self._L.confkv_paged_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc):
        if rc:
            from . import ConfKVError
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
        import torch
        if page_table.dim() != 2:
            raise ValueError("page_table: want [batch, blocks]")
        B, blocks = page_table.shape
        s = BatchStruct(B, blocks, self._ints(page_table, (B, blocks), "page_table"),
                        self._ints(ctx_len, (B,), "ctx_len"), self._ints(q_start, (B + 1,), "q_start"),
                        None, 0)
        rows = None
        if mask is not None:
            if mask.dim() != 2 or mask.dtype is not torch.int32:
                raise ValueError("mask: want int32 [rows, words]")
            rows = mask.shape[0]
            s.mask = self._ints(mask, tuple(mask.shape), "mask")
            s.mask_words = mask.shape[1]
            if rows and mask.shape[1] < 1:
                raise ValueError("mask: want at least one word per row")
        return PagedBatch(s, (page_table, ctx_len, q_start, mask), B, rows)

    def append(self, layer, batch, k, v, *, q=None, q_out=None, positions=None, inv_freq=None,
               interleaved=False, stream=None):
        """Stores k, v [rows, kv_heads, head_dim] of the batch's new tokens in
        layer `layer`, k rotated by `positions` (int32 [rows]; None: places in
        the sequence) x `inv_freq` (fp32 [rotary / 2]; None: not rotated), and
        rotates q [rows, heads, head_dim] into q_out (q itself allowed)."""
        rows = k.shape[0]
        kp, ks = self._rows(k, rows, self.kv_heads, "k")
        vp, vs = self._rows(v, rows, self.kv_heads, "v")
        qp = op = None
        qs = os_ = 0
        if q is not None or q_out is not None:
            if q is None or q_out is None:
                raise ValueError("q and q_out go together")
            qp, qs = self._rows(q, rows, self.heads, "q")
            op, os_ = self._rows(q_out, rows, self.heads, "q_out")
        fp, rotary = None, 0
        if inv_freq is not None:
            import torch
            if inv_freq.dtype is not torch.float32 or inv_freq.get_device() != self._index \
                    or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
                raise ValueError(f"inv_freq: want contiguous float32 [rotary / 2] on {self.device}")
            fp, rotary = inv_freq.data_ptr(), 2 * inv_freq.shape[0]
        pp = None if positions is None else self._ints(positions, (rows,), "positions")
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
        qp, qs = self._rows(q, rows, self.heads, "q")
        op, _ = self._rows(out, rows, self.heads, "out")
        if not out.is_contiguous():
            raise ValueError("out: want a contiguous tensor")
        lp = None
        if lse is not None:
            import torch
            if lse.dtype is not torch.float32 or lse.get_device() != self._index \
                    or lse.shape != (rows, self.heads) or not lse.is_contiguous():
                raise ValueError(f"lse: want contiguous float32 {(rows, self.heads)} on {self.device}")
            lp = lse.data_ptr()
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
        rc = self._L.confkv_paged_commit(
            self._h, B, blocks, self._ints(page_table, (B, blocks), "page_table"),
            self._ints(ctx_len, (B,), "ctx_len"), self._ints(path, (B, path.shape[1]), "path"),
            path.shape[1], self._ints(path_len, (B,), "path_len"), self._ints(new_len, (B,), "new_len"),
            self._stream(stream))
        if rc:
            self._check(rc)

    def fork(self, parent, beams, table_in, len_in, tail_pages, table_out, len_out, stream=None):
        """Reorders beams: row r of [batch x beams] takes over its parent's pages,
        the part-filled last one as a copy in tail_pages[r]."""
        if table_in.dim() != 2:
            raise ValueError("table_in: want [rows, blocks]")
        n, blocks = table_in.shape
        rc = self._L.confkv_paged_fork(
            self._h, n, beams, blocks, self._ints(parent.view(-1), (n,), "parent"),
            self._ints(table_in, (n, blocks), "table_in"), self._ints(len_in, (n,), "len_in"),
            self._ints(tail_pages, (n,), "tail_pages"), self._ints(table_out, (n, blocks), "table_out"),
            self._ints(len_out, (n,), "len_out"), self._stream(stream))
        if rc:
            self._check(rc)


class BeamSelect(_Device):
    """The `keep` best continuations of `batch` sequences of `beams` beams over
    `vocab` tokens.  Keeps the scratch: calls on one object must be ordered."""

    def __init__(self, batch, beams, vocab, keep, dtype=None, device=None):
        import torch
        from . import ConfKVError, ERR_INVALID_ARG, load_library
        self._L = load_library()
        self.logits_dtype = torch.float32 if dtype is None else dtype
        self._code = _dtype_code(self.logits_dtype)
        if self._code is None:
            raise ValueError("dtype: want float16, bfloat16 or float32")
        self.sizes = (batch, beams, vocab, keep)
        n = self._L.confkv_beam_workspace(batch, beams, vocab, keep, self._code)
        if not n:
            raise ConfKVError(ERR_INVALID_ARG, f"beam sizes {self.sizes} are not supported")
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index if not isinstance(device, int) else device)
        self._index = self.device.index
        self._ws = torch.zeros(n, dtype=torch.uint8, device=self.device)
        # the zeroes must be there whichever stream the first call comes on
        torch.cuda.current_stream(self.device).synchronize()

    def select(self, logits, scores, score_out, parent_out, token_out, *, finished=None, pad_token=0,
               flags_out=None, stream=None):
        """logits [batch, beams, vocab] (rows may be strided), scores fp32
        [batch, beams]; score_out fp32, parent_out and token_out int32 [batch,
        keep]; finished bool [batch, beams]; flags_out int32 [batch, beams]."""
        import torch
        B, W, V, K = self.sizes
        s = logits.stride()
        if logits.dtype is not self.logits_dtype or logits.get_device() != self._index \
                or logits.shape != (B, W, V) or s[2] != 1 or (s[0] != W * s[1] and B > 1):
            raise ValueError(f"logits: want {self.logits_dtype} {(B, W, V)} on {self.device} with evenly "
                             f"spaced rows, got {logits.dtype} {tuple(logits.shape)} strides {s} on {logits.device}")
        stride = s[1] if W > 1 else s[0] if B > 1 else max(V, s[1])
        for t, n, name in ((scores, W, "scores"), (score_out, K, "score_out")):
            if t.dtype is not torch.float32 or t.get_device() != self._index or t.shape != (B, n) \
                    or not t.is_contiguous():
                raise ValueError(f"{name}: want contiguous float32 {(B, n)} on {self.device}")
        fp = None
        if finished is not None:
            if finished.dtype not in (torch.bool, torch.uint8) or finished.get_device() != self._index \
                    or finished.shape != (B, W) or not finished.is_contiguous():
                raise ValueError(f"finished: want contiguous bool {(B, W)} on {self.device}")
            fp = finished.data_ptr()
        gp = None if flags_out is None else self._ints(flags_out, (B, W), "flags_out")
        cur = torch.cuda.current_device()
        if cur != self._index:
            torch.cuda.set_device(self._index)
        try:
            rc = self._L.confkv_beam_select(
                logits.data_ptr(), self._code, stride, B, W, V, K, scores.data_ptr(), fp, pad_token,
                score_out.data_ptr(), self._ints(parent_out, (B, K), "parent_out"),
                self._ints(token_out, (B, K), "token_out"), gp, self._ws.data_ptr(), self._ws.numel(),
                self._stream(stream))
        finally:
            if cur != self._index:
                torch.cuda.set_device(cur)
        if rc:
            from . import ConfKVError
            raise ConfKVError(rc, "confkv_beam_select refused its arguments" if rc == -1 else "confkv_beam_select")
