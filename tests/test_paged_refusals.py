"""Refusals of the paged-cache and beam entry points (CPU: nothing reaches a
GPU), and the bad metadata that only the GPU can see (flags, nothing touched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pkg():
    from confidence_gated_kv_logits_gb300 import build as B
    B.build()
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


GOOD = dict(layers=2, heads=8, kv_heads=2, dim=128, pages=10, page=16, dtype=0, device=0, k=1 << 12, v=1 << 12, scratch=1 << 16)


@pytest.mark.parametrize("bad", [
    dict(layers=0), dict(layers=40000), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(heads=34),
    dict(dim=96), dict(dim=0), dict(pages=0), dict(page=8), dict(page=48), dict(page=512), dict(dtype=2),
    dict(dtype=-1), dict(k=None), dict(v=None), dict(k=(1 << 12) + 16), dict(pages=1 << 27),
    dict(layers=30000, pages=1 << 30), dict(scratch=None), dict(scratch=(1 << 16) + 128)])
def test_create_refuses(pkg, bad):
    a = {**GOOD, **bad}
    h = ctypes.c_void_p(7)
    rc = pkg.load_library().confkv_paged_create(
        a["layers"], a["heads"], a["kv_heads"], a["dim"], a["pages"], a["page"], a["dtype"], a["device"],
        a["k"], a["v"], a["scratch"], 1 << 40, ctypes.byref(h))
    assert rc == pkg.ERR_INVALID_ARG and not h.value


def test_null_handles(pkg):
    L = pkg.load_library()
    assert L.confkv_paged_create(2, 8, 2, 128, 10, 16, 0, 0, 4096, 4096, 65536, 1 << 40, None) == pkg.ERR_INVALID_ARG
    assert L.confkv_paged_last_error(None) == b"null handle"
    assert L.confkv_paged_status(None, None) == pkg.ERR_INVALID_ARG
    assert L.confkv_paged_append(None, None, 0, 1, *([0] * 8), None, None, 0, 0, None) == pkg.ERR_INVALID_ARG
    assert L.confkv_paged_attend(None, None, 0, 1, None, 0, None, None, 0.0, None) == pkg.ERR_INVALID_ARG
    assert L.confkv_paged_commit(None, 1, 1, None, None, None, 1, None, None, None) == pkg.ERR_INVALID_ARG
    assert L.confkv_paged_fork(None, 1, 1, 1, *([None] * 7)) == pkg.ERR_INVALID_ARG
    L.confkv_paged_free(None)
    assert L.confkv_paged_scratch(96, 0) == 0


BEAM = dict(batch=2, beams=4, vocab=100, keep=8, dtype=2, stride=100, logits=4096, scores=1 << 20, pad=0,
            so=1 << 21, po=1 << 22, to=1 << 23, ws=1 << 24, bytes=None)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(beams=0), dict(beams=33), dict(batch=40000, beams=2), dict(vocab=1), dict(vocab=(1 << 24) + 1),
    dict(keep=0), dict(keep=65), dict(dtype=3), dict(dtype=-1), dict(stride=99), dict(logits=None), dict(logits=4098),
    dict(scores=None), dict(pad=-1), dict(pad=100), dict(so=None), dict(po=None), dict(to=None), dict(ws=None),
    dict(ws=(1 << 24) + 4), dict(bytes=16), dict(so=1 << 20), dict(to=(1 << 20) + 4)])
def test_beam_refuses(pkg, bad):
    L = pkg.load_library()
    a = {**BEAM, **bad}
    need = L.confkv_beam_workspace(a["batch"], a["beams"], a["vocab"], a["keep"], a["dtype"])
    rc = L.confkv_beam_select(a["logits"], a["dtype"], a["stride"], a["batch"], a["beams"], a["vocab"], a["keep"],
                              a["scores"], None, a["pad"], a["so"], a["po"], a["to"], None, a["ws"],
                              need if a["bytes"] is None else a["bytes"], -1, None)
    assert rc == (pkg.ERR_CAPACITY if a["bytes"] == 16 else pkg.ERR_INVALID_ARG)
    if set(bad) & {"batch", "beams", "vocab", "keep", "dtype"}:
        assert need == 0


def test_beam_workspace_grows_with_its_sizes(pkg):
    n = lambda *a: pkg.load_library().confkv_beam_workspace(*a)  # noqa: E731
    assert 0 < n(1, 4, 50257, 8, 2) < n(16, 4, 50257, 8, 2) <= n(16, 4, 50257, 16, 2)


def test_beam_outputs_may_not_overlap(pkg):
    """flags_out, the outputs and finished against each other and against the scores."""
    L = pkg.load_library()
    a = BEAM
    need = L.confkv_beam_workspace(a["batch"], a["beams"], a["vocab"], a["keep"], a["dtype"])

    def call(so=a["so"], po=a["po"], to=a["to"], flags=1 << 25, finished=1 << 26):
        return L.confkv_beam_select(a["logits"], a["dtype"], a["stride"], a["batch"], a["beams"], a["vocab"], a["keep"],
                                    a["scores"], finished, a["pad"], so, po, to, flags, a["ws"], need, -1, None)

    for bad in (dict(flags=a["scores"]), dict(flags=a["scores"] + 28), dict(flags=a["so"]), dict(flags=1 << 26),
                dict(po=a["so"]), dict(to=a["po"] + 4), dict(finished=a["to"] + 8), dict(so=a["ws"] + 16),
                dict(flags=a["ws"]), dict(so=a["logits"] + 64)):
        assert call(**bad) == pkg.ERR_INVALID_ARG, bad


def run_alone(code):
    """In a process of its own, which an exception that crosses a C entry would end."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_tensors_without_plain_memory_raise(pkg):
    """Sparse, nested, quantised and other tensors that have no sizes, strides or address raise; nothing ends."""
    run_alone("""
import torch, pytest
from confidence_gated_kv_logits_gb300 import _paged_ops as ops
ob = ops.make(4096, 0, 0, 0, 2, 1, 64, 0, 0, 0)
nested = torch.nested.nested_tensor([torch.zeros(2), torch.zeros(3)])
three = torch.nested.nested_tensor([torch.zeros(2, 64), torch.zeros(3, 64)])
sparse = torch.zeros(2, 3, dtype=torch.int32).to_sparse()
meta = torch.zeros(2, 3, dtype=torch.int32, device="meta")
i = torch.zeros(2, dtype=torch.int32)
for t in (nested, sparse, meta, i, 3, None):
    for call in (lambda: ops.commit(ob, t, i, t, i, i, None), lambda: ops.fork(ob, i, 2, t, i, i, t, i, None),
                 lambda: ops.fork(ob, t, 2, meta, i, i, t, i, None), lambda: ops.append(ob, 0, 0, t, t, None, None, None, t, 0, None),
                 lambda: ops.attend(ob, 0, -1, 0, t, t, t, 0.0, None)):
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            call()
for t in (three, nested, sparse, meta):
    with pytest.raises((ValueError, RuntimeError, TypeError)):
        ops.attend(ob, 0, -1, 0, t, t, None, 0.0, None)
bs = ops.make(1, 4096, 1, 0, 1, 2, 3, 1, 0, 2)
for t in (three, nested, sparse, meta):
    with pytest.raises((ValueError, RuntimeError, TypeError)):
        ops.select(bs, t, t, t, 0, t, t, t, t, None)
ops.release(ob)
ops.release(bs)
""")


def test_a_batch_of_another_device_is_refused(pkg):
    from confidence_gated_kv_logits_gb300.paged import PagedBatch, PagedKV, _load
    _load()
    kv = PagedKV.__new__(PagedKV)
    kv._h, kv._ob, kv._index = None, None, 0
    from confidence_gated_kv_logits_gb300.paged import BatchStruct
    batch = PagedBatch(BatchStruct(), (), 1, -1, 1)
    with pytest.raises(ValueError, match="device"):
        kv.append(0, batch, None, None)
    with pytest.raises(ValueError, match="device"):
        kv.attend(0, batch, None, None)
