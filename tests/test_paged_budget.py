"""Refusals of normed appends, attention over shared prefixes, accumulated weights and eviction
(CPU: argument checks come before any work; the tensors' checks are the binding's)."""
import ctypes
import subprocess
import sys

import pytest


@pytest.fixture(scope="module")
def pkg():
    from confidence_gated_kv_logits_gb300 import build as B
    B.build()
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


def test_null_handles(pkg):
    L = pkg.load_library()
    bad = pkg.ERR_INVALID_ARG
    assert L.confkv_paged_append_normed(None, None, 0, 1, *([0] * 8), None, None, 0, 0, None, None) == bad
    assert L.confkv_paged_attend_shared(None, None, None, 0, 1, None, 0, None, None, 0.0, None) == bad
    assert L.confkv_paged_weigh(None, None, 0, 1, None, 0, None, None, None, None, 1, None, 1.0, 1.0, 0.0, None) == bad
    assert L.confkv_paged_evict(None, 1, 1, None, None, 0, None, None, 1, None, None, 0, None, None, None, None) == bad


@pytest.mark.parametrize("rows,heads,d,want", [
    (1, 8, 128, 8 * 130 * 4), (0, 8, 64, 8 * 66 * 4), (-1, 8, 128, 0), (1, 0, 128, 0), (1, 8, 96, 0), (1 << 30, 8, 64, 0),
    (1000, 40, 128, 1000 * 40 * 130 * 4)])
def test_partial_bytes(pkg, rows, heads, d, want):
    assert pkg.load_library().confkv_paged_partial(rows, heads, d) == want


def test_binding_refuses_tensors(pkg):
    """On tensors of the CPU every call of the binding raises before the library is reached."""
    code = """
import torch, pytest
from confidence_gated_kv_logits_gb300 import _paged_ops as ops
ob = ops.make(4096, 0, 0, 0, 2, 1, 64, 0, 0, 0)
i = torch.zeros(2, dtype=torch.int32)
f = torch.zeros(2, 1, 8)
nested = torch.nested.nested_tensor([torch.zeros(2, 64), torch.zeros(3, 64)])
sparse = torch.zeros(2, 3, dtype=torch.int32).to_sparse()
meta = torch.zeros(2, 2, 64, dtype=torch.float16, device="meta")
half = torch.zeros(2, 2, 64, dtype=torch.float16)
for t in (nested, sparse, meta, half, i, 3, None):
    for call in (lambda: ops.append_normed(ob, 0, 0, t, t, None, None, None, None, 0, t, t, 1e-6, None, None),
                 lambda: ops.append_normed(ob, 0, 0, t, t, t, t, t, t, 0, None, None, 1e-6, t, None),
                 lambda: ops.attend_shared(ob, 0, 0, -1, 0, t, t, t, 0.0, None),
                 lambda: ops.weigh(ob, 0, 2, -1, 0, t, t, f, f, None, None, 1.0, 1.0, 0.0, None),
                 lambda: ops.evict(ob, 2, t, i, f, i, i, f, i, i, 0, None, None),
                 lambda: ops.evict(ob, 2, i.view(1, 2), t, f, i, i, f, i, i, 0, None, None)):
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            call()
for n, call in ((15, ops.append_normed), (10, ops.attend_shared), (15, ops.weigh), (13, ops.evict)):
    with pytest.raises(TypeError):
        call(*([None] * (n - 1)))
    with pytest.raises(ValueError, match="closed"):
        call(*([0] * n))
with pytest.raises(ValueError):
    ops.weigh(ob, 0, 2, -1, 0, half, i, f, f, None, None, 1.0, 1.0, 1e-60, None)     # a scale that is zero in 32 bits
ops.release(ob)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_handles_of_another_device_are_refused(pkg):
    from confidence_gated_kv_logits_gb300.paged import BatchStruct, PagedBatch, PagedKV, PrefixStruct, SharedPrefix, _load
    _load()
    kv = PagedKV.__new__(PagedKV)
    kv._h, kv._ob, kv._index = None, None, 0
    far, near = PagedBatch(BatchStruct(), (), 1, -1, 1), PagedBatch(BatchStruct(), (), 1, -1, 0)
    with pytest.raises(ValueError, match="device"):
        kv.append(0, far, None, None, axis=1)
    with pytest.raises(ValueError, match="device"):
        kv.weigh(0, far, None, None, None, None)
    with pytest.raises(ValueError, match="device"):
        kv.attend(0, near, None, None, prefix=SharedPrefix(PrefixStruct(), (), 1, 1))


def test_structures_have_the_headers_layout(pkg):
    from confidence_gated_kv_logits_gb300.paged import NormStruct, PrefixStruct
    assert ctypes.sizeof(NormStruct) == 40 and NormStruct.axis.offset == 24 and NormStruct.eps.offset == 20
    assert ctypes.sizeof(PrefixStruct) == 40 and PrefixStruct.partial_bytes.offset == 32
