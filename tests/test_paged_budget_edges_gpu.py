"""Normed appends, attention over shared prefixes, accumulated weights and eviction where calls meet the ends
of their ranges and one another.  Tolerances: those of test_paged_budget_gpu.py."""
import math

import numpy as np
import pytest
import torch

from tests.test_paged_budget_gpu import check_append
from tests.test_paged_gpu import DT, Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


# ---------------------------------------------------------------------------
# append with norms
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("r", [0, 64])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("low,high", [(-24, -17), (-10, 0), (0, 10), (60, 100)])
def test_append_normed_huge_rows_under_any_weights(pkg, low, high, wide, r):
    """Rows from 2^118 to the type's largest value: 1 / rms is small or subnormal, and weights from 1e-7 to 2^100 times it
    would leave fp32's range, in which the normed values and the results lie."""
    c = Case(torch.bfloat16, 4, 4, 64, 16, [0], [10], seed=high + r, extra_rows=0)
    x = c.randn(10, 4, 64).float().clamp(-0.99, 0.99) * 2.0 ** torch.arange(119, 129, device=DEV).float()[:, None, None]
    x = x.to(torch.bfloat16)
    x[9] = torch.finfo(torch.bfloat16).max
    assert torch.isfinite(x).all()
    w = [(2.0 ** (low + (high - low) * torch.rand(64, generator=c.g, device=DEV))).to(torch.float32 if wide else torch.bfloat16) for _ in range(2)]
    check_append(pkg, c, r, False, 0, w[0], w[1], q=x, k=x.flip(0).contiguous())


@pytest.mark.parametrize("wide", [False, True])
def test_append_normed_tiny_rows_under_huge_weights(pkg, wide):
    """Rows so small that eps alone counts: 1 / sqrt(eps) = 1e6 times a weight of 1e33 leaves fp32, the results (1e20 and less) do not."""
    c = Case(torch.bfloat16, 4, 4, 64, 16, [0], [6], seed=3, extra_rows=0)
    x = (c.randn(6, 4, 64).float() * 10.0 ** -torch.arange(20, 26, device=DEV).float()[:, None, None]).to(torch.bfloat16)
    w = [(1e33 * (1 + torch.rand(64, generator=c.g, device=DEV))).to(torch.float32 if wide else torch.bfloat16) for _ in range(2)]
    check_append(pkg, c, 64, True, 0, w[0], w[1], eps=1e-12, q=x, k=x.flip(0).contiguous())
