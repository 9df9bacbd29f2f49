"""Norms of rows that fp32 holds as subnormal numbers only. Tolerances as in test_gpu_block.py: 2^-8 for the bf16 result,
2^-18 for the sums, and the half step of the smallest bf16 or fp32 number where y is that small.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from test_gpu_attention import _bf16, _gen, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


@pytest.mark.parametrize("d", [8, 264, 2560, 8200, 16400])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-42, 1e-6])
@pytest.mark.parametrize("top", [2.0 ** -126, 2.0 ** -132, 2.0 ** -140, 2.0 ** -147])
def test_rows_of_subnormal_numbers(mx, d, eps, top):
    g = _gen(d)
    eps = float(np.float32(eps))
    x = (torch.rand((3, d), generator=g, device="cuda") + 0.5) * top
    x[:, ::3] *= -1
    w = _bf16(g, d)
    ref = ob.block_norm(_np(x), eps=eps, pre=_np(w))["h"]
    _, h = mx.moe_block_norm(x, eps=eps, pre_weight=w)
    assert np.all(np.abs(_np(h) - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref) + 2.0 ** -134)
    if top < 2.0 ** -132:
        return
    # and of the half's output, as bf16: its norm is added to a row of ordinary size
    a, z = x.to(torch.bfloat16), torch.randn((3, d), generator=g, device="cuda")
    r = ob.block_norm(_np(z), _np(a), _np(w), eps=eps)
    y, _ = mx.moe_block_norm(z, a, post_weight=w, eps=eps)
    assert np.all(np.abs(_np(y) - r["y"]) <= 2.0 ** -18 * np.abs(r["add"]) + 2.0 ** -23 * np.abs(_np(z)) + 2.0 ** -24 * np.abs(r["y"]) + 1e-38)


def test_the_smallest_number(mx):
    x = torch.full((2, 64), 2.0 ** -149, device="cuda")
    x[1, 1:] = 0.0
    _, h = mx.moe_block_norm(x, eps=0.0)
    assert torch.all(h[0] == 1.0) and float(h[1, 0]) == 8.0 and not h[1, 1:].any()
