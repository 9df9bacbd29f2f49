"""Routing by groups whose biases force experts, mask them or are as large as fp32 holds: experts by the definition in fp64,
no expert twice."""
import math

import numpy as np
import pytest
import torch

from oracle import block as ob
from test_gpu_attention import _gen, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _check(mx, l, k, bias, score, n, top, best):
    idx, w = mx.moe_route_groups(l, k, bias, score, n, top, best)
    got = idx.cpu().numpy()
    assert all(len(set(row)) == k for row in got.tolist())
    want = ob.route_groups(_np(l), k, _np(bias), score, n, top, best)
    assert np.array_equal(got, want[0])
    assert np.all(np.abs(_np(w) - want[1]) <= 2.0 ** -18 * np.abs(want[1]) + 2.0 ** -120)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
def test_forced_and_masked_in_one_group(mx, score, best):
    l = torch.randn((30, 64), generator=_gen(1), device="cuda")
    for forced in ([8], [8, 41], [8, 9], [0, 8, 41, 63]):
        bias = torch.randn(64, generator=_gen(2), device="cuda") * 0.1
        for e in forced:
            bias[e // 8 * 8:e // 8 * 8 + 8] = -math.inf
        for e in forced:
            bias[e] = math.inf
        for top in (1, 2, 5):
            for k in (1, 4, 8):
                _check(mx, l, k, bias, score, 8, top, best)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups_that_are_masked_whole(mx, score):
    l = torch.randn((30, 64), generator=_gen(3), device="cuda")
    bias = torch.randn(64, generator=_gen(4), device="cuda") * 0.1
    bias[:40] = -math.inf
    bias[50] = math.nan
    for top in (1, 3, 4):
        _check(mx, l, 8, bias, score, 8, top, 2)
    # one group with a single expert left
    bias[40:47] = -math.inf
    _check(mx, l, 4, bias, score, 8, 3, 2)
    l[:5, 47] = math.nan
    _check(mx, l, 4, bias, score, 8, 4, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sums_beyond_fp32(mx, score, sign):
    """Two keys of a group add up to more than fp32 holds; their order is that of the sums."""
    l = torch.randn((20, 64), generator=_gen(5), device="cuda")
    bias = sign * (2.0 + torch.randperm(64, generator=torch.Generator().manual_seed(6)).float().cuda() / 64) * 1e38
    for top in (1, 3, 5):
        _check(mx, l, 8, bias, score, 8, top, 2)
        _check(mx, l, 2, bias, score, 32, 2 * top, 2)      # groups of two
        bias[::5] = 0.25
