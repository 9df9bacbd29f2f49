"""Routing by groups where keys crowd at the cut: experts that share logit and bias next to others that fp32 cannot tell
from them.

Experts are held to the definition in fp64. Distinct keys lie at least 2^-40 of a score apart, which the sums of two fp32
numbers resolve; equal ones go to the lower expert.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from mxfp4_expert_gb300 import synthetic
from oracle import block as ob
from test_gpu_attention import _gen, _np
from test_gpu_block import _check_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


@pytest.mark.parametrize("logits", [[20.0, 20.0, 30.0], [16.0, 16.0, 16.125], [30.0, 20.0, 20.0, 25.0, 20.0], [18.0] * 40 + [19.0]])
@pytest.mark.parametrize("k", [1, 2])
def test_sigmoids_next_to_one(mx, logits, k):
    """Scores that fp32 rounds to 1, two of them of one logit."""
    l = torch.tensor([logits], device="cuda")
    idx, _ = _check_route(mx, l, k, torch.zeros(len(logits), device="cuda"), group_best=1)
    assert int(idx[0, 0]) == int(l[0].argmax())


def _crowd(score, twins, others, E, seed, far=-3.0):
    """One token's logits and a bias: `twins` experts of one logit and bias, `others` of other ones, all with keys within
    2^-24 of 0.75 and distinct ones 2^-38 apart; the rest far below. The best key is one of the others."""
    for tries in range(1000):
        g = torch.Generator().manual_seed(1000 * seed + tries)
        l, bias = torch.randn(E, generator=g), torch.full((E,), far)
        at = torch.randperm(E, generator=g)[:twins + others]
        same = at[:twins].sort().values
        l[same] = l[same[0]].clone()
        s = ob.scores(l[None].numpy(), score)[0][0]
        bias[at] = torch.from_numpy(0.75 - s[at.numpy()]).float()
        key = s + bias.double().numpy()
        near = np.sort(key[at.numpy()])
        gaps = np.diff(near)
        gaps = gaps[gaps > 0]
        if len(gaps) == others and gaps.min() > 2.0 ** -38 and near[-1] - near[0] < 2.0 ** -24 and near[-1] > near[-2]:
            return l, bias, same
    raise AssertionError("no such crowd")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("twins,others", [(2, 1), (2, 3), (3, 2), (5, 6), (12, 9), (40, 2)])
def test_twins_at_the_cut(mx, score, twins, others):
    for seed in range(12):
        l, bias, _ = _crowd(score, twins, others, 128, seed)
        for k in {1, 2, 3, min(twins, 31), min(twins + others - 1, 32)}:
            _check_route(mx, l[None].cuda(), k, bias.cuda(), score, group_best=1)
            if k <= 16:
                _check_route(mx, l[None].cuda(), k, bias.cuda(), score, 4, 4, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_twins_in_the_groups_taken(mx, score):
    """The crowd lies in groups that are taken for a larger key of theirs."""
    for seed in range(12):
        l, bias, same = _crowd(score, 2, 3, 128, seed)
        bias[torch.arange(8) * 16 + 5] += 2.0 + 0.125 * torch.arange(8)
        for k in (2, 3, 4, 5, 8):
            _check_route(mx, l[None].cuda(), k, bias.cuda(), score, 8, 5, 1)


@pytest.mark.parametrize("T", [1, 3, 4, 6])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_the_layer_with_twins(mx, T, score):
    """Router rows that are alike give logits that are; in the single launch and by the per-stage kernels."""
    w = wl.get("tiny", E=128, k=4)
    layer = synthetic.build_layer(w, 0)
    layer.router_w[1::2] = layer.router_w[::2]
    x = torch.randn((T, w.d), generator=_gen(T), device="cuda").to(torch.bfloat16)
    logits, idx = torch.empty((T, w.E), device="cuda"), torch.empty((T, w.k), dtype=torch.int32, device="cuda")
    mx.moe_forward_groups(layer, x, logits_out=logits)
    assert torch.equal(logits[:, 1::2], logits[:, ::2])
    for t in range(T):
        s = ob.scores(_np(logits[t:t + 1]), score)[0][0]
        bias = torch.from_numpy(0.75 - s).float().cuda()
        bias[16:] = -3.0             # eight pairs are left, of this token
        again = torch.empty_like(logits)
        mx.moe_forward_groups(layer, x, bias, score=score, logits_out=again, idx_out=idx, group_best=1)
        assert torch.equal(again, logits)
        want = ob.route_groups(_np(logits), w.k, _np(bias), score)[0]
        assert np.array_equal(idx[t].cpu().numpy(), want[t])
