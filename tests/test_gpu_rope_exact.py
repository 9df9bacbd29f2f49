"""Codes and scales of rotated keys are those of the exact values: an error of the fp32 rotation decides neither.

The oracle turns in fp64 and rounds once. A value lies within fp64's own error of a border between two codes once in
2^40, which no case here meets.
"""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import block as ob
from test_gpu_attention import _Cache, _bf16, _cu, _gen, _i32, _np, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _both(mx, k, f, lens, start, P, interleaved, seed):
    """Append on the GPU and in the oracle's cache; codes and scales of both."""
    H, D = k.shape[1:]
    width = max((n + s - 1) // P + 1 for n, s in zip(lens, start))
    table = _tables(len(lens), width, seed)
    c = _Cache(mx, len(lens) * width, P, H, D)
    mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu(lens), _i32(start), table, f, interleaved=interleaved)
    pos = np.concatenate([np.arange(n) + s for n, s in zip(lens, start)])
    kr, tab, t0 = ob.rotate(_np(k), pos, _np(f), interleaved), table.cpu().numpy(), 0
    for b, n in enumerate(lens):
        oa.append(c.codes["k"], c.scales["k"], kr[t0:t0 + n], start[b], tab[b])
        t0 += n
    return (c.gpu.k_codes.cpu().numpy(), c.gpu.k_scales.cpu().numpy()), (c.codes["k"], c.scales["k"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("P,D,r,lens,start", [(64, 128, 128, [4100], [70016]), (16, 64, 32, [1999, 1500], [0, 160]),
                                              (128, 128, 64, [3000, 1, 257], [0, 0, 1 << 20]), (32, 64, 64, [1] * 400, [64] * 400),
                                              (64, 128, 128, [2] * 150, [128] * 150)])
def test_codes(mx, P, D, r, lens, start, interleaved):
    k = _bf16(_gen(r + len(lens)), sum(lens), 8, D)
    f = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
    start = [s - s % P for s in start]       # whole pages: no older codes
    got, want = _both(mx, k, f, lens, start, P, interleaved, 3)
    assert np.array_equal(got[1], want[1])
    same = (got[0] == want[0]) | ((got[0] | want[0]) & 0x7F == 0)
    assert same.all(), int((~same).sum())


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("interleaved", [False, True])
def test_scales_next_to_a_border(mx, tokens, interleaved):
    """A page's largest value within a few 2^-25 of 448, on both sides of it, for one angle after another."""
    theta = np.float32(math.acos(448 / 500))
    seen = set()
    for step in range(-12, 13):
        t = theta
        for _ in range(abs(step)):
            t = np.nextafter(t, np.float32(9.0 if step > 0 else 0.0))
        k = torch.zeros((tokens, 2, 64), dtype=torch.bfloat16, device="cuda")
        k[0, :, 0] = 500.0                  # at position 1 below
        f = torch.full((8,), float(t), device="cuda")
        table = _i32([[0, 1]])
        c = _Cache(mx, 2, 16, 2, 64)
        mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu([tokens]), _i32([0]), table, f, interleaved=interleaved, rope_start=_i32([1]))
        exact = 500.0 * math.cos(float(t))
        want = 127 if max(exact, 500.0 * math.sin(float(t))) <= 448.0 else 128
        assert c.gpu.k_scales[0].tolist() == [want, want], (step, exact)
        seen.add(want)
    assert seen == {127, 128}


@pytest.mark.parametrize("tokens", [1, 5])
def test_scales_next_to_a_border_of_a_page_in_use(mx, tokens):
    """The older codes of the page are rescaled once, to the scale that the exact value needs."""
    theta = np.float32(math.acos(448 / 500))
    for step in range(-3, 4):
        t = theta
        for _ in range(abs(step)):
            t = np.nextafter(t, np.float32(9.0 if step > 0 else 0.0))
        f = torch.full((8,), float(t), device="cuda")
        table = _i32([[1, 0]])
        c = _Cache(mx, 2, 16, 2, 64)
        first = _bf16(_gen(9), 1, 2, 64)
        k = torch.zeros((tokens, 2, 64), dtype=torch.bfloat16, device="cuda")
        k[0, :, 0], k[0, 1, 20] = 500.0, 3.0
        mx.moe_kv_append_rope_fp8(c.gpu, first, first, _cu([1]), _i32([0]), table, f)
        mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu([tokens]), _i32([1]), table, f)
        tab = table.cpu().numpy()
        oa.append(c.codes["k"], c.scales["k"], ob.rotate(_np(first), np.array([0.0]), _np(f), False), 0, tab[0])
        oa.append(c.codes["k"], c.scales["k"], ob.rotate(_np(k), np.arange(1.0, tokens + 1), _np(f), False), 1, tab[0])
        assert np.array_equal(c.gpu.k_scales.cpu().numpy(), c.scales["k"]), step
        got = c.gpu.k_codes.cpu().numpy()
        assert ((got == c.codes["k"]) | ((got | c.codes["k"]) & 0x7F == 0)).all(), step


@pytest.mark.parametrize("lens", [[300], [1] * 70, [2] * 40])
def test_every_group_in_doubt(mx, lens):
    """Without an angle many bf16 values lie on a border exactly: more than a CTA lists."""
    k = _bf16(_gen(11), sum(lens), 8, 128)
    f = torch.zeros(64, device="cuda")
    got, want = _both(mx, k, f, lens, [0] * len(lens), 128, False, 5)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0] & 0x7F, want[0] & 0x7F)
