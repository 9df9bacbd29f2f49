"""Codes and scales of rotated keys are those of the exact values, also inside pages in use, beside values that are not
finite, at far positions and for frequencies of any sign.

The oracle turns in fp64 and rounds once; where position times frequency has more than 53 bits, the angle comes from whole
numbers.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import block as ob
from test_gpu_attention import _Cache, _bf16, _cu, _gen, _i32, _np, _tables

pytestmark = pytest.mark.gpu
TURN = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
BEYOND = 2.0 ** 128 - 2.0 ** 103      # from here on fp32 rounds to infinity


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _freq(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def _append(mx, c, k, lens, start, table, f, interleaved, rope_start=None, turned=None):
    """On the GPU and in the oracle's cache (turned: the exact keys where fp64 products do not give them); the status."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = start if rope_start is None else rope_start
    mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu(lens), _i32(start), table, f, interleaved=interleaved, dev_status=status,
                              rope_start=None if rope_start is None else _i32(rope_start))
    if turned is None:
        pos = np.concatenate([np.arange(n) + p for n, p in zip(lens, at)])
        assert pos.max(initial=0) < 2 ** 29
        with np.errstate(invalid="ignore"):
            turned = ob.rotate(_np(k), pos, _np(f), interleaved)
    turned = np.where(np.abs(turned) >= BEYOND, np.inf, turned)
    tab, t0 = table.cpu().numpy(), 0
    for b, n in enumerate(lens):
        oa.append(c.codes["k"], c.scales["k"], turned[t0:t0 + n], start[b], tab[b])
        t0 += n
    return int(status)


def _same(c):
    assert np.array_equal(c.gpu.k_scales.cpu().numpy(), c.scales["k"])
    got, want = c.gpu.k_codes.cpu().numpy(), c.codes["k"]
    got, want = (np.where(x & 0x7F == 0x7F, 0x7F, x) for x in (got, want))       # NaN of either sign
    same = (got == want) | ((got | want) & 0x7F == 0)
    assert same.all(), (int((~same).sum()), np.argwhere(~same)[:4].tolist())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("P,d,r,n_seq", [(16, 64, 32, 600), (64, 128, 128, 120), (128, 128, 64, 60), (32, 64, 64, 300)])
def test_pages_in_use(mx, P, d, r, n_seq, interleaved):
    """Tokens behind others of the same page: one and two a sequence, and more; scales that stay and that grow."""
    g, H = _gen(P + d), 8
    c, table, f = _Cache(mx, n_seq * 3, P, H, d), _tables(n_seq, 3), _freq(r)
    at = [0] * n_seq
    for step, spread in ((lambda b: 3 + b % (P // 2), 1.0), (lambda b: 1, 1.0), (lambda b: 1, 4.0), (lambda b: 2, 0.25),
                         (lambda b: 5 + b % 9, 16.0), (lambda b: b % 3, 60.0), (lambda b: 1 + b % 7, 1.0)):
        lens = [step(b) for b in range(n_seq)]
        _append(mx, c, _bf16(g, sum(lens), H, d, spread=spread), lens, at, table, f, interleaved)
        _same(c)
        at = [a + n for a, n in zip(at, lens)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,start", [([3000, 700], [0, 21]), ([1] * 500, [37] * 500), ([2] * 300, [64] * 300)])
def test_beside_values_that_are_not_finite(mx, lens, start, interleaved):
    """One such channel in a fifth of the rows: its pair becomes NaN, the rest of the head keeps exact codes."""
    g, H, d, P = _gen(len(lens)), 8, 128, 64
    width = max(n + s for n, s in zip(lens, start)) // P + 1
    c, table, f = _Cache(mx, len(lens) * width, P, H, d), _tables(len(lens), width), _freq(96)
    k = _bf16(g, sum(start), H, d, spread=0.5)
    _append(mx, c, k, start, [0] * len(lens), table, f, interleaved)
    k = _bf16(g, sum(lens), H, d)
    for i, bad in enumerate((math.inf, -math.inf, math.nan)):
        rows = torch.arange(i, sum(lens), 15, device="cuda")
        k[rows, rows % H, rows * 7 % d] = bad
    assert _append(mx, c, k, lens, start, table, f, interleaved) == mx.DEV_NONFINITE_INPUT
    _same(c)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens", [[400], [1] * 200])
def test_keys_next_to_the_largest_number(mx, lens, interleaved):
    """Pairs whose turned channels lie on both sides of what fp32 holds."""
    g = _gen(5)
    k = (torch.rand((sum(lens), 4, 64), generator=g, device="cuda") * 0.6 + 0.4) * 3.38e38
    k = (k * (torch.randint(0, 2, k.shape, generator=g, device="cuda") * 2 - 1)).to(torch.bfloat16)
    c, table = _Cache(mx, 16 * len(lens), 32, 4, 64), _tables(len(lens), 16)
    assert _append(mx, c, k, lens, [0] * len(lens), table, _freq(64), interleaved, rope_start=[1000] * len(lens)) == mx.DEV_NONFINITE_INPUT
    _same(c)


@pytest.mark.parametrize("tokens", [1, 5])
def test_a_key_within_an_fp32_step_of_infinity(mx, tokens):
    """Angles that put the larger channel of a pair right below and right above it."""
    a = float(torch.tensor(3.38e38).to(torch.bfloat16))
    theta = np.float32(math.pi / 4 - math.acos(BEYOND / (a * math.sqrt(2.0))))     # a (cos t + sin t) = BEYOND
    seen = set()
    for step in range(-8, 9):
        t = theta
        for _ in range(abs(step)):
            t = np.nextafter(t, np.float32(9.0 if step > 0 else 0.0))
        k = torch.zeros((tokens, 2, 64), dtype=torch.bfloat16, device="cuda")
        k[0, :, 0], k[0, :, 8] = a, a
        c, f = _Cache(mx, 2, 16, 2, 64), torch.full((8,), float(t), device="cuda")
        status = _append(mx, c, k, [tokens], [0], _i32([[0, 1]]), f, False, rope_start=[1])
        big = a * (math.cos(float(t)) + math.sin(float(t)))
        assert (status != 0) == (big >= BEYOND), step
        _same(c)
        seen.add(status)
    assert len(seen) == 2


def _exact(k, pos, f, interleaved):
    """Keys turned by angles that whole numbers reduce."""
    x, r = _np(k), 2 * len(f)
    y = x.copy()
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    for t, p in enumerate(pos):
        z = [Fraction(fj) * int(p) / TURN for fj in f.tolist()]
        w = np.array([float((v - round(v)) * TURN) for v in z])
        co, si = np.cos(w), np.sin(w)
        y[t][:, i] = x[t][:, i] * co - x[t][:, j] * si
        y[t][:, j] = x[t][:, j] * co + x[t][:, i] * si
    return y


# position, pair (of 32), channels: values that an angle wrong by 2^-31 of a radian puts on the other side of a border
FAR = [(2138202708, 1, 36.0, -2.046875), (2144234721, 8, 59.0, -3.6875), (2146559153, 3, 39.75, 25.75), (2146559153, 3, 51.5, -79.5)]


@pytest.mark.parametrize("p,j,a,b", FAR)
@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(mx, p, j, a, b, tokens, interleaved):
    k = torch.zeros((tokens, 1, 128), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 127] = 448.0                     # the scale: one
    k[0, 0, 2 * j if interleaved else j], k[0, 0, 2 * j + 1 if interleaved else j + 32] = a, b
    c, f = _Cache(mx, 1, 16, 1, 128), _freq(64)
    _append(mx, c, k, [tokens], [0], _i32([[0]]), f, interleaved, rope_start=[p], turned=_exact(k, p + np.arange(tokens), f, interleaved))
    assert int(c.scales["k"][0, 0]) == 127
    _same(c)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,factor", [([4000], -1.0), ([1] * 2000, -1.0), ([1500], 1000.0), ([1500], -1234.5), ([700], 1e6), ([700], 1e-6)])
def test_frequencies_of_any_size_and_sign(mx, lens, factor, interleaved):
    g, P, n = _gen(7), 64, len(lens)
    width = lens[0] // P + 1
    c, table, f = _Cache(mx, n * width, P, 8, 128), _tables(n, width), _freq(128) * factor
    bits = 2 ** 53 / 2 ** 24
    assert bits == 2 ** 29
    at = [2 ** 29 - lens[0] - 64 * b for b in range(n)]
    _append(mx, c, _bf16(g, sum(lens), 8, 128), lens, [0] * n, table, f, interleaved, rope_start=at)
    _same(c)


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan, 2.0 ** 41])
def test_frequencies_that_are_no_angles(mx, bad, tokens, interleaved):
    """They give NaN, for keys and queries, and nothing else does."""
    f = _freq(32)
    f[3] = bad
    k, q = _bf16(_gen(8), tokens, 2, 64), _bf16(_gen(9), tokens, 4, 64)
    c, status = _Cache(mx, 1, 16, 2, 64), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu([tokens]), _i32([0]), _i32([[0]]), f, q=q, interleaved=interleaved,
                                    rope_start=_i32([1000]), dev_status=status)
    assert int(status) == mx.DEV_NONFINITE_INPUT
    pair = [6, 7] if interleaved else [3, 19]
    want = torch.zeros(64, dtype=torch.bool, device="cuda")
    want[pair] = True
    assert torch.equal(torch.isnan(out), want.expand_as(out))
    assert torch.equal(c.gpu.k_codes[0, :, :tokens] & 0x7F == 0x7F, want.expand(2, tokens, 64))
