"""Append with the position rotation, and attention of chunks over the cache, on the GPU against the fp64 oracles.

Tolerances. The rotation: cosine and sine err by at most 2^-23 (an angle reduced to 2^-32 of a turn, rounded to fp32, and
a series), products and their sum are rounded to fp32, so a turned channel errs by u = 2^-22 (|a| + |b|) of its pair. A
query adds the half step of bf16, 2^-8 of it. A key's code is the nearest of a value that lies within u of the exact
one: it may be the exact one's neighbour where that lies within u of the middle between them, so
|code's value - exact| <= |oracle code's value - exact| + 2 u; scales are equal unless the page's largest value lies
within u of a power of two times 448. Values are compared bit for bit.

Attention: outputs are bf16 (2^-8 of them at most); probabilities enter the second product as f16, 2^-11 of each, where
they are above 2^-22 of the row's largest product with its page's scale, and to 2^-32 of that below; scores are fp32
sums of at most 128 products, 2^-17 of their size, and change a probability by that factor twice:
  |y - ref| <= 2^-8 |ref| + (2^-10 + 2^-15 (1 + size)) sum p |v| + n 2^-32 448 max (p 2^scale)
  |lse - ref| <= 2^-16 (1 + size).
"""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import block as ob
from test_gpu_attention import _Cache, _bf16, _cu, _filled, _gen, _i32, _np, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


# ---- append with rotation ---------------------------------------------------------------------------------------

def _freq(r, base=10000.0):
    return (base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def _decode(codes, scales):
    with np.errstate(invalid="ignore"):
        return oa.decode(codes, scales[:, :, None, None].astype(np.int64))


def _check_append(mx, c, k, v, q, lens, start, table, f, interleaved, rope_start=None, want_status=0):
    """Append on the GPU and in the oracle's copy of the cache; compare everything."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda") if q is not None else None
    got = mx.moe_kv_append_rope_fp8(c.gpu, k, v, _cu(lens), _i32(start), table, f, q=q, interleaved=interleaved,
                                    rope_start=None if rope_start is None else _i32(rope_start), q_out=q_out,
                                    dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == want_status and got is q_out
    r, fn = 2 * len(f), _np(f)
    pos = np.concatenate([np.arange(n) + p for n, p in zip(lens, start if rope_start is None else rope_start)]).astype(np.float64)
    if q is not None:
        ref, size = ob.rotate(_np(q), pos, fn, interleaved), ob.pair_size(_np(q), r, interleaved)
        assert np.all(np.abs(_np(q_out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size)
    kr, ks = ob.rotate(_np(k), pos, fn, interleaved), ob.pair_size(_np(k), r, interleaved)
    tab, t0, P = table.cpu().numpy(), 0, c.codes["k"].shape[2]
    exact, slack = _decode(c.codes["k"], c.scales["k"]), np.zeros(c.codes["k"].shape)
    for b, n in enumerate(lens):
        oa.append(c.codes["k"], c.scales["k"], kr[t0:t0 + n], start[b], tab[b])
        oa.append(c.codes["v"], c.scales["v"], _np(v[t0:t0 + n]), start[b], tab[b])
        for i in range(n):
            p = start[b] + i
            exact[tab[b, p // P], :, p % P] = kr[t0 + i]
            slack[tab[b, p // P], :, p % P] = 2.0 ** -21 * ks[t0 + i]
        t0 += n
    assert np.array_equal(c.gpu.v_scales.cpu().numpy(), c.scales["v"])
    assert np.array_equal(c.gpu.v_codes.cpu().numpy(), c.codes["v"])
    assert np.array_equal(c.gpu.k_scales.cpu().numpy(), c.scales["k"])
    mine = c.gpu.k_codes.cpu().numpy()
    differ = mine != c.codes["k"]
    far = np.abs(_decode(mine, c.scales["k"]) - exact) > np.abs(_decode(c.codes["k"], c.scales["k"]) - exact) + slack
    assert not np.any(differ & (far | (slack == 0))), np.argwhere(differ & far)[:4].tolist()
    assert differ.mean() < 1e-3
    c.codes["k"][:] = mine


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("P,d,r", [(16, 64, 64), (16, 128, 48), (32, 64, 16), (32, 128, 128), (64, 64, 32), (64, 128, 64),
                                   (128, 64, 48), (128, 128, 128), (128, 128, 112)])
def test_rope_prompts_and_tokens(mx, P, d, r, interleaved):
    """Prompts, single tokens behind them, and more; spreads that make scales grow."""
    g = _gen(P + d + r)
    H = 3
    c = _Cache(mx, 4 * 7, P, H, d)
    table, at, f = _tables(4, 7), [0, 0, 0, 0], _freq(r)
    for lens, spread in [([P + 1, 0, 2 * P, 5], 0.01), ([1, 1, 1, 1], 0.5), ([1, 3, P, 2 * P + 3], 40.0),
                         ([1, 1, 1, 1], 1e-3), ([0, 0, 0, 1], 1e4), ([2, P - 1, 1, 0], 1e-9)]:
        n = sum(lens)
        k, v, q = _bf16(g, n, H, d, spread=spread), _bf16(g, n, H, d, spread=3 * spread), _bf16(g, n, 2 * H, d)
        _check_append(mx, c, k, v, q, lens, at, table, f, interleaved)
        at = [a + n for a, n in zip(at, lens)]


@pytest.mark.parametrize("heads", [1, 3, 4, 5, 8, 20])
def test_rope_query_heads(mx, heads):
    g = _gen(heads)
    c = _Cache(mx, 6, 32, 1, 128)
    kv = _bf16(g, 70, 2 + heads, 128)
    _check_append(mx, c, kv[:, :1], kv[:, 1:2], kv[:, 2:], [40, 30], [0, 0], _tables(2, 3), _freq(128), False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions(mx, interleaved):
    """Angles of positions up to the largest int, by the definition in integers."""
    g = _gen(2)
    c = _Cache(mx, 8, 16, 2, 64)
    n = 5
    x, q = _bf16(g, 4 * n, 2, 64), _bf16(g, 4 * n, 2, 64)
    at = [0, 1 << 20, (1 << 30) + 12345, (1 << 31) - n]
    f = _freq(64)
    out = mx.moe_kv_append_rope_fp8(c.gpu, x, x, _cu([n] * 4), _i32([0] * 4), _tables(4, 2), f, q=q, interleaved=interleaved,
                                    rope_start=_i32(at))
    # the angle modulo 2 pi in long integers: 2 pi to 40 digits
    from fractions import Fraction
    turn = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
    t = np.zeros((4 * n, 32))
    for b, p0 in enumerate(at):
        for i in range(n):
            for j, fj in enumerate(f.tolist()):
                z = Fraction(fj) * (p0 + i) / turn
                t[b * n + i, j] = float((z - math.floor(z)) * turn)
    # the fraction of a turn is exact to p 2^-52 of the turns a step makes, 2^-53 / pi for the fastest: 2^-21 of a radian
    # at 2^31, to which comes the rounding's share
    one = torch.ones(1)  # rotate() takes angles as positions times one frequency
    ref = np.empty((4 * n, 2, 64))
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    qn, co, si = _np(q), np.cos(t)[:, None], np.sin(t)[:, None]
    ref[..., a], ref[..., b] = qn[..., a] * co - qn[..., b] * si, qn[..., b] * co + qn[..., a] * si
    size = ob.pair_size(qn, 64, interleaved)
    assert np.all(np.abs(_np(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size), one


def test_rope_start_apart_from_the_cache(mx):
    """After an eviction the cache holds fewer positions than the sequence had."""
    g = _gen(3)
    c = _Cache(mx, 8, 32, 2, 128)
    k, v, q = (_bf16(g, 50, h, 128) for h in (2, 2, 4))
    _check_append(mx, c, k, v, q, [20, 30], [0, 0], _tables(2, 4), _freq(64), False, rope_start=[1000, 77777])


def test_rope_at_position_zero_is_the_plain_append(mx):
    g = _gen(4)
    a, b = _Cache(mx, 12, 16, 2, 64), _Cache(mx, 12, 16, 2, 64)
    k, v = _bf16(g, 6, 2, 64), _bf16(g, 6, 2, 64)
    lens, table = [1] * 6, _tables(6, 2)
    q = _bf16(g, 6, 4, 64)
    out = mx.moe_kv_append_rope_fp8(a.gpu, k, v, _cu(lens), _i32([0] * 6), table, _freq(64), q=q)
    mx.moe_kv_append_fp8(b.gpu, k, v, _cu(lens), _i32([0] * 6), table)
    assert torch.equal(out, q)
    for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(a.gpu, n), getattr(b.gpu, n))


def test_rope_many_sequences_without_queries(mx):
    g = _gen(5)
    n_seq = 100
    c = _Cache(mx, n_seq * 3, 32, 2, 128)
    table = _tables(n_seq, 3)
    lens, start = [(i * 13) % 4 for i in range(n_seq)], [(i * 29) % 60 for i in range(n_seq)]
    kv = _bf16(g, sum(start), 4, 128)
    _check_append(mx, c, kv[:, :2], kv[:, 2:], None, start, [0] * n_seq, table, _freq(128), False)
    kv = _bf16(g, sum(lens), 4, 128, spread=5.0)
    _check_append(mx, c, kv[:, 1:3], kv[:, 2:], None, lens, start, table, _freq(128), True)


def test_rope_special_values(mx):
    """Zeros; inf and NaN become NaN with their pairs and are reported; rows outside every sequence stay."""
    c = _Cache(mx, 8, 16, 2, 64)
    table, f = _tables(2, 4), _freq(64)
    x = torch.zeros((20, 2, 64), dtype=torch.bfloat16, device="cuda")
    _check_append(mx, c, x, x, x, [20, 0], [0, 0], table, f, False)
    z = _bf16(_gen(0), 3, 2, 64)
    z[0, 0, 3], z[1, 1, 4], z[2, 0, 5] = math.inf, -math.inf, math.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mx.moe_kv_append_rope_fp8(c.gpu, z, z, _cu([3, 0]), _i32([20, 0]), table, f, q=z, dev_status=status)
    assert int(status) == mx.DEV_NONFINITE_INPUT
    codes = c.gpu.k_codes[int(table[0, 1]), :, 4:7].cpu().numpy() & 0x7F
    bad = {(0, 0, 3), (0, 0, 35), (1, 1, 4), (1, 1, 36), (0, 2, 5), (0, 2, 37)}
    assert {tuple(i) for i in np.argwhere(codes == 0x7F).tolist()} == bad
    assert {(h, t, ch) for t, h, ch in np.argwhere(~np.isfinite(_np(out))).tolist()} == bad
    q_out = torch.full((6, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    y = _bf16(_gen(1), 6, 2, 64)
    mx.moe_kv_append_rope_fp8(c.gpu, y, y, _i32([0, 2, 4]), _i32([0, 0]), table, f, q=y[:, :1], q_out=q_out)
    assert torch.all(q_out[4:] == 3.0) and not torch.any(q_out[:4] == 3.0)


def test_rope_reports_what_it_cannot_place(mx):
    c = _Cache(mx, 4, 16, 1, 64)
    x, f = _bf16(_gen(1), 4, 1, 64), _freq(64)
    for bad, start, cu in (([[4, 1]], 0, [0, 4]), ([[-1, 1]], 0, [0, 4]), ([[0, 1]], -1, [0, 4]), ([[0, 1]], 30, [0, 4]),
                           ([[0, 1]], 0, [3, 1]), ([[0, 1]], 2 ** 31 - 2, [0, 4])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mx.moe_kv_append_rope_fp8(c.gpu, x, x, _i32(cu), _i32([start]), _i32(bad), f, q=x, dev_status=status)
        assert int(status) == mx.DEV_INDEX_OOB, (bad, start, cu)


def test_rope_binding_refusals(mx):
    c = _Cache(mx, 4, 16, 2, 64)
    x, f = _bf16(_gen(1), 4, 2, 64), _freq(64)
    args = (c.gpu, x, x, _cu([4]), _i32([0]), _i32([[0, 1]]))
    for bad in (dict(inv_freq=f.double()), dict(inv_freq=f, q=x.float()), dict(inv_freq=f, rope_start=_i32([0]).long())):
        with pytest.raises(TypeError):
            mx.moe_kv_append_rope_fp8(*args, **bad)
    for bad in (dict(inv_freq=f, q=x[:3]), dict(inv_freq=f, q_out=x), dict(inv_freq=f[None]), dict(inv_freq=f, rope_start=_i32([0, 1])),
                dict(inv_freq=f, q=x, q_out=x[:, :1])):
        with pytest.raises(ValueError):
            mx.moe_kv_append_rope_fp8(*args, **bad)
    for bad in (f[:4], f[:20], torch.cat([f, f])):
        with pytest.raises(mx.MoeError):
            mx.moe_kv_append_rope_fp8(*args, bad)


# ---- attention of chunks ------------------------------------------------------------------------------------------

def _check_chunk(mx, c, table, new, lens, hq, seed=0, scale=None, q=None, heads=None, rows=None):
    """All outputs against the oracle. heads, rows: those that are compared (all by default)."""
    H, P, D = c.codes["k"].shape[1:]
    G, total = hq // H, sum(new)
    q = _bf16(_gen(seed), total, hq, D) if q is None else q
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((total, hq), 7.0, device="cuda")
    ws = torch.full((mx.moe_attn_chunk_workspace_bytes(c.gpu, hq, total, len(new)),), 0xFF, dtype=torch.uint8, device="cuda")
    args = (c.gpu, q, _cu(new), _i32(lens), table)
    out = mx.moe_attn_chunk_fp8(*args, scale=scale, lse=lse, workspace=ws, dev_status=status)
    again = mx.moe_attn_chunk_fp8(*args, scale=scale)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    s = D ** -0.5 if scale is None else scale
    y, ls, tab, t0 = _np(out), _np(lse), table.cpu().numpy(), 0
    for b, (nq, nk) in enumerate(zip(new, lens)):
        which = [r for r in range(nq) if rows is None or r in rows or r - nq in rows]
        seen = np.array([nk - nq + r + 1 for r in which], dtype=np.int64)
        for h in range(H):
            with np.errstate(invalid="ignore"):
                k = oa.sequence(c.codes["k"], c.scales["k"], tab[b], h, nk)
                v = oa.sequence(c.codes["v"], c.scales["v"], tab[b], h, nk)
            step = np.repeat(2.0 ** (c.scales["v"][tab[b, :-(-nk // P)], h].astype(np.float64) - 127), P)[:nk] if nk else np.zeros(0)
            for i in range(h * G, (h + 1) * G):
                if heads is not None and i not in heads:
                    continue
                with np.errstate(invalid="ignore"):
                    ref = oa.attend(_np(q[t0:t0 + nq, i])[which], k, v, seen, s)
                got, gl = y[t0:t0 + nq, i][which], ls[t0:t0 + nq, i][which]
                none = np.isneginf(ref["lse"])
                assert np.array_equal(np.isneginf(gl), none) and np.all(got[none] == 0)
                tail = nk * 2.0 ** -32 * 448 * (ref["weights"] * step).max(-1, initial=0.0)
                bound = (2.0 ** -8 * np.abs(ref["out"]) + (2.0 ** -10 + 2.0 ** -15 * (1 + ref["size"][:, None])) * ref["mass"]
                         + tail[:, None] + 1e-38)
                err = np.abs(got - ref["out"])
                assert np.all(err <= bound), (b, i, float(np.max(err / bound)), np.argwhere(err > bound)[:4].tolist())
                ok = ~none
                assert np.all(np.abs(gl[ok] - ref["lse"][ok]) <= 2.0 ** -16 * (1 + ref["size"][ok]))
        t0 += nq
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 385])
def test_chunk_of_a_whole_sequence(mx, n, d):
    c, table = _filled(mx, [n], 32, 1, d, -(-n // 32), n)
    _check_chunk(mx, c, table, [n], [n], 2, seed=n)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (8, 2), (20, 4), (16, 1), (40, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_head_layouts(mx, hq, hkv, d):
    lens = [190, 33]
    c, table = _filled(mx, lens, 64, hkv, d, 3, hq)
    _check_chunk(mx, c, table, [70, 3], lens, hq, seed=hq)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_pages_and_lengths(mx, P, d):
    """Empty chunks and caches, one token, chunks behind long and short prefixes, ends on both sides of tiles."""
    new = [0, 1, 128, 0, 37, 5, 1, 130, 2]
    lens = [0, 1, 128, 40, 700, 133, 513, 257, 1000]
    c, table = _filled(mx, lens, P, 2, d, -(-1000 // P), P)
    _check_chunk(mx, c, table, new, lens, 4, seed=P)


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_rows_that_see_nothing(mx, d):
    """More new tokens than positions: the first ones see none; and an empty cache."""
    c, table = _filled(mx, [100, 0, 130], 16, 2, d, 9, 4)
    out, lse = _check_chunk(mx, c, table, [300, 7, 130], [100, 0, 130], 4, seed=4)
    assert torch.all(out[:200] == 0) and torch.all(torch.isneginf(lse[:200])) and torch.all(out[300:307] == 0)
    # a table without columns
    empty = torch.empty((1, 0), dtype=torch.int32, device="cuda")
    q = _bf16(_gen(1), 5, 4, d)
    assert not mx.moe_attn_chunk_fp8(c.gpu, q, _cu([5]), _i32([0]), empty).any()
    assert mx.moe_attn_chunk_fp8(c.gpu, q[:0], _cu([0]), _i32([0]), table[:1]).shape == (0, 4, d)


@pytest.mark.parametrize("n,lens,hq,hkv,d,P", [([37], [20011], 4, 1, 128, 64), ([3, 1, 20], [9000, 17, 12345], 8, 2, 64, 16),
                                               ([1], [30000], 1, 1, 128, 128), ([600], [5000], 16, 2, 128, 32)])
def test_chunk_long_caches(mx, n, lens, hq, hkv, d, P):
    """Few rows over many positions: the positions are shared out and the parts joined."""
    c, table = _filled(mx, lens, P, hkv, d, -(-max(lens) // P), 5)
    _check_chunk(mx, c, table, n, lens, hq, seed=6, rows={0, 1, 13, -2, -1})


@pytest.mark.parametrize("d,P", [(64, 16), (128, 128)])
def test_chunk_items_without_a_second_tile_between_others(mx, d, P):
    """Sequences of more and of fewer rows than a query tile by turns, each long enough for a CTA's stretch to end in it."""
    new = [150, 3, 90, 20, 130, 1, 64, 100]
    lens = [4000, 6442, 3797, 5000, 3708, 4500, 2900, 7099]
    c, table = _filled(mx, lens, P, 1, d, -(-max(lens) // P), 3)
    _check_chunk(mx, c, table, new, lens, 4, seed=8, heads=[0, 3], rows={0, 1, 30, 33, 50, 63, -30, -2, -1})


def test_chunk_many_sequences(mx):
    new = [(i * 37) % 23 for i in range(200)]
    lens = [n + (i * 53) % 90 for i, n in enumerate(new)]
    c, table = _filled(mx, lens, 32, 2, 64, 4, 7)
    _check_chunk(mx, c, table, new, lens, 4, seed=7, heads=[0, 3])


def test_chunk_strided_queries(mx):
    g = _gen(11)
    c, table = _filled(mx, [150, 90], 32, 2, 64, 5, 8)
    qkv = _bf16(g, 150, 8, 64)
    _check_chunk(mx, c, table, [100, 50], [150, 90], 4, q=qkv[:, 2:6])
    _check_chunk(mx, c, table, [100, 50], [150, 90], 4, q=_bf16(g, 4, 150, 64).transpose(0, 1))
    _check_chunk(mx, c, table, [100, 50], [150, 90], 4, q=_bf16(g, 150, 1, 64).expand(150, 4, 64))
    _check_chunk(mx, c, table, [100, 50], [150, 90], 4, q=_bf16(g, 1, 4, 64).expand(150, 4, 64))


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("spread", [15, 60, 120])
def test_chunk_scales_that_differ(mx, what, spread):
    """Pages whose scales lie 2^spread apart, in keys (with queries as small) and in values, zeros among them."""
    c, table = _filled(mx, [300, 300], 16, 2, 64, 19, 9)
    rng = np.random.default_rng(1)
    s = c.scales[what]
    if what == "v":
        s[:] = 127 + rng.integers(-spread, spread // 4 + 1, size=s.shape)
        zero = rng.random(s.shape) < 0.2
        c.codes["v"][zero] = 0
        s[zero] = 0
    else:
        s[:] = np.clip(127 - 8 + rng.integers(-spread, 1, size=s.shape), 1, 254)
    getattr(c.gpu, what + "_scales").copy_(torch.tensor(s))
    c.gpu.v_codes.copy_(torch.tensor(c.codes["v"]))
    _check_chunk(mx, c, table, [60, 300], [300, 300], 4, seed=spread)


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_scores_of_any_size(mx, d):
    """Scores that grow along the row, huge ones, all alike, scales of 0 and below."""
    n = 400
    c, table = _filled(mx, [n], 16, 1, d, 25, 3)
    tab = table[0].cpu().numpy()
    c.scales["k"][tab, 0] = 127 - 8 + np.arange(25) // 3
    c.gpu.k_scales.copy_(torch.tensor(c.scales["k"]))
    _check_chunk(mx, c, table, [150], [n], 2, seed=21)
    _check_chunk(mx, c, table, [150], [n], 2, seed=22, scale=0.0)
    _check_chunk(mx, c, table, [150], [n], 2, seed=23, scale=-1.0)
    q = _bf16(_gen(24), 150, 2, d)
    q[::3] *= 0
    q[1::3] *= 2.0 ** -100
    _check_chunk(mx, c, table, [150], [n], 2, q=q)
    # every key alike
    c.codes["k"][:] = 0x38
    c.gpu.k_codes.fill_(0x38)
    _check_chunk(mx, c, table, [150], [n], 2, seed=25)


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 2.0 ** 100])
def test_chunk_scores_beyond_fp32_exponentials(mx, size):
    """Queries so large that only the largest score counts: the output is that position's value."""
    n, d = 300, 64
    c, table = _filled(mx, [n], 16, 1, d, 19, 3)
    q = (_bf16(_gen(26), 40, 2, d).float() * size).to(torch.bfloat16)
    out = _np(mx.moe_attn_chunk_fp8(c.gpu, q, _cu([40]), _i32([n]), table))
    tab = table[0].cpu().numpy()
    k, v = (oa.sequence(c.codes[x], c.scales[x], tab, 0, n) for x in "kv")
    for r in range(40):
        for h in range(2):
            s = k[:n - 40 + r + 1] @ _np(q[r, h])
            top = int(np.argmax(s))
            # the runner-up is behind by more than the error of an fp32 sum of 64 products and by exp(30)
            gap = np.sort(s)[-1] - np.sort(s)[-2]
            assert gap * d ** -0.5 > 30 or size < 2.0 ** 40
            if gap * d ** -0.5 > 30 and gap > 2.0 ** -17 * (np.abs(k) @ np.abs(_np(q[r, h]))).max():
                assert np.all(np.abs(out[r, h] - v[top]) <= 2.0 ** -8 * np.abs(v[top]) + 1e-11 * np.abs(v).max())


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("at,new,n", [(129, 100, 200), (60, 100, 100), (255, 256, 256), (320, 600, 700), (10, 30, 400)])
def test_chunk_masked_places_hold_anything(mx, where, at, new, n):
    """A NaN code changes only what the queries that see it get; a scale byte of a masked page nothing."""
    d = 128
    c, table = _filled(mx, [n], 16, 1, d, -(-n // 16), at)
    q = _bf16(_gen(at), new, 2, d)
    args = (q, _cu([new]), _i32([n]), table)
    clean = mx.moe_attn_chunk_fp8(c.gpu, *args)
    page = int(table[0, at // 16])
    (c.gpu.k_codes if where == "k" else c.gpu.v_codes)[page, 0, at % 16, 5] = 0x7F
    out = mx.moe_attn_chunk_fp8(c.gpu, *args)
    sees = torch.arange(new, device="cuda") + n - new >= at
    assert torch.equal(out[~sees].view(torch.int16), clean[~sees].view(torch.int16))
    if where == "v":
        assert torch.isnan(out[sees][:, :, 5]).all()
        rest = [x for x in range(d) if x != 5]
        assert torch.isfinite(out[sees][:, :, rest]).all()
    else:
        assert torch.isnan(out[sees]).all()


def test_chunk_masked_pages_with_huge_scales(mx):
    """The page of the last tokens has scales far above the others': the rows before them do not notice."""
    n, new, d = 96, 40, 64
    c, table = _filled(mx, [n], 16, 1, d, 6, 3)
    q = _bf16(_gen(5), new, 2, d)
    args = (q, _cu([new]), _i32([n]), table)
    clean = mx.moe_attn_chunk_fp8(c.gpu, *args)
    last = int(table[0, 5])
    c.gpu.k_scales[last], c.gpu.v_scales[last] = 230, 230
    out = mx.moe_attn_chunk_fp8(c.gpu, *args)
    assert torch.equal(out[:new - 16].view(torch.int16), clean[:new - 16].view(torch.int16))


def test_chunk_pages_outside_the_cache_are_masked(mx):
    n, new, d = 300, 50, 64
    c, table = _filled(mx, [n], 32, 2, d, 10, 6)
    bad = table.clone()
    bad[0, 3], bad[0, 8] = -1, 99
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = _bf16(_gen(6), new, 4, d)
    lse = torch.empty((new, 4), device="cuda")
    out = mx.moe_attn_chunk_fp8(c.gpu, q, _cu([new]), _i32([n]), bad, lse=lse, dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB
    tab = table[0].cpu().numpy()
    gone = np.zeros(n, dtype=bool)
    gone[96:128], gone[256:288] = True, True
    for i in range(4):
        k, v = (oa.sequence(c.codes[x], c.scales[x], tab, i // 2, n) for x in "kv")
        for r in range(new):
            keep = ~gone[:n - new + r + 1]
            ref = oa.attend(_np(q[r, i])[None], k[:n - new + r + 1][keep], v[:n - new + r + 1][keep], [keep.sum()], d ** -0.5)
            err = np.abs(_np(out[r, i]) - ref["out"][0])
            assert np.all(err <= 2.0 ** -8 * np.abs(ref["out"][0]) + (2.0 ** -10 + 2.0 ** -15 * (1 + ref["size"])) * ref["mass"][0]
                          + n * 2.0 ** -32 * 448)
    out = mx.moe_attn_chunk_fp8(c.gpu, q, _cu([new]), _i32([n]), torch.full_like(table, -1), lse=lse)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("cu,lens", [([0, 200], [60]), ([-3, 20], [60]), ([0, 30, 20], [60, 60]), ([0, 50], [-1]), ([0, 50], [1000])])
def test_chunk_reports_bad_offsets(mx, cu, lens):
    c, table = _filled(mx, [64] * len(lens), 16, 1, 64, 4, 2)
    q = _bf16(_gen(42), 50, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.moe_attn_chunk_fp8(c.gpu, q, _i32(cu), _i32(lens), table, dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB


def test_chunk_rows_outside_sequences_stay(mx):
    c, table = _filled(mx, [64, 40], 16, 1, 64, 4, 2)
    q = _bf16(_gen(41), 50, 2, 64)
    out = torch.full((50, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((50, 2), 3.0, device="cuda")
    mx.moe_attn_chunk_fp8(c.gpu, q, _i32([0, 10, 30]), _i32([64, 40]), table, out=out, lse=lse)
    assert torch.all(out[30:] == 3.0) and torch.all(lse[30:] == 3.0) and not torch.any(out[:30] == 3.0)


def test_chunk_agrees_with_decode_and_prompt(mx):
    """One token: as moe_attn_decode_fp8; and two chunks as one, to the tolerance of both."""
    c, table = _filled(mx, [700, 90], 16, 2, 64, 44, 3)
    q = _bf16(_gen(95), 2, 8, 64)
    a = mx.moe_attn_chunk_fp8(c.gpu, q, _cu([1, 1]), _i32([700, 90]), table)
    b = mx.moe_attn_decode_fp8(c.gpu, q[:, None], _i32([700, 90]), table)[:, 0]
    top = 448 * 2.0 ** (int(c.scales["v"].max()) - 127)
    assert (a.float() - b.float()).abs().max() <= top * 2.0 ** -7
    q = _bf16(_gen(96), 300, 8, 64)
    whole = mx.moe_attn_chunk_fp8(c.gpu, q, _cu([300, 0]), _i32([700, 90]), table)
    first = mx.moe_attn_chunk_fp8(c.gpu, q[:130], _cu([130, 0]), _i32([530, 90]), table)
    rest = mx.moe_attn_chunk_fp8(c.gpu, q[130:], _cu([170, 0]), _i32([700, 90]), table)
    assert (whole.float() - torch.cat([first, rest]).float()).abs().max() <= top * 2.0 ** -7


def test_chunk_streams_and_graphs(mx):
    """Two calls at once on their own streams and workspaces; a captured one replayed with other lengths."""
    lens = [2000, 500]
    c, table = _filled(mx, lens, 64, 2, 128, 32, 3)
    q, cu, ln = _bf16(_gen(43), 90, 8, 128), _cu([60, 30]), _i32(lens)
    want = mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table, stream=s) for s in (s1, s2, s1, s2)]
    s1.synchronize()
    s2.synchronize()
    assert all(torch.equal(x, want) for x in got)
    ws = torch.empty(mx.moe_attn_chunk_workspace_bytes(c.gpu, 8, 90, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table, out=out, workspace=ws)
    for lens2 in ([2000, 500], [61, 31], [1999, 30]):
        ln.copy_(_i32(lens2))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table))


def test_chunk_binding_refusals(mx):
    c, table = _filled(mx, [64], 16, 2, 64, 4, 2)
    q = _bf16(_gen(44), 10, 4, 64)
    cu, ln = _cu([10]), _i32([64])
    with pytest.raises(TypeError):
        mx.moe_attn_chunk_fp8(c.gpu, q.float(), cu, ln, table)
    with pytest.raises(TypeError):
        mx.moe_attn_chunk_fp8(c.gpu, q, cu.long(), ln, table)
    for bad in (dict(q=q[0]), dict(cu_q=_i32([0])), dict(out=q[:, :2]), dict(page_table=table[0]), dict(lse=torch.empty(3, device="cuda")),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            mx.moe_attn_chunk_fp8(**{"cache": c.gpu, "q": q, "cu_q": cu, "lengths": ln, "page_table": table, **bad})
    for bad in (dict(q=q[:, :3]), dict(scale=math.inf), dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
                dict(q=_bf16(_gen(1), 10, 4, 65)[:, :, 1:])):
        with pytest.raises(mx.MoeError):
            mx.moe_attn_chunk_fp8(**{"cache": c.gpu, "q": q, "cu_q": cu, "lengths": ln, "page_table": table, **bad})
