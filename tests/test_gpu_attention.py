"""Prompt attention, the 8-bit key/value cache, attention over it and eviction,
on the GPU against oracle.attention (fp64).

Tolerances. Outputs are bf16 (8 significant bits): half a unit in the last
place is at most 2^-8 |y|. The probabilities enter the second product as bf16
(prompt; relative error at most 2^-8 each) or f16 (cache; 2^-11, plus f16's
subnormal step where they are small): an error of at most that times sum p |v|,
to which fp32 scores add their own: a sum of D products errs by at most D 2^-24
sum |q k| scale =: 2^-17 size for D <= 128, and changes p by that factor twice
(numerator and denominator). So
  |y - ref| <= 2^-8 |ref| + (e_p + 2^-15 (1 + size)) sum p |v|,
e_p = 2^-8 for the prompt and 2^-10 for the cache; |lse - ref| <= 2^-16 (1 +
size); accumulated weights within a factor 2^-15 (1 + size) of the sum. Codes,
scales and positions are compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _bf16(g, *shape, spread=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(torch.bfloat16)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _near(y, lse, ref, e_p, rows=slice(None)):
    y, lse = _np(y)[rows], _np(lse)[rows]
    bound = 2.0 ** -8 * np.abs(ref["out"]) + (e_p + 2.0 ** -15 * (1 + ref["size"][:, None])) * ref["mass"] + 1e-30
    err = np.abs(y - ref["out"])
    assert np.all(err <= bound), (float(np.max(err / bound)), np.argwhere(err > bound)[:4].tolist())
    none = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), none)
    assert np.all(np.abs(lse[~none] - ref["lse"][~none]) <= 2.0 ** -16 * (1 + ref["size"][~none]))
    assert np.all(y[none] == 0)


# ---- prompts ----------------------------------------------------------------------------------------------------

def _check_prompt(mx, lq, lk, hq, hkv, d, causal, seed=0, scale=None, q=None, k=None, v=None, heads=None):
    g = _gen(seed)
    tq, tk = sum(lq), sum(lk)
    q = _bf16(g, tq, hq, d) if q is None else q
    k = _bf16(g, tk, hkv, d) if k is None else k
    v = _bf16(g, tk, hkv, d) if v is None else v
    lse = torch.full((tq, hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mx.moe_attn_prefill(q, k, v, _cu(lq), _cu(lk), causal=causal, scale=scale, lse=lse, dev_status=status)
    again = mx.moe_attn_prefill(q, k, v, _cu(lq), _cu(lk), causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    s = d ** -0.5 if scale is None else scale
    for h in (range(hq) if heads is None else heads):
        q0 = k0 = 0
        for nq, nk in zip(lq, lk):
            seen = np.arange(nq) + nk - nq + 1 if causal else np.full(nq, nk)
            kk, vv = _np(k[k0:k0 + nk, h // (hq // hkv)]), _np(v[k0:k0 + nk, h // (hq // hkv)])
            with np.errstate(invalid="ignore"):
                ref = oa.attend(_np(q[q0:q0 + nq, h]), kk, vv, seen, s)
            _near(out[:, h], lse[:, h], ref, 2.0 ** -8, slice(q0, q0 + nq))
            q0, k0 = q0 + nq, k0 + nk
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 385])
def test_prompt_one_sequence(mx, n, d):
    _check_prompt(mx, [n], [n], 2, 1, d, True, seed=n)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (8, 2), (20, 4), (16, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_head_layouts(mx, hq, hkv, d):
    _check_prompt(mx, [130, 3], [130, 3], hq, hkv, d, True, seed=hq)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_packed_sequences(mx, causal, d):
    """Empty sequences, one token, lengths on both sides of the tiles."""
    lens = [0, 1, 128, 0, 129, 31, 257, 2, 127, 0]
    _check_prompt(mx, lens, lens, 4, 2, d, causal, seed=9)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([5], [300]), ([128], [129]), ([130, 1, 64], [700, 256, 64]), ([1, 1, 1], [1, 128, 129])])
def test_prompt_with_earlier_keys(mx, lq, lk, causal):
    _check_prompt(mx, lq, lk, 4, 2, 128, causal, seed=3)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rows_that_see_nothing(mx, d):
    """More queries than keys: the first ones see none; and a sequence without keys."""
    out, lse = _check_prompt(mx, [300, 7, 130], [100, 0, 130], 4, 2, d, True, seed=4)
    assert torch.all(out[:200] == 0) and torch.all(torch.isneginf(lse[:200]))
    assert torch.all(out[300:307] == 0)
    _check_prompt(mx, [20, 7], [0, 5], 4, 2, d, False, seed=5)


def test_prompt_without_any_key(mx):
    out = mx.moe_attn_prefill(torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda"),
                              torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"),
                              torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"), _cu([3]), _cu([0]))
    assert torch.all(out == 0)
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert mx.moe_attn_prefill(empty, empty, empty, _cu([0])).shape == (0, 2, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_strided_views(mx, d):
    """Slices of one projection, and heads before tokens in memory."""
    g = _gen(11)
    qkv = _bf16(g, 150, 4 + 2 + 2, d)
    _check_prompt(mx, [100, 50], [100, 50], 4, 2, d, True, q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:])
    hm = [_bf16(g, h, 150, d).transpose(0, 1) for h in (4, 2, 2)]
    _check_prompt(mx, [100, 50], [100, 50], 4, 2, d, True, q=hm[0], k=hm[1], v=hm[2])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("at,lens", [(129, [200]), (60, [100]), (255, [256]), (100, [64, 90, 64]), (320, [700])])
def test_prompt_masked_places_hold_anything(mx, bad, where, at, lens):
    """A non-finite key or value changes only what the queries that see it get."""
    g = _gen(at)
    n = sum(lens)
    q, k, v = _bf16(g, n, 2, 128), _bf16(g, n, 1, 128), _bf16(g, n, 1, 128)
    clean = mx.moe_attn_prefill(q, k, v, _cu(lens))
    (k if where == "k" else v)[at, 0, 5] = bad
    lse = torch.empty((n, 2), device="cuda")
    out = mx.moe_attn_prefill(q, k, v, _cu(lens), lse=lse)
    torch.cuda.synchronize()
    ends = np.cumsum(lens)
    end = int(ends[np.searchsorted(ends, at, side="right")])
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    sees[at:end] = True
    assert torch.equal(out[~sees].view(torch.int16), clean[~sees].view(torch.int16))
    if where == "v":
        # p * inf is inf where p > 0, NaN is NaN; the other channels stand
        assert not torch.isfinite(out[sees][:, :, 5]).any()
        rest = [c for c in range(128) if c != 5]
        near = (out[sees][:, :, rest].float() - clean[sees][:, :, rest].float()).abs()
        assert torch.all(near <= 2.0 ** -6 * clean[sees][:, :, rest].float().abs() + 2.0 ** -7)
        if math.isinf(bad):
            assert torch.all(out[sees][:, :, 5] == bad)


def test_prompt_many_bad_values_of_both_signs(mx):
    """Infinities of both signs and NaN in one masked tile of values."""
    n, d = 128, 64
    g = _gen(5)
    q, k, v = _bf16(g, n, 2, d), _bf16(g, n, 1, d), _bf16(g, n, 1, d)
    v[40, 0, 3], v[50, 0, 3], v[60, 0, 4], v[127, 0, 63] = math.inf, -math.inf, math.nan, -math.inf
    _check = mx.moe_attn_prefill(q, k, v, _cu([n]))
    y = _check.float()
    assert torch.isfinite(y[:40]).all()
    assert torch.all(y[40:50, :, 3] == math.inf) and torch.all(torch.isnan(y[50:, :, 3]))
    assert torch.all(torch.isnan(y[60:, :, 4])) and torch.isfinite(y[:60, :, 4]).all()
    assert torch.all(y[127, :, 63] == -math.inf) and torch.isfinite(y[:, :, 5:63]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_scores_of_any_size(mx, d):
    """Scores that grow along the row (the maximum is raised again and again), huge and all alike."""
    g = _gen(21)
    n = 400
    q = _bf16(g, n, 2, d)
    k = (_bf16(g, n, 1, d).float() * torch.linspace(0.1, 8, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    _check_prompt(mx, [n], [n], 2, 1, d, True, q=q, k=k, seed=21)
    q1 = torch.ones((n, 2, d), dtype=torch.bfloat16, device="cuda")
    ramp = torch.linspace(-3, 3, n, device="cuda")[:, None, None].expand(n, 1, d).to(torch.bfloat16).contiguous()
    _check_prompt(mx, [n], [n], 2, 1, d, True, q=q1, k=ramp, seed=22)
    _check_prompt(mx, [n], [n], 2, 1, d, True, q=q1, k=-ramp, seed=23)
    _check_prompt(mx, [n], [n], 2, 1, d, False, q=q1, k=torch.zeros_like(ramp), seed=24)
    _check_prompt(mx, [n], [n], 2, 1, d, True, seed=25, scale=0.0)
    _check_prompt(mx, [n], [n], 2, 1, d, True, seed=26, scale=-1.0)


def test_prompt_longer(mx):
    """Several tiles of keys per query tile, and many sequences at once."""
    _check_prompt(mx, [1100], [1100], 8, 2, 128, True, seed=31, heads=[0, 3, 7])
    _check_prompt(mx, [700], [2300], 4, 4, 64, True, seed=32, heads=[1])
    lens = [(i * 37) % 71 for i in range(300)]
    _check_prompt(mx, lens, lens, 2, 1, 64, True, seed=33, heads=[0])


def test_prompt_rows_outside_sequences_stay(mx):
    g = _gen(41)
    q, k = _bf16(g, 50, 2, 64), _bf16(g, 50, 1, 64)
    out = torch.full((50, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((50, 2), 3.0, device="cuda")
    mx.moe_attn_prefill(q, k, k, _i32([0, 10, 30]), out=out, lse=lse)
    assert torch.all(out[30:] == 3.0) and torch.all(lse[30:] == 3.0) and not torch.any(out[:30] == 3.0)


@pytest.mark.parametrize("cu", [[0, 200], [-3, 20], [0, 30, 20], [0, 60, 70]])
def test_prompt_reports_bad_offsets(mx, cu):
    g = _gen(42)
    q, k = _bf16(g, 50, 2, 64), _bf16(g, 50, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.moe_attn_prefill(q, k, k, _i32(cu), dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB


def test_prompt_on_another_stream(mx):
    g = _gen(43)
    q, k, v = _bf16(g, 300, 4, 128), _bf16(g, 300, 2, 128), _bf16(g, 300, 2, 128)
    want = mx.moe_attn_prefill(q, k, v, _cu([300]))
    s = torch.cuda.Stream()
    cu = _cu([300])
    torch.cuda.synchronize()
    got = torch.empty_like(want)
    mx.moe_attn_prefill(q, k, v, cu, out=got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_prompt_refusals(mx):
    g = _gen(44)
    q, k = _bf16(g, 10, 4, 64), _bf16(g, 10, 2, 64)
    cu = _cu([10])
    with pytest.raises(TypeError):
        mx.moe_attn_prefill(q.float(), k, k, cu)
    with pytest.raises(TypeError):
        mx.moe_attn_prefill(q, k, k, cu.long())
    with pytest.raises(ValueError):
        mx.moe_attn_prefill(q, k, k[:9], cu)
    with pytest.raises(ValueError):
        mx.moe_attn_prefill(q, k, k, cu, cu[:1])
    with pytest.raises(ValueError):
        mx.moe_attn_prefill(q, k, k, cu, out=q[:, :2])
    with pytest.raises(ValueError):
        mx.moe_attn_prefill(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_prefill(q[:, :3], k, k, cu)                 # 3 heads over 2
    with pytest.raises(mx.MoeError):
        mx.moe_attn_prefill(_bf16(g, 10, 4, 96), _bf16(g, 10, 2, 96), _bf16(g, 10, 2, 96), cu)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_prefill(q, k, k, cu, scale=math.nan)
    wide = _bf16(g, 10, 4, 65)[:, :, 1:]                         # rows not 16-byte aligned
    with pytest.raises(mx.MoeError):
        mx.moe_attn_prefill(wide, k, k, cu)


# ---- the cache --------------------------------------------------------------------------------------------------

class _Cache:
    """A cache on the GPU beside the oracle's copy of it."""

    def __init__(self, mx, n_pages, P, H, D):
        self.gpu = mx.KVCache.alloc(n_pages, P, H, D)
        for t in (self.gpu.k_codes, self.gpu.v_codes, self.gpu.k_scales, self.gpu.v_scales):
            t.fill_(0xFF)   # what is not written may hold anything: NaN codes here
        self.codes = {n: np.full((n_pages, H, P, D), 0xFF, np.uint8) for n in "kv"}
        self.scales = {n: np.full((n_pages, H), 0xFF, np.uint8) for n in "kv"}

    def append(self, mx, k, v, lens, start, table, want_status=0):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mx.moe_kv_append_fp8(self.gpu, k, v, _cu(lens), _i32(start), table, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == want_status
        tab, t0 = table.cpu().numpy(), 0
        for b, n in enumerate(lens):
            for name, x in (("k", k), ("v", v)):
                oa.append(self.codes[name], self.scales[name], _np(x[t0:t0 + n]), start[b], tab[b])
            t0 += n

    def check(self):
        assert np.array_equal(self.gpu.k_scales.cpu().numpy(), self.scales["k"])
        assert np.array_equal(self.gpu.v_scales.cpu().numpy(), self.scales["v"])
        assert np.array_equal(self.gpu.k_codes.cpu().numpy(), self.codes["k"])
        assert np.array_equal(self.gpu.v_codes.cpu().numpy(), self.codes["v"])


def _tables(n_seq, width, seed=0):
    """Disjoint page tables in shuffled order."""
    p = torch.randperm(n_seq * width, generator=torch.Generator().manual_seed(seed))
    return p.view(n_seq, width).to(torch.int32).cuda()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_prompts_and_tokens(mx, P, d):
    """Prompts, then single tokens, then more tokens behind them; spreads that make scales grow."""
    g = _gen(P + d)
    H = 3
    c = _Cache(mx, 4 * 7, P, H, d)
    table = _tables(4, 7)
    at = [0, 0, 0, 0]
    for step, (lens, spread) in enumerate([([P + 1, 0, 2 * P, 5], 0.01), ([1, 1, 1, 1], 0.5), ([1, 3, P, 2 * P + 3], 40.0),
                                           ([1, 1, 1, 1], 1e-3), ([0, 0, 0, 1], 1e4), ([2, P - 1, 1, 0], 1e-9)]):
        n = sum(lens)
        k, v = _bf16(g, n, H, d, spread=spread), _bf16(g, n, H, d, spread=3 * spread)
        c.append(mx, k, v, lens, at, table)
        c.check()
        at = [a + n for a, n in zip(at, lens)]


def test_append_special_values(mx):
    """Zeros, the largest and the smallest bf16, ties, inf and NaN."""
    c = _Cache(mx, 8, 16, 2, 64)
    table = _tables(2, 4)
    x = torch.zeros((20, 2, 64), dtype=torch.bfloat16, device="cuda")
    c.append(mx, x, x, [20, 0], [0, 0], table)
    c.check()
    y = torch.zeros((33, 2, 64), dtype=torch.bfloat16, device="cuda")
    y[0, 0, 0] = 3.38e38
    y[1, 1, 1] = 9.2e-41
    y[17, 0] = torch.arange(64, device="cuda").to(torch.bfloat16) * 4 + 200
    y[18, 0, 7] = -448.0
    y[17:19, 1, :3] = torch.tensor([[1.0625, -1.1875, 0.001], [17.0, 449.0, -1e-6]], device="cuda").to(torch.bfloat16)
    c.append(mx, y, -y, [0, 33], [0, 0], table)
    c.check()
    z = _bf16(_gen(0), 3, 2, 64)
    z[0, 0, 3], z[1, 1, 4], z[2, 0, 5] = math.inf, -math.inf, math.nan
    c.append(mx, z, z, [3, 0], [20, 0], table, want_status=mx.DEV_NONFINITE_INPUT)
    c.check()


def test_append_strided_and_many_sequences(mx):
    g = _gen(3)
    n_seq = 100
    c = _Cache(mx, n_seq * 3, 32, 2, 128)
    table = _tables(n_seq, 3)
    lens = [(i * 13) % 4 for i in range(n_seq)]
    start = [(i * 29) % 60 for i in range(n_seq)]
    kv = _bf16(g, sum(start), 4, 128)
    c.append(mx, kv[:, :2], kv[:, 2:], start, [0] * n_seq, table)
    kv = _bf16(g, sum(lens), 4, 128, spread=5.0)
    c.append(mx, kv[:, 1:3], kv[:, 2:], lens, start, table)
    c.check()


def test_append_reports_what_it_cannot_place(mx):
    c = _Cache(mx, 4, 16, 1, 64)
    x = _bf16(_gen(1), 40, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.moe_kv_append_fp8(c.gpu, x, x, _cu([40]), _i32([0]), _i32([[0, 1]]), dev_status=status)   # 2 pages hold 32
    assert int(status) == mx.DEV_INDEX_OOB
    oa.append(c.codes["k"], c.scales["k"], _np(x[:32]), 0, [0, 1])
    oa.append(c.codes["v"], c.scales["v"], _np(x[:32]), 0, [0, 1])
    c.check()
    for bad, start, cu in (([[4, 1]], 0, [0, 4]), ([[-1, 1]], 0, [0, 4]), ([[0, 1]], -1, [0, 4]), ([[0, 1]], 0, [0, 41]),
                           ([[0, 1]], 0, [3, 1]), ([[0, 1]], 2 ** 31 - 2, [0, 4])):
        status.zero_()
        before = [t.clone() for t in (c.gpu.k_codes, c.gpu.v_codes)]
        mx.moe_kv_append_fp8(c.gpu, x, x, _i32(cu), _i32([start]), _i32(bad), dev_status=status)
        assert int(status) == mx.DEV_INDEX_OOB, (bad, start, cu)
        if cu != [0, 41]:
            assert torch.equal(before[0], c.gpu.k_codes) and torch.equal(before[1], c.gpu.v_codes)


# ---- attention over the cache -------------------------------------------------------------------------------------

def _filled(mx, lens, P, H, D, width, seed, spread=None, n_pages=None):
    """A cache of random codes with scales that differ from page to page."""
    rng = np.random.default_rng(seed)
    table = _tables(len(lens), width, seed)
    n_pages = len(lens) * width
    c = _Cache(mx, n_pages, P, H, D)
    for name in "kv":
        x = rng.normal(size=(n_pages, H, P, D))
        byte = 127 - 8 + rng.integers(-2, 3, size=(n_pages, H)) if spread is None else spread(rng, (n_pages, H))
        c.codes[name] = np.stack([oa.encode(x[i] * 2.0 ** 7, 127) for i in range(n_pages)])
        c.scales[name] = byte.astype(np.uint8)
        for b, n in enumerate(lens):      # past the end: NaN codes
            tab = table[b].cpu().numpy()
            for p in range(width):
                m = min(max(n - p * P, 0), P)
                c.codes[name][tab[p], :, m:] = 0x7F
    c.gpu.k_codes.copy_(torch.tensor(c.codes["k"]))
    c.gpu.v_codes.copy_(torch.tensor(c.codes["v"]))
    c.gpu.k_scales.copy_(torch.tensor(c.scales["k"]))
    c.gpu.v_scales.copy_(torch.tensor(c.scales["v"]))
    return c, table


def _ref_decode(c, table, q, lens, scale):
    """Oracle's answers: {(b, h): dict over the rows (token, head of the group)}."""
    B, T, Hq, D = q.shape
    H = c.codes["k"].shape[1]
    G = Hq // H
    res = {}
    for b, n in enumerate(lens):
        tab = table[b].cpu().numpy()
        for h in range(H):
            with np.errstate(invalid="ignore"):
                k = oa.sequence(c.codes["k"], c.scales["k"], tab, h, n)
                v = oa.sequence(c.codes["v"], c.scales["v"], tab, h, n)
            rows = _np(q[b, :, h * G:(h + 1) * G]).reshape(T * G, D)
            seen = np.repeat(np.arange(T) + n - T + 1, G)
            with np.errstate(invalid="ignore"):
                res[b, h] = oa.attend(rows, k, v, seen, scale)
    return res


def _check_decode(mx, lens, T, hq, H, D, P, width=None, seed=0, weights=False, q=None, scale=None, made=None,
                  spread=None, workspace=None):
    width = max(-(-max(lens) // P), 1) if width is None else width
    c, table = _filled(mx, lens, P, H, D, width, seed, spread) if made is None else made
    q = _bf16(_gen(seed + 1), len(lens), T, hq, D) if q is None else q
    lse = torch.full((len(lens), T, hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = w0 = None
    if weights:
        w0 = torch.rand((len(lens), H, width * P), generator=_gen(seed + 2), device="cuda")
        w = w0.clone()
    out = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table, scale=scale, lse=lse, weights=w, workspace=workspace,
                                 dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ref = _ref_decode(c, table, q, lens, D ** -0.5 if scale is None else scale)
    G = hq // H
    for (b, h), r in ref.items():
        _near(out[b, :, h * G:(h + 1) * G].reshape(T * G, D), lse[b, :, h * G:(h + 1) * G].reshape(T * G), r, 2.0 ** -10)
        if weights:
            n = lens[b]
            add = r["weights"].sum(0)
            err = np.abs(_np(w[b, h]) - _np(w0[b, h]) - np.pad(add, (0, width * P - n)))
            top = r["size"].max() if len(r["size"]) else 0.0
            assert np.all(err[:n] <= 2.0 ** -15 * (1 + top) * add + 2.0 ** -23), float(err[:n].max())
            assert np.all(err[n:] == 0)
    return c, table, q, out


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_lengths(mx, n, d):
    _check_decode(mx, [n], 1, 8, 1, d, 64, seed=n, weights=True)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_ragged_batch(mx, P, d):
    _check_decode(mx, [0, 1, 300, 17, 64, 0, 515, 128, 129], 1, 10, 2, d, P, seed=P, weights=True)


@pytest.mark.parametrize("T,hq,H", [(1, 1, 1), (1, 3, 3), (1, 5, 1), (1, 16, 2), (1, 9, 1), (1, 64, 4), (1, 24, 1), (1, 64, 1),
                                    (2, 8, 2), (3, 15, 3), (4, 20, 4), (4, 32, 4), (8, 8, 1), (8, 16, 4), (5, 3, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_rows(mx, T, hq, H, d, weights):
    _check_decode(mx, [200, 9, 77], T, hq, H, d, 32, seed=T + hq, weights=weights)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_more_tokens_than_positions(mx, d):
    """The first tokens of a sequence shorter than n_new see nothing."""
    *_, out = _check_decode(mx, [3, 0, 8, 1], 8, 4, 2, d, 16, seed=2, weights=True)
    assert torch.all(out[0, :5] == 0) and torch.all(out[1] == 0) and torch.all(out[3, :7] == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq", [(1, 4), (4, 8), (4, 32)])
def test_decode_nan_values_stay_with_those_who_see_them(mx, d, T, hq):
    """A NaN code among the newest positions reaches the tokens that see it, and no others."""
    lens, H, P = [45, 33], 2, 16
    made = _filled(mx, lens, P, H, d, 3, 7)
    c, table = made
    q = _bf16(_gen(8), 2, T, hq, d)
    clean = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table)
    G = hq // H
    for b, n in enumerate(lens):
        page, slot = int(table[b, (n - 1) // P]), (n - 1) % P
        for codes in (c.gpu.k_codes, c.gpu.v_codes):
            codes[page, 1, slot, 9] = 0xFF
        out = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table)
        assert torch.equal(out[b, :T - 1], clean[b, :T - 1])
        assert torch.equal(out[b, :, :G], clean[b, :, :G])
        assert torch.isnan(out[b, T - 1, G:]).all()        # a NaN key: the whole row
        c.gpu.k_codes[page, 1, slot, 9] = 0x11
        ref = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table)
        assert torch.isnan(ref[b, T - 1, G:, 9]).all()     # a NaN value: its channel
        rest = [i for i in range(d) if i != 9]
        assert torch.isfinite(ref[b, T - 1, G:][:, rest]).all()
        assert torch.equal(ref[b, :T - 1], clean[b, :T - 1])
        c.gpu.v_codes[page, 1, slot, 9] = 0x11


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scales_far_apart(mx, d):
    """Pages whose scales differ by up to 2^60, rising and falling: no page is rounded for another's sake."""
    wild = lambda rng, shape: 127 - 8 + rng.integers(-30, 31, size=shape)   # noqa: E731
    calm = lambda rng, shape: 127 - 30 + 0 * rng.integers(0, 2, size=shape)   # noqa: E731
    lens, P, H = [300, 129], 16, 1
    c, table = _filled(mx, lens, P, H, d, 19, 3, wild)
    c.scales["k"] = calm(np.random.default_rng(0), c.scales["k"].shape).astype(np.uint8)
    c.gpu.k_scales.copy_(torch.tensor(c.scales["k"]))
    _check_decode(mx, lens, 1, 4, H, d, P, 19, seed=3, made=(c, table))
    # the extreme bytes
    c.scales["v"][:] = 0
    c.scales["v"][::2] = 200
    c.gpu.v_scales.copy_(torch.tensor(c.scales["v"]))
    _check_decode(mx, lens, 1, 4, H, d, P, 19, seed=3, made=(c, table))


def test_decode_scores_of_any_size(mx):
    """Rising and falling scores, large ones, queries of very different magnitudes, no scale at all."""
    d, H, P, lens = 128, 2, 16, [400, 399]
    g = _gen(5)
    mag = torch.tensor([1e-30, 1e-3, 1.0, 30.0], device="cuda").repeat(2)[None, None, :, None]
    q = (_bf16(g, 2, 1, 8, d).float() * mag).to(torch.bfloat16)
    for spread in (lambda rng, s: 127 - 8 + 0 * rng.integers(0, 2, size=s), lambda rng, s: 127 - 5 + rng.integers(0, 3, size=s)):
        made = _filled(mx, lens, P, H, d, 25, 6, spread)
        _check_decode(mx, lens, 1, 8, H, d, P, 25, seed=6, q=q, made=made, weights=True)
        _check_decode(mx, lens, 1, 8, H, d, P, 25, seed=6, made=made, scale=0.0, weights=True)
        _check_decode(mx, lens, 1, 8, H, d, P, 25, seed=6, made=made, scale=-0.7)


def test_decode_long_and_workspace_reuse(mx):
    """Work split over many CTAs; one workspace for calls of different lengths; equal bits every time."""
    H, d, P = 2, 128, 64
    c, table = _filled(mx, [20000, 70, 9000], P, H, d, 313, 11)
    n = mx.moe_attn_decode_workspace_bytes(c.gpu, 3, 1, 16, 313, True)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for lens in ([20000, 70, 9000], [1, 70, 0], [12345, 64, 8999], [0, 0, 0], [20000, 70, 9000]):
        for name in "kv":
            pass
        q = _bf16(_gen(12), 3, 1, 16, d)
        w = torch.zeros((3, H, 313 * P), device="cuda")
        out = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table, weights=w, workspace=ws)
        w2 = torch.zeros_like(w)
        out2 = mx.moe_attn_decode_fp8(c.gpu, q, _i32(lens), table, weights=w2, workspace=ws)
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(w, w2)
        _check_decode(mx, lens, 1, 16, H, d, P, 313, seed=11, q=q, made=(c, table), workspace=ws)


def test_decode_strided_q_and_stream(mx):
    lens, H, d, P = [50, 70], 2, 128, 16
    made = _filled(mx, lens, P, H, d, 5, 13)
    qkv = _bf16(_gen(14), 2 * 3, 8 + 4, d)
    q = qkv.view(2, 3, 12, d)[:, :, :8]
    *_, out = _check_decode(mx, lens, 3, 8, H, d, P, 5, seed=13, q=q, made=made)
    s = torch.cuda.Stream()
    got = torch.empty_like(out)
    ln, ws = _i32(lens), torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    mx.moe_attn_decode_fp8(made[0].gpu, q, ln, made[1], out=got, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got, out)


def test_decode_reports_what_it_cannot_reach(mx):
    lens, H, d, P = [50], 1, 64, 16
    c, table = _filled(mx, lens, P, H, d, 4, 15)
    q = _bf16(_gen(16), 1, 1, 4, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = mx.moe_attn_decode_fp8(c.gpu, q, _i32([64]), table)
    got = mx.moe_attn_decode_fp8(c.gpu, q, _i32([65]), table, dev_status=status)     # 4 pages hold 64
    assert int(status) == mx.DEV_INDEX_OOB and torch.equal(got.view(torch.int16), want.view(torch.int16))
    status.zero_()
    got = mx.moe_attn_decode_fp8(c.gpu, q, _i32([-1]), table, dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB and torch.all(got == 0)
    status.zero_()
    w = torch.zeros((1, 1, 20), device="cuda")
    mx.moe_attn_decode_fp8(c.gpu, q, _i32([50]), table, weights=w, dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB
    status.zero_()
    bad = table.clone()
    bad[0, 1] = 4
    out = mx.moe_attn_decode_fp8(c.gpu, q, _i32([50]), bad, dev_status=status)
    assert int(status) == mx.DEV_INDEX_OOB and torch.isfinite(out).all()


def test_decode_refusals(mx):
    c, table = _filled(mx, [20], 16, 2, 64, 2, 17)
    g, ln = _gen(18), _i32([20])
    q = _bf16(g, 1, 1, 4, 64)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_decode_fp8(c.gpu, _bf16(g, 1, 1, 3, 64), ln, table)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_decode_fp8(c.gpu, _bf16(g, 1, 9, 4, 64), ln, table)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_decode_fp8(c.gpu, _bf16(g, 1, 1, 130, 64), ln, table)
    with pytest.raises(mx.MoeError):
        mx.moe_attn_decode_fp8(c.gpu, q, ln, table, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mx.moe_attn_decode_fp8(c.gpu, _bf16(g, 1, 1, 4, 128), ln, table)
    with pytest.raises(ValueError):
        mx.moe_attn_decode_fp8(c.gpu, q, _i32([20, 20]), table)
    with pytest.raises(ValueError):
        mx.moe_attn_decode_fp8(c.gpu, q, ln, table, weights=torch.zeros((1, 3, 32), device="cuda"))
    with pytest.raises(TypeError):
        mx.moe_attn_decode_fp8(c.gpu, q.float(), ln, table)


def test_decode_in_a_graph(mx):
    """Captured once, replayed on other data: nothing is kept from one call for the next."""
    lens, H, d, P = [700, 90], 2, 128, 64
    c, table = _filled(mx, lens, P, H, d, 11, 19)
    q, ln = _bf16(_gen(20), 2, 1, 16, d), _i32(lens)
    w, ws = torch.zeros((2, H, 704), device="cuda"), torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    run = lambda: mx.moe_attn_decode_fp8(c.gpu, q, ln, table, out=out, weights=w, workspace=ws)   # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.copy_(_bf16(_gen(21), 2, 1, 16, d))
    ln.copy_(_i32([333, 11]))
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want_w = torch.zeros_like(w)
    want = mx.moe_attn_decode_fp8(c.gpu, q, ln, table, weights=want_w)
    assert torch.equal(out, want) and torch.equal(w, want_w)


# ---- eviction -----------------------------------------------------------------------------------------------------

def _check_evict(mx, lens, keep, recent, H, D, P, seed, w, made=None):
    width = max(-(-max(lens) // P), 1)
    n_dst = -(-min(keep, width * P) // P)
    rng = np.random.default_rng(seed)
    table_all = _tables(len(lens), width + n_dst, seed)
    table, dst = table_all[:, :width].contiguous(), table_all[:, width:].contiguous()
    c = _Cache(mx, len(lens) * (width + n_dst), P, H, D)
    n_pages = c.codes["k"].shape[0]
    for name in "kv":
        x = rng.normal(size=(n_pages, H, P, D)) * np.exp(rng.normal(size=(n_pages, H, P, 1)) * 2)
        c.codes[name] = np.stack([oa.encode(np.clip(x[i] * 40, -448, 448), 127) for i in range(n_pages)])
        c.scales[name] = (127 - 8 + rng.integers(-4, 5, size=(n_pages, H))).astype(np.uint8)
    c.codes["v"][int(table[0, 0]), 0, 0, 3] = 0x7F
    for name, t in (("k", c.gpu.k_codes), ("v", c.gpu.v_codes)):
        t.copy_(torch.tensor(c.codes[name]))
    c.gpu.k_scales.copy_(torch.tensor(c.scales["k"]))
    c.gpu.v_scales.copy_(torch.tensor(c.scales["v"]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, kw, ln = mx.moe_kv_evict_fp8(c.gpu, table, _i32(lens), w, keep, recent, dst, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert ln.tolist() == [min(n, keep) for n in lens]
    kept, kwn, wn = kept.cpu().numpy(), kw.cpu().numpy(), w.cpu().numpy()
    for b, n in enumerate(lens):
        tab, to = table[b].cpu().numpy(), dst[b].cpu().numpy()
        for h in range(H):
            ids = oa.select(wn[b, h, :n], keep, recent)
            assert kept[b, h, :len(ids)].tolist() == ids
            assert np.all(kept[b, h, len(ids):] == -1)
            assert np.array_equal(kwn[b, h, :len(ids)], wn[b, h, ids], equal_nan=True) and np.all(kwn[b, h, len(ids):] == 0)
            for name in "kv":
                with np.errstate(invalid="ignore"):
                    x = oa.sequence(c.codes[name], c.scales[name], tab, h, n)[ids]
                for i, (codes, byte) in enumerate(oa.repage(x, P)):
                    c.codes[name][to[i], h, :len(codes)] = codes
                    c.scales[name][to[i], h] = byte
    # NaN codes keep their sign when they are copied without a change of scale
    for t in (c.gpu.k_codes, c.gpu.v_codes):
        t[(t & 0x7F) == 0x7F] = 0x7F
    c.check()


def _weights(seed, *shape):
    return torch.round(torch.exp(torch.randn(shape, generator=_gen(seed), device="cuda")) * 8) / 8


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_evict_pages(mx, P, d):
    lens = [300, 1, 0, 129, 128, 257]
    _check_evict(mx, lens, 128, 17, 2, d, P, P + d, _weights(P, 6, 2, 384))


@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (2, 1), (64, 64), (64, 0), (199, 3), (200, 0), (500, 20)])
def test_evict_counts(mx, keep, recent):
    _check_evict(mx, [200, 64, 65], keep, recent, 2, 64, 16, keep, _weights(keep, 3, 2, 208))


@pytest.mark.parametrize("kind", ["equal", "zero", "negative", "special", "two", "spread"])
def test_evict_weights_of_any_kind(mx, kind):
    w = _weights(1, 2, 2, 5000)
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "zero":
        w.zero_()
        w[:, :, ::2] = -0.0
    elif kind == "negative":
        w -= 2.0
    elif kind == "special":
        w[:, :, ::7], w[:, :, 1::7], w[:, :, 2::11], w[:, :, 3::50] = math.nan, -math.inf, math.inf, 1e-42
    elif kind == "two":
        w = (w > 1).float()
    else:
        w = torch.exp(20 * torch.randn(w.shape, generator=_gen(3), device="cuda"))
    _check_evict(mx, [5000, 4097], 1000, 100, 2, 64, 128, 5, w)


def test_evict_reports_bad_pages(mx):
    c = _Cache(mx, 8, 16, 1, 64)
    w = _weights(1, 1, 1, 64)
    for table, dst, n in (([[0, 1, 9, 3]], [[4, 5]], 64), ([[0, 1, 2, 3]], [[4, 8]], 64), ([[0, 1, 2, 3]], [[4, 5]], 65)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.gpu.k_codes.zero_(), c.gpu.v_codes.zero_(), c.gpu.k_scales.zero_(), c.gpu.v_scales.zero_()
        mx.moe_kv_evict_fp8(c.gpu, _i32(table), _i32([n]), w, 32, 32, _i32(dst), dev_status=status)
        assert int(status) == mx.DEV_INDEX_OOB
    with pytest.raises(mx.MoeError):
        mx.moe_kv_evict_fp8(c.gpu, _i32([[0, 1, 2, 3]]), _i32([64]), w, 33, 0, _i32([[4, 5]]))
    with pytest.raises(ValueError):
        mx.moe_kv_evict_fp8(c.gpu, _i32([[0, 1, 2, 3]]), _i32([64]), w, 32, 33, _i32([[4, 5]]))
    with pytest.raises(ValueError):
        mx.moe_kv_evict_fp8(c.gpu, _i32([[0, 1, 2, 3]]), _i32([64]), w[0], 32, 3, _i32([[4, 5]]))


def test_decode_evict_decode(mx):
    """The operators together: keys with almost all of the attention stay, and so does the output."""
    P, H, d, n = 16, 2, 64, 200
    g = _gen(50)
    c = mx.KVCache.alloc(32, P, H, d)
    k, v = _bf16(g, n, H, d), _bf16(g, n, H, d)
    q = _bf16(g, 1, 1, 4, d)
    heavy = [3, 50, 51, 120, 199]
    for i in heavy:      # aligned with the queries of each group
        k[i] = (q[0, 0].view(H, 2, d).float().mean(1) * 6).to(torch.bfloat16)
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None]
    mx.moe_kv_append_fp8(c, k, v, _cu([n]), _i32([0]), table)
    w = torch.zeros((1, H, 208), device="cuda")
    before = mx.moe_attn_decode_fp8(c, q, _i32([n]), table, weights=w)
    assert torch.allclose(w.sum(-1), torch.full((1, H), 2.0, device="cuda"), rtol=1e-4)
    dst = torch.arange(20, 24, dtype=torch.int32, device="cuda")[None]
    kept, kw, ln = mx.moe_kv_evict_fp8(c, table, _i32([n]), w, 64, 8, dst)
    assert ln.tolist() == [64] and all(set(heavy) <= set(kept[0, h].tolist()) for h in range(H))
    after = mx.moe_attn_decode_fp8(c, q, ln, dst)
    lost = 1 - kw.sum(-1) / 2.0          # the share of the weight that was dropped
    assert float((after.float() - before.float()).abs().max()) <= 2 * float(lost.max()) * 4.0 * 2 + 0.05


def test_evict_refuses_to_write_over_what_it_reads(mx):
    c = _Cache(mx, 8, 16, 1, 64)
    w, ln = _weights(1, 1, 1, 64), _i32([64])
    with pytest.raises(mx.MoeError):
        mx.moe_kv_evict_fp8(c.gpu, _i32([[0, 1, 2, 3]]), ln, w, 32, 8, _i32([[4, 5]]), new_lengths=ln)
    with pytest.raises(mx.MoeError):
        mx.moe_kv_evict_fp8(c.gpu, _i32([[0, 1, 2, 3]]), ln, w, 64, 8, _i32([[4, 5, 6, 7]]), kept_weights=w)


@pytest.mark.parametrize("lens,keep,recent,H,ties", [([70001, 40000], 1500, 100, 2, False), ([70001], 1500, 0, 1, True),
                                                     ([17003], 64, 5, 80, False), ([33000, 9], 700, 31, 3, True)])
def test_evict_long(mx, lens, keep, recent, H, ties):
    """More positions than a pair's CTAs keep in registers; several CTAs and one; ties across their borders."""
    w = _weights(7, len(lens), H, -(-max(lens) // 128) * 128)
    if ties:
        w = (w * 4).round() / 4
    _check_evict(mx, lens, keep, recent, H, 64, 128, 11, w)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_scores_that_leave_the_reference_behind(mx, d):
    """Every 64 keys the scores rise by more than 2^64, for some queries only and in many items of a CTA."""
    g = _gen(61)
    n = 700
    scale = 256.0 / d
    ramp = torch.linspace(-3, 3, n, device="cuda")[:, None, None].expand(n, 1, d).to(torch.bfloat16).contiguous()
    q = torch.ones((n, 2, d), dtype=torch.bfloat16, device="cuda")
    q[::3] *= 0.25
    q[1::7] *= -1
    _check_prompt(mx, [n], [n], 2, 1, d, True, q=q, k=ramp, seed=62, scale=scale)
    _check_prompt(mx, [n], [n], 2, 1, d, False, q=q, k=ramp, seed=63, scale=scale)
    # a step at one key, in the first or the second half of a tile, the last key among them
    for at in (1, 63, 64, 70, 127, 128, 200, 299):
        k = torch.zeros((300, 1, d), dtype=torch.bfloat16, device="cuda")
        k[at:] = 1.0
        _check_prompt(mx, [300], [300], 2, 1, d, at % 2 == 0, q=q[:300], k=k, seed=at, scale=scale)
    lens = [300, 129, 64, 257, 300, 31]
    total = sum(lens)
    k = (ramp[:1] * 0 + torch.randint(-3, 4, (total, 8, 1), generator=g, device="cuda")).to(torch.bfloat16).expand(
        total, 8, d).contiguous()
    q = torch.ones((total, 64, d), dtype=torch.bfloat16, device="cuda")
    _check_prompt(mx, lens, lens, 64, 8, d, True, q=q, k=k, seed=64, scale=scale, heads=[0, 31, 63])


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_many_sequences_of_many_costs(mx, causal):
    """More items than CTAs, of many costs, from more sequences than a warp has lanes."""
    lens = [(i * 97) % 410 for i in range(50)]
    _check_prompt(mx, lens, lens, 8, 4, 128, causal, seed=71, heads=[0, 5])
    longer = [n + 300 * (i % 3) for i, n in enumerate(lens)]
    _check_prompt(mx, lens, longer, 6, 2, 64, causal, seed=72, heads=[4])


@pytest.mark.parametrize("d", [64, 128])
def test_decode_one_workspace_for_batches_of_any_size(mx, d):
    """A workspace zeroed once, for calls whose sequences, heads and new tokens grow and shrink: as with a new one."""
    P, big = 32, 200
    g = _gen(d)
    pools = {}
    for H in (8, 2):
        c, table = _filled(mx, [320] * big, P, H, d, 10, H)
        pools[H] = c.gpu, table
    ws = torch.zeros(max(mx.moe_attn_decode_workspace_bytes(pools[H][0], big, 4, 2 * H, 10, True) for H in pools),
                     dtype=torch.uint8, device="cuda")
    for H, n_seq, T, G in ((8, 4, 1, 2), (8, big, 1, 2), (2, 3, 4, 2), (8, big, 1, 1), (2, 1, 1, 1), (8, 150, 4, 2),
                           (8, 8, 1, 2), (2, big, 2, 2), (8, big, 1, 2)):
        cache, table = pools[H]
        lens = _i32([1 + (i * 97) % 320 for i in range(n_seq)])
        q = _bf16(g, n_seq, T, H * G, d)
        got = []
        for w in (ws, None):
            out = torch.full_like(q, math.nan)
            lse = torch.full(q.shape[:3], math.nan, device="cuda")
            weights = torch.zeros((n_seq, H, 320), device="cuda")
            mx.moe_attn_decode_fp8(cache, q, lens, table[:n_seq].contiguous(), out=out, lse=lse, weights=weights,
                                   workspace=w)
            got.append((out, lse, weights))
        torch.cuda.synchronize()
        assert torch.isfinite(got[1][0]).all()
        for a, b in zip(*got):
            assert torch.equal(a, b), (H, n_seq, T, G)


@pytest.mark.parametrize("T,hq", [(1, 2), (3, 4), (5, 4), (8, 5), (8, 8)])
def test_decode_many_sequences(mx, T, hq):
    """More sequences than a CTA has threads, empty ones among them."""
    lens = [(i * 37) % 70 if i % 5 else 0 for i in range(900)]
    _check_decode(mx, lens, T, hq, 1, 64, 16, 5, seed=91, weights=True)


def test_evict_pages_with_the_largest_values(mx):
    """A page whose largest value is bf16's largest (its code stands for 2^128), or near it; and codes of every magnitude."""
    P, n = 16, 40
    for top in (3.3895e38, 2.0 ** 127, 1e38):
        c = _Cache(mx, 6, P, 1, 64)
        k = _bf16(_gen(7), n, 1, 64, spread=1e36)
        k[3, 0, 5], k[20, 0, 1], k[39, 0, 63] = top, -top, top
        table, dst = _i32([[2, 0, 4]]), _i32([[1, 3, 5]])
        c.append(mx, k, -k, [n], [0], table)
        mx.moe_kv_evict_fp8(c.gpu, table, _i32([n]), torch.ones((1, 1, 48), device="cuda"), 48, 0, dst)
        for name in "kv":
            x = oa.sequence(c.codes[name], c.scales[name], [2, 0, 4], 0, n)
            for i, (codes, byte) in enumerate(oa.repage(x, P)):
                c.codes[name][[1, 3, 5][i], 0, :len(codes)] = codes
                c.scales[name][[1, 3, 5][i], 0] = byte
        c.check()


def test_evict_page_scale_of_every_code(mx):
    """The scale follows from the page's largest code and scale byte alone, whatever they are."""
    P, srcs = 16, [0, 1, 17, 18, 130, 247, 254]
    table = torch.arange(len(srcs), dtype=torch.int32, device="cuda")[:, None].contiguous()
    for top in range(1, 127):
        c = _Cache(mx, 2 * len(srcs), P, 1, 64)
        for name in "kv":
            c.codes[name][:] = np.random.default_rng(top).integers(0, top + 1, size=c.codes[name].shape)
            c.codes[name][:, 0, 5, 9] = top | (0x80 if name == "v" else 0)
            c.scales[name][:len(srcs), 0] = srcs
        for name, codes, scales in (("k", c.gpu.k_codes, c.gpu.k_scales), ("v", c.gpu.v_codes, c.gpu.v_scales)):
            codes.copy_(torch.tensor(c.codes[name]))
            scales.copy_(torch.tensor(c.scales[name]))
        mx.moe_kv_evict_fp8(c.gpu, table, _i32([P] * len(srcs)), torch.ones((len(srcs), 1, P), device="cuda"), P, 0,
                            table + len(srcs))
        for name in "kv":
            for b, byte in enumerate(srcs):
                [(codes, new)] = oa.repage(oa.decode(c.codes[name][b, 0], byte), P)
                c.codes[name][len(srcs) + b, 0], c.scales[name][len(srcs) + b, 0] = codes, new
        c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_decode_values_of_any_size(mx, d):
    """Values near the ends of bf16's range, where scores and scales rise together in the middle of a warp's work."""
    H, P, n = 8, 32, 20000
    g = _gen(98)
    c = mx.KVCache.alloc(n // P, P, H, d)
    table = torch.arange(n // P, dtype=torch.int32, device="cuda")[None]
    q = torch.ones((1, 1, H, d), dtype=torch.bfloat16, device="cuda")
    for big in (2.0 ** 119, 2.0 ** 60):
        k = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda")
        v = _bf16(g, n, H, d, spread=1e-3)
        for h in range(H):
            at = 32 * (40 + 61 * h)
            k[at:at + 32, h] = 17.0 / d            # e^17 is 2^24.5
            v[at:at + 32, h] = (_bf16(g, 32, d).clamp(-4, 4).float() * big).to(torch.bfloat16)
        mx.moe_kv_append_fp8(c, k, v, _cu([n]), _i32([0]), table)
        _range_check(mx, c, table, q, n, 1.0)
    # and small ones: the results stay normal bf16 numbers
    v = (_bf16(g, n, H, d).clamp(-4, 4).float() * 2.0 ** -122).to(torch.bfloat16)
    v = torch.where(v == 0, torch.full_like(v, 2.0 ** -122), v).abs()
    mx.moe_kv_append_fp8(c, k, v, _cu([n]), _i32([0]), table)
    _range_check(mx, c, table, q, n, 1.0)


def _range_check(mx, c, table, q, n, scale):
    out = _np(mx.moe_attn_decode_fp8(c, q, _i32([n]), table, scale=scale))
    codes = [t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
    tab = table[0].cpu().numpy()
    for h in range(c.n_kv_heads):
        k, v = oa.sequence(codes[0], codes[2], tab, h, n), oa.sequence(codes[1], codes[3], tab, h, n)
        r = oa.attend(_np(q[0, :, h]), k, v, [n], scale)
        err = np.abs(out[0, :, h] - r["out"])
        bound = 2.0 ** -8 * np.abs(r["out"]) + (2.0 ** -10 + 2.0 ** -15 * (1 + r["size"][:, None])) * r["mass"]
        assert np.all(err <= bound), (h, float(np.max(err / bound)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_large_values(mx, d, causal):
    """Values of any size, near the largest bf16 too, while the scores rise by up to 2^60 within a tile."""
    g = _gen(97)
    n = 400
    q = torch.ones((n, 2, d), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    for at, x in ((30, 0.25), (90, 0.5), (127, 0.75), (200, 1.0), (300, 1.25), (399, 1.4)):
        k[at:] = x
    scale = 40.0 / d    # a step of 0.25 is 14 in log2
    for spread in (2.0 ** -77, 2.0 ** 60, 2.0 ** 100, 2.0 ** 123):
        v = _bf16(g, n, 1, d, spread=1.0).clamp(-8, 8) * spread
        _check_prompt(mx, [n], [n], 2, 1, d, causal, q=q, k=k, v=v, scale=scale)
        _check_prompt(mx, [n], [n], 2, 1, d, causal, q=q, k=k, v=v, scale=4 * scale)
        out, _ = _check_prompt(mx, [n], [n], 2, 1, d, causal, q=q, k=0 * k, v=v, scale=scale)
        assert torch.isfinite(out).all()


def test_prompt_equal_keys_and_the_largest_values(mx):
    """A mean over many keys whose values' sum is beyond fp32."""
    n, d = 5000, 64
    q, k = _bf16(_gen(99), 3, 2, d), torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    v = torch.full((n, 1, d), 2.0 ** 127, dtype=torch.bfloat16, device="cuda")
    out = mx.moe_attn_prefill(q, k, v, _cu([3]), _cu([n]))
    assert torch.all(out == 2.0 ** 127)


@pytest.mark.parametrize("T,hq,H", [(5, 7, 1), (5, 16, 2), (6, 8, 1), (7, 14, 2), (7, 8, 1), (8, 24, 4), (7, 27, 3), (1, 49, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_more_than_32_rows(mx, T, hq, H, d, weights):
    """Every number of row tiles and blocks above 32 query rows, work split over CTAs or not."""
    _check_decode(mx, [200, 9, 77, 1500], T, hq, H, d, 32, seed=T + hq, weights=weights)


@pytest.mark.parametrize("mag", [1e3, 1e4, 1e5, 1e9, 1e15])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("hq", [4, 48])
def test_decode_scores_beyond_24_bits(mx, mag, mixed, hq):
    """Equal values give that value whatever the scores are, and every query's weights sum to 1; the leading key is there
    twice. Value scales alike, and different ones for the same values."""
    n, d, P, H = 3000, 64, 16, 2
    g = _gen(101)
    pages = -(-n // P)
    c = mx.KVCache.alloc(pages, P, H, d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q, k = (_bf16(g, 1, 1, hq, d).float() * mag).to(torch.bfloat16), (_bf16(g, n, H, d).float() * mag).to(torch.bfloat16)
    k[1] = k[2900] = (2 * q[0, 0, ::hq // H].float()).to(torch.bfloat16)   # leads for the first query of each group
    v = torch.full((n, H, d), 1.5, dtype=torch.bfloat16, device="cuda")
    mx.moe_kv_append_fp8(c, k, v, _cu([n]), _i32([0]), table)
    # key pages of one scale, so that the two leading keys are equal
    c.k_scales.fill_(int(c.k_scales.max()))
    if mixed:
        c.v_codes.fill_(0x3C), c.v_scales.fill_(127)          # 1.5
        c.v_codes[::3], c.v_scales[::3] = 0x74, 120           # 192 * 2^-7
    for codes in (c.k_codes.view(pages, H, P, d),):
        codes[2900 // P, :, 2900 % P] = codes[0, :, 1]
    w = torch.zeros((1, H, n), device="cuda")
    lse = torch.empty((1, 1, hq), device="cuda")
    out = mx.moe_attn_decode_fp8(c, q, _i32([n]), table, weights=w, lse=lse)
    assert torch.all(out == 1.5)
    assert torch.all((w.double().sum(-1) - hq // H).abs() <= 1e-4 * hq)
    # the leading pair of the first query shares its weight evenly
    one = torch.zeros_like(w)
    for h in range(H):
        alone = q[:, :, [h * (hq // H)] * H].contiguous()
        mx.moe_attn_decode_fp8(c, alone, _i32([n]), table, weights=one.zero_())
        assert abs(float(one[0, h, 1]) - 0.5) < 1e-6 and abs(float(one[0, h, 2900]) - 0.5) < 1e-6
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,rise", [(16, False), (16, True), (80, True)])
def test_decode_small_and_huge_scores_side_by_side(mx, d, hq, rise):
    """Queries of very different sizes in one warp, several chunks each: the small ones keep their accuracy, the huge ones
    give the value of the key that leads, wherever it lies."""
    n, P, H = 20000, 16, 8
    g = _gen(102)
    pages, G = n // P, hq // H
    c = mx.KVCache.alloc(pages, P, H, d)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    k, v = _bf16(g, n, H, d), _bf16(g, n, H, d)
    v *= torch.exp2(torch.randint(-3, 4, (n, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)   # scales differ
    if rise:
        k = (k.float() * torch.linspace(0.01, 8, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    mx.moe_kv_append_fp8(c, k, v, _cu([n]), _i32([0]), table)
    size = torch.tensor([0.05, 3e4, 1.0, 1e9, 1e6], device="cuda").repeat(-(-G // 2))[:G].repeat(H)
    q = (_bf16(g, 1, 1, hq, d).float() * size[None, None, :, None]).to(torch.bfloat16)
    lse = torch.empty((1, 1, hq), device="cuda")
    out = mx.moe_attn_decode_fp8(c, q, _i32([n]), table, lse=lse)
    codes = {x: t.cpu().numpy() for x, t in (("k", c.k_codes), ("v", c.v_codes))}
    scales = {x: t.cpu().numpy() for x, t in (("k", c.k_scales), ("v", c.v_scales))}
    tab, huge = table[0].cpu().numpy(), 0
    for h in (0, 3, 7):
        kk, vv = (oa.sequence(codes[x], scales[x], tab, h, n) for x in "kv")
        for i in range(h * G, (h + 1) * G):
            r = oa.attend(_np(q[0, 0, i:i + 1]), kk, vv, [n], d ** -0.5)
            s = np.sort(kk @ _np(q[0, 0, i]) * d ** -0.5)
            if s[-1] - s[-2] > 100 + 2.0 ** -17 * r["size"][0]:     # one key leads, whatever fp32 rounds
                err = np.abs(_np(out[0, 0, i]) - r["out"][0])
                assert np.all(err <= (2.0 ** -8 + 2.0 ** -10) * np.abs(r["out"][0]) + 1e-30), (h, i, float(err.max()))
                huge += 1
            else:
                _near(out[0, 0, i:i + 1], lse[0, 0, i:i + 1], r, 2.0 ** -10)
    assert huge >= 3


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mag", [1e3, 1e4, 3e4, 1e5, 1e9, 1e15])
def test_prompt_scores_beyond_31_bits(mx, d, mag):
    """Equal values give that value whatever the scores are; where one key leads by far, or two equal ones, the result is
    its value, or their mean, in every tile."""
    g = _gen(103)
    n = 700
    q, k = (_bf16(g, n, 2, d).float() * mag).to(torch.bfloat16), (_bf16(g, n, 1, d).float() * mag).to(torch.bfloat16)
    lse = torch.empty((n, 2), device="cuda")
    same = torch.full((n, 1, d), 1.5, dtype=torch.bfloat16, device="cuda")
    for scale in (None, -d ** -0.5, 3.0):
        out = mx.moe_attn_prefill(q, k, same, _cu([n]), lse=lse, scale=scale)
        assert torch.all((out.float() - 1.5).abs() <= 2.0 ** -7) and torch.isfinite(lse).all(), scale
    # keys of falling, then rising size, the first 64 of them twice in the last tile
    k = (k.float() * (torch.arange(n, device="cuda") % 200 - 100).abs()[:, None, None] / 50).to(torch.bfloat16)
    k[-64:] = k[:64]
    v = _bf16(g, n, 1, d)
    out = mx.moe_attn_prefill(q, k, v, _cu([n]), causal=False)
    for h in range(2):
        s = (q[:, h].double() @ k[:, 0].double().T) * d ** -0.5
        top = s.amax(-1, keepdim=True)
        leads = s == top
        rest = s.masked_fill(leads, -math.inf).amax(-1)
        clear = top[:, 0] - rest > 100 + 2.0 ** -17 * mag * mag * d ** 0.5 * 50
        w = (leads / leads.sum(-1, keepdim=True)).double()
        want, mass = w @ v[:, 0].double(), w @ v[:, 0].double().abs()
        err = (out[:, h].double() - want).abs()
        assert int(clear.sum()) > n // 4 and int((leads.sum(-1) == 2)[clear].sum()) > 3
        assert torch.all(err[clear] <= 2.0 ** -8 * want[clear].abs() + 2.0 ** -8 * mass[clear] + 1e-30)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_small_and_huge_scores_side_by_side(mx, d):
    """Queries of very different sizes in one tile: the small ones keep their accuracy."""
    g = _gen(104)
    n = 600
    size = torch.tensor([0.05, 3e5, 1.0, 1e9, 2.0, 1e14], device="cuda").repeat(n // 6)
    q = (_bf16(g, n, 2, d).float() * size[:, None, None]).to(torch.bfloat16)
    k, v = _bf16(g, n, 1, d), _bf16(g, n, 1, d)
    lse = torch.empty((n, 2), device="cuda")
    out = mx.moe_attn_prefill(q, k, v, _cu([n]), lse=lse)
    ref = oa.attend(_np(q[:, 1]), _np(k[:, 0]), _np(v[:, 0]), np.arange(n) + 1, d ** -0.5)
    _near(out[:, 1], lse[:, 1], ref, 2.0 ** -8)
    assert torch.isfinite(out).all()
