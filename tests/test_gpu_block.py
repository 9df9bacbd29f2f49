"""The norms around a block's halves and routing by groups, on the GPU against oracle.block (fp64).

Tolerances. A sum of squares adds at most 32 products in a thread and 10 steps of a tree, each rounded by 2^-24 of terms
of one sign: 2^-18 of the sum, so a norm's factor errs by 2^-19 and its reciprocal square root's 2^-22. With the
products around it a normalised term errs by at most 2^-18 of itself: y before its rounding by
  u = 2^-18 |scale gate n| + 2^-23 |x|,
and y by that and the half step of its type (2^-8 of it for bf16, 2^-24 for fp32). The norm of y then has the factor's
own 2^-18 and rms(u) / rms(y):
  |h - ref| <= 2^-8 |ref| + |w| r u + |ref| (2^-18 + rms(u) / rms(y)).
Weights of a route: scores to 2^-23, a sum of at most 32 and a division: 2^-18 of the weight. Indices are equal.
"""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _bf16(g, *shape, spread=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(BF16)


def _rms(z):
    return np.sqrt((z * z).mean(-1, keepdims=True))


def _near(y, h, x, ref, eps):
    u = 2.0 ** -18 * np.abs(ref["add"]) + 2.0 ** -23 * np.abs(_np(x))
    if y is not None:
        half = 2.0 ** -8 if y.dtype == BF16 else 2.0 ** -24
        err = np.abs(_np(y) - ref["y"])
        assert np.all(err <= half * np.abs(ref["y"]) + u + 1e-38), float(err.max())
    if h is not None:
        r = ob.rstd(ref["sum"], eps)
        bound = 2.0 ** -8 * np.abs(ref["h"]) + np.abs(ref["w"]) * r * u + np.abs(ref["h"]) * (2.0 ** -18 + r * _rms(u))
        err = np.abs(_np(h) - ref["h"])
        assert np.all(err <= bound + 1e-38), float((err / (bound + 1e-38)).max())


def _check(mx, x, a=None, eps=1e-6, **kw):
    y, h = mx.moe_block_norm(x, a, eps=eps, **kw)
    y2, h2 = mx.moe_block_norm(x, a, eps=eps, **kw)
    for p, q in ((y, y2), (h, h2)):
        assert p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    ref = ob.block_norm(_np(x), _np(a), _np(kw.get("post_weight")), _np(kw.get("gate")), kw.get("residual_scale", 1.0),
                        _np(kw.get("pre_weight")), eps, kw.get("weight_offset", 0.0))
    _near(y, h, x, ref, eps)
    return y, h


# ---- norms ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d", [8, 16, 72, 248, 256, 264, 512, 1000, 2048, 2056, 2560, 4104, 8192, 8200, 16384, 16392, 32768])
def test_norm_widths(mx, d, wide):
    g = _gen(d)
    x = torch.randn((5, d), generator=g, device="cuda") * 3
    x = x if wide else x.to(BF16)
    _check(mx, x, _bf16(g, 5, d), post_weight=_bf16(g, d), gate=_bf16(g, d), residual_scale=0.25, pre_weight=_bf16(g, d))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 151, 152, 153, 1000, 5000])
def test_norm_rows(mx, T, wide):
    g = _gen(T)
    x = torch.randn((T, 320), generator=g, device="cuda")
    _check(mx, x if wide else x.to(BF16), _bf16(g, T, 320), post_weight=_bf16(g, 320), gate=_bf16(g, T, 320),
           pre_weight=_bf16(g, 320))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("pre", [False, True])
def test_norm_options(mx, wide, post, gate, pre):
    g = _gen(7)
    T, d = 9, 640
    x = torch.randn((T, d), generator=g, device="cuda")
    kw = {}
    if post:
        kw["post_weight"] = _bf16(g, d)
    if gate:
        kw["gate"] = _bf16(g, d) if gate == 1 else _bf16(g, T, d)
    if pre:
        kw["pre_weight"] = _bf16(g, d)
    y, h = _check(mx, x if wide else x.to(BF16), _bf16(g, T, d), residual_scale=-1.5, weight_offset=1.0, eps=1e-5, **kw)
    assert (h is not None) == pre and y.dtype == (torch.float32 if wide else BF16)


def test_norm_alone_and_weightless(mx):
    g = _gen(8)
    x = _bf16(g, 6, 96)
    y, h = _check(mx, x, pre_weight=_bf16(g, 96))
    assert y is None
    _check(mx, x)
    h = torch.empty_like(x)
    y, got = mx.moe_block_norm(x, _bf16(g, 6, 96), h=h)
    assert got is h and y is not None
    assert mx.moe_block_norm(x[:0], x[:0], pre_weight=_bf16(g, 96))[1].shape == (0, 96)


@pytest.mark.parametrize("wide", [False, True])
def test_norm_in_place_and_strided(mx, wide):
    g = _gen(9)
    T, d = 70, 256
    big = torch.randn((T, 3 * d), generator=g, device="cuda")
    big = big if wide else big.to(BF16)
    x, a, gate = big[:, d:2 * d], _bf16(g, T, 2 * d)[:, 16:16 + d], _bf16(g, T, d + 8)[:, 8:]
    kw = dict(post_weight=_bf16(g, d), gate=gate, residual_scale=0.5, pre_weight=_bf16(g, d))
    want = mx.moe_block_norm(x.contiguous(), a.contiguous(), **{**kw, "gate": gate.contiguous()})
    rest = big.clone()
    y, h = mx.moe_block_norm(x, a, y=x, h=a, **kw)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    assert torch.equal(big[:, :d], rest[:, :d]) and torch.equal(big[:, 2 * d:], rest[:, 2 * d:])


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1.0, 1e15, 1e20, 1e38])
@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-6])
@pytest.mark.parametrize("wide", [False, True])
def test_norm_of_values_of_any_size(mx, size, eps, wide):
    """Squares leave fp32 on both sides; bf16 and fp32 rows, and rows of zeros."""
    g = _gen(10)
    x = torch.rand((4, 264), generator=g, device="cuda") * size * 2 + size / 2
    x[:, ::3] *= -1
    x = x if wide else x.to(BF16)
    _check(mx, x, eps=eps, pre_weight=_bf16(g, 264))
    a = (torch.rand((4, 264), generator=g, device="cuda") * size * 2 + size / 2).to(BF16)
    # x above 2^-14 of y, so that its rounding shows, but y below the largest number
    _check(mx, x, a, eps=eps, post_weight=torch.full((264,), 0.5, dtype=BF16, device="cuda"))


def test_norm_of_zeros_and_of_nothing_finite(mx):
    x = torch.zeros((3, 64), dtype=BF16, device="cuda")
    _, h = mx.moe_block_norm(x, eps=1e-6)
    assert not h.any()
    x[1, 5], x[2, 7] = math.inf, math.nan
    y, h = mx.moe_block_norm(x, x.clone(), pre_weight=torch.ones(64, dtype=BF16, device="cuda"))
    assert not h[0].any() and torch.isnan(h[1, 5]) and torch.isnan(h[2]).all()
    assert torch.isfinite(y[0]).all() and y[1, 5] == math.inf and torch.isnan(y[2, 7])


def test_norm_on_another_stream(mx):
    g = _gen(11)
    x, a, w = _bf16(g, 300, 512), _bf16(g, 300, 512), _bf16(g, 512)
    want = mx.moe_block_norm(x, a, pre_weight=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mx.moe_block_norm(x, a, pre_weight=w, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_norm_refusals(mx):
    g = _gen(12)
    x, a, w = _bf16(g, 4, 64), _bf16(g, 4, 64), _bf16(g, 64)
    for bad in (dict(x=x.half()), dict(a=a.float()), dict(pre_weight=w.float()), dict(gate=a.float()), dict(y=x.float())):
        with pytest.raises(TypeError):
            mx.moe_block_norm(**{"x": x, "a": a, **bad})
    for bad in (dict(x=x[0]), dict(a=a[:3]), dict(pre_weight=w[:32]), dict(gate=w[:32]), dict(gate=a[:3]), dict(h=a[:, :32]),
                dict(a=a.t().contiguous().t()), dict(a=None, y=x)):
        with pytest.raises(ValueError):
            mx.moe_block_norm(**{"x": x, "a": a, **bad})
    wide = _bf16(g, 4, 70)
    for bad in (dict(x=_bf16(g, 4, 60), a=None), dict(a=wide[:, 6:]), dict(eps=-1.0), dict(residual_scale=math.inf),
                dict(a=None, gate=w), dict(a=None, post_weight=w)):
        with pytest.raises(mx.MoeError):
            mx.moe_block_norm(**{"x": x, "a": a, **bad})


# ---- routing by groups --------------------------------------------------------------------------------------------

def _check_route(mx, logits, k, bias=None, score="sigmoid", n_groups=1, top_groups=1, group_best=2, renormalise=True,
                 scale=1.0):
    idx, w = mx.moe_route_groups(logits, k, bias, score, n_groups, top_groups, group_best, renormalise, scale)
    ref = ob.route_groups(_np(logits), k, _np(bias), score, n_groups, top_groups, group_best, renormalise, scale)
    got = idx.cpu().numpy()
    for t in np.flatnonzero((got != ref[0]).any(-1)):
        # s(x) + s(-x) = 1, and sums with the biases of others may be equal as well: groups then tie as real numbers, and
        # 64 bits are not enough to see it. The kernel's sums are good to 2^-40; which of such groups it takes is free.
        assert group_best == 2
        rank = ob.group_ranks(_np(logits[t]), _np(bias), score, n_groups)
        cut = np.sort(rank)[-top_groups]
        sure, maybe = np.flatnonzero(rank > cut + 2.0 ** -40), np.flatnonzero(np.abs(rank - cut) <= 2.0 ** -40)
        for more in itertools.combinations(maybe, top_groups - len(sure)):
            one = ob.route_groups(_np(logits[t:t + 1]), k, _np(bias), score, n_groups, top_groups, group_best, renormalise,
                                  scale, groups=sorted([*sure, *more]))
            if np.array_equal(got[t], one[0][0]):
                ref[1][t] = one[1][0]
                break
        else:
            raise AssertionError((t, got[t].tolist(), ref[0][t].tolist(), rank.tolist()))
    err = np.abs(_np(w) - ref[1])
    assert np.all(err <= 2.0 ** -18 * np.abs(ref[1]) + 2.0 ** -120), float(err.max())
    return idx, w


SHAPES = [(1, 1, 1, 1), (5, 3, 1, 1), (31, 4, 1, 1), (32, 8, 2, 1), (33, 2, 3, 2), (64, 8, 8, 4), (96, 6, 12, 5),
          (160, 6, 8, 3), (256, 8, 8, 4), (384, 8, 1, 1), (512, 8, 8, 4), (512, 32, 16, 16), (1000, 10, 4, 3),
          (1024, 32, 32, 8), (1023, 7, 1, 1)]


@pytest.mark.parametrize("E,k,n,top", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_shapes(mx, E, k, n, top, score, with_bias):
    g = _gen(E + k)
    logits = torch.randn((37, E), generator=g, device="cuda") * 2
    bias = torch.randn(E, generator=g, device="cuda") * 0.2 if with_bias else None
    for best in (1, 2):
        if E // n >= best:
            _check_route(mx, logits, k, bias, score, n, top, best, scale=2.5)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 63, 300, 1111])
def test_route_tokens(mx, T):
    g = _gen(T)
    _check_route(mx, torch.randn((T, 128), generator=g, device="cuda"), 4, torch.randn(128, generator=g, device="cuda") * 0.1,
                 "sigmoid", 4, 2, 2)
    _check_route(mx, torch.randn((T, 128), generator=g, device="cuda"), 4, renormalise=False, scale=-0.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_go_to_the_lower_index(mx, score):
    g = _gen(3)
    logits = torch.randint(-2, 3, (200, 96), generator=g, device="cuda").float()
    bias = torch.randint(-2, 3, (96,), generator=g, device="cuda").float() / 8
    for b in (None, bias):
        for n, top, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (12, 12, 2)):
            _check_route(mx, logits, 9, b, score, n, top, best)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_keys_closer_than_fp32_tells(mx, score):
    """Scores and biases whose sums differ by far less than an fp32 step still rank by their exact size."""
    g = _gen(4)
    T, E = 64, 128
    logits = torch.randn((T, E), generator=g, device="cuda")
    if score == "sigmoid":
        # key = sigmoid(l) + b with b = fp32(c - sigmoid(l)): sums within 2^-25 of c
        s = torch.sigmoid(logits[:1].double())
        logits = logits[:1].expand(T, E).contiguous()
    else:
        logits = logits[:1].expand(T, E).contiguous()
        s = torch.softmax(logits[:1].double(), -1)
    bias = (0.75 - s[0]).float()
    sums = (s[0] + bias.double()).sort().values
    assert (sums[-1] - sums[0]) < 2.0 ** -23 and (sums[1:] - sums[:-1]).min() > 2.0 ** -42
    _check_route(mx, logits, 16, bias, score)
    _check_route(mx, logits, 5, bias, score, 8, 2, 2)
    _check_route(mx, logits, 5, bias, score, 8, 2, 1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_special_logits(mx, score):
    g = _gen(5)
    l = torch.randn((40, 64), generator=g, device="cuda")
    l[0] = math.nan
    l[1, ::2] = math.nan
    l[2] = -math.inf
    l[3, 5:] = -math.inf
    l[4, 7], l[4, 9] = math.inf, math.inf
    l[5, :] = 0.0
    l[5, 1::2] = -0.0
    l[6] *= 30
    l[7, 3], l[7, 60] = 3e38, -3e38
    l[8] = torch.arange(64, device="cuda") - 32.0
    _check_route(mx, l, 8, None, score)
    _check_route(mx, l, 8, None, score, 8, 3, 1)
    bias = torch.randn(64, generator=g, device="cuda") * 0.1
    _check_route(mx, l, 8, bias, score)
    bias[3], bias[17] = -math.inf, 1e30
    _check_route(mx, l, 8, bias, score, 8, 3, 2)


def test_route_large_and_small_logits(mx):
    g = _gen(6)
    for size in (1e-6, 1.0, 20.0, 60.0):
        l = torch.randn((50, 256), generator=g, device="cuda") * size
        b = torch.randn(256, generator=g, device="cuda") * 1e-3
        for score in ("sigmoid", "softmax"):
            _check_route(mx, l, 8, b, score, 8, 4, 2)


def test_route_outputs_and_stream(mx):
    g = _gen(7)
    l = torch.randn((100, 64), generator=g, device="cuda")
    want = mx.moe_route_groups(l, 4, n_groups=4, top_groups=2)
    idx, w = torch.empty((100, 4), dtype=torch.int32, device="cuda"), torch.empty((100, 4), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mx.moe_route_groups(l, 4, n_groups=4, top_groups=2, idx=idx, w=w, stream=s)
    s.synchronize()
    assert got[0] is idx and got[1] is w and torch.equal(idx, want[0]) and torch.equal(w, want[1])
    assert mx.moe_route_groups(l[:0], 4)[0].shape == (0, 4)
    # the experts of a route are what the sort by expert takes
    assert int(mx.moe_sort_by_expert(idx, 64)["offsets"][64]) == 400


def test_route_refusals(mx):
    l = torch.zeros((4, 64), device="cuda")
    with pytest.raises(TypeError):
        mx.moe_route_groups(l.half(), 2)
    for bad in (dict(logits=l[0]), dict(bias=l[0, :32].contiguous()), dict(score="tanh"), dict(idx=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            mx.moe_route_groups(**{"logits": l, "k": 2, **bad})
    for bad in (dict(k=0), dict(k=40), dict(n_groups=3), dict(n_groups=4, top_groups=5), dict(group_best=3), dict(scale=math.nan)):
        with pytest.raises(mx.MoeError):
            mx.moe_route_groups(**{"logits": l, "k": 2, **bad})


# ---- the layer with it ------------------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def tiny(mx):
    import workloads as wl
    from mxfp4_expert_gb300 import synthetic
    w = wl.get("tiny")
    return w, synthetic.build_layer(w, 0)


@pytest.mark.parametrize("T", [1, 4, 5, 40, 200])
@pytest.mark.parametrize("score,n,top,best", [("sigmoid", 8, 3, 2), ("softmax", 4, 2, 1), ("sigmoid", 1, 1, 1)])
def test_layer_routed_by_groups(mx, tiny, T, score, n, top, best):
    """Against the oracle's experts, with the routing that the oracle finds for the layer's own logits. Tolerances as for
    moe_forward: relative L2 5e-3, 2e-2 of the rms an element (or the nearest bf16)."""
    import oracle_par
    import workloads as wl
    from oracle import moe as omoe
    w, layer = tiny
    g = _gen(T)
    x, bias = _bf16(g, T, w.d), torch.randn(w.E, generator=g, device="cuda") * 0.1
    logits = torch.empty((T, w.E), device="cuda")
    idx, wts = torch.empty((T, w.k), dtype=torch.int32, device="cuda"), torch.empty((T, w.k), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(score=score, n_groups=n, top_groups=top, group_best=best, scale=2.5)
    y = mx.moe_forward_groups(layer, x, bias, logits_out=logits, idx_out=idx, w_out=wts, dev_status=status, **kw)
    assert int(status) == 0
    alone = mx.moe_route_groups(logits, w.k, bias, **kw)
    assert torch.equal(alone[0], idx) and torch.equal(alone[1], wts)
    ri, rw = ob.route_groups(_np(logits), w.k, _np(bias), score, n, top, best, True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    xs = x.cpu()
    sg, su, sd = (omoe.as_f64(t) for t in wl.gen_shared(w, 0, "cuda"))
    ref = omoe.swiglu_ffn(omoe.as_f64(xs), sg, su, sd)
    for e in np.unique(ri):
        gu, dn = wl.gen_experts(w, 0, int(e), 1, "cuda")
        t, j = np.nonzero(ri == e)
        ref[t] += rw[t, j][:, None] * omoe.expert_outputs(xs[t], gu[0].cpu(), dn[0].cpu())
    got = _np(y)
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
    rms = np.sqrt(np.mean(ref ** 2))
    assert np.all((np.abs(got - ref) <= 2e-2 * rms) | (got == oracle_par.bf16_rne(ref)))


def test_layer_routed_by_groups_refusals(mx, tiny):
    w, layer = tiny
    x = torch.zeros((2, w.d), dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        mx.moe_forward_groups(layer, x, score="tanh")
    with pytest.raises(ValueError):
        mx.moe_forward_groups(layer, x, torch.zeros((2, w.E), device="cuda"))
    with pytest.raises(ValueError):
        mx.moe_forward_groups(layer, x[:, :64])
    for bad in (dict(n_groups=5), dict(n_groups=8, top_groups=9), dict(group_best=0), dict(scale=math.nan),
                dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(mx.MoeError):
            mx.moe_forward_groups(layer, x, **bad)
