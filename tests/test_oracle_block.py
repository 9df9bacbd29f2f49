"""Pins of oracle.block, and the refusals of the operators around a block's halves (CPU only)."""
import ctypes
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block as ob


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_expert_gb300 as mx
    return mx


def test_norm_against_torch():
    g = torch.Generator().manual_seed(1)
    x, a = torch.randn((5, 48), generator=g, dtype=torch.float64), torch.randn((5, 48), generator=g, dtype=torch.float64)
    wp, wn, gate = (torch.randn(48, generator=g, dtype=torch.float64) for _ in range(3))
    r = ob.block_norm(x, a, wp, gate, 0.5, wn, 1e-5, 1.0)
    y = x + 0.5 * gate * torch.nn.functional.rms_norm(a, (48,), 1 + wp, 1e-5)
    assert np.allclose(r["y"], y, rtol=1e-13, atol=1e-13)
    assert np.allclose(r["h"], torch.nn.functional.rms_norm(y, (48,), 1 + wn, 1e-5), rtol=1e-13, atol=1e-13)
    r = ob.block_norm(x, eps=0.0)
    assert r["y"] is None and np.allclose((r["h"] ** 2).mean(-1), 1.0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_routing_against_a_search(kind, best, with_bias):
    """The chosen groups and experts maximise the sums of their keys over all choices."""
    rng = np.random.default_rng(3)
    l, bias = rng.normal(size=(6, 12)), rng.normal(size=12) * 0.3 if with_bias else None
    idx, w = ob.route_groups(l, 3, bias, kind, 4, 2, best, True, 2.0)
    s = torch.sigmoid(torch.tensor(l)).numpy() if kind == "sigmoid" else torch.softmax(torch.tensor(l), -1).numpy()
    key = s + (0 if bias is None else bias)
    for t in range(6):
        def score(g):
            return sum(sorted(key[t, 3 * g:3 * g + 3])[-best:])
        groups = max(itertools.combinations(range(4), 2), key=lambda c: sum(score(g) for g in c))
        inside = [e for g in groups for e in range(3 * g, 3 * g + 3)]
        want = max(itertools.combinations(inside, 3), key=lambda c: sum(key[t, e] for e in c))
        assert set(idx[t]) == set(want)
        assert list(key[t, idx[t]]) == sorted(key[t, idx[t]], reverse=True)
        assert np.allclose(w[t], 2.0 * s[t, idx[t]] / s[t, idx[t]].sum(), rtol=1e-12)


def test_routing_ties_and_specials():
    idx, w = ob.route_groups(np.zeros((1, 8)), 3, None, "softmax", 4, 2)
    assert idx.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 3)
    l = np.array([[math.nan, 1.0, -math.inf, math.inf]])
    idx, w = ob.route_groups(l, 4)
    assert idx.tolist() == [[3, 1, 2, 0]] and w[0, 3] == 0 and w[0, 0] > w[0, 1]
    idx, w = ob.route_groups(np.full((1, 4), math.nan), 2, None, "softmax")
    assert idx.tolist() == [[0, 1]] and not w.any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_against_complex_numbers(interleaved):
    rng = np.random.default_rng(5)
    x, f, pos = rng.normal(size=(4, 2, 24)), 10.0 ** -np.arange(8.0), np.array([0, 1, 77, 100000])
    y = ob.rotate(x, pos, f, interleaved)
    z = x[..., 0:16:2] + 1j * x[..., 1:16:2] if interleaved else x[..., :8] + 1j * x[..., 8:16]
    z = z * np.exp(1j * pos[:, None] * f)[:, None]
    got = y[..., 0:16:2] + 1j * y[..., 1:16:2] if interleaved else y[..., :8] + 1j * y[..., 8:16]
    assert np.allclose(got, z, atol=1e-11)
    assert np.array_equal(y[..., 16:], x[..., 16:]) and np.allclose(y[0], x[0])
    assert np.all(np.abs(y) <= ob.pair_size(x, 16, interleaved) + 1e-12)


def test_angles_in_integers():
    """The reduction in turns by 64-bit integers: p F modulo 2^64 is the angle's fraction of a turn to p 2^-64."""
    # 2 pi to 40 digits
    turn = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
    for f in (1.0, 0.1, 1e-4, 0.7498942, 3.3e-6):
        f = float(np.float32(f))
        turns = f * 0.15915494309189533577
        F = int((turns - math.floor(turns)) * 18446744073709551616.0)
        for p in (1, 2, 4095, 1 << 20, (1 << 31) - 1):
            got = Fraction((p * F) % (1 << 64), 1 << 64)
            want = Fraction(f) * p / turn
            want -= math.floor(want)
            err = abs(got - want)
            # the product by 1 / 2 pi is rounded twice: 2^-52 of the turns that a step makes
            assert min(err, 1 - err) <= p * (Fraction(turns) / 2 ** 52 + Fraction(1, 2 ** 64))


def test_norm_refusals(mx):
    L, p = mx.lib, ctypes.c_void_p(64)
    ok = dict(x=p, xs=64, f32=0, a=p, as_=64, T=2, d=64, wp=p, g=p, gs=0, s=1.0, wn=p, eps=1e-6, off=0.0, y=p, ys=64, h=p,
              hs=64)

    def call(**kw):
        v = {**ok, **kw}
        return L.moe_block_norm(*(v[n] for n in ok), None)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(d=0), dict(f32=2), dict(s=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(off=math.nan),
               dict(a=None), dict(y=None), dict(a=None, y=None), dict(h=None), dict(xs=63), dict(as_=60), dict(gs=8),
               dict(hs=32), dict(x=None), dict(x=ctypes.c_void_p(8)), dict(wn=ctypes.c_void_p(4)),
               dict(a=None, y=None, wp=None, g=None, wn=None, h=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(d=60), dict(d=32776, xs=32776, as_=32776, ys=32776, hs=32776)):
        assert call(**kw) == -2, kw


def test_routing_refusals(mx):
    L, p = mx.lib, ctypes.c_void_p(64)
    rule = dict(score=0, n=8, top=4, best=2, renorm=1, scale=1.0)
    ok = dict(l=p, T=2, E=64, k=4, b=None, idx=p, w=p)

    def call(**kw):
        r = mx.moe_group_rule(*({**rule, **{n: v for n, v in kw.items() if n in rule}}[n] for n in rule))
        v = {**ok, **kw}
        return L.moe_route_groups(v["l"], v["T"], v["E"], v["k"], v["b"], ctypes.byref(r), v["idx"], v["w"], None)
    assert L.moe_route_groups(p, 2, 64, 4, None, None, p, p, None) == -1
    assert L.moe_forward_groups(None, None, p, 2, p, None, None, None, None, p, 0, None, None) == -1
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(n=0), dict(top=0), dict(top=9), dict(score=2), dict(best=0),
               dict(best=3), dict(renorm=2), dict(scale=math.nan), dict(l=None), dict(idx=None), dict(w=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(E=1032), dict(k=33), dict(n=7, top=4), dict(E=128, n=64, top=4), dict(k=9, top=1), dict(E=8, top=8),
               dict(E=1020, n=17, top=4)):
        assert call(**kw) == -2, kw


def _cache(mx, **kw):
    d = dict(n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, k_codes=64, v_codes=64, k_scales=64, v_scales=64)
    d.update(kw)
    return mx.moe_kv_cache(*(d[n] for n, _ in mx.moe_kv_cache._fields_))


def test_append_with_rotation_refusals(mx):
    L, p = mx.lib, ctypes.c_void_p(64)
    r = mx.moe_rows(64, 128, 64)
    ok = dict(c=_cache(mx), k=r, v=r, cu=p, st=p, n=2, total=5, tab=p, width=2, f=p, rot=64, il=0, rs=None, q=r, nh=4, qo=p)

    def call(**kw):
        v = {**ok, **kw}
        return L.moe_kv_append_rope_fp8(*(v[n] for n in ok), None, None)
    assert call(n=0) == 0 and call(total=0) == 0
    bad = mx.moe_rows(64, 127, 64)
    for kw in (dict(il=2), dict(k=None), dict(v=bad), dict(q=bad), dict(f=None), dict(qo=None), dict(qo=ctypes.c_void_p(8)),
               dict(cu=None), dict(st=None), dict(tab=None), dict(total=-1), dict(n=-1), dict(width=-1), dict(c=None),
               dict(c=_cache(mx, k_codes=8))):
        assert call(**kw) == -1, kw
    for kw in (dict(rot=0), dict(rot=8), dict(rot=40), dict(rot=80), dict(rot=128), dict(nh=0), dict(nh=70000),
               dict(n=65537), dict(total=2 ** 31 - 65535), dict(c=_cache(mx, page_size=8))):
        assert call(**kw) == -2, kw


def test_chunk_refusals(mx):
    L, p = mx.lib, ctypes.c_void_p(256)
    r = mx.moe_rows(64, 256, 64)
    ok = dict(c=_cache(mx), q=r, nh=4, cu=p, n=2, total=5, ln=p, tab=p, width=2, s=0.1, out=p, lse=None, ws=p, wn=1 << 30)

    def call(**kw):
        v = {**ok, **kw}
        return L.moe_attn_chunk_fp8(*(v[n] for n in ok), None, None)
    assert call(n=0) == 0 and call(total=0) == 0
    for kw in (dict(c=None), dict(nh=0), dict(n=-1), dict(total=-1), dict(q=None), dict(cu=None), dict(ln=None), dict(tab=None),
               dict(out=None), dict(out=ctypes.c_void_p(8)), dict(ws=None), dict(ws=ctypes.c_void_p(64)), dict(s=math.nan),
               dict(width=-1), dict(q=mx.moe_rows(64, 4, 64)), dict(c=_cache(mx, v_scales=None))):
        assert call(**kw) == -1, kw
    for kw in (dict(nh=3), dict(nh=65536), dict(n=65537), dict(total=2 ** 31 - 65535), dict(nh=64, total=1 << 27),
               dict(c=_cache(mx, head_dim=96))):
        assert call(**kw) == -2, kw
    assert L.moe_attn_chunk_workspace_bytes(ctypes.byref(_cache(mx)), 3, 5, 2) == 0


def test_binding_checks_before_the_gpu(mx):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError, RuntimeError, AssertionError)):
        mx.moe_block_norm(x)
    with pytest.raises(ValueError):
        mx.moe_route_groups(x, 2, score="tanh")


def test_rope_refuses_more_heads_than_a_grid_has(mx):
    p, r = ctypes.c_void_p(64), mx.moe_rows(64, 128, 64)
    c = _cache(mx)
    n = 65536 - 2 * c.n_kv_heads
    assert mx.lib.moe_kv_append_rope_fp8(c, r, r, p, p, 2, 5, p, 2, p, 64, 0, None, r, n, p, None, None) == -2
