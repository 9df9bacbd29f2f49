"""Pins of oracle.attention, and the attention entry points' checks that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import mxfp8


def test_attend_against_torch_softmax():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(7, 16)), g.normal(size=(11, 16)), g.normal(size=(11, 16))
    seen = np.arange(7) + 5
    r = oa.attend(q, k, v, seen, 0.3)
    s = torch.tensor(q) @ torch.tensor(k).T * 0.3
    s = s.masked_fill(torch.arange(11)[None] >= torch.tensor(seen)[:, None], -math.inf)
    assert np.allclose(r["out"], (torch.softmax(s, -1) @ torch.tensor(v)).numpy(), rtol=1e-13, atol=1e-13)
    assert np.allclose(r["lse"], torch.logsumexp(s, -1).numpy(), rtol=1e-13)
    assert np.allclose(r["weights"].sum(1), 1.0)


def test_attend_equal_keys_is_a_mean_and_empty_rows_are_zero():
    g = np.random.default_rng(1)
    k, v = np.tile(g.normal(size=(1, 8)), (5, 1)), g.normal(size=(5, 8))
    r = oa.attend(g.normal(size=(3, 8)), k, v, [5, 2, 0], 1.0)
    assert np.allclose(r["out"][0], v.mean(0)) and np.allclose(r["out"][1], v[:2].mean(0))
    assert np.all(r["out"][2] == 0) and r["lse"][2] == -np.inf


def test_attend_ignores_what_is_not_seen():
    g = np.random.default_rng(2)
    k, v = g.normal(size=(6, 8)), g.normal(size=(6, 8))
    q = g.normal(size=(2, 8))
    want = oa.attend(q, k, v, [3, 4], 1.0)["out"]
    k[4:], v[4:] = np.nan, np.inf
    assert np.array_equal(oa.attend(q, k, v, [3, 4], 1.0)["out"], want)


def test_scale_byte_is_the_smallest_that_fits():
    g = np.random.default_rng(3)
    for x in [1e-38, 448.0, 448.0000001, 447.9, 224.0, 225.0, 3e38, 2.0 ** -118, 1.0] + list(np.exp(g.normal(size=200) * 20)):
        b = oa.scale_byte(float(x))
        fits = [e for e in range(-127, 128) if x <= 448 * 2.0 ** e]
        assert b == fits[0] + 127, x
    assert oa.scale_byte(0.0) == 0


def test_encode_against_torch():
    g = np.random.default_rng(4)
    x = g.normal(size=4000) * np.exp(g.normal(size=4000) * 2)
    x = np.clip(x, -440, 440)
    want = torch.tensor(x, dtype=torch.float64).float()
    x = want.double().numpy()
    assert np.array_equal(oa.encode(x, 127), want.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(oa.encode(np.array([np.inf, -np.inf, np.nan]), 127)) == [0x7F] * 3


def test_rescale_is_exact_above_the_subnormals():
    codes = np.array([c for c in range(256) if (c & 0x7F) != 0x7F and ((c >> 3) & 15) > 3], dtype=np.uint8)
    new = oa.rescale(codes, 130, 132)
    assert np.array_equal(oa.decode(new, 132), oa.decode(codes, 130))
    assert list(oa.rescale(np.array([0x7F, 0xFF], dtype=np.uint8), 1, 9)) == [0x7F, 0xFF]


def test_append_in_steps_and_at_once_agree_while_the_scale_stands():
    g = np.random.default_rng(5)
    x = g.normal(size=(40, 2, 64))
    x[0, :, 0] = 400.0   # the first page's scale from its first token on
    x[16, :, 0] = x[32, :, 0] = 400.0
    table = [2, 0, 1]
    a = np.zeros((3, 2, 16, 64), np.uint8), np.zeros((3, 2), np.uint8)
    b = np.zeros((3, 2, 16, 64), np.uint8), np.zeros((3, 2), np.uint8)
    oa.append(*a, x, 0, table)
    for lo, hi in ((0, 1), (1, 15), (15, 17), (17, 33), (33, 40)):
        oa.append(*b, x[lo:hi], lo, table)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    got = oa.sequence(*a, table, 1, 40)
    assert np.all(np.abs(got - x[:, 1]) <= np.maximum(np.abs(x[:, 1]) * 2.0 ** -4, 2.0 ** -10))
    # 400 lies halfway between 384 and 416; 384 has the even code
    assert a[1][2, 0] == 127 and mxfp8.e4m3_decode(a[0][2, 0, 0, :1])[0] == 384.0


def test_select_against_a_sort():
    w = np.array([3.0, 1.0, 3.0, np.nan, -0.0, 0.0, 5.0, 2.0, 9.0, 9.0])
    assert oa.select(w, 10, 3) == list(range(10))
    assert oa.select(w, 5, 2) == [0, 2, 6, 8, 9]
    assert oa.select(w, 4, 2) == [0, 6, 8, 9]      # of equal weights the lower position
    assert oa.select(w, 3, 3) == [7, 8, 9]
    assert oa.select(w, 8, 1) == [0, 1, 2, 4, 6, 7, 8, 9]   # -0 is +0: the lower position
    assert oa.select(w, 2, 0) == [8, 9]


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_expert_gb300 as mx
    return mx


def test_argument_checks_return_before_cuda(mx):
    """Statuses of calls that are refused for their arguments alone."""
    L, p = mx.lib, ctypes.c_void_p(256)
    rows = mx.moe_rows(256, 128, 128)
    r = ctypes.byref(rows)
    odd = ctypes.byref(mx.moe_rows(256, 129, 128))
    off = ctypes.byref(mx.moe_rows(264, 128, 128))
    pre = lambda q=r, k=r, v=r, h=4, hk=2, d=128, cq=p, ck=p, n=1, tq=8, tk=8, c=1, s=1.0, o=p: L.moe_attn_prefill(  # noqa: E731
        q, k, v, h, hk, d, cq, ck, n, tq, tk, c, s, o, None, None, None)
    assert pre(q=None) == pre(k=None) == pre(v=None) == pre(cq=None) == pre(ck=None) == pre(o=None) == -1
    assert pre(q=odd) == pre(k=odd) == pre(v=off) == -1
    assert pre(n=-1) == pre(tq=-1) == pre(tk=-1) == pre(c=2) == pre(h=0) == pre(hk=0) == -1
    assert pre(s=math.nan) == pre(s=math.inf) == -1
    assert pre(d=96) == pre(d=256) == pre(h=5) == -2
    assert pre(n=0) == pre(tq=0) == 0      # nothing to do

    good = mx.moe_kv_cache(4, 64, 2, 128, 256, 256, 256, 256)
    c = ctypes.byref(good)
    bad_page, bad_dim = mx.moe_kv_cache(4, 48, 2, 128, 256, 256, 256, 256), mx.moe_kv_cache(4, 64, 2, 96, 256, 256, 256, 256)
    null = mx.moe_kv_cache(4, 64, 2, 128, None, 256, 256, 256)
    app = lambda cc=c, k=r, n=1, t=8, w=4, tab=p, st=p: L.moe_kv_append_fp8(cc, k, r, p, st, n, t, tab, w, None, None)  # noqa: E731
    assert app(cc=None) == app(cc=ctypes.byref(null)) == app(k=None) == app(k=odd) == app(tab=None) == app(st=None) == -1
    assert app(n=-1) == app(t=-1) == app(w=-1) == app(w=1 << 30) == -1
    assert app(cc=ctypes.byref(bad_page)) == app(cc=ctypes.byref(bad_dim)) == -2
    assert app(n=0) == app(t=0) == 0

    dec = lambda cc=c, q=r, h=8, n=1, t=1, ln=p, tab=p, w=4, s=1.0, o=p, wt=None, ws=0, wp=p: L.moe_attn_decode_fp8(  # noqa: E731
        cc, q, h, n, t, ln, tab, w, s, o, None, wt, ws, wp, 1 << 40, None, None)
    assert dec(cc=None) == dec(q=None) == dec(q=odd) == dec(ln=None) == dec(tab=None) == dec(o=None) == dec(wp=None) == -1
    assert dec(n=-1) == dec(t=0) == dec(s=math.nan) == dec(wt=p, ws=-1) == dec(wp=ctypes.c_void_p(16)) == -1
    assert dec(h=7) == dec(t=9) == dec(h=130) == dec(n=4097) == dec(cc=ctypes.byref(bad_dim)) == -2
    assert dec(n=0) == 0
    assert L.moe_attn_decode_workspace_bytes(c, 1, 9, 8, 4, 0) == 0

    ev = lambda cc=c, n=1, keep=64, rec=8, dw=1, w=4, kept=p, nl=p, wt=p, ws=256: L.moe_kv_evict_fp8(  # noqa: E731
        cc, p, w, p, n, wt, ws, keep, rec, p, dw, kept, None, nl, None, None)
    assert ev(cc=None) == ev(keep=0) == ev(rec=-1) == ev(rec=65) == ev(n=-1) == ev(ws=-1) == ev(kept=None) == ev(nl=None) == ev(wt=None) == -1
    assert ev(cc=ctypes.byref(bad_page)) == ev(n=65536) == -2
    assert ev(keep=65) == -5               # the destination's pages hold 64
    assert ev(n=0) == 0


def test_binding_refuses_wrong_tensors(mx):
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        mx.moe_attn_prefill(q, q, q, cu)
    with pytest.raises(TypeError, match="k_codes must be a CUDA tensor"):
        mx.KVCache.alloc(1, 64, 1, 64, device="cpu")


def test_more_rows_than_32_bits_can_step_over_are_refused(mx):
    """The kernels count positions in 32 bits and look a tile past the last one."""
    L, p, most = mx.lib, ctypes.c_void_p(256), 2 ** 31 - 65536
    r = ctypes.byref(mx.moe_rows(256, 128, 128))
    for page in (16, 128):
        cache = mx.moe_kv_cache(4, page, 2, 128, 256, 256, 256, 256)
        c, w = ctypes.byref(cache), most // page + 1
        assert L.moe_kv_append_fp8(c, r, r, p, p, 1, 8, p, w, None, None) == -1
        assert L.moe_attn_decode_fp8(c, r, 8, 1, 1, p, p, w, 1.0, p, None, None, 0, p, 1 << 62, None, None) == -1
        assert L.moe_attn_decode_workspace_bytes(c, 1, 1, 8, w, 0) == 0
        assert L.moe_kv_evict_fp8(c, p, w, p, 1, p, 1 << 40, 64, 8, p, 8, p, None, p, None, None) == -1
        # every table fits, but not the chunks of all sequences in one count
        w = 2 ** 30 // page
        assert L.moe_attn_decode_fp8(c, r, 8, 64, 1, p, p, w, 1.0, p, None, None, 0, p, 1 << 62, None, None) == -2
    assert L.moe_kv_append_fp8(c, r, r, p, p, 1, most + 1, p, 8, None, None) == -2
    for tq, tk in ((8, most + 1), (most + 1, 8)):
        assert L.moe_attn_prefill(r, r, r, 4, 2, 128, p, p, 1, tq, tk, 1, 1.0, p, None, None, None) == -2


def test_eviction_refuses_outputs_that_overlap(mx):
    """Any overlap, not only equal addresses: 2 sequences, 2 heads, keep 8, weights of 64 positions each."""
    c = ctypes.byref(mx.moe_kv_cache(4, 64, 2, 128, 256, 256, 256, 256))
    names = ["table", "lengths", "weights", "dst", "kept", "kept_weights", "new_lengths"]
    size = dict(table=8, lengths=8, weights=2 * 2 * 64 * 4, dst=8, kept=2 * 2 * 8 * 4, kept_weights=2 * 2 * 8 * 4, new_lengths=8)

    def call(**at):
        a = {n: ctypes.c_void_p(at.get(n, 4096 * (i + 1))) for i, n in enumerate(names)}
        return mx.lib.moe_kv_evict_fp8(c, a["table"], 1, a["lengths"], 2, a["weights"], 64, 8, 2, a["dst"], 1, a["kept"],
                                       a["kept_weights"], a["new_lengths"], None, None)

    for out in names[4:]:
        for other in names:
            if other != out:
                base = 1 << 16
                for shift in (0, size[other] - 4, 4 - size[out]):
                    assert call(**{other: base, out: base + shift}) == -1, (out, other, shift)


def test_prompt_refuses_what_its_header_says(mx):
    """Limits of moe_attn_prefill alone: a broadcast token stride, many heads."""
    p, r, one = ctypes.c_void_p(256), ctypes.byref(mx.moe_rows(256, 128, 128)), ctypes.byref(mx.moe_rows(256, 0, 128))
    pre = lambda q=r, k=r, v=r, h=4, tq=8, tk=8: mx.lib.moe_attn_prefill(  # noqa: E731
        q, k, v, h, 1, 128, p, p, 1, tq, tk, 1, 1.0, p, None, None, None)
    assert pre(q=one) == pre(k=one) == pre(v=one) == pre(h=65536) == -2


def test_eviction_refuses_more_places_than_32_bits_can_step_over(mx):
    c = ctypes.byref(mx.moe_kv_cache(4, 64, 2, 128, 256, 256, 256, 256))
    at = [ctypes.c_void_p((i + 1) << 40) for i in range(6)]
    assert mx.lib.moe_kv_evict_fp8(c, at[0], 1, at[1], 1, at[2], 64, 2 ** 31 - 65535, 8, at[3], 1, at[4], None, at[5], None,
                                   None) == -1
