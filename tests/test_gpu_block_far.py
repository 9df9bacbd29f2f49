"""The rest of a block at addresses far apart, with pages that sequences share, and with queries that are not finite.

Everything is compared bit for bit with the same call on tensors that lie close together.
"""
import math

import pytest
import torch

from test_gpu_attention import _bf16, _cu, _filled, _gen, _i32

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
FAR = 2 ** 28   # elements: ten rows pass 2^32 bytes


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _spread(t, stride=FAR):
    """The same values with rows that far apart."""
    big = torch.empty((t.shape[0] - 1) * stride + t[0].numel(), dtype=t.dtype, device="cuda")
    v = big.as_strided(t.shape, (stride, *t[0].contiguous().stride()))
    v.copy_(t)
    return v


def test_norm_of_rows_far_apart(mx):
    g = _gen(1)
    x, a, w = _bf16(g, 11, 256), _bf16(g, 11, 256), _bf16(g, 256)
    y, h = mx.moe_block_norm(x, a, post_weight=w, pre_weight=w)
    far = _spread(x)
    y2, h2 = mx.moe_block_norm(far, _spread(a), post_weight=w, pre_weight=w, y=far, h=_spread(a))
    assert _equal(y2, y) and _equal(h2, h)


def test_queries_far_apart(mx):
    c, table = _filled(mx, [700, 90], 16, 2, 64, 44, 3)
    q, cu, ln = _bf16(_gen(2), 11, 8, 64), _cu([8, 3]), _i32([700, 90])
    want = mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table)
    assert _equal(mx.moe_attn_chunk_fp8(c.gpu, _spread(q), cu, ln, table), want)
    f, k = torch.rand(32, generator=_gen(3), device="cuda"), _bf16(_gen(4), 11, 2, 64)
    small = mx.KVCache.alloc(8, 16, 2, 64)
    pages = _i32([[1, 2], [5, 6]])
    want = mx.moe_kv_append_rope_fp8(small, k, k, cu, _i32([0, 16]), pages, f, q=q)
    other = mx.KVCache.alloc(8, 16, 2, 64)
    for t in (*_fields(small), *_fields(other)):
        t.zero_()
    mx.moe_kv_append_rope_fp8(small, k, k, cu, _i32([0, 16]), pages, f, q=q)
    got = mx.moe_kv_append_rope_fp8(other, _spread(k), _spread(k), cu, _i32([0, 16]), pages, f, q=_spread(q))
    assert _equal(got, want) and all(_equal(a, b) for a, b in zip(_fields(small), _fields(other)))


def _fields(c):
    return c.k_codes, c.v_codes, c.k_scales, c.v_scales


@pytest.mark.parametrize("few", [False, True])
def test_pages_beyond_32_bits(mx, few):
    """Codes of the last pages lie past 2^32 bytes (one page of all heads has 2^17)."""
    n, P, H, D = 33000, 128, 8, 128
    g = _gen(5)
    lens = [1, 1] if few else [300, 140]
    total = sum(lens)
    k, v, q = _bf16(g, total, H, D), _bf16(g, total, H, D), _bf16(g, total, 16, D)
    f = torch.rand(64, generator=g, device="cuda")
    big, small = mx.KVCache.alloc(n, P, H, D), mx.KVCache.alloc(6, P, H, D)
    far, near = _i32([[n - 1, n - 3, n - 2], [n - 200, n - 5, n - 4]]), _i32([[0, 1, 2], [3, 4, 5]])
    outs = []
    for c, table in ((big, far), (small, near)):
        for t in _fields(c):
            t[table.flatten().long()] = 0
        cu, start = _cu(lens), _i32([0, 128])
        q_out = mx.moe_kv_append_rope_fp8(c, k, v, cu, start, table, f, q=q)
        ln = _i32([a + b for a, b in zip(lens, [0, 128])])
        outs.append([q_out, mx.moe_attn_chunk_fp8(c, q_out, cu, ln, table), *(t[table.flatten().long()] for t in _fields(c))])
    assert all(_equal(a, b) for a, b in zip(*outs))
    assert outs[0][1].float().abs().max() > 0


def test_sequences_that_share_pages(mx):
    """A cached prefix that two sequences see is read by both."""
    c, table = _filled(mx, [700, 700], 16, 2, 64, 44, 3)
    q = _bf16(_gen(6), 60, 8, 64)
    shared = table.clone()
    shared[1, :30] = table[0, :30]
    got = mx.moe_attn_chunk_fp8(c.gpu, q, _cu([30, 30]), _i32([700, 600]), shared)
    first = mx.moe_attn_chunk_fp8(c.gpu, q[:30], _cu([30]), _i32([700]), shared[:1].contiguous())
    second = mx.moe_attn_chunk_fp8(c.gpu, q[30:], _cu([30]), _i32([600]), shared[1:].contiguous())
    # cuts differ with the batch: f16 probabilities (2^-11) and bf16 results (2^-8) of at most max |v|
    top = 448 * 2.0 ** (int(c.scales["v"].max()) - 127)
    assert (got.float() - torch.cat([first, second]).float()).abs().max() <= top * 2.0 ** -7


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_queries_that_are_not_finite_reach_their_own_rows_only(mx, bad):
    c, table = _filled(mx, [900, 300], 64, 2, 128, 16, 3)
    q = _bf16(_gen(7), 300, 8, 128)
    cu, ln = _cu([200, 100]), _i32([900, 300])
    want, lse = torch.empty_like(q), torch.empty((300, 8), device="cuda")
    mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table, out=want, lse=lse)
    q2, lse2 = q.clone(), torch.empty_like(lse)
    rows = [(0, 0), (77, 3), (199, 7), (250, 4)]
    for t, h in rows:
        q2[t, h, 5] = bad
    got = mx.moe_attn_chunk_fp8(c.gpu, q2, cu, ln, table, lse=lse2)
    keep = torch.ones((300, 8), dtype=torch.bool, device="cuda")
    for t, h in rows:
        keep[t, h] = False
        assert not torch.isfinite(got[t, h].float()).any()
    assert _equal(got[keep], want[keep]) and _equal(lse2[keep], lse[keep])
