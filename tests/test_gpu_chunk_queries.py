"""Attention of chunks over the cache for queries that are not finite: every row that sees a position then is not finite
either, whatever the keys' signs are, and a row that sees none stays zero.
"""
import math

import pytest
import torch

from test_gpu_attention import _Cache, _bf16, _cu, _gen, _i32, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _signed(mx, lens, P, H, d, sign, channel=5):
    """A cache whose keys have one sign in a channel."""
    width = max(-(-n // P) for n in lens)
    c, table = _Cache(mx, len(lens) * width, P, H, d), _tables(len(lens), width)
    k, v = (_bf16(_gen(i), sum(lens), H, d) for i in (1, 2))
    k[..., channel] = sign * (k[..., channel].abs() + 1)
    mx.moe_kv_append_fp8(c.gpu, k, v, _cu(lens), _i32([0] * len(lens)), table)
    return c.gpu, table


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 128)])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([4, 2], [4, 2]), ([200, 70], [900, 300]), ([3], [20000]), ([300], [100])])
def test_keys_of_one_sign(mx, bad, sign, P, d, new, lens):
    cache, table = _signed(mx, [max(a, b) for a, b in zip(new, lens)], P, 2, d, sign)
    total, hq = sum(new), 8
    q = _bf16(_gen(3), total, hq, d)
    args = (_cu(new), _i32(lens), table)
    want, lse = torch.empty_like(q), torch.empty((total, hq), device="cuda")
    mx.moe_attn_chunk_fp8(cache, q, *args, out=want, lse=lse)
    q2, lse2 = q.clone(), torch.empty_like(lse)
    hit = torch.zeros((total, hq), dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (0, 7), (total // 2, 3), (total - 1, 4)):
        hit[t, h] = True
    q2[..., 5][hit] = bad
    got = mx.moe_attn_chunk_fp8(cache, q2, *args, lse=lse2)
    sees = hit & ~torch.isneginf(lse)
    blind = hit & torch.isneginf(lse)
    assert sees.any() and not torch.isfinite(got[sees].float()).any() and torch.isnan(lse2[sees]).all()
    assert not got[blind].any() and torch.isneginf(lse2[blind]).all()
    assert torch.equal(got[~hit].view(torch.int16), want[~hit].view(torch.int16)) and torch.equal(lse2[~hit], lse[~hit])


def test_pages_outside_the_cache(mx):
    """Positions of such pages are masked for these queries, too."""
    cache, table = _signed(mx, [48], 16, 1, 64, -1.0)
    q = _bf16(_gen(4), 2, 2, 64)
    q[:, 0, 5] = math.inf
    none, some = torch.full_like(table, -1), table.clone()
    some[0, 1:] = -1
    for t, blind in ((none, True), (some, False)):
        lse = torch.empty((2, 2), device="cuda")
        out = mx.moe_attn_chunk_fp8(cache, q, _cu([2]), _i32([48]), t, lse=lse)
        if blind:
            assert not out.any() and torch.isneginf(lse).all()
        else:
            assert torch.isnan(out[:, 0]).all() and torch.isfinite(out[:, 1].float()).all()
