"""The example block on the GPU: the attention operators and the expert layer, run together.

The operators have their own tests; here their states have to fit together over
prompts, steps and evictions.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_block
    finally:
        sys.path.pop(0)
    return decoder_block


def _values(block, b, h):
    """fp64 keys and values of one sequence and head, read back from the cache."""
    n = int(block.lengths[b])
    pages = block.tables[0][b].long()
    out = []
    for codes, scales in ((block.cache.k_codes, block.cache.k_scales), (block.cache.v_codes, block.cache.v_scales)):
        c = codes[pages, h].view(torch.float8_e4m3fn).double()
        c = c * torch.exp2(scales[pages, h].double() - 127)[:, None, None]
        out.append(c.flatten(0, 1)[:n])
    return out


def test_without_eviction_the_weights_sum_to_the_query_heads(example):
    steps = 9
    block, x, evictions = example.run([33, 5], steps, keep=64, limit=200)
    assert evictions == 0 and int(block.status) == 0
    assert block.lengths.tolist() == [33 + steps, 5 + steps]
    assert torch.isfinite(x.float()).all()
    # every step adds probabilities that sum to 1 for each of the group's query heads: fp32 sums of
    # steps * group terms near 1, each of at most 42 products, stay within 42 * 2^-23 of it
    group = block.n_heads // block.n_kv
    total = block.weights.double().sum(-1)
    assert (total / (steps * group) - 1).abs().max() < 2e-5
    for b in range(2):
        assert not block.weights[b, :, int(block.lengths[b]):].any()


@pytest.mark.parametrize("prompts,steps,keep,limit", [([150, 40, 1], 40, 32, 47), ([65], 70, 64, 64)])
def test_evictions_keep_the_newest_and_leave_a_cache_that_serves(example, prompts, steps, keep, limit):
    block, x, evictions = example.run(prompts, steps, keep, limit)
    assert evictions >= 2 and int(block.status) == 0
    assert torch.isfinite(x.float()).all()
    # one more step, its attention recomputed in 64 bits from the cache's own values
    q = torch.randn((len(prompts), 1, block.n_heads, block.hd), device="cuda").to(torch.bfloat16)
    got = example.mx.moe_attn_decode_fp8(block.cache, q, block.lengths, block.tables[0]).double()
    group = block.n_heads // block.n_kv
    for b in range(len(prompts)):
        for h in range(block.n_kv):
            k, v = _values(block, b, h)
            for i in range(h * group, (h + 1) * group):
                p = torch.softmax(k @ q[b, 0, i].double() * block.hd ** -0.5, 0)
                # f16 probabilities (2^-11) and a bf16 result (2^-8), both relative to at most max |v|
                assert (got[b, 0, i] - p @ v).abs().max() <= v.abs().max() * (2.0 ** -8 + 2.0 ** -10)
    # an eviction's result: ascending positions that end with the newest ones, weights that follow them
    before = block.lengths.tolist()
    old = block.weights.clone()
    kept = block.evict(8, recent=3).cpu()
    for b, n in enumerate(before):
        m = min(n, 8)
        for h in range(block.n_kv):
            row = kept[b, h]
            assert (row[1:m] > row[:m - 1]).all() and (row[m:] == -1).all()
            assert row[m - min(m, 3):m].tolist() == list(range(n - min(m, 3), n))
            assert torch.equal(block.weights[b, h, :m], old[b, h, row[:m].long().cuda()])
            assert not block.weights[b, h, m:].any()
        assert int(block.lengths[b]) == m


def test_equal_runs_give_equal_bits(example):
    a = example.run([70, 9, 31], 24, keep=32, limit=64)
    b = example.run([70, 9, 31], 24, keep=32, limit=64)
    assert torch.equal(a[1], b[1]) and torch.equal(a[0].lengths, b[0].lengths)
