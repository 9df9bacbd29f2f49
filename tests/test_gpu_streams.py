"""Calls on a stream of the caller's, with outputs and workspaces that they allocate themselves.

The current stream is kept busy meanwhile: what a call allocates must neither
wait for that stream's work nor be overwritten by it.
"""
import math

import pytest
import torch

import workloads as wl
from test_gpu_attention import _bf16, _cu, _filled, _gen, _i32, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _busy():
    torch.cuda._sleep(200_000_000)   # cycles: about a tenth of a second


def _beside_earlier_work(call, like):
    """call(stream)'s results, while freed tensors of the shapes and types `like` are still to be written."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in like]
    torch.cuda.synchronize()
    _busy()
    for t in old:
        t.fill_(7)
    del old, t
    got = call(s)
    torch.cuda.synchronize()
    return got


def test_decode_workspace_is_zeroed_on_the_launch_stream(mx):
    s = torch.cuda.Stream()
    c, table = _filled(mx, [700, 90], 16, 2, 64, 44, 3)
    q, ln = _bf16(_gen(95), 2, 1, 8, 64), _i32([700, 90])
    want = mx.moe_attn_decode_fp8(c.gpu, q, ln, table)
    n = mx.moe_attn_decode_workspace_bytes(c.gpu, 2, 1, 8, 44, False)
    junk = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # what the allocator may hand out again
    out = torch.full_like(q, math.nan)
    torch.cuda.synchronize()
    del junk
    _busy()
    mx.moe_attn_decode_fp8(c.gpu, q, ln, table, out=out, stream=s)
    with torch.cuda.stream(s):
        got = out.clone()
    s.synchronize()
    assert torch.equal(got, want)


def test_forward_workspace_is_zeroed_on_the_launch_stream(mx):
    s = torch.cuda.Stream()
    from mxfp4_expert_gb300 import synthetic
    layer = synthetic.build_layer(wl.get("tiny"), 0)
    x = _bf16(_gen(1), 2, layer.d)
    want = mx.moe_forward(layer, x)
    y = torch.full_like(x, math.nan)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    _busy()
    mx.moe_forward(layer, x, y=y, dev_status=status, stream=s)
    with torch.cuda.stream(s):
        got = y.clone()
    s.synchronize()
    assert torch.equal(got, want) and int(status) == 0


def test_attention_outputs(mx):
    g = _gen(96)
    q, k, v, cu = _bf16(g, 300, 4, 64), _bf16(g, 300, 2, 64), _bf16(g, 300, 2, 64), _cu([300])
    want = mx.moe_attn_prefill(q, k, v, cu)
    assert torch.equal(_beside_earlier_work(lambda s: mx.moe_attn_prefill(q, k, v, cu, stream=s), [want]), want)
    c, table = _filled(mx, [700, 90], 16, 2, 64, 44, 3)
    q, ln = _bf16(g, 2, 1, 8, 64), _i32([700, 90])
    want = mx.moe_attn_decode_fp8(c.gpu, q, ln, table)
    assert torch.equal(_beside_earlier_work(lambda s: mx.moe_attn_decode_fp8(c.gpu, q, ln, table, stream=s), [want]), want)


def test_eviction_outputs(mx):
    c, tables = _filled(mx, [300, 90], 16, 2, 64, 40, 3)
    table, dst = tables[:, :20].contiguous(), tables[:, 20:].contiguous()
    w, ln = _weights(5, 2, 2, 320), _i32([300, 90])
    want = mx.moe_kv_evict_fp8(c.gpu, table, ln, w, 64, 5, dst)
    got = _beside_earlier_work(lambda s: mx.moe_kv_evict_fp8(c.gpu, table, ln, w, 64, 5, dst, stream=s), want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layer_outputs(mx):
    g = _gen(97)
    from mxfp4_expert_gb300 import synthetic
    layer = synthetic.build_layer(wl.get("tiny"), 0)
    x, logits = _bf16(g, 40, layer.d), torch.randn((40, 64), generator=g, device="cuda")
    want = mx.moe_forward(layer, x)
    assert torch.equal(_beside_earlier_work(lambda s: mx.moe_forward(layer, x, stream=s), [want]), want)
    want = mx.moe_route_topk(logits, 4)
    got = _beside_earlier_work(lambda s: mx.moe_route_topk(logits, 4, stream=s), want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ids = want[0]
    want = mx.moe_sort_by_expert(ids, 64)
    got = _beside_earlier_work(lambda s: mx.moe_sort_by_expert(ids, 64, stream=s), want.values())
    n = int(want["n_active"])
    assert all(torch.equal(got[k][:n], want[k][:n]) if k == "active" else torch.equal(got[k], want[k]) for k in want)
    want = mx.moe_quant_mxfp8(x)
    got = _beside_earlier_work(lambda s: mx.moe_quant_mxfp8(x, stream=s), want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
