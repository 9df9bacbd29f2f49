"""The rest of a block on a caller's stream with outputs that the calls allocate, and captured into a graph."""
import pytest
import torch

from test_gpu_attention import _bf16, _cu, _filled, _gen, _i32
from test_gpu_streams import _beside_earlier_work

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


def _equal(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_outputs_allocated_for_the_callers_stream(mx):
    g = _gen(1)
    x, a = _bf16(g, 300, 512), _bf16(g, 300, 512)
    want = mx.moe_block_norm(x, a, post_weight=a[0], pre_weight=x[0])
    got = _beside_earlier_work(lambda s: mx.moe_block_norm(x, a, post_weight=a[0], pre_weight=x[0], stream=s), want)
    assert all(_equal(p, q) for p, q in zip(got, want))
    logits = torch.randn((300, 64), generator=g, device="cuda")
    want = mx.moe_route_groups(logits, 4, n_groups=4, top_groups=2)
    got = _beside_earlier_work(lambda s: mx.moe_route_groups(logits, 4, n_groups=4, top_groups=2, stream=s), want)
    assert all(_equal(p, q) for p, q in zip(got, want))


def test_attention_outputs_and_workspaces(mx):
    g = _gen(2)
    c, table = _filled(mx, [700, 90], 16, 2, 64, 44, 3)
    q, cu, ln = _bf16(g, 150, 8, 64), _cu([90, 60]), _i32([700, 90])
    want = mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table)
    ws = torch.empty(mx.moe_attn_chunk_workspace_bytes(c.gpu, 8, 150, 2), dtype=torch.uint8, device="cuda")
    got = _beside_earlier_work(lambda s: mx.moe_attn_chunk_fp8(c.gpu, q, cu, ln, table, stream=s), [want, ws])
    assert _equal(got, want)
    k, f = _bf16(g, 20, 2, 64), torch.rand(16, generator=g, device="cuda")
    qs, table, at = q[:20], table[:, :8].contiguous(), _i32([0, 0])   # an append from position 0 gives the same cache again
    want = mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu([15, 5]), at, table, f, q=qs)
    codes, scales = c.gpu.k_codes.clone(), c.gpu.k_scales.clone()
    got = _beside_earlier_work(lambda s: mx.moe_kv_append_rope_fp8(c.gpu, k, k, _cu([15, 5]), at, table, f, q=qs, stream=s),
                               [want])
    assert _equal(got, want) and torch.equal(c.gpu.k_codes, codes) and torch.equal(c.gpu.k_scales, scales)


def test_layer_by_groups(mx):
    import workloads as wl
    from mxfp4_expert_gb300 import synthetic
    layer = synthetic.build_layer(wl.get("tiny"), 0)
    x = _bf16(_gen(3), 40, layer.d)
    kw = dict(n_groups=4, top_groups=2)
    want = mx.moe_forward_groups(layer, x, **kw)
    ws = torch.empty(layer.workspace_bytes(40), dtype=torch.uint8, device="cuda")
    assert _equal(_beside_earlier_work(lambda s: mx.moe_forward_groups(layer, x, stream=s, **kw), [want, ws]), want)


def test_two_streams_at_once(mx):
    """Calls that share inputs only, at the same time."""
    g = _gen(4)
    x, a, w = _bf16(g, 2000, 1024), _bf16(g, 2000, 1024), _bf16(g, 1024)
    logits = torch.randn((3000, 256), generator=g, device="cuda")
    norm = lambda s: mx.moe_block_norm(x, a, post_weight=w, pre_weight=w, stream=s)  # noqa: E731
    route = lambda s: mx.moe_route_groups(logits, 8, n_groups=8, top_groups=4, stream=s)  # noqa: E731
    want = [*norm(None), *route(None)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[*norm(s), *route(s)] for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(_equal(p, q) for one in got for p, q in zip(one, want))


def test_replayed_with_other_contents(mx):
    """Captured calls read shapes from their arguments and everything else from memory."""
    g = _gen(5)
    x, a, logits = _bf16(g, 33, 256), _bf16(g, 33, 256), torch.randn((33, 96), generator=g, device="cuda")
    c, table = _filled(mx, [200, 40], 16, 2, 64, 16, 3)
    k, q, f = _bf16(g, 9, 2, 64), _bf16(g, 9, 4, 64), torch.rand(32, generator=g, device="cuda")
    cu, start = _cu([5, 4]), _i32([0, 16])

    def calls():
        y, h = mx.moe_block_norm(x, a, post_weight=a[0], pre_weight=a[1])
        return [y, h, *mx.moe_route_groups(logits, 6, n_groups=4, top_groups=2),
                mx.moe_kv_append_rope_fp8(c.gpu, k, k, cu, start, table, f, q=q)]
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for lens, at in (([5, 4], [0, 16]), ([9, 0], [32, 0]), ([1, 3], [48, 64])):
        cu.copy_(_cu(lens))
        start.copy_(_i32(at))
        for t in (x, a, logits, k, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        once = [t.clone() for t in got]
        codes, scales, n = c.gpu.k_codes.clone(), c.gpu.k_scales.clone(), sum(lens)
        want = calls()
        assert all(_equal(p, w) for p, w in zip(once[:4], want[:4])) and _equal(once[4][:n], want[4][:n])
        assert torch.equal(c.gpu.k_codes, codes) and torch.equal(c.gpu.k_scales, scales)
