"""The layer routed by groups for one to four tokens: the single launch, and the shapes that it leaves to the per-stage kernels.

Experts and weights are those that moe_route_groups gives for the layer's own logits, bit for bit. Outputs of the single
launch and of the per-stage kernels are each within 5e-3 (relative L2) of the exact ones, so within 1e-2 of one another.
"""
import pytest
import torch

import workloads as wl
from mxfp4_expert_gb300 import synthetic

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


@pytest.fixture(scope="module")
def layers():
    made = {}

    def get(E):
        if E not in made:
            w = wl.get("tiny", E=E, k=8)
            made[E] = (w, synthetic.build_layer(w, 0))
        return made[E]
    return get


def _routed(mx, w, layer, x, bias, **rule):
    T = x.shape[0]
    logits = torch.empty((T, w.E), device="cuda")
    idx, wts = torch.empty((T, w.k), dtype=torch.int32, device="cuda"), torch.empty((T, w.k), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mx.moe_forward_groups(layer, x, bias, logits_out=logits, idx_out=idx, w_out=wts, dev_status=status, **rule)
    assert int(status) == 0
    want = mx.moe_route_groups(logits, w.k, bias, **rule)
    assert torch.equal(idx, want[0]) and torch.equal(wts, want[1])
    return y, idx


RULES = [(512, dict(n_groups=8, top_groups=4, scale=2.5)), (512, dict(n_groups=1, group_best=1, score="softmax")),
         (512, dict(n_groups=16, top_groups=11, score="softmax", renormalise=False)), (512, dict(n_groups=32, top_groups=3)),
         (96, dict(n_groups=12, top_groups=5)), (480, dict(n_groups=20, top_groups=7)), (33, dict(n_groups=3, top_groups=2))]


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("E,rule", RULES)
def test_few_tokens(mx, layers, E, rule, T):
    w, layer = layers(E)
    g = torch.Generator(device="cuda").manual_seed(10 * T + E)
    x = torch.randn((8, w.d), generator=g, device="cuda").to(BF16)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    few, idx = _routed(mx, w, layer, x[:T].contiguous(), bias, **rule)
    many, idx8 = _routed(mx, w, layer, x, bias, **rule)        # per-stage kernels
    same = (idx == idx8[:T]).all(1)     # logits differ by roundings: a token may route otherwise
    assert same.float().mean() >= 0.5
    a, b = few[same].double(), many[:T][same].double()
    assert (a - b).norm() <= 1e-2 * b.norm()


def test_keys_that_fp32_cannot_tell_apart(mx, layers):
    """A bias that makes nearly all keys equal: the selection ranks by pairs inside the launch, too."""
    w, layer = layers(512)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, w.d), generator=g, device="cuda").to(BF16)
    logits = torch.empty((1, 512), device="cuda")
    mx.moe_forward_groups(layer, x, logits_out=logits)
    for score in ("sigmoid", "softmax"):
        s = torch.sigmoid(logits[0].double()) if score == "sigmoid" else torch.softmax(logits[0].double(), 0)
        bias = (0.75 - s).float()
        _routed(mx, w, layer, x, bias, score=score)
        _routed(mx, w, layer, x, bias, score=score, n_groups=8, top_groups=2)


def test_special_biases(mx, layers):
    w, layer = layers(512)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((3, w.d), generator=g, device="cuda").to(BF16)
    bias = torch.randn(512, generator=g, device="cuda") * 0.1
    bias[3], bias[100], bias[400] = float("-inf"), float("nan"), 1e30
    _routed(mx, w, layer, x, bias, n_groups=8, top_groups=3)


def test_calls_of_both_kinds_take_turns(mx, layers):
    """One workspace, whose counters every launch leaves as it found them; captured and replayed as well."""
    w, layer = layers(512)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((2, w.d), generator=g, device="cuda").to(BF16)
    rule = dict(n_groups=8, top_groups=4)
    want = mx.moe_forward(layer, x), mx.moe_forward_groups(layer, x, **rule)
    ws = torch.zeros(layer.workspace_bytes(2), dtype=torch.uint8, device="cuda")

    def pair(y):
        mx.moe_forward(layer, x, y=y[0], workspace=ws)
        mx.moe_forward_groups(layer, x, y=y[1], workspace=ws, **rule)
    ys = [(torch.empty_like(x), torch.empty_like(x)) for _ in range(4)]
    for y in ys:
        pair(y)
    assert all(torch.equal(a, b) for y in ys for a, b in zip(y, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for y in ys:
            pair(y)
    for _ in range(3):
        for y in ys:
            for t in y:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for y in ys for a, b in zip(y, want))
