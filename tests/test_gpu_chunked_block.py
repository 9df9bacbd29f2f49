"""The example that takes prompts in chunks, on the GPU: norms, rotation, attention of chunks, groups and evictions together.

The operators have their own tests; here every call of a run is checked against 64 bits with what the calls before it left.
"""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import block as ob
from test_gpu_block import _near, _np

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import chunked_block
    finally:
        sys.path.pop(0)
    return chunked_block


def _decoded(cache, which, pages, h):
    """fp64 values of the pages of one head, and half the smallest step of each page: positions in a row."""
    codes, scales = getattr(cache, which + "_codes"), getattr(cache, which + "_scales")
    step = torch.exp2(scales[pages, h].double() - 127)[:, None, None]
    return (codes[pages, h].view(torch.float8_e4m3fn).double() * step).flatten(0, 1), (
        step * 2.0 ** -10).expand(-1, cache.page_size, 1).flatten(0, 1)


class _Checked:
    """The library's calls of the example, each compared with 64 bits as it is made."""

    def __init__(self, mx, monkeypatch):
        self.mx, self.calls = mx, {}
        for name in ("moe_block_norm", "moe_kv_append_rope_fp8", "moe_attn_chunk_fp8", "moe_attn_decode_fp8",
                     "moe_forward_groups"):
            monkeypatch.setattr(mx, name, self._wrap(name, getattr(mx, name)))

    def _wrap(self, name, call):
        check = getattr(self, name)

        def run(*args, **kw):
            self.calls[name] = self.calls.get(name, 0) + 1
            return check(call, *args, **kw)
        return run

    def moe_block_norm(self, call, x, a=None, **kw):
        ref = ob.block_norm(_np(x), _np(a), _np(kw.get("post_weight")), _np(kw.get("gate")), kw.get("residual_scale", 1.0),
                            _np(kw.get("pre_weight")), 1e-6)
        before = x.clone()
        y, h = call(x, a, **kw)
        _near(y, h, before, ref, 1e-6)
        return y, h

    def moe_kv_append_rope_fp8(self, call, cache, k, v, cu, start, table, f, q, rope_start, dev_status):
        out = call(cache, k, v, cu, start, table, f, q=q, rope_start=rope_start, dev_status=dev_status)
        rows = cu.tolist()
        for b, (t0, t1) in enumerate(zip(rows, rows[1:])):
            pos, at = int(rope_start[b]) + np.arange(t1 - t0), int(start[b])
            kr, qr = (ob.rotate(_np(t[t0:t1]), pos, _np(f), False) for t in (k, q))
            ks, qs = (ob.pair_size(_np(t[t0:t1]), 2 * len(f), False) for t in (k, q))
            assert np.all(np.abs(_np(out[t0:t1]) - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -22 * qs)
            for h in range(cache.n_kv_heads):
                # a code is off by half a step: 2^-4 of it, or half of the smallest code's step
                for which, ref, slack in (("k", kr, ks), ("v", _np(v[t0:t1]), 0 * ks)):
                    got, half = _decoded(cache, which, table[b].long(), h)
                    got, half = _np(got[at:at + t1 - t0]), _np(half[at:at + t1 - t0])
                    bound = 2.0 ** -4 * np.abs(ref[:, h]) + half + 2.0 ** -21 * slack[:, h]
                    assert np.all(np.abs(got - ref[:, h]) <= bound)
        return out

    def _attention(self, cache, q, cu, lengths, table, out):
        rows, group = cu.tolist(), q.shape[1] // cache.n_kv_heads
        for b, (t0, t1) in enumerate(zip(rows, rows[1:])):
            n = int(lengths[b])
            seen = torch.arange(n, device="cuda") <= (n - (t1 - t0) + torch.arange(t1 - t0, device="cuda"))[:, None]
            for h in range(cache.n_kv_heads):
                k, v = (_decoded(cache, w, table[b].long(), h)[0][:n] for w in "kv")
                for i in range(h * group, (h + 1) * group):
                    s = (q[t0:t1, i].double() @ k.T) * q.shape[2] ** -0.5
                    ref = torch.softmax(s.masked_fill(~seen, float("-inf")), -1) @ v
                    # a bf16 result (2^-8), f16 probabilities and their sum (2^-10) and scores that err by 2^-16 of their
                    # size, in a probability and in the sum: all relative to at most max |v|
                    size = (q[t0:t1, i].double().abs() @ k.abs().T).max() * q.shape[2] ** -0.5
                    bound = v.abs().max() * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -15 * (1 + size))
                    assert (out[t0:t1, i].double() - ref).abs().max() <= bound

    def moe_attn_chunk_fp8(self, call, cache, q, cu, lengths, table, **kw):
        out = call(cache, q, cu, lengths, table, **kw)
        self._attention(cache, q, cu, lengths, table, out)
        return out

    def moe_attn_decode_fp8(self, call, cache, q, lengths, table, **kw):
        out = call(cache, q, lengths, table, **kw)
        cu = torch.arange(q.shape[0] + 1)
        self._attention(cache, q[:, 0], cu, lengths, table, out[:, 0])
        return out

    def moe_forward_groups(self, call, layer, x, bias, dev_status, **rule):
        E, k = layer.shape.n_experts, layer.shape.top_k
        logits = torch.empty((x.shape[0], E), device="cuda")
        idx, w = torch.empty((x.shape[0], k), dtype=torch.int32, device="cuda"), torch.empty((x.shape[0], k), device="cuda")
        y = call(layer, x, bias, dev_status=dev_status, logits_out=logits, idx_out=idx, w_out=w, **rule)
        # the weights of the selected, from the layer's logits; which are selected is the routing tests' part
        s = 1 / (1 + np.exp(-_np(logits)))
        s = np.take_along_axis(s, idx.cpu().numpy().astype(np.int64), 1)
        ref = rule["scale"] * s / s.sum(1, keepdims=True)
        assert np.all(np.abs(_np(w) - ref) <= 2.0 ** -18 * ref)
        groups = idx.cpu().numpy() // (E // rule["n_groups"])
        assert all(len(set(g)) <= rule["top_groups"] for g in groups.tolist())
        return y


@pytest.mark.parametrize("hd,page", [(64, 16), (128, 64)])
def test_every_call_of_a_run(example, monkeypatch, hd, page):
    mx = _Checked(example.mx, monkeypatch)
    prompts, steps, chunk = [150, 1, 70, 37], 16, 32
    block, y, evictions = example.run(prompts, steps, chunk, keep=24, limit=153, head_dim=hd, page_size=page)
    assert int(block.status) == 0 and torch.isfinite(y).all() and evictions >= 1
    taken = [n + steps - -(-n // chunk) for n in prompts]   # a step for each chunk, one token in each of the others
    assert block.positions.tolist() == taken
    assert all(n <= m for n, m in zip(block.lengths.tolist(), taken)) and block.lengths[0] < block.positions[0]
    assert mx.calls["moe_attn_chunk_fp8"] == 5 and mx.calls["moe_attn_decode_fp8"] == steps - 5
    assert mx.calls["moe_block_norm"] == 3 * steps and mx.calls["moe_forward_groups"] == steps


def test_equal_runs_give_equal_bits(example):
    a = example.run([90, 9, 131], 24, 64, keep=32, limit=140)
    b = example.run([90, 9, 131], 24, 64, keep=32, limit=140)
    assert a[2] == b[2] >= 1
    assert torch.equal(a[1], b[1]) and torch.equal(a[0].positions, b[0].positions)


@pytest.mark.parametrize("new,decoding", [([1, 1, 1], True), ([40, 1, 7], False)])
def test_steps_replayed_from_a_graph(example, new, decoding):
    wl = example.wl
    gen = torch.Generator(device="cuda").manual_seed(5)
    cu = torch.tensor([0, *new], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    eager, replayed = (example.ChunkedBlock(wl.get("tiny"), 8, 2, 64, 3, 400) for _ in range(2))
    xs = torch.randn((6, sum(new), eager.d), generator=gen, device="cuda")
    want = [eager.forward(x, cu, decoding).clone() for x in xs]
    buffer = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = replayed.forward(buffer, cu, decoding)
    for x, y in zip(xs, want):
        buffer.copy_(x)
        graph.replay()
        assert torch.equal(got, y)
    assert int(replayed.status) == 0
    assert torch.equal(replayed.lengths, eager.lengths) and torch.equal(replayed.positions, eager.positions)
