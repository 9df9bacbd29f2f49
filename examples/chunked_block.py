"""One decoder block that takes long prompts in chunks beside the sequences that already decode.

    python examples/chunked_block.py [--prompts 700 3 260] [--steps 64] [--chunk 128] [--keep 128] [--limit 320]

Each step takes the next --chunk tokens of every prompt that is not through yet
and one token of every other sequence, packed one after another:
moe_block_norm, the projection, moe_kv_append_rope_fp8 (rotation of keys and
queries, keys and values into the paged FP8 cache), moe_attn_chunk_fp8,
moe_block_norm with the gated residual sum and the norm of the experts' input,
moe_forward_groups, and the residual sum behind it. Once every sequence decodes,
moe_attn_decode_fp8 takes the place of moe_attn_chunk_fp8 and sums the
probabilities that moe_kv_evict_fp8 ranks; positions then run ahead of the
cache's lengths (rope_start). The residual stream is fp32.

Weights and inputs are random. The projections are torch products, as a caller
would have them.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from decoder_block import DecoderBlock, mx, wl  # noqa: E402


class ChunkedBlock(DecoderBlock):
    """The block with norms on both sides of its halves, rotated positions and experts routed by groups."""

    def __init__(self, *args, n_groups: int = 8, top_groups: int = 4, residual_scale: float = 0.5, **kw):
        super().__init__(*args, **kw)
        device = self.w_qkv.device
        gen = torch.Generator(device=device).manual_seed(kw.get("seed", 0) + 17)
        d = self.d

        def near_one(*shape):
            return (1 + 0.1 * torch.randn(shape, generator=gen, device=device)).to(torch.bfloat16)

        self.norm_in, self.norm_attn, self.norm_mid, self.norm_out = (near_one(d) for _ in range(4))
        self.gate = near_one(d)
        self.bias = 0.01 * torch.randn(self.layer.shape.n_experts, generator=gen, device=device)
        self.residual_scale = residual_scale
        self.rule = dict(n_groups=n_groups, top_groups=top_groups, scale=2.5)
        self.inv_freq = 10000.0 ** (-torch.arange(0, self.hd, 2, device=device, dtype=torch.float32) / self.hd)
        self.positions = torch.zeros_like(self.lengths)   # tokens taken; lengths counts those still in the cache

    def forward(self, x, cu, decoding: bool):
        """x fp32 [total, d]: the new tokens of every sequence, cu int32 [n_seq + 1]; decoding: one of each."""
        _, h = mx.moe_block_norm(x, pre_weight=self.norm_in)
        q, k, v = (h @ self.w_qkv).view(x.shape[0], -1, self.hd).split((self.n_heads, self.n_kv, self.n_kv), dim=1)
        q = mx.moe_kv_append_rope_fp8(self.cache, k, v, cu, self.lengths, self.tables[0], self.inv_freq, q=q,
                                      rope_start=self.positions, dev_status=self.status)
        new = cu[1:] - cu[:-1]
        self.lengths += new
        self.positions += new
        if decoding:
            attn = mx.moe_attn_decode_fp8(self.cache, q.unsqueeze(1), self.lengths, self.tables[0],
                                          weights=self.weights, workspace=self.workspace, dev_status=self.status)
        else:
            attn = mx.moe_attn_chunk_fp8(self.cache, q, cu, self.lengths, self.tables[0], dev_status=self.status)
        x, h = mx.moe_block_norm(x, attn.reshape(x.shape[0], -1) @ self.w_out, post_weight=self.norm_attn,
                                 gate=self.gate, residual_scale=self.residual_scale, pre_weight=self.norm_mid)
        m = mx.moe_forward_groups(self.layer, h, self.bias, dev_status=self.status, **self.rule)
        return mx.moe_block_norm(x, m, post_weight=self.norm_out, residual_scale=self.residual_scale, y=x)[0]


def run(prompts, steps, chunk, keep, limit, workload="tiny", n_heads=8, n_kv_heads=2, head_dim=64, page_size=64, seed=0):
    """Serve the prompts for some steps; returns (block, outputs of the last step, number of evictions).

    A sequence that decodes feeds its last output back. Evictions wait until every prompt is through.
    """
    n_seq = len(prompts)
    longest = max(max(prompts) + steps, limit) + 1
    block = ChunkedBlock(wl.get(workload), n_heads, n_kv_heads, head_dim, n_seq, longest, page_size=page_size, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    inputs = [torch.randn((n, block.d), generator=gen, device="cuda") for n in prompts]
    taken, held, evictions, last = [0] * n_seq, [0] * n_seq, 0, [None] * n_seq
    for _ in range(steps):
        rows = []
        for b, n in enumerate(prompts):
            rows.append(inputs[b][taken[b]:taken[b] + chunk] if taken[b] < n else last[b])
        counts = [r.shape[0] for r in rows]
        decoding = all(t >= n for t, n in zip(taken, prompts))
        cu = torch.tensor([0, *counts], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        y = block.forward(torch.cat(rows), cu, decoding)
        end = 0
        for b, n in enumerate(counts):
            end, taken[b], held[b] = end + n, taken[b] + n, held[b] + n
            last[b] = y[end - 1:end]
        if decoding and max(held) > limit:
            block.evict(keep, recent=keep // 4)
            held, evictions = [min(n, keep) for n in held], evictions + 1
    return block, y, evictions


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 3, 260], help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--chunk", type=int, default=128, help="tokens of a prompt that one step takes")
    ap.add_argument("--keep", type=int, default=128, help="positions that an eviction keeps")
    ap.add_argument("--limit", type=int, default=320, help="positions after which it runs")
    ap.add_argument("--workload", default="tiny", help="the expert layer's shape")
    a = ap.parse_args()
    block, y, evictions = run(a.prompts, a.steps, a.chunk, a.keep, a.limit, a.workload)
    torch.cuda.synchronize()
    print(f"{len(a.prompts)} sequences, {a.steps} steps, {evictions} evictions, lengths {block.lengths.tolist()}, "
          f"device status {int(block.status.item())}, output rms {y.square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
