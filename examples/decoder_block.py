"""One decoder block served with this library: attention with a paged FP8 cache, then the MXFP4 expert layer.

    python examples/decoder_block.py [--prompts 300 77] [--steps 96] [--keep 128] [--limit 192]

Prompts of different lengths run packed (moe_attn_prefill) and fill the cache
(moe_kv_append_fp8). Each step then appends one token of every sequence,
attends over the cache (moe_attn_decode_fp8) while summing the probabilities
that every position receives, and runs the experts (moe_forward). Once any
sequence holds more than --limit positions, moe_kv_evict_fp8 keeps the heaviest
and the newest --keep of each, in other pages. Everything runs on the current
stream; lengths stay on the device, and the host knows them by counting.

Weights and inputs are random. The projections are torch products, as a caller
would have them; positional encoding is left out.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_expert_gb300 as mx  # noqa: E402
import workloads as wl  # noqa: E402
from mxfp4_expert_gb300 import synthetic  # noqa: E402


def _norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class DecoderBlock:
    """Attention of n_heads over n_kv_heads and one expert layer, with the cache of n_seq sequences.

    Every sequence owns two runs of pages, one in use and one that an eviction writes to.
    """

    def __init__(self, workload, n_heads: int, n_kv_heads: int, head_dim: int, n_seq: int, max_positions: int,
                 page_size: int = 64, seed: int = 0, device="cuda"):
        self.n_heads, self.n_kv, self.hd, self.n_seq = n_heads, n_kv_heads, head_dim, n_seq
        self.layer = synthetic.build_layer(workload, 0, device=device)
        self.d = self.layer.d
        gen = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape):
            return (torch.randn(shape, generator=gen, device=device) * shape[0] ** -0.5).to(torch.bfloat16)

        self.w_qkv = draw(self.d, (n_heads + 2 * n_kv_heads) * head_dim)
        self.w_out = draw(n_heads * head_dim, self.d)
        width = -(-max_positions // page_size)
        self.cache = mx.KVCache.alloc(2 * n_seq * width, page_size, n_kv_heads, head_dim, device)
        pages = torch.randperm(2 * n_seq * width, generator=gen, device=device).to(torch.int32)
        self.tables = list(pages.view(2, n_seq, width))  # [0] in use, [1] free
        self.lengths = torch.zeros(n_seq, dtype=torch.int32, device=device)
        self.weights = torch.zeros((n_seq, n_kv_heads, max_positions), device=device)
        self.one_each = torch.arange(n_seq + 1, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.zeros(
            mx.moe_attn_decode_workspace_bytes(self.cache, n_seq, 1, n_heads, width, True),
            dtype=torch.uint8, device=device)

    def _qkv(self, x):
        """q, k and v as slices of one projection; the kernels take their strides."""
        rows = (_norm(x) @ self.w_qkv).view(x.shape[0], -1, self.hd)
        return rows.split((self.n_heads, self.n_kv, self.n_kv), dim=1)

    def _finish(self, x, attn):
        x = x + attn.reshape(x.shape[0], -1) @ self.w_out
        return x + mx.moe_forward(self.layer, _norm(x), dev_status=self.status)

    def prompt(self, x, cu):
        """x bf16 [total, d], the prompts one after another; cu int32 [n_seq + 1]. Fills the cache."""
        q, k, v = self._qkv(x)
        attn = mx.moe_attn_prefill(q, k, v, cu, dev_status=self.status)
        mx.moe_kv_append_fp8(self.cache, k, v, cu, self.lengths, self.tables[0], dev_status=self.status)
        self.lengths += cu[1:] - cu[:-1]
        return self._finish(x, attn)

    def step(self, x):
        """x bf16 [n_seq, d], one new token of every sequence."""
        q, k, v = self._qkv(x)
        mx.moe_kv_append_fp8(self.cache, k, v, self.one_each, self.lengths, self.tables[0], dev_status=self.status)
        self.lengths += 1
        attn = mx.moe_attn_decode_fp8(self.cache, q.unsqueeze(1), self.lengths, self.tables[0], weights=self.weights,
                                      workspace=self.workspace, dev_status=self.status)
        return self._finish(x, attn)

    def evict(self, keep: int, recent: int):
        """Keep `keep` positions of every sequence and head. Returns the positions kept, int32 [n_seq, n_kv, keep]."""
        kept, kept_weights, self.lengths = mx.moe_kv_evict_fp8(
            self.cache, self.tables[0], self.lengths, self.weights, keep, recent, self.tables[1],
            dev_status=self.status)
        self.tables.reverse()
        self.weights.zero_()  # positions to come start from nothing
        self.weights[:, :, :keep] = kept_weights
        return kept


def run(prompts, steps, keep, limit, workload="tiny", n_heads=8, n_kv_heads=2, head_dim=64, seed=0):
    """Serve the prompts for some steps; returns (block, outputs of the last step, number of evictions)."""
    n_seq = len(prompts)
    block = DecoderBlock(wl.get(workload), n_heads, n_kv_heads, head_dim, n_seq, max(max(prompts), limit) + 1,
                         seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    cu = torch.tensor([0, *prompts], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    x = torch.randn((sum(prompts), block.d), generator=gen, device="cuda").to(torch.bfloat16)
    x = block.prompt(x, cu)[(cu[1:] - 1).long()]
    longest, evictions = max(prompts), 0
    for _ in range(steps):
        x = block.step(_norm(x))
        longest += 1
        if longest > limit:
            block.evict(keep, recent=keep // 4)
            longest, evictions = keep, evictions + 1
    return block, x, evictions


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[300, 77], help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=96)
    ap.add_argument("--keep", type=int, default=128, help="positions that an eviction keeps")
    ap.add_argument("--limit", type=int, default=192, help="positions after which it runs")
    ap.add_argument("--workload", default="tiny", help="the expert layer's shape")
    a = ap.parse_args()
    block, x, evictions = run(a.prompts, a.steps, a.keep, a.limit, a.workload)
    torch.cuda.synchronize()
    print(f"{len(a.prompts)} sequences, {a.steps} steps, {evictions} evictions, lengths {block.lengths.tolist()}, "
          f"device status {int(block.status.item())}, output rms {x.float().square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
