"""Timed cases of the attention operators: prompt attention, the 8-bit key/value cache's append, attention of new
tokens over that cache, and eviction from it.

Where ``own`` is false, ``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded
once at the end); where it is true, ``run`` makes the package's calls. ``exact`` gives the same outputs from the
definitions in 64 bits.

The cache's format: E4M3 codes ``[n_pages, kv_heads, page_size, head_dim]`` and one E8M0 byte (the value
``2**(byte - 127)``) for each (page, kv head), for keys and for values; position p of a sequence is slot
``p % page_size`` of page ``page_table[sequence, p // page_size]``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a short question, alone on the machine: latency counts. 20 query heads of 128 (d_model 2560), 4 kv heads
        dict(name="prompt_17", op="prompt", n_seq=1, tokens=17, prior=0, hq=20, hkv=4, d=128, causal=True, split=1),
        # a batch of short and middling prompts packed without padding, every head its own keys, heads of 64
        dict(name="prompt_packed_24", op="prompt", n_seq=24, tokens=6001, prior=0, hq=16, hkv=16, d=64, causal=True,
             split=2),
        # one chunk of 4096 tokens of a long prompt whose first 4096 tokens are there already
        dict(name="prompt_chunk_4096", op="prompt", n_seq=1, tokens=4096, prior=4096, hq=32, hkv=4, d=128,
             causal=True, split=3),
        # one long prompt, the largest
        dict(name="prompt_16384", op="prompt", n_seq=1, tokens=16384, prior=0, hq=16, hkv=2, d=128, causal=True,
             split=4),
        # a decode step of 64 sequences: one token each into the cache
        dict(name="append_64x1", op="append", n_seq=64, tokens=64, start=4000, hkv=4, d=128, page=64, split=5),
        # prompts of different lengths behind cached prefixes that end inside a page
        dict(name="append_prompts", op="append", n_seq=5, tokens=12345, start=700, hkv=8, d=128, page=64, split=6),
        # one sequence, one token, a short cache: latency counts
        dict(name="decode_1x1000", op="decode", n_seq=1, new=1, length=1000, hq=32, hkv=4, d=128, page=64,
             weights=False, split=7),
        # a batch of 64 of different lengths with the weights that eviction needs
        dict(name="decode_64x8192", op="decode", n_seq=64, new=1, length=8192, hq=32, hkv=4, d=128, page=64,
             weights=True, split=8),
        # verification of 4 drafted tokens for 16 sequences, 5 query heads to each kv head, short pages
        dict(name="decode_verify_16", op="decode", n_seq=16, new=4, length=20011, hq=20, hkv=4, d=128, page=16,
             weights=False, split=9),
        # long contexts, heads of 64: the largest read of the cache
        dict(name="decode_32x65536", op="decode", n_seq=32, new=1, length=65536, hq=64, hkv=8, d=64, page=128,
             weights=False, split=10),
        # one sequence halves its cache
        dict(name="evict_1x4096", op="evict", n_seq=1, length=4096, keep=2048, recent=256, hkv=4, d=128, page=64,
             split=11),
        # sixteen long sequences keep an eighth
        dict(name="evict_16x32768", op="evict", n_seq=16, length=32768, keep=4096, recent=512, hkv=4, d=128, page=64,
             split=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "append", "decode", "evict"])
    d = rng.choice([64, 128])
    split = rng.randrange(1 << 20)
    if op == "prompt":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 8]) if hkv < 8 else hkv * rng.choice([1, 2, 4])
        tokens = _log_int(rng, 16, 12000)
        n_seq = min(tokens, _log_int(rng, 1, 40))
        prior = rng.choice([0, 0, _log_int(rng, 1, 4000)])
        c = dict(op=op, n_seq=n_seq, tokens=tokens, prior=prior, hq=hq, hkv=hkv, d=d, causal=rng.random() < 0.8,
                 split=split)
        while work(c)["flops"] > 1e12:   # no more than the largest listed case
            c["tokens"] = max(c["n_seq"], c["tokens"] * 3 // 4)
        return c
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        n_seq = _log_int(rng, 1, 128)
        tokens = n_seq if rng.random() < 0.5 else _log_int(rng, n_seq, 16000)
        return dict(op=op, n_seq=n_seq, tokens=tokens, start=_log_int(rng, 1, 8000), hkv=hkv, d=d, page=page,
                    split=split)
    if op == "decode":
        n_seq = _log_int(rng, 1, 128)
        length = _log_int(rng, 16, max(64, min(65536, (1 << 23) // (n_seq * hkv))))
        return dict(op=op, n_seq=n_seq, new=rng.choice([1, 1, 2, 4]), length=length,
                    hq=hkv * rng.choice([1, 4, 5, 8]), hkv=hkv, d=d, page=page, weights=rng.random() < 0.5, split=split)
    n_seq = _log_int(rng, 1, 64)
    length = _log_int(rng, 64, max(256, min(65536, (1 << 21) // (n_seq * hkv))))
    keep = _log_int(rng, 16, length)
    return dict(op=op, n_seq=n_seq, length=length, keep=keep, recent=rng.randrange(0, keep // 2 + 1), hkv=hkv, d=d,
                page=page, split=split)


def _parts(total, n, split):
    """total cut into n lengths >= 1 of different sizes."""
    if n == 1:
        return [total]
    rng = random.Random(split)
    w = [rng.uniform(0.2, 1.0) ** 2 for _ in range(n)]
    left = total - n
    lens = [1 + int(left * x / sum(w)) for x in w]
    lens[0] += total - sum(lens)
    return lens


def _lengths(c):
    """Cache lengths of a decode or evict case: up to c["length"], the first one exactly that."""
    rng = random.Random(c["split"])
    lo = 0.5 if c["n_seq"] > 1 else 1.0
    return [c["length"]] + [max(1, int(c["length"] * rng.uniform(lo, 1.0))) for _ in range(c["n_seq"] - 1)]


def _starts(c):
    rng = random.Random(c["split"] + 1)
    return [rng.randrange(0, c["start"] + 1) for _ in range(c["n_seq"])]


def _prompt_lens(c):
    lq = _parts(c["tokens"], c["n_seq"], c["split"])
    return lq, [n + c["prior"] for n in lq]


# ---- inputs -----------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return _i32(cu)


def _activations(g, rows, heads, d, spread=1.0):
    """bf16 [rows, heads, d]: normal, with a magnitude for each channel as keys and values have it."""
    ch = torch.exp(0.5 * torch.randn((1, heads, d), generator=g, device=DEV))
    return (torch.randn((rows, heads, d), generator=g, device=DEV) * ch * spread).to(torch.bfloat16)


def _tables(g, n_pages_of, width, first=0):
    """Page tables of sequences with n_pages_of[b] pages each, the pages shuffled over the pool from `first` on."""
    total = sum(n_pages_of)
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32) + first
    pt = torch.zeros((len(n_pages_of), width), dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)[None]
    n = torch.tensor(n_pages_of, device=DEV)[:, None]
    pt[col < n] = perm
    return pt, first + total


def _filled(g, n_pages, hkv, page, d):
    """A pool of codes and scales as an append leaves it."""
    codes = torch.empty((n_pages, hkv, page, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n_pages, hkv), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (hkv * page * d))
    ch = torch.exp(0.5 * torch.randn((1, hkv, 1, d), generator=g, device=DEV))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn((n, hkv, page, d), generator=g, device=DEV) * ch
        x *= torch.exp(0.7 * torch.randn((n, hkv, 1, 1), generator=g, device=DEV))
        e = torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0))
        codes[i:i + n] = (x * torch.exp2(-e)[:, :, None, None]).clamp(-448, 448).to(F8).view(torch.uint8)
        scales[i:i + n] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "prompt":
        lq, lk = _prompt_lens(c)
        tq, tk = sum(lq), sum(lk)
        if c["prior"] == 0:   # slices of one fused projection
            hq, hkv = c["hq"], c["hkv"]
            qkv = _activations(g, tq, hq + 2 * hkv, c["d"])
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"] = _activations(g, tq, c["hq"], c["d"])
            s["k"] = _activations(g, tk, c["hkv"], c["d"])
            s["v"] = _activations(g, tk, c["hkv"], c["d"])
        s["cu_q"], s["cu_k"] = _cu(lq), _cu(lk)
        s["out"] = torch.empty((tq, c["hq"], c["d"]), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((tq, c["hq"]), dtype=torch.float32, device=DEV)
        s["max_q"], s["max_k"] = max(lq), max(lk)
        return s
    page, hkv, d = c["page"], c["hkv"], c["d"]
    if c["op"] == "append":
        ln, st = _parts(c["tokens"], c["n_seq"], c["split"]), _starts(c)
        pages = [-(-(a + b) // page) for a, b in zip(ln, st)]
        s["pt"], n_pages = _tables(g, pages, max(pages))
        s["k"] = _activations(g, c["tokens"], hkv, d)
        s["v"] = _activations(g, c["tokens"], hkv, d, 2.0)
        s["cu"], s["start"] = _cu(ln), _i32(st)
        s["max_new"] = max(ln)
    elif c["op"] == "decode":
        ln = _lengths(c)
        pages = [-(-n // page) for n in ln]
        s["pt"], n_pages = _tables(g, pages, max(pages))
        s["q"] = _activations(g, c["n_seq"] * c["new"], c["hq"], d).view(c["n_seq"], c["new"], c["hq"], d)
        s["lengths"] = _i32(ln)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device=DEV)
        if c["weights"]:   # what earlier steps have left
            s["weights"] = torch.rand((c["n_seq"], hkv, max(ln)), generator=g, device=DEV) * 0.01
    else:
        ln = _lengths(c)
        pages = [-(-n // page) for n in ln]
        s["pt"], first = _tables(g, pages, max(pages))
        to = [-(-min(n, c["keep"]) // page) for n in ln]
        s["dst"], n_pages = _tables(g, to, max(to), first)
        s["first"] = first
        s["lengths"] = _i32(ln)
        # heavy-tailed, as accumulated weights are; coarse, so that there are ties
        w = torch.exp(2 * torch.randn((c["n_seq"], hkv, max(ln)), generator=g, device=DEV))
        s["weights"] = torch.round(w * 64) / 64
        s["kept"] = torch.empty((c["n_seq"], hkv, c["keep"]), dtype=torch.int32, device=DEV)
        s["kept_weights"] = torch.empty((c["n_seq"], hkv, c["keep"]), dtype=torch.float32, device=DEV)
        s["new_lengths"] = torch.empty(c["n_seq"], dtype=torch.int32, device=DEV)
    s["kc"], s["ks"] = _filled(g, n_pages, hkv, page, d)
    s["vc"], s["vs"] = _filled(g, n_pages, hkv, page, d)
    if c["op"] == "evict":   # pages that nothing has been written to yet
        for n in ("kc", "vc", "ks", "vs"):
            s[n][s["first"]:] = 0
    if own:
        import mxfp4_expert_gb300 as mx
        s["cache"] = mx.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] == "decode":
            s["ws"] = torch.zeros(mx.moe_attn_decode_workspace_bytes(s["cache"], c["n_seq"], c["new"], c["hq"],
                                                                     s["pt"].shape[1], c["weights"]),
                                  dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    return (_run_own if own else _run_plain)[c["op"]](state)


def _visible(rows, lq, lk, cols, causal):
    """[B, rows, cols] truth values: query row r of a sequence sees key j (aligned at the sequences' ends)."""
    r, j = rows[None, :, None], cols[None, None, :]
    ok = (j < lk[:, None, None]) & (r < lq[:, None, None])
    return ok & (j <= r + (lk - lq)[:, None, None]) if causal else ok


def _softmax_out(s, ok, v):
    """s: scores [B, Hkv, G, R, L] in natural units (overwritten); ok broadcastable; v [B, Hkv, L, D]."""
    s.masked_fill_(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + m)[..., 0]
    b, h, g, r, n = p.shape
    out = torch.matmul(p.reshape(b, h, g * r, n), v).reshape(b, h, g, r, -1)
    return out, lse, p


def _plain_prompt(s):
    c = s["case"]
    d, hkv, g = c["d"], c["hkv"], c["hq"] // c["hkv"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    rows, cols = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at_q = (cu_q[:-1, None] + rows).clamp_(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + cols).clamp_(max=s["k"].shape[0] - 1)
    q = s["q"].float()[at_q].view(len(lq), -1, hkv, g, d).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[at_k].permute(0, 2, 1, 3)
    v = s["v"].float()[at_k].permute(0, 2, 1, 3)
    b, _, _, r, _ = q.shape
    sc = torch.matmul(q.reshape(b, hkv, g * r, d), k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(b, hkv, g, r, -1)
    ok = _visible(rows, lq, lk, cols, c["causal"])
    out, lse, _ = _softmax_out(sc, ok[:, None, None], v)
    here = rows[None] < lq[:, None]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(b, r, c["hq"], d)[here].to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(b, r, c["hq"])[here]}


def _own_prompt(s):
    import mxfp4_expert_gb300 as mx
    c = s["case"]
    mx.moe_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _exp2i(byte):
    """2**(byte - 127) for bytes 0 .. 254, from the bits of a 32-bit number."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _scale_byte(amax):
    """Byte of the smallest 2**e (e >= -127) with amax <= 448 * 2**e; 0 for amax 0."""
    m, e = torch.frexp(amax)                      # amax = m 2**e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)           # 448 = 0.875 * 2**9
    return torch.where(amax > 0, (e + 127).clamp(0, 254), 0)


def _plain_append(s):
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    cu, start = s["cu"].long(), s["start"].long()
    n_seq = len(start)
    end = start + cu[1:] - cu[:-1]
    width = s["max_new"] // page + 2              # pages that one sequence can touch
    blk = start[:, None] // page + torch.arange(width, device=DEV)
    pos = blk[:, :, None] * page + torch.arange(page, device=DEV)
    new = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    old = (pos < start[:, None, None])
    touched = new.any(-1)
    at = (cu[:-1, None, None] + pos - start[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    pages = s["pt"].long().gather(1, blk.clamp(max=s["pt"].shape[1] - 1))[touched]
    new, old, at = new[touched], old[touched], at[touched]
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()[at].permute(0, 2, 1, 3)                         # [touched, hkv, page, d]
        amax = (x.abs() * new[:, None, :, None]).amax((2, 3))
        had = torch.where(old.any(-1)[:, None], scales[pages].long(), 0)
        byte = torch.maximum(_scale_byte(amax).long(), had)
        was = codes[pages].view(F8).float() * _exp2i(had)[:, :, None, None]
        val = torch.where(new[:, None, :, None], x, torch.where(old[:, None, :, None], was, 0.0))
        coded = (val * _exp2i(254 - byte)[:, :, None, None]).to(F8).view(torch.uint8)
        keep = (new | old)[:, None, :, None]
        codes[pages] = torch.where(keep, coded, codes[pages])
        scales[pages] = byte.to(torch.uint8)
    return _cache_out(s)


def _cache_out(s, first=0):
    return {"k": s["kc"][first:].view(F8), "v": s["vc"][first:].view(F8), "k_scales": s["ks"][first:],
            "v_scales": s["vs"][first:]}


def _own_append(s):
    import mxfp4_expert_gb300 as mx
    mx.moe_kv_append_fp8(s["cache"], s["k"], s["v"], s["cu"], s["start"], s["pt"])
    return _cache_out(s)


def _dequant(codes, scales, pt, n):
    """fp32 [B, Hkv, n, D] of the first n positions of every sequence."""
    b, w = pt.shape
    _, h, p, d = codes.shape
    x = codes[pt].view(F8).float() * _exp2i(scales[pt])[..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, w * p, d)[:, :, :n]


def _plain_decode(s):
    c = s["case"]
    d, hkv, g, t = c["d"], c["hkv"], c["hq"] // c["hkv"], c["new"]
    n = c["length"]
    pt, lengths = s["pt"].long(), s["lengths"].long()
    b = len(lengths)
    q = s["q"].float().view(b, t, hkv, g, d).permute(0, 2, 3, 1, 4)
    k = _dequant(s["kc"], s["ks"], pt, n)
    sc = torch.matmul(q.reshape(b, hkv, g * t, d), k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(b, hkv, g, t, n)
    del k
    tq = torch.full((b,), t, device=DEV)
    ok = _visible(torch.arange(t, device=DEV), tq, lengths, torch.arange(n, device=DEV), True)
    out, lse, p = _softmax_out(sc, ok[:, None, None], _dequant(s["vc"], s["vs"], pt, n))
    res = {"out": out.permute(0, 3, 1, 2, 4).reshape(b, t, c["hq"], d).to(torch.bfloat16),
           "lse": lse.permute(0, 3, 1, 2).reshape(b, t, c["hq"])}
    if c["weights"]:
        s["weights"] += p.sum((2, 3))
        res["weights"] = s["weights"]
    return res


def _own_decode(s):
    import mxfp4_expert_gb300 as mx
    w = s.get("weights")
    mx.moe_attn_decode_fp8(s["cache"], s["q"], s["lengths"], s["pt"], out=s["out"], lse=s["lse"], weights=w,
                           workspace=s["ws"])
    res = {"out": s["out"], "lse": s["lse"]}
    if w is not None:
        res["weights"] = w
    return res


def _plain_evict(s):
    c = s["case"]
    page, hkv, d, keep, recent = c["page"], c["hkv"], c["d"], c["keep"], c["recent"]
    pt, dst, ln = s["pt"].long(), s["dst"].long(), s["lengths"].long()
    b, n = len(ln), s["weights"].shape[2]
    j = torch.arange(n, device=DEV)
    w = s["weights"].masked_fill((j >= ln[:, None])[:, None], -math.inf)
    w = w.masked_fill(((j >= (ln - recent)[:, None]) & (j < ln[:, None]))[:, None], math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :keep]
    m = torch.minimum(ln, torch.full_like(ln, keep))
    here = torch.arange(order.shape[2], device=DEV) < m[:, None, None]
    here = here.expand(order.shape)
    kept = torch.sort(order.masked_fill(~here, n), dim=-1)[0]
    if kept.shape[2] < keep:
        pad = (b, hkv, keep - kept.shape[2])
        kept = torch.cat([kept, torch.full(pad, n, device=DEV)], -1)
        here = torch.cat([here, torch.zeros(pad, dtype=torch.bool, device=DEV)], -1)
    src = kept.clamp(max=n - 1)
    s["kept"].copy_(kept.masked_fill(~here, -1))
    s["kept_weights"].copy_(s["weights"].gather(2, src).masked_fill(~here, 0.0))
    s["new_lengths"].copy_(m)
    wide = dst.shape[1] * page
    src = torch.nn.functional.pad(src, (0, max(0, wide - keep)))[..., :wide]
    here = torch.nn.functional.pad(here, (0, max(0, wide - keep)))[..., :wide]
    at_page = pt[:, None].expand(b, hkv, pt.shape[1]).gather(2, src // page)
    at_slot, head = src % page, torch.arange(hkv, device=DEV)[None, :, None]
    used = torch.arange(dst.shape[1], device=DEV) * page < m[:, None]
    for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = codes[at_page, head, at_slot].view(F8).float() * _exp2i(scales[at_page, head])[..., None]
        x = x.masked_fill(~here[..., None], 0.0).view(b, hkv, -1, page, d).permute(0, 2, 1, 3, 4)[used]
        byte = _scale_byte(x.abs().amax((2, 3))).long()
        codes[dst[used]] = (x * _exp2i(254 - byte)[:, :, None, None]).to(F8).view(torch.uint8)
        scales[dst[used]] = byte.to(torch.uint8)
    return _evict_out(s)


def _evict_out(s):
    return {**_cache_out(s, s["first"]), "kept": s["kept"], "kept_weights": s["kept_weights"],
            "new_lengths": s["new_lengths"]}


def _own_evict(s):
    import mxfp4_expert_gb300 as mx
    c = s["case"]
    mx.moe_kv_evict_fp8(s["cache"], s["pt"], s["lengths"], s["weights"], c["keep"], c["recent"], s["dst"],
                        kept=s["kept"], kept_weights=s["kept_weights"], new_lengths=s["new_lengths"])
    return _evict_out(s)


_run_plain = {"prompt": _plain_prompt, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}
_run_own = {"prompt": _own_prompt, "append": _own_append, "decode": _own_decode, "evict": _own_evict}


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "prompt":
        lq, lk = _prompt_lens(c)
        pairs = sum(sum(range(k - q + 1, k + 1)) if c["causal"] else q * k for q, k in zip(lq, lk))
        tq, tk = sum(lq), sum(lk)
        return {"bytes": 2 * c["d"] * (2 * tq * c["hq"] + 2 * tk * c["hkv"]) + 4 * tq * c["hq"],
                "flops": 4 * c["d"] * c["hq"] * pairs}
    row = c["hkv"] * c["d"]
    if c["op"] == "append":
        return {"bytes": 2 * c["tokens"] * row * 3, "flops": 0}
    ln = _lengths(c)
    if c["op"] == "decode":
        rows = c["n_seq"] * c["new"] * c["hq"]
        return {"bytes": sum(ln) * (2 * row + (8 * c["hkv"] if c["weights"] else 0)) + rows * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * c["new"] * sum(ln)}
    kept = sum(min(n, c["keep"]) for n in ln)
    return {"bytes": 4 * sum(ln) * c["hkv"] + kept * (4 * row + 12 * c["hkv"]), "flops": 0}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"prompt": _exact_prompt, "append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[
        case["op"]](s)


def _attend64(q, k, v, first_seen):
    """One head in 64 bits: q [R, D], k, v [L, D]; row r sees keys [0, first_seen[r]). Returns out, lse, weights."""
    s = (q @ k.T) / math.sqrt(q.shape[1])
    s = torch.where(torch.arange(k.shape[0], device=DEV)[None] < first_seen[:, None], s, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[:, None])
    return p @ v, lse, p.sum(0)


def _exact_prompt(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    lq, lk = _prompt_lens(c)
    out = torch.zeros((sum(lq), c["hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(lq), c["hq"]), dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for nq, nk in zip(lq, lk):
        seen = torch.arange(nq, device=DEV) + (nk - nq) + 1 if c["causal"] else torch.full((nq,), nk, device=DEV)
        for h in range(c["hq"]):
            k, v = (s[n][k0:k0 + nk, h // g].double() for n in ("k", "v"))
            out[q0:q0 + nq, h], lse[q0:q0 + nq, h], _ = _attend64(s["q"][q0:q0 + nq, h].double(), k, v, seen)
        q0, k0 = q0 + nq, k0 + nk
    return {"out": out, "lse": lse}


_E4M3 = None


def _values64(codes):
    """E4M3 codes -> 64-bit values, by the format's definition (1 sign, 4 exponent bits of bias 7, 3 fraction bits)."""
    global _E4M3
    if _E4M3 is None:
        t = []
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
            t.append(-x if c & 128 else x)
        _E4M3 = torch.tensor(t, dtype=torch.float64, device=DEV)
    return _E4M3[codes.long()]


def _round64(x):
    """64-bit values rounded to the E4M3 grid, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _power64(amax):
    """The smallest power of two 2**e, e >= -127, with amax <= 448 * 2**e."""
    if amax == 0:
        return -127
    e = math.ceil(math.log2(amax / 448))
    while amax > 448 * 2.0 ** e:
        e += 1
    while amax <= 448 * 2.0 ** (e - 1):
        e -= 1
    return max(e, -127)


def _exact_append(s):
    c = s["case"]
    if c["tokens"] * c["hkv"] // c["page"] + c["n_seq"] * c["hkv"] > 20000:
        return None
    page = c["page"]
    ln, st = _parts(c["tokens"], c["n_seq"], c["split"]), _starts(c)
    pt = s["pt"].tolist()
    res = {}
    for n, x, codes, scales in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        val, byte = _values64(codes), scales.tolist()
        t0 = 0
        for b, (m, p0) in enumerate(zip(ln, st)):
            at = p0
            while at < p0 + m:
                pg, slot = pt[b][at // page], at % page
                n_here = min(page - slot, p0 + m - at)
                xs = x[t0 + at - p0:t0 + at - p0 + n_here].double()
                top = xs.abs().amax((0, 2)).tolist()
                for h in range(c["hkv"]):
                    e = max(_power64(top[h]), byte[pg][h] - 127 if slot else -127)
                    if slot:
                        val[pg, h, :slot] = _round64(val[pg, h, :slot] * 2.0 ** (byte[pg][h] - 127 - e))
                    val[pg, h, slot:slot + n_here] = _round64(xs[:, h] * 2.0 ** -e)
                at += n_here
            t0 += m
        res[n] = val
    return {"k": res["k"], "v": res["v"], "k_scales": None, "v_scales": None}


def _sequence64(s, b, h, n):
    """Keys and values [n, D] of sequence b, kv head h, in 64 bits."""
    pages = s["pt"][b, :-(-n // s["case"]["page"])].long()
    got = []
    for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = _values64(codes[pages, h]) * torch.exp2(scales[pages, h].double() - 127)[:, None, None]
        got.append(x.reshape(-1, x.shape[-1])[:n])
    return got


def _exact_decode(s):
    c = s["case"]
    g, t, d = c["hq"] // c["hkv"], c["new"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    w = s["weights"].double() if c["weights"] else None
    for b, n in enumerate(_lengths(c)):
        seen = (n - t + 1 + torch.arange(t, device=DEV))[:, None].expand(t, g).reshape(-1)
        for h in range(c["hkv"]):
            k, v = _sequence64(s, b, h, n)
            q = s["q"][b, :, h * g:(h + 1) * g].double().reshape(t * g, d)
            o, l, p = _attend64(q, k, v, seen)
            out[b, :, h * g:(h + 1) * g] = o.view(t, g, d)
            lse[b, :, h * g:(h + 1) * g] = l.view(t, g)
            if w is not None:
                w[b, h, :n] += p
    return {"out": out, "lse": lse, **({"weights": w} if w is not None else {})}


def _exact_evict(s):
    c = s["case"]
    page, keep, recent = c["page"], c["keep"], c["recent"]
    if sum(min(n, keep) // page + 1 for n in _lengths(c)) * c["hkv"] > 20000:
        return None
    shape = (s["kc"].shape[0] - s["first"], c["hkv"], page, c["d"])
    res = {n: torch.zeros(shape, dtype=torch.float64, device=DEV) for n in ("k", "v")}
    kept_w = torch.zeros((c["n_seq"], c["hkv"], keep), dtype=torch.float64)
    w, dst = s["weights"].double().cpu(), s["dst"].tolist()
    for b, n in enumerate(_lengths(c)):
        for h in range(c["hkv"]):
            ids = list(range(n))
            if n > keep:
                ws = w[b, h].tolist()
                ids = sorted(sorted(range(n - recent), key=lambda i: (-ws[i], i))[:keep - recent]) + ids[n - recent:]
            kept_w[b, h, :len(ids)] = w[b, h, ids]
            at = torch.tensor(ids, device=DEV)
            for name, x in zip(("k", "v"), _sequence64(s, b, h, n)):
                x = x[at]
                for i in range(0, len(ids), page):
                    part = x[i:i + page]
                    e = _power64(float(part.abs().max()))
                    res[name][dst[b][i // page] - s["first"], h, :len(part)] = _round64(part * 2.0 ** -e)
    return {**res, "k_scales": None, "v_scales": None, "kept": None, "kept_weights": kept_w, "new_lengths": None}
