"""Timed cases of the rest of a served decoder block: the norms around its halves with gate and residual, the append to
the 8-bit key/value cache with the position rotation on the way, attention of a chunk of new tokens over that cache, and
routing by groups of experts.

Where ``own`` is false, ``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles
and routing scores in 64, rounded once at the end); where it is true, ``run`` makes the package's calls. ``exact`` gives
the same outputs from the definitions in 64 bits.

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
EPS = 1e-6


# ---- cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # between the halves of a block in a decode step of one sequence: latency counts
        dict(name="norm_1x2560", op="norm", tokens=1, d=2560, stream="bf16", post=True, gate="none", pre=True),
        # the same for a prompt of 4096 tokens, with a gate per channel
        dict(name="norm_4096x2560", op="norm", tokens=4096, d=2560, stream="bf16", post=True, gate="channel", pre=True),
        # a wide model that keeps its residual stream in 32 bits and gates every token
        dict(name="norm_1001x7168", op="norm", tokens=1001, d=7168, stream="fp32", post=True, gate="token", pre=True),
        # a decode step of 64 sequences over 512 experts in 8 groups
        dict(name="route_64x512", op="route", tokens=64, experts=512, k=8, score="sigmoid", groups=8, top=4, best=2,
             bias=True),
        # a prompt of 4096 tokens over the same experts
        dict(name="route_4096x512", op="route", tokens=4096, experts=512, k=8, score="sigmoid", groups=8, top=4,
             best=2, bias=True),
        # softmax scores, groups by their best expert, no bias
        dict(name="route_16384x160", op="route", tokens=16384, experts=160, k=6, score="softmax", groups=8, top=3,
             best=1, bias=False),
        # a decode step of 64 sequences: one token each into the cache, its queries rotated too
        dict(name="rope_64x1", op="rope", n_seq=64, tokens=64, start=4000, hq=32, hkv=4, d=128, rot=128, page=64,
             pairs="halves", split=5),
        # prompts of different lengths behind cached prefixes that end inside a page; half of each head is rotated
        dict(name="rope_prompts", op="rope", n_seq=5, tokens=12345, start=70000, hq=16, hkv=8, d=128, rot=64, page=64,
             pairs="neighbours", split=6),
        # a short follow-up question over a conversation in the cache, alone on the machine
        dict(name="chunk_37", op="chunk", n_seq=1, tokens=37, prior=5000, hq=20, hkv=4, d=128, page=64, split=7),
        # follow-ups of different lengths in one batch, heads of 64, short pages
        dict(name="chunk_24x", op="chunk", n_seq=24, tokens=1501, prior=9000, hq=16, hkv=4, d=64, page=16, split=8),
        # a chunk of 256 tokens at the end of each of 4 long documents
        dict(name="chunk_4x256", op="chunk", n_seq=4, tokens=1024, prior=65536, hq=32, hkv=4, d=128, page=128, split=9),
        # the last 4096 tokens of a prompt of 32768 that is taken in chunks, the largest
        dict(name="chunk_4096", op="chunk", n_seq=1, tokens=4096, prior=28672, hq=32, hkv=4, d=128, page=64, split=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "rope", "chunk"])
    if op == "norm":
        d = 8 * _log_int(rng, 16, 1536)
        return dict(op=op, tokens=_log_int(rng, 1, min(8192, 10500000 // d)), d=d, stream=rng.choice(["bf16", "fp32"]),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]), pre=rng.random() < 0.8)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        experts = groups * _log_int(rng, 4, 1024 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(16, experts // groups * top))
        return dict(op=op, tokens=_log_int(rng, 1, min(16384, 2600000 // experts)), experts=experts, k=k,
                    score=rng.choice(["sigmoid", "softmax"]), groups=groups, top=top, best=rng.choice([1, 2]),
                    bias=rng.random() < 0.6)
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    split = rng.randrange(1 << 20)
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        n_seq = _log_int(rng, 1, 128)
        tokens = n_seq if rng.random() < 0.5 else _log_int(rng, n_seq, 8000)
        return dict(op=op, n_seq=n_seq, tokens=tokens, start=_log_int(rng, 1, 100000 // n_seq + 2000), hq=hq, hkv=hkv,
                    d=d, rot=rng.choice([d, d, d // 2, 16]), page=page, pairs=rng.choice(["halves", "neighbours"]),
                    split=split)
    tokens = _log_int(rng, 1, 4000)
    n_seq = min(tokens, _log_int(rng, 1, 48))
    c = dict(op=op, n_seq=n_seq, tokens=tokens, prior=_log_int(rng, 1, 65536), hq=hq, hkv=hkv, d=d, page=page,
             split=split)
    while work(c)["flops"] > 1e12 or n_seq * c["prior"] * hkv > 1 << 22:   # no more than the largest listed case
        c["prior"] = max(1, c["prior"] * 3 // 4)
    return c


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


def _starts(c):
    """Positions that each sequence of a rope case holds already."""
    rng = random.Random(c["split"] + 1)
    return [rng.randrange(0, c["start"] + 1) for _ in range(c["n_seq"])]


def _chunk_lens(c):
    """New tokens and all positions of each sequence of a chunk case; the first sequence's prior ones are the most."""
    new = _parts(c["tokens"], c["n_seq"], c["split"])
    rng = random.Random(c["split"] + 2)
    prior = [c["prior"]] + [int(c["prior"] * rng.uniform(0.3, 1.0)) for _ in range(c["n_seq"] - 1)]
    return new, [a + b for a, b in zip(new, prior)]


# ---- inputs -----------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return _i32(cu)


def _activations(g, rows, heads, d, spread=1.0):
    """bf16 [rows, heads, d]: normal, with a magnitude for each channel as queries, keys and values have it."""
    ch = torch.exp(0.5 * torch.randn((1, heads, d), generator=g, device=DEV))
    return (torch.randn((rows, heads, d), generator=g, device=DEV) * ch * spread).to(torch.bfloat16)


def _tables(g, n_pages_of, width):
    """Page tables of sequences with n_pages_of[b] pages each, the pages shuffled over the pool."""
    total = sum(n_pages_of)
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    pt = torch.zeros((len(n_pages_of), width), dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)[None]
    pt[col < torch.tensor(n_pages_of, device=DEV)[:, None]] = perm
    return pt, total


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
    if c["op"] == "norm":
        t, d = c["tokens"], c["d"]
        wide = torch.float32 if c["stream"] == "fp32" else torch.bfloat16
        ch = torch.exp(0.5 * torch.randn((1, d), generator=g, device=DEV))   # channels differ in a residual stream
        s["x"] = (4 * torch.randn((t, d), generator=g, device=DEV) * ch).to(wide)
        s["a"] = torch.randn((t, d), generator=g, device=DEV).to(torch.bfloat16)
        for n in ("post", "pre"):
            s[n] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if c[n] else None
        s["gate"] = None
        if c["gate"] != "none":
            s["gate"] = torch.rand((t, d) if c["gate"] == "token" else d, generator=g, device=DEV).to(torch.bfloat16)
        s["scale"] = 0.22
        s["y"] = torch.empty_like(s["x"])
        s["h"] = torch.empty((t, d), dtype=torch.bfloat16, device=DEV) if c["pre"] else None
        return s
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        popular = 0.5 * torch.randn((1, e), generator=g, device=DEV)
        s["logits"] = 1.5 * torch.randn((t, e), generator=g, device=DEV) + popular
        s["bias"] = -0.1 * popular[0] + 0.02 * torch.randn(e, generator=g, device=DEV) if c["bias"] else None
        s["scale"] = 2.5
        s["idx"] = torch.empty((t, c["k"]), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty((t, c["k"]), dtype=torch.float32, device=DEV)
        return s
    page, hq, hkv, d = c["page"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        ln, st = _parts(c["tokens"], c["n_seq"], c["split"]), _starts(c)
        pages = [-(-(a + b) // page) for a, b in zip(ln, st)]
        s["pt"], n_pages = _tables(g, pages, max(pages))
        qkv = _activations(g, c["tokens"], hq + 2 * hkv, d)   # slices of one fused projection
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["cu"], s["start"] = _cu(ln), _i32(st)
        s["max_new"] = max(ln)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float32) / c["rot"])
        s["q_out"] = torch.empty((c["tokens"], hq, d), dtype=torch.bfloat16, device=DEV)
    else:
        new, ln = _chunk_lens(c)
        pages = [-(-n // page) for n in ln]
        s["pt"], n_pages = _tables(g, pages, max(pages))
        s["q"] = _activations(g, c["tokens"], hq, d)
        s["cu"], s["lengths"] = _cu(new), _i32(ln)
        s["out"] = torch.empty((c["tokens"], hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((c["tokens"], hq), dtype=torch.float32, device=DEV)
    s["kc"], s["ks"] = _filled(g, n_pages, hkv, page, d)
    s["vc"], s["vs"] = _filled(g, n_pages, hkv, page, d)
    if own:
        import mxfp4_expert_gb300 as mx
        s["cache"] = mx.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] == "chunk":
            s["ws"] = torch.empty(mx.moe_attn_chunk_workspace_bytes(s["cache"], hq, c["tokens"], c["n_seq"]),
                                  dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    n = s["a"].float()
    if s["post"] is not None:
        n = _rms(n) * s["post"].float()
    if s["gate"] is not None:
        n = n * s["gate"].float()
    y = s["x"].float() + s["scale"] * n
    res = {"y": y.to(s["x"].dtype)}
    if s["pre"] is not None:
        res["h"] = (_rms(y) * s["pre"].float()).to(torch.bfloat16)
    return res


def _own_norm(s):
    import mxfp4_expert_gb300 as mx
    mx.moe_block_norm(s["x"], s["a"], post_weight=s["post"], gate=s["gate"], residual_scale=s["scale"],
                      pre_weight=s["pre"], eps=EPS, y=s["y"], h=s["h"])
    return {"y": s["y"], "h": s["h"]} if s["h"] is not None else {"y": s["y"]}


def _first_sorted(x, n):
    """The n largest along the last dimension, equal ones by the lower index: (values, indices)."""
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    return v[..., :n], i[..., :n]


def _plain_route(s):
    c = s["case"]
    l = s["logits"].double()      # two keys may lie closer than 32 bits tell
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["top"] < c["groups"]:
        t = key.view(len(key), c["groups"], -1)
        rank = _first_sorted(t, c["best"])[0].sum(-1)
        chosen = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, _first_sorted(rank, c["top"])[1], True)
        key = t.masked_fill(~chosen[..., None], -math.inf).view_as(key)
    idx = _first_sorted(key, c["k"])[1]
    w = score.gather(1, idx)
    w = w / (w.sum(-1, keepdim=True) + 1e-20) * s["scale"]
    return {"idx": idx.to(torch.int32), "w": w.float()}


def _own_route(s):
    import mxfp4_expert_gb300 as mx
    c = s["case"]
    mx.moe_route_groups(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_groups=c["groups"],
                        top_groups=c["top"], group_best=c["best"], scale=s["scale"], idx=s["idx"], w=s["w"])
    return {"idx": s["idx"], "w": s["w"]}


def _exp2i(byte):
    """2**(byte - 127) for bytes 0 .. 254, from the bits of a 32-bit number."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _scale_byte(amax):
    """Byte of the smallest 2**e (e >= -127) with amax <= 448 * 2**e; 0 for amax 0."""
    m, e = torch.frexp(amax)                      # amax = m 2**e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)           # 448 = 0.875 * 2**9
    return torch.where(amax > 0, (e + 127).clamp(0, 254), 0)


def _token_positions(s):
    cu, start = s["cu"].long(), s["start"].long()
    n = s["q"].shape[0]
    row = torch.arange(n, device=DEV)
    b = torch.searchsorted(cu[1:], row, right=True)
    return row - cu[b] + start[b]


def _turned(c, x, cos, sin):
    """fp32 rows x [n, heads, d] with their first rot channels rotated."""
    r = c["rot"]
    y = x.clone()
    a, b = (slice(0, r // 2), slice(r // 2, r)) if c["pairs"] == "halves" else (slice(0, r, 2), slice(1, r, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope(s):
    c = s["case"]
    page = c["page"]
    cu, start = s["cu"].long(), s["start"].long()
    angle = _token_positions(s).double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
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
    for x, codes, scales in ((_turned(c, s["k"].float(), cos, sin), s["kc"], s["ks"]),
                             (s["v"].float(), s["vc"], s["vs"])):
        x = x[at].permute(0, 2, 1, 3)                                 # [touched, hkv, page, d]
        amax = (x.abs() * new[:, None, :, None]).amax((2, 3))
        had = torch.where(old.any(-1)[:, None], scales[pages].long(), 0)
        byte = torch.maximum(_scale_byte(amax).long(), had)
        was = codes[pages].view(F8).float() * _exp2i(had)[:, :, None, None]
        val = torch.where(new[:, None, :, None], x, torch.where(old[:, None, :, None], was, 0.0))
        coded = (val * _exp2i(254 - byte)[:, :, None, None]).to(F8).view(torch.uint8)
        keep = (new | old)[:, None, :, None]
        codes[pages] = torch.where(keep, coded, codes[pages])
        scales[pages] = byte.to(torch.uint8)
    s["q_out"].copy_(_turned(c, s["q"].float(), cos, sin))
    return _rope_out(s)


def _rope_out(s):
    return {"k": s["kc"].view(F8), "v": s["vc"].view(F8), "k_scales": s["ks"], "v_scales": s["vs"], "q": s["q_out"]}


def _own_rope(s):
    import mxfp4_expert_gb300 as mx
    mx.moe_kv_append_rope_fp8(s["cache"], s["k"], s["v"], s["cu"], s["start"], s["pt"], s["inv_freq"], q=s["q"],
                              q_out=s["q_out"], interleaved=s["case"]["pairs"] == "neighbours")
    return _rope_out(s)


def _values(codes, scales, pages, n):
    """fp32 [hkv, n, d] of the first n positions on these pages."""
    x = codes[pages].view(F8).float() * _exp2i(scales[pages])[..., None, None]
    return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def _plain_chunk(s):
    c = s["case"]
    d, hkv, g, page = c["d"], c["hkv"], c["hq"] // c["hkv"], c["page"]
    new, lens = _chunk_lens(c)
    t0 = 0
    for b, (nq, nk) in enumerate(zip(new, lens)):
        pages = s["pt"][b, :-(-nk // page)].long()
        q = s["q"][t0:t0 + nq].float().view(nq, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * nq, d)
        p = torch.matmul(q, _values(s["kc"], s["ks"], pages, nk).transpose(1, 2)).mul_(1 / math.sqrt(d))
        hidden = torch.arange(nk, device=DEV)[None] > torch.arange(nq, device=DEV)[:, None] + (nk - nq)
        p.view(hkv, g, nq, nk).masked_fill_(hidden, -math.inf)
        m = p.amax(-1, keepdim=True)
        total = p.sub_(m).exp_().sum(-1, keepdim=True)
        out = torch.matmul(p, _values(s["vc"], s["vs"], pages, nk)) / total
        s["out"][t0:t0 + nq] = out.view(hkv, g, nq, d).permute(2, 0, 1, 3).reshape(nq, c["hq"], d)
        s["lse"][t0:t0 + nq] = (torch.log(total) + m).view(c["hq"], nq).T
        t0 += nq
    return {"out": s["out"], "lse": s["lse"]}


def _own_chunk(s):
    import mxfp4_expert_gb300 as mx
    mx.moe_attn_chunk_fp8(s["cache"], s["q"], s["cu"], s["lengths"], s["pt"], out=s["out"], lse=s["lse"],
                          workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


_run_plain = {"norm": _plain_norm, "route": _plain_route, "rope": _plain_rope, "chunk": _plain_chunk}
_run_own = {"norm": _own_norm, "route": _own_route, "rope": _own_rope, "chunk": _own_chunk}


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * c["d"]
        wide = 4 if c["stream"] == "fp32" else 2
        gate = {"none": 0, "channel": 2 * c["d"], "token": 2 * n}[c["gate"]]
        return {"bytes": n * (2 + 2 * wide + (2 if c["pre"] else 0)) + gate + 2 * c["d"] * (c["post"] + c["pre"]),
                "flops": 0}
    if c["op"] == "route":
        return {"bytes": 4 * c["tokens"] * c["experts"] + 8 * c["tokens"] * c["k"] + 4 * c["experts"] * c["bias"],
                "flops": 0}
    if c["op"] == "rope":
        return {"bytes": c["tokens"] * c["d"] * (2 * c["hkv"] * 3 + 4 * c["hq"]), "flops": 0}
    new, lens = _chunk_lens(c)
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(new, lens))
    return {"bytes": 2 * c["hkv"] * c["d"] * sum(lens) + c["tokens"] * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "route": _exact_route, "rope": _exact_rope, "chunk": _exact_chunk}[case["op"]](s)


def _exact_norm(s):
    def normed(x, w):
        return x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * w.double()

    n = s["a"].double()
    if s["post"] is not None:
        n = normed(n, s["post"])
    y = s["x"].double() + s["scale"] * n * (1.0 if s["gate"] is None else s["gate"].double())
    return {"y": y, "h": normed(y, s["pre"])} if s["pre"] is not None else {"y": y}


def _exact_route(s):
    """Weights by repeated selection of the largest key that is left."""
    c = s["case"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
    key = score + (0.0 if s["bias"] is None else s["bias"].double())
    each = c["experts"] // c["groups"]
    if c["top"] < c["groups"]:
        left, rank = key.clone().view(-1, c["groups"], each), 0.0
        for _ in range(c["best"]):
            top, at = left.max(-1, keepdim=True)
            rank = rank + top[..., 0]
            left.scatter_(-1, at, -math.inf)
        keep = torch.zeros_like(key)
        for _ in range(c["top"]):
            at = rank.argmax(-1, keepdim=True)
            rank = rank.scatter(-1, at, -math.inf)
            keep += torch.nn.functional.one_hot(at[:, 0], c["groups"]).repeat_interleave(each, -1)
        key = torch.where(keep > 0, key, -math.inf)
    picked = []
    for _ in range(c["k"]):
        at = key.argmax(-1, keepdim=True)
        picked.append(score.gather(-1, at))
        key = key.scatter(-1, at, -math.inf)
    w = torch.cat(picked, -1)
    return {"idx": None, "w": s["scale"] * w / (w.sum(-1, keepdim=True) + 1e-20)}


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


def _turned64(c, x, pos, inv_freq):
    """Rows x [n, heads, d] as complex numbers times e**(i p f)."""
    r = c["rot"]
    z = x[..., :r].double()
    z = torch.complex(z[..., :r // 2], z[..., r // 2:]) if c["pairs"] == "halves" else torch.view_as_complex(
        z.unflatten(-1, (r // 2, 2)).contiguous())
    t = pos.double()[:, None] * inv_freq.double()
    z = z * torch.polar(torch.ones_like(t), t)[:, None]
    z = torch.cat([z.real, z.imag], -1) if c["pairs"] == "halves" else torch.view_as_real(z).flatten(-2)
    return torch.cat([z, x[..., r:].double()], -1)


def _exact_rope(s):
    c = s["case"]
    if c["tokens"] * c["hkv"] // c["page"] + c["n_seq"] * c["hkv"] > 20000:
        return None
    page = c["page"]
    ln, st = _parts(c["tokens"], c["n_seq"], c["split"]), _starts(c)
    pos = torch.cat([torch.arange(a, a + n, device=DEV) for a, n in zip(st, ln)])
    pt = s["pt"].tolist()
    res = {"k_scales": None, "v_scales": None, "q": _turned64(c, s["q"], pos, s["inv_freq"])}
    for n, x, codes, scales in (("k", _turned64(c, s["k"], pos, s["inv_freq"]), s["kc"], s["ks"]),
                                ("v", s["v"].double(), s["vc"], s["vs"])):
        val, byte = _values64(codes), scales.tolist()
        t0 = 0
        for b, (m, p0) in enumerate(zip(ln, st)):
            at = p0
            while at < p0 + m:
                pg, slot = pt[b][at // page], at % page
                n_here = min(page - slot, p0 + m - at)
                xs = x[t0 + at - p0:t0 + at - p0 + n_here]
                top = xs.abs().amax((0, 2)).tolist()
                for h in range(c["hkv"]):
                    e = max(_power64(top[h]), byte[pg][h] - 127 if slot else -127)
                    if slot:
                        val[pg, h, :slot] = _round64(val[pg, h, :slot] * 2.0 ** (byte[pg][h] - 127 - e))
                    val[pg, h, slot:slot + n_here] = _round64(xs[:, h] * 2.0 ** -e)
                at += n_here
            t0 += m
        res[n] = val
    return res


def _exact_chunk(s):
    c = s["case"]
    g, d, page = c["hq"] // c["hkv"], c["d"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    new, lens = _chunk_lens(c)
    t0 = 0
    for b, (nq, nk) in enumerate(zip(new, lens)):
        pages = s["pt"][b, :-(-nk // page)].long()
        seen = torch.arange(nk, device=DEV)[None] <= torch.arange(nq, device=DEV)[:, None] + (nk - nq)
        for h in range(c["hkv"]):
            k, v = ((_values64(x[pages, h]) * torch.exp2(sc[pages, h].double() - 127)[:, None, None]).reshape(-1, d)[:nk]
                    for x, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for i in range(h * g, (h + 1) * g):
                sc = (s["q"][t0:t0 + nq, i].double() @ k.T) / math.sqrt(d)
                sc = torch.where(seen, sc, -math.inf)
                lse[t0:t0 + nq, i] = torch.logsumexp(sc, -1)
                out[t0:t0 + nq, i] = torch.exp(sc - lse[t0:t0 + nq, i, None]) @ v
        t0 += nq
    return {"out": out, "lse": lse}
