"""Norms around a block's halves, routing by groups and the position rotation in fp64 — TEST INFRASTRUCTURE.

Only tests may use it. Pins (tests/test_oracle_block.py): the norm against torch's rms_norm in float64, routing against
a search over all subsets of groups and experts, the rotation against complex multiplication and exact integers.
"""
from __future__ import annotations

import numpy as np

FMAX = float(np.finfo(np.float32).max)


def rstd(z, eps):
    z = np.asarray(z, dtype=np.float64)
    return 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)


def block_norm(x, a=None, post=None, gate=None, scale=1.0, pre=None, eps=1e-6, offset=0.0):
    """y (None without a) and h of the definition; also the term scale * gate * n that is added."""
    x = np.asarray(x, dtype=np.float64)
    if a is None:
        y, add = x, np.zeros_like(x)
    else:
        n = np.asarray(a, dtype=np.float64)
        if post is not None:
            n = n * rstd(n, eps) * (offset + np.asarray(post, dtype=np.float64))
        add = scale * n * (1.0 if gate is None else np.asarray(gate, dtype=np.float64))
        y = x + add
    w = 1.0 if pre is None else offset + np.asarray(pre, dtype=np.float64)
    return {"y": None if a is None else y, "h": y * rstd(y, eps) * w, "add": add, "w": w, "sum": y}


def scores(logits, kind):
    """(scores, whether a logit is NaN): infinities count as the largest finite numbers, NaN scores 0."""
    l = np.asarray(logits, dtype=np.float64)
    nan = np.isnan(l)
    l = np.clip(np.where(nan, 0.0, l), -FMAX, FMAX)
    if kind == "sigmoid":
        e = np.exp(-np.abs(l))
        s = np.where(l >= 0, 1 / (1 + e), e / (1 + e))
    else:
        l = np.where(nan, -np.inf, l)
        top = l.max(-1, keepdims=True)
        e = np.where(nan, 0.0, np.exp(l - np.where(np.isfinite(top), top, 0.0)))
        s = e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
    return np.where(nan, 0.0, s), nan


def _keys(l, s, nan, bias, best):
    """Keys of one token's experts, and what counts for their groups."""
    # without a bias the logits rank: scores are monotone in them, and they tell more of them apart
    key = np.clip(l, -FMAX, FMAX) if bias is None else s + np.asarray(bias, dtype=np.float64)
    key = np.where(nan | np.isnan(key), -np.inf, key)
    return key, key if bias is not None or best == 1 else np.where(nan, -np.inf, s)


def _ranks(member, n_groups, best):
    """Sums of each group's best; with an infinite one it is that, the larger of two."""
    best_of = [sorted(m, reverse=True)[:best] for m in np.asarray(member).reshape(n_groups, -1)]
    return np.array([m[0] if np.isposinf(m[0]) else sum(m) for m in best_of])


def group_ranks(l, bias, kind, n_groups, best=2):
    """The scores of one token's groups."""
    s, nan = scores(l[None], kind)
    return _ranks(_keys(np.asarray(l, dtype=np.float64), s[0], nan[0], bias, best)[1], n_groups, best)


def route_groups(logits, k, bias=None, kind="sigmoid", n_groups=1, top=1, best=2, renormalise=True, scale=1.0, groups=None):
    """idx int [T, k], w fp64 [T, k]; plain Python per token. groups: these instead of the best ones."""
    l = np.asarray(logits, dtype=np.float64)
    s, nan = scores(l, kind)
    T, E = l.shape
    size = E // n_groups
    idx, w = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    for t in range(T):
        key, member = _keys(l[t], s[t], nan[t], bias, best)
        rank = _ranks(member, n_groups, best)
        chosen = groups or sorted(range(n_groups), key=lambda g: (-rank[g], g))[:top]
        left = [e for g in sorted(chosen) for e in range(g * size, (g + 1) * size)]
        idx[t] = sorted(left, key=lambda e: (-key[e], e))[:k]
        w[t] = s[t, idx[t]]
        if renormalise:
            w[t] /= w[t].sum() + 1e-20
    return idx, w * scale


def rotate(x, pos, inv_freq, interleaved):
    """Rows x [n, heads, d] at positions pos [n]: their first 2 len(inv_freq) channels turned."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    r = 2 * len(f)
    t = np.asarray(pos, dtype=np.float64)[:, None] * f
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def pair_size(x, r, interleaved):
    """|a| + |b| of the pair that a channel belongs to (its own size beyond the first r)."""
    m = np.abs(np.asarray(x, dtype=np.float64))
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    y = m.copy()
    y[..., i] = y[..., j] = m[..., i] + m[..., j]
    return y
