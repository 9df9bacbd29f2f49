"""Attention, the 8-bit key/value cache and eviction in fp64 — TEST INFRASTRUCTURE.

Only tests may use it. The formulas are softmax(scale q K^T) V over what a
query sees, E4M3 codes with one E8M0 scale per (page, key/value head) (OCP MX
v1.0 element and scale formats), and a selection by accumulated weight.

Pins (tests/test_oracle_attention.py): attention against torch's softmax in
float64, against a dense matrix product where all keys are equal, and for
rows that see nothing; the scale rule against a search over all powers of two;
codes against torch's float8_e4m3fn conversion; selection against a sort.
"""
from __future__ import annotations

import math

import numpy as np

from . import mxfp8


def attend(q, k, v, seen, scale):
    """One head: q [R, D], k, v [L, D]; row r sees keys [0, seen[r]).

    Returns a dict of fp64 arrays: out [R, D]; lse [R]; mass [R, D] = sum p |v|
    (what an error in p is multiplied with); size [R] = the largest
    scale * sum |q k| over the keys seen (what an error in a score grows
    with); weights [R, L] = the probabilities (0 where not seen)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    R, L = q.shape[0], k.shape[0]
    r = {"out": np.zeros((R, v.shape[1])), "lse": np.full(R, -np.inf), "mass": np.zeros((R, v.shape[1])),
         "size": np.zeros(R), "weights": np.zeros((R, L))}
    for i in range(R):
        n = int(min(max(seen[i], 0), L))
        if n == 0:
            continue
        s = scale * (k[:n] @ q[i])
        m = np.max(s)
        e = np.exp(s - m)
        p = e / e.sum()
        r["out"][i] = p @ v[:n]
        r["lse"][i] = m + math.log(e.sum()) if np.isfinite(m) else m
        r["mass"][i] = p @ np.abs(v[:n])
        r["size"][i] = abs(scale) * np.max(np.abs(k[:n]) @ np.abs(q[i]))
        r["weights"][i, :n] = p
    return r


def scale_byte(amax: float) -> int:
    """E8M0 byte of the smallest 2^e >= 2^-127 with amax <= 448 * 2^e; 0 for 0."""
    if not amax > 0:
        return 0
    m, e = math.frexp(amax)
    e = e - 9 + (1 if m > 448 / 512 else 0)
    return min(max(e + 127, 0), 254)


def encode(x, byte):
    """E4M3 codes of x in units of 2^(byte - 127); inf and NaN become 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    c = mxfp8.round_to_e4m3(np.where(ok, x, 0.0) * math.ldexp(1.0, 127 - byte))
    return np.where(ok, c, 0x7F).astype(np.uint8)


def decode(codes, byte):
    """Values of codes; the byte broadcasts."""
    return mxfp8.e4m3_decode(codes) * np.ldexp(1.0, np.asarray(byte, dtype=np.int64) - 127)


def rescale(codes, old, new):
    """Codes of one scale in units of a larger one: rounded once more, NaN kept."""
    v = mxfp8.e4m3_decode(codes)
    c = mxfp8.round_to_e4m3(np.where(np.isnan(v), 0.0, v) * math.ldexp(1.0, old - new))
    return np.where(np.isnan(v), np.asarray(codes) & 0x80 | 0x7F, c).astype(np.uint8)


def append(codes, scales, x, start, table, first_row=0):
    """Append rows x [n, H, D] of one sequence at position `start` (arrays changed in place)."""
    x = np.asarray(x, dtype=np.float64)
    P, H = codes.shape[2], codes.shape[1]
    at, n = start, x.shape[0]
    while at < start + n:
        page, slot = int(table[at // P]), at % P
        m = min(P - slot, start + n - at)
        part = x[at - start:at - start + m]
        for h in range(H):
            fin = np.abs(part[:, h][np.isfinite(part[:, h])])
            byte = scale_byte(float(fin.max()) if fin.size else 0.0)
            if slot:
                old = int(scales[page, h])
                byte = max(byte, old)
                if byte != old:
                    codes[page, h, :slot] = rescale(codes[page, h, :slot], old, byte)
            codes[page, h, slot:slot + m] = encode(part[:, h], byte)
            scales[page, h] = byte
        at += m


def sequence(codes, scales, table, h, n):
    """Values [n, D] of a sequence's first n positions, head h."""
    P = codes.shape[2]
    out = np.zeros((n, codes.shape[3]))
    for p0 in range(0, n, P):
        page = int(table[p0 // P])
        m = min(P, n - p0)
        out[p0:p0 + m] = decode(codes[page, h, :m], int(scales[page, h]))
    return out


def select(weights, keep, recent):
    """Positions kept of len(weights), ascending."""
    w = np.asarray(weights, dtype=np.float64)
    n = len(w)
    if n <= keep:
        return list(range(n))
    w = np.where(np.isnan(w), -np.inf, w)
    best = sorted(range(n - recent), key=lambda i: (-w[i], i))[:keep - recent]
    return sorted(best) + list(range(n - recent, n))


def repage(x, P):
    """Values [n, D] -> list of (codes [m, D], byte) per page of P positions."""
    out = []
    for i in range(0, len(x), P):
        part = x[i:i + P]
        fin = np.abs(part[np.isfinite(part)])
        byte = scale_byte(float(fin.max()) if fin.size else 0.0)
        out.append((encode(part, byte), byte))
    return out
