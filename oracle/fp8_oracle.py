"""Plain float64 oracle of the grouped router, the grouping, the 8-bit quantiser and the block-scaled 8-bit layer.

Test infrastructure only: loops and tables in numpy, sharing no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
from scipy import special

NONE_ID = 0x7FFFFFFF
BLOCK = 128
LOWEST = {"float32": float(np.finfo(np.float32).min), "bfloat16": -float(2.0 ** 128 - 2.0 ** 120)}


# ---------------------------------------------------------------------------- router

def scores(row, score, lowest):
    """float64 scores of one token's logits and which experts may be chosen."""
    l = [float(v) for v in row]
    masked = [v <= lowest for v in l]
    if score == "sigmoid":
        s = [0.0 if m else (math.nan if math.isnan(v) else float(special.expit(v))) for v, m in zip(l, masked)]
    else:
        live = [v for v, m in zip(l, masked) if not m]
        if any(math.isnan(v) or v == math.inf for v in live):
            s = [0.0 if m else math.nan for m in masked]
        elif not live:
            s = [0.0] * len(l)
        else:
            top = max(live)
            ex = [0.0 if m else math.exp(v - top) for v, m in zip(l, masked)]
            total = math.fsum(ex)
            s = [v / total for v in ex]
    may = [not m and not math.isnan(v) for v, m in zip(s, masked)]
    return [v if ok else 0.0 for v, ok in zip(s, may)], may


def choose(s, may, bias, K, groups, top_groups, group_top):
    """The ids chosen for one token (NONE_ID where no expert is left)."""
    E = len(s)
    c = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in range(E) if may[e]}
    size = E // groups
    if top_groups < groups:
        ranked = []
        for g in range(groups):
            best = sorted((c[e] for e in range(g * size, (g + 1) * size) if e in c), reverse=True)[:group_top]
            if best:
                ranked.append((-sum(best), g))
        keep = {g for _, g in sorted(ranked)[:top_groups]}
        c = {e: v for e, v in c.items() if e // size in keep}
    order = sorted(c, key=lambda e: (-c[e], e))[:K]
    return order + [NONE_ID] * (K - len(order))


def gates(s, idx, renorm, scale, row=None):
    """row: the token's logits, for softmax scores (whose renormalised gates are the softmax of the chosen logits)."""
    sel = [s[e] if 0 <= e < len(s) else 0.0 for e in idx]
    if renorm and row is not None:
        top = max((float(row[e]) for e in idx if 0 <= e < len(s)), default=0.0)
        sel = [math.exp(float(row[e]) - top) if 0 <= e < len(s) else 0.0 for e in idx]
        total = math.fsum(sel)
        sel = [v / total for v in sel] if total else sel
    elif renorm:
        D = max(math.fsum(sel), 2.0 ** -126)
        sel = [v / D for v in sel]
    return [scale * v for v in sel]


def route(logits, dtype, bias, K, score, renorm, scale, groups, top_groups, group_top):
    idx, gate = [], []
    for row in logits:
        s, may = scores(row, score, LOWEST[dtype])
        idx.append(choose(s, may, bias, K, groups, top_groups, group_top))
        gate.append(gates(s, idx[-1], renorm, scale, row if score == "softmax" else None))
    return np.array(idx, np.int64).reshape(-1, K), np.array(gate, np.float64).reshape(-1, K)


def route_grad(logits, dtype, idx, dgate, score, renorm, scale):
    """Gradient of sum(dgate * gates), and the magnitude of the terms each element is formed from."""
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s, may = scores(logits[t], score, LOWEST[dtype])
        s = np.array(s)
        live = [(int(e), scale * float(u)) for e, u in zip(idx[t], dgate[t]) if 0 <= e < E and may[int(e)]]
        ds, ad = np.zeros(E), np.zeros(E)
        if score == "softmax" and renorm:
            top = max((float(logits[t, e]) for e, _ in live), default=0.0)
            g = [math.exp(float(logits[t, e]) - top) for e, _ in live]
            D = math.fsum(g) or 1.0
            us, aus = (math.fsum(v / D * f(u) for v, (_, u) in zip(g, live)) for f in (float, abs))
            for v, (e, u) in zip(g, live):
                out[t, e] += v / D * (u - us)
                mag[t, e] += v / D * (abs(u) + aus)
            continue
        D = max(math.fsum(s[e] for e, _ in live), 2.0 ** -126)
        us = math.fsum(u * s[e] for e, u in live)
        aus = math.fsum(abs(u) * s[e] for e, u in live)
        for e, u in live:
            ds[e] += (u - us / D) / D if renorm else u
            ad[e] += (abs(u) + aus / D) / D if renorm else abs(u)
        if score == "sigmoid":
            out[t], mag[t] = ds * s * (1 - s), ad * s
        else:
            out[t] = s * (ds - math.fsum(ds * s))
            mag[t] = s * (ad + math.fsum(ad * s))
    return out, mag


# ---------------------------------------------------------------------------- grouping

def group(topk_idx, E):
    T, K = topk_idx.shape
    slots = [(int(e), t * K + j) for t in range(T) for j, e in enumerate(topk_idx[t]) if 0 <= e < E]
    slots.sort()
    counts = np.zeros(E, np.int64)
    for e, _ in slots:
        counts[e] += 1
    slot_token = np.full(T * K, -1, np.int64)
    token_slot = np.full(T * K, -1, np.int64)
    for r, (_, s) in enumerate(slots):
        slot_token[r] = s // K
        token_slot[s] = r
    return counts, np.concatenate([[0], np.cumsum(counts)]), slot_token, token_slot.reshape(T, K)


# ---------------------------------------------------------------------------- 8-bit values

def e4m3(byte):
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
    return -v if s else v


TABLE = np.array([e4m3(b) for b in range(256)])
_POS = TABLE[:127]  # 0 .. 448, ascending


def nearest(v):
    """Bytes of the nearest e4m3 values (ties to even); |v| <= 448."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    b = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (b + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def exponent(top):
    """Smallest e >= -127 with top <= 448 2^e."""
    e = -127
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x, block_rows):
    """[R][C] -> bytes [R][C], scale bytes; finite values."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    q = np.zeros((R, C), np.uint8)
    sc = np.zeros((-(-R // block_rows), -(-C // BLOCK)), np.uint8)
    for i in range(sc.shape[0]):
        for j in range(sc.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
            e = exponent(np.abs(x[at]).max())
            sc[i, j] = e + 127
            q[at] = nearest(x[at] * 2.0 ** -e)
    return q, sc


def values(q, sc, block_rows):
    R, C = q.shape
    f = 2.0 ** (sc.astype(np.float64) - 127)
    return TABLE[q] * f.repeat(block_rows, 0)[:R].repeat(BLOCK, 1)[:, :C]


# ---------------------------------------------------------------------------- experts

def grouped_product(x, W, offsets, bias=None):
    """x [S][Kd] and W [E][N][Kd] as values: out [S][N] (NaN where no expert holds the row) and sums of magnitudes."""
    S, N = x.shape[0], W.shape[1]
    out, mag = np.full((S, N), np.nan), np.zeros((S, N))
    for e in range(W.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        out[r] = x[r] @ W[e].T
        mag[r] = np.abs(x[r]) @ np.abs(W[e]).T
        if bias is not None:
            out[r] += bias[e]
            mag[r] += np.abs(bias[e])
    return out, mag


def expert_ffn(x, W1, W3, W2, b1, b2, offsets, gelu):
    """Grouped rows through each expert's MLP, the hidden activation rounded to 8 bits per 128 columns."""
    S = int(offsets[-1])
    z, _ = grouped_product(x[:S], W1, offsets, b1)
    if gelu:
        a = 0.5 * z * (1.0 + special.erf(z / math.sqrt(2.0)))
    else:
        a = z * special.expit(z) * grouped_product(x[:S], W3, offsets)[0]
    a = values(*quantize(a, 1), 1) if S else a
    return grouped_product(a, W2, offsets, b2)[0]


def layer(h, logits, dtype, bias, W1, W3, W2, b1, b2, K, gelu, **router):
    E, d = W1.shape[0], h.shape[1]
    idx, gate = route(logits, dtype, bias, K, **router)
    counts, offsets, slot_token, token_slot = group(idx, E)
    x = values(*quantize(h, 1), 1)
    o = expert_ffn(x[slot_token[:offsets[-1]]], W1, W3, W2, b1, b2, offsets, gelu)
    y = np.zeros((h.shape[0], d))
    for t in range(h.shape[0]):
        for j in range(K):
            if token_slot[t, j] >= 0:
                y[t] += gate[t, j] * o[token_slot[t, j]]
    return y, idx, counts
