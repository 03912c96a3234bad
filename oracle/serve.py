"""A serving step of drafted trees in fp64 numpy: norms and rotation of queries
and keys, append to and attention over a cache held in 8 bits, and the verify of
a tree against probabilities.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Everything is written row by
row and node by node from the definitions in include/sd_serve.h.  Parity: pinned
by closed forms, identities and brute force in tests/test_oracle_serve.py.
"""
import math
from fractions import Fraction

import numpy as np

from .tree import attend, visible_nodes

TOP = {"i8": 127.0, "e4m3": 448.0}
MIN_SCALE, MAX_SCALE = np.float32(2.0 ** -50), np.float32(2.0 ** 50)


# 2 pi times 2^200, to the nearest (pi to 64 digits).
TWO_PI = round(2 * Fraction("3.141592653589793238462643383279502884197169399375105820974944592") * 2 ** 200)


def turned(position, freq):
    """position * freq (an fp32 number) reduced to one turn, in whole numbers: products of
    far positions lose bits in fp64."""
    num, den = (int(position) * Fraction(float(freq))).as_integer_ratio()
    return ((num << 200) // den % TWO_PI) / 2 ** 200


def norm_rope_ref(x, weight, positions, inv_freq, eps, interleaved=False):
    """Heads x [N][H][D] normed and rotated."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    half = len(inv_freq)
    out = y.copy()
    for n, pos in enumerate(positions):
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            t = turned(pos, inv_freq[j])
            c, s = math.cos(t), math.sin(t)
            out[n, :, a] = y[n, :, a] * c - y[n, :, b] * s
            out[n, :, b] = y[n, :, b] * c + y[n, :, a] * s
    return out


def e4m3_round(x):
    """Nearest e4m3 value of fp64 numbers within +-448, ties to even mantissa."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(x / step) * step


def quant_scale(amax, code):
    """fp32 scale of a largest magnitude."""
    if not amax > 0:
        return np.float32(0)
    return np.clip(np.float32(amax) / np.float32(TOP[code]), MIN_SCALE, MAX_SCALE)


def quant_codes(x, scale, code):
    """fp32 numbers x as codes of a scale; in fp32, as the definition has it."""
    x = np.asarray(x, dtype=np.float32)
    inv = np.float32(1) / np.float32(scale) if scale > 0 else np.float32(0)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.clip(x * inv, -np.float32(TOP[code]), np.float32(TOP[code]))
    y = np.where(np.isnan(x), 0, np.where(np.isinf(x), np.sign(x) * TOP[code], y)).astype(np.float64)
    return np.rint(y) if code == "i8" else e4m3_round(y)


def quant_append_ref(new, codes, scales, table, ctx, block, code):
    """Rows `new` [m][H][D] of one request appended in place to codes
    [pages][H][page][D] and scales [pages][H][page / block]."""
    pages, H, page, _ = codes.shape
    m = len(new)
    for start in range(ctx // block * block, ctx + m, block):
        p = int(table[start // page])
        if not 0 <= p < pages:
            continue
        lo, hi = max(ctx, start), min(ctx + m, start + block)
        at, blk = start % page, start % page // block
        for h in range(H):
            rows = np.asarray(new[lo - ctx:hi - ctx, h], dtype=np.float32)
            fine = np.abs(rows[np.isfinite(rows)])
            old = np.float32(scales[p, h, blk]) if lo > start else np.float32(0)
            if not (old == 0 or MIN_SCALE <= old <= MAX_SCALE):
                old = np.float32(0)
            scale = np.maximum(old, quant_scale(fine.max() if fine.size else 0, code))
            if lo > start and scale > old:
                was = codes[p, h, at:at + lo - start]
                codes[p, h, at:at + lo - start] = quant_codes(was.astype(np.float32) * old, scale, code)
            codes[p, h, at + lo - start:at + hi - start] = quant_codes(rows, scale, code)
            scales[p, h, blk] = scale


def depths(T, parents=None):
    return visible_nodes(T, parents).sum(1) - 1


def quant_rows(codes, scales, other, table, n, h, block):
    """Slots 0..n-1 of a request for head h as fp64 [n][D], and which of them are
    there: on a page of the pool, both scales (`other`: those of the values for the
    keys and the other way round) within their range."""
    pages, _, page, D = codes.shape
    out, there = np.zeros((n, D)), np.zeros(n, dtype=bool)
    for t in range(n):
        p = int(table[t // page])
        if not 0 <= p < pages:
            continue
        s = [np.float32(x[p, h, t % page // block]) for x in (scales, other)]
        there[t] = all(v == 0 or MIN_SCALE <= v <= MAX_SCALE for v in s)
        if there[t] and s[0] > 0:
            out[t] = np.nan_to_num(codes[p, h, t % page].astype(np.float64)) * float(s[0])
    return out, there


def quant_attention_ref(q, k_new, v_new, k, v, ks, vs, table, lens, offsets, block, scale, parents=None,
                        window=0, sinks=0):
    """(out, lse, weighted |v|) of all packed nodes; rows of no request are NaN."""
    N, Hq, D = q.shape
    H = k_new.shape[1]
    out, lse, mag = np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan), np.full((N, Hq, D), np.nan)
    for b in range(len(lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(lens[b])
        up = None if parents is None else parents[lo:hi]
        sees, deep = visible_nodes(hi - lo, up), depths(hi - lo, up)
        at = np.concatenate([np.arange(n), n + deep])
        for h in range(H):
            kc, there = quant_rows(k, ks, vs, table[b], n, h, block)
            vc, _ = quant_rows(v, vs, ks, table[b], n, h, block)
            kk, vv = np.concatenate([kc, k_new[lo:hi, h]]), np.concatenate([vc, v_new[lo:hi, h]])
            for i in range(lo, hi):
                seen = np.concatenate([there, sees[i - lo]])
                if window:
                    seen &= (at < sinks) | (n + deep[i - lo] - at < window)
                for g in range(h * Hq // H, (h + 1) * Hq // H):
                    out[i, g], lse[i, g], mag[i, g] = attend(q[i, g], kk, vv, seen, scale)
    return out, lse, mag


def tree_sample_ref(p, q, tokens, parents, offsets, max_nodes, u, v, no_bonus=False, no_replacement=False):
    """(accepted, path, tokens, margin) of requests without defects: p [N][V], q
    [N][V_draft] or None.  margin [B]: how near the nearest decision of the
    request came to going the other way."""
    B, V = len(offsets) - 1, p.shape[1]
    acc = np.zeros(B, dtype=np.int32)
    path, out = np.full((B, max_nodes), -1, dtype=np.int32), np.full((B, max_nodes), -1, dtype=np.int32)
    margin = np.full(B, np.inf)
    for b in range(B):
        lo, T = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        cur, n = 0, 0
        while True:
            path[b, n] = cur
            kids = [c for c in range(cur + 1, T) if parents[lo + c] == cur]
            P = p[lo + cur].astype(np.float64)
            if no_bonus and not kids:
                break
            left = P.copy()                  # the residual, not normalised
            Z = 1.0
            Q = np.zeros(V)
            if q is not None:
                Q[:q.shape[1]] = q[lo + cur]
            cut, rate, gone, took = 0.0, 1.0, 0.0, None
            for c in kids:
                x, r = int(tokens[lo + c]), float(u[lo + c])
                need, have = (r * Q[x] * rate * Z, left[x]) if q is not None else (r * Z, left[x])
                margin[b] = min(margin[b], abs(need - have))
                if need < have:
                    took = c
                    break
                if q is not None:
                    cut += Z * rate
                    gone += Q[x]
                    left = np.maximum(P - cut * Q, 0)
                    Z = left.sum()
                    if no_replacement:
                        rate = 1.0 / (1.0 - gone) if gone < 1.0 else 0.0
                    if Z == 0:
                        left = P.copy()
                        break
                else:
                    Z -= left[x]
                    left[x] = 0.0
            if took is None:
                if kids and not left.any():      # (without draft rows: all that p holds was given and rejected)
                    left = P.copy()
                C = np.cumsum(left)
                t = float(v[b]) * C[-1]
                out[b, n] = min(int(np.searchsorted(C, t, side="right")), V - 1)
                while out[b, n] > 0 and left[out[b, n]] == 0:      # rounding at the last of the sum
                    out[b, n] -= 1
                if v[b] > 0:
                    margin[b] = min(margin[b], np.abs(C[C > 0] - t).min())
                break
            out[b, n] = tokens[lo + took]
            cur, n = took, n + 1
        acc[b] = n
    return acc, path, out, margin

