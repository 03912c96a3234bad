"""Tree drafting in fp64 numpy: attention of a drafted tree over a paged
cache, greedy verify of a tree, append of the kept branch with the weight it
gives to the cached tokens, eviction by that weight, and a beam step.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Everything is written
slot by slot and node by node from the definitions in include/sd_tree.h; no
page names no tile.  Parity: pinned by closed forms and brute force in
tests/test_oracle_tree.py.
"""
import math

import numpy as np


def visible_nodes(T, parents=None, mask=None):
    """[T][T] bool: which nodes of its tree node i sees."""
    sees = np.zeros((T, T), dtype=bool)
    for i in range(T):
        if mask is not None:
            for j in range(T):
                sees[i, j] = (int(mask[i]) >> j) & 1
        elif parents is None:
            sees[i, :i + 1] = True
        else:
            j = i
            while j >= 0:
                sees[i, j] = True
                j = int(parents[j]) if -1 <= parents[j] < j else -1
    return sees


def cache_rows(cache, table, n, h):
    """Slots 0..n-1 of a request for head h as fp64 [n][D], and which of them
    are on a page of the pool."""
    pages, _, page, D = cache.shape
    out, there = np.zeros((n, D)), np.zeros(n, dtype=bool)
    for t in range(n):
        p = int(table[t // page])
        if 0 <= p < pages:
            out[t], there[t] = cache[p, h, t % page], True
    return out, there


def attend(q, k, v, seen, scale):
    """One row: (out [D], lse, sum of |v| weighted by the softmax)."""
    if not seen.any():
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1])
    x = scale * (k[seen] @ q)
    m = x.max()
    p = np.exp(x - m)
    s = p.sum()
    return (p @ v[seen]) / s, m + math.log(s), (p @ np.abs(v[seen])) / s


def tree_attention_ref(q, k_new, v_new, k_cache, v_cache, table, lens, offsets, scale,
                       parents=None, mask=None):
    """(out, lse, weighted |v|) of all packed nodes; rows of no request are NaN."""
    N, Hq, D = q.shape
    H = k_new.shape[1]
    out, lse, mag = np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan), np.full((N, Hq, D), np.nan)
    for b in range(len(lens)):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        sees = visible_nodes(hi - lo, None if parents is None else parents[lo:hi],
                             None if mask is None else mask[lo:hi])
        for h in range(H):
            kc, there = cache_rows(k_cache, table[b], int(lens[b]), h)
            vc, _ = cache_rows(v_cache, table[b], int(lens[b]), h)
            k, v = np.concatenate([kc, k_new[lo:hi, h]]), np.concatenate([vc, v_new[lo:hi, h]])
            for g in range(h * Hq // H, (h + 1) * Hq // H):
                for i in range(lo, hi):
                    out[i, g], lse[i, g], mag[i, g] = attend(
                        q[i, g], k, v, np.concatenate([there, sees[i - lo]]), scale)
    return out, lse, mag


def tree_verify_greedy_ref(logits, tokens, parents, offsets, max_nodes, no_bonus=False):
    """(accepted, path, tokens) of requests without defects."""
    B = len(offsets) - 1
    acc = np.zeros(B, dtype=np.int32)
    path, out = np.full((B, max_nodes), -1, dtype=np.int32), np.full((B, max_nodes), -1, dtype=np.int32)
    for b in range(B):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        cur, n = 0, 0
        while True:
            path[b, n] = cur
            kids = [c for c in range(cur + 1, hi - lo) if parents[lo + c] == cur]
            if no_bonus and not kids:
                break
            best = int(np.argmax(logits[lo + cur]))     # the first of equal maxima
            out[b, n] = best
            kids = [c for c in kids if tokens[lo + c] == best]
            if not kids:
                break
            cur, n = kids[0], n + 1
        acc[b] = n
    return acc, path, out


def commit_weights_ref(q, lse, k_new, k_cache, table_row, ctx, rows, h, scale):
    """Weight of slots 0..ctx+len(rows)-1 of one request and KV head: q and
    lse of that head's group [N][G][D], [N][G]; rows: the branch's packed rows."""
    k, there = cache_rows(k_cache, table_row, ctx, h)
    w = np.zeros(ctx + len(rows))
    for i, r in enumerate(rows):
        for g in range(q.shape[1]):
            if lse[r, g] == -math.inf:      # the row saw nothing
                continue
            w[:ctx] += np.where(there, np.exp(scale * (k @ q[r, g]) - lse[r, g]), 0.0)
            for j in range(i + 1):
                w[ctx + j] += math.exp(scale * float(k_new[rows[j], h] @ q[r, g]) - lse[r, g])
    return w


def evict_ref(mass, positions, n, seen, budget, recent, sinks):
    """(source slot of each of the slots kept, in their new order)."""
    def rank(t):
        if positions is not None and (positions[t] < sinks or positions[t] >= seen - recent):
            return (0, 0.0, t)
        return (1, math.inf if math.isnan(mass[t]) else -float(mass[t]), t)
    kept = set(sorted(range(n), key=rank)[:budget])
    late = [t for t in range(n) if t in kept and t >= budget]
    return [t if t in kept else late.pop(0) for t in range(min(n, budget))]


def beam_select_ref(logits, scores, n_out, ended=None, eos=-1):
    """[(score, beam, token)] of one request, best first; logits fp64 [W][V]."""
    cand = []
    for w in range(len(scores)):
        if not scores[w] > -math.inf:
            continue
        if ended is not None and ended[w]:
            cand.append((float(scores[w]), w, eos))
            continue
        z = logits[w]
        m = z.max()
        x = float(scores[w]) + ((z - m) - math.log(np.exp(z - m).sum()))     # the level cancels first
        order = np.argsort(-z, kind="stable")[:n_out]
        cand += [(float(x[i]), w, int(i)) for i in order if z[i] > -math.inf]
    cand.sort(key=lambda c: (-c[0], c[1], c[2]))
    return cand[:n_out]
