"""Plain 64-bit models of what a decode loop does with the paged cache besides attending to it (accumulated
weights, eviction, beam selection, reordering), written from their definitions (numpy, on the CPU)."""

from __future__ import annotations

import math

import numpy as np

import cache_reference as R

D = 512


def weights(q, codes, scales, table, cu, lens, lse, earlier, decay, before, page, block, scale=None):
    """(weights [B, W], their bound): `before` is what the output tensor holds before the call.

    The bound counts, for a term w = exp(s - lse): s is an fp32 sum of 512 exact products, off by at most
    512 * 2^-23 * sum |q x| (truncating adders count) and, where q's parts do not hold a small value, by
    2^-22 of its row's largest a product; the factors scale, block scale and log2(e), lse times log2(e), their
    difference and the base-2 exponential a few 2^-23 of their sizes. Together d: the term is off by w (e^d - 1). The
    sum of n terms and of decay * earlier (two roundings) adds n + 4 of its own roundings.
    """
    scale = scale if scale is not None else 1.0 / math.sqrt(D)
    out = before.astype(np.float64).copy()
    bound = np.zeros_like(out)
    for b in range(table.shape[0]):
        mine = [t for t in range(cu[b], cu[b + 1]) if lens[t] > 0]
        n = max([int(lens[t]) for t in mine], default=0)
        if n == 0:
            continue
        x, _, _ = R.rows_of(codes, scales, table[b], np.arange(n), page, block)
        total, off, terms = np.zeros(n), np.zeros(n), 0
        for t in mine:
            xs = x[: lens[t]]
            s = scale * (q[t] @ xs.T)
            l = lse[t][:, None].astype(np.float64)
            fine = ~np.isneginf(l)
            d = scale * (512 * 2.0 ** -23 * (np.abs(q[t]) @ np.abs(xs).T)
                         + 2.0 ** -22 * np.abs(q[t]).max(axis=1)[:, None] * np.abs(xs).sum(axis=1)[None, :])
            d = d + 2.0 ** -20 * (np.abs(s) + np.where(fine, np.abs(l), 0.0) + 1.0)
            w = np.where(fine, np.exp(s - np.where(fine, l, 0.0)), 0.0)
            total[: lens[t]] += w.sum(axis=0)
            off[: lens[t]] += (w * np.expm1(d)).sum(axis=0)
            terms += q.shape[1]
        e = decay * earlier[b, :n].astype(np.float64) if decay else np.zeros(n)
        out[b, :n] = e + total
        bound[b, :n] = 1.01 * off + (terms + 4) * 2.0 ** -23 * (np.abs(e) + total) + 1e-37
    return out, bound


def choose(w, n, keep, first, recent):
    """Positions of a sequence of n that stay, ascending (w: its weights)."""
    if n <= keep:
        return list(range(n))
    forced = set(range(first)) | set(range(n - recent, n))
    rest = [p for p in range(n) if p not in forced]
    rest.sort(key=lambda p: (not math.isnan(w[p]), 0.0 if math.isnan(w[p]) else w[p], -p), reverse=True)
    return sorted(forced | set(rest[: keep - first - recent]))


def evict(codes, scales, refcount, table, lens, w, keep, first, recent, page, block):
    """(new_table, new_lens, new_weights, kept), in place on the pool; None (nothing changed) with too few pages."""
    B = len(lens)
    picks = [choose(w[b], int(lens[b]), keep, first, recent) for b in range(B)]
    free = [i for i, c in enumerate(refcount) if c == 0]
    if sum(-(-len(p) // page) for p in picks) > len(free):
        return None
    new_table = np.full_like(table, -1)
    new_weights = np.zeros_like(w)
    kept = np.full((B, keep), -1, dtype=np.int32)
    for b, at in enumerate(picks):
        kept[b, : len(at)] = at
        new_weights[b, : len(at)] = w[b, at]
        for j in range(0, len(at), page):
            to = free.pop(0)
            new_table[b, j // page], refcount[to] = to, 1
            for k in range(j, min(j + page, len(at)), block):
                src = at[k: min(k + block, j + page, len(at))]
                pg = [int(table[b, p // page]) for p in src]
                there = [0 <= g < len(codes) for g in pg]
                sc = np.array([scales[g, p % page // block] if ok else 0.0 for g, p, ok in zip(pg, src, there)],
                              dtype=np.float32)
                big = sc.max()
                for r, (g, p) in enumerate(zip(pg, src)):
                    row = codes[g, p % page] if there[r] else np.zeros(D, np.uint8)
                    if sc[r] != big:
                        row = R.encode(R.VALUES[row] * (float(sc[r]) / float(big)))
                    codes[to, k - j + r] = row
                scales[to, (k - j) // block] = big
    return new_table, np.array([len(p) for p in picks], dtype=np.int32), new_weights, kept


def select(logits, scores, n, done=None, eos=-1):
    """(parents, tokens, scores in 64 bits) of logits [B*K, V] float64."""
    B, K = scores.shape
    V = logits.shape[1]
    parents, tokens = np.full((B, n), -1), np.full((B, n), -1)
    best = np.full((B, n), -np.inf)
    with np.errstate(all="ignore"):
        for b in range(B):
            score, flat = [], []
            for k in range(K):
                s = float(scores[b, k])
                if done is not None and done[b, k]:
                    score.append(np.array([s])), flat.append(np.array([k * V + eos]))
                    continue
                x = logits[b * K + k]
                top = x.max() if not np.isnan(x).any() else np.nan
                lse = top + np.log(np.exp(x - top).sum())
                score.append(s + (x - lse)), flat.append(k * V + np.arange(V))
            score, flat = np.concatenate(score), np.concatenate(flat)
            fine = np.isfinite(score)
            score, flat = score[fine], flat[fine]
            order = np.lexsort((flat, -score))[:n]
            m = len(order)
            parents[b, :m], tokens[b, :m], best[b, :m] = b * K + flat[order] // V, flat[order] % V, score[order]
    return parents, tokens, best


def reorder(codes, scales, refcount, table, lens, parents, page, w=None):
    """(new_table, new_lens, new_weights), in place on the pool; None (nothing changed) with too few pages."""
    n = len(parents)
    heir = {}
    for i, p in enumerate(parents):
        if p >= 0:
            heir.setdefault(int(p), i)
    ended = [p for p in range(len(lens)) if p not in heir]
    spare = []
    for p in ended:
        if lens[p] % page:
            e = int(table[p, lens[p] // page])
            if refcount[e] == 1:
                spare.append(e)
    copies = [i for i, p in enumerate(parents) if p >= 0 and heir[int(p)] != i and lens[p] % page]
    free = [i for i, c in enumerate(refcount) if c == 0]
    if len(copies) > len(spare) + len(free):
        return None
    to = dict(zip(copies, spare + free))
    new = np.full((n, table.shape[1]), -1, dtype=np.int32)
    new_w = None if w is None else np.zeros((n, w.shape[1]), dtype=w.dtype)
    for p in ended:
        for e in table[p]:
            if e >= 0:
                refcount[e] -= 1
    for i, p in enumerate(parents):
        if p < 0:
            continue
        full = lens[p] // page
        if heir[int(p)] == i:
            new[i] = table[p]
        else:
            new[i, :full] = table[p, :full]
            for e in table[p, :full]:
                refcount[e] += 1
            if i in to:
                new[i, full] = to[i]
                refcount[to[i]] = 1
                codes[to[i]], scales[to[i]] = codes[table[p, full]], scales[table[p, full]]
        if w is not None:
            new_w[i, : lens[p]] = w[p, : lens[p]]
    return new, np.array([lens[p] if p >= 0 else 0 for p in parents], dtype=np.int32), new_w
