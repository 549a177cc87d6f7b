"""Plain 64-bit models of the paged-cache operators, written from their
definitions (numpy, on the CPU), for the GPU tests."""

from __future__ import annotations

import math

import numpy as np

D = 512


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 e4m3 codes (0x7f and 0xff: NaN)."""
    v = np.zeros(256)
    for c in range(256):
        s, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        v[c] = s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        if e == 15 and m == 7:
            v[c] = np.nan
    return v


VALUES = e4m3_values()


def encode(y: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 values nearest to y (ties to even), saturated; NaN -> 0x7f."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    out = np.zeros(y.shape, dtype=np.uint8)
    nan = np.isnan(y)
    a = np.where(nan, 0.0, np.minimum(a, 448.0))
    e = np.frexp(a)[1] - 1                       # a = m 2^e, 1 <= m < 2
    e = np.maximum(np.where(a > 0, e, -6), -6)
    k = np.rint(np.ldexp(a, 3 - e)).astype(np.int64)            # eighths of 2^e, 0..16
    code = np.where(a < 2.0 ** -6, k, ((e + 6) * 8 + k))         # 8 eighths carry into the exponent
    out[...] = code
    out |= np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    out[nan] = 0x7F
    return out


def block_scale(amax: float) -> float:
    """The least 2^e, e >= -100, with amax <= 448 * 2^e."""
    e = -100
    if amax > 0:
        e = max(-100, math.frexp(amax)[1] - 10)
        while amax > math.ldexp(448.0, e):
            e += 1
    return math.ldexp(1.0, e)


def write(codes, scales, table, start, cu, rows, page, block):
    """In place on codes [P,page,512] uint8 and scales [P,page/block]; rows float64 [n,512]."""
    for b in range(len(start)):
        pos, end = int(start[b]), int(start[b]) + int(cu[b + 1]) - int(cu[b])
        while pos < end:
            upto = min(end, (pos // block + 1) * block)
            pg, lo = int(table[b][pos // page]), pos % page
            k, kept = lo // block, lo % block
            x = rows[cu[b] + pos - start[b]: cu[b] + upto - start[b]]
            fin = np.abs(x[np.isfinite(x)])
            sc = block_scale(float(fin.max()) if fin.size else 0.0)
            if kept:
                old = float(scales[pg, k])
                if old >= sc:
                    sc = old
                else:
                    h = slice(k * block, k * block + kept)
                    codes[pg, h] = encode(VALUES[codes[pg, h]] * (old / sc))
            with np.errstate(over="ignore"):
                codes[pg, lo: lo + upto - pos] = encode(x / sc)
            scales[pg, k] = sc
            pos = upto


def rows_of(codes, scales, table_row, positions, page, block):
    """float64 rows [n,512], their scales [n] and codes' values [n,512] of positions of one sequence."""
    pg = np.asarray(table_row)[positions // page]
    slot = positions % page
    sc = scales[pg, slot // block].astype(np.float64)
    val = VALUES[codes[pg, slot]]
    return val * sc[:, None], sc, val


def attend(q, codes, scales, table, lens, page, block, topk=None, seq=None, sink=None, scale=None):
    """(o [T,H,512], lse [T,H], o_bound, lse_bound) in 64 bits.

    The bounds count, for each output element:
    * the output's rounding to bf16: 2^-8 |o|;
    * scores: q and the codes are exact, the fp32 sum over 512 products is off by at most
      gamma * sum |q x|, gamma = 512 * 2^-23 (truncating adders count), doubled for the factors scale and
      block scale, log2(e) and the base-2 exponential (each a few 2^-23 of the score): ds;
    * weights: a weight w (scaled so that the running maximum's, at the largest block scale, is at least 2^4 and none
      passes 2^8.75) is held as an e4m3 value plus an e5m2 value of what is left: 2^-4 * 2^-3 = 2^-7 of w, and for w
      below e4m3's normal range (2^-6) the rest is at most 2^-10, off by 2^-13 at most: 2^-17 of the largest weight, a
      block's scale being part of the weight and the largest block scale of the sequence its unit; 2^-16 is allowed;
    * fp32 accumulation over n ranks: n * 2^-23 of sum w |x| (and of the denominator).
    """
    T, H, _ = q.shape
    scale = scale if scale is not None else 1.0 / math.sqrt(D)
    o, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    ob, lb = np.zeros((T, H, D)), np.zeros((T, H))
    for t in range(T):
        b = t if seq is None else int(seq[t])
        pos = np.arange(lens[t]) if topk is None else topk[t][topk[t] >= 0]
        x, sc, val = rows_of(codes, scales, table[b], pos.astype(np.int64), page, block)
        n = len(pos)
        s = scale * (q[t] @ x.T)
        ds = 2 * 512 * 2.0 ** -23 * scale * (np.abs(q[t]) @ np.abs(x).T)
        if sink is not None:
            s = np.concatenate([s, sink[:, None]], axis=1)
            ds = np.concatenate([ds, np.zeros((H, 1))], axis=1)
        if s.shape[1] == 0:
            continue
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        tot = p.sum(axis=1, keepdims=True)
        lse[t] = (m + np.log(tot))[:, 0]
        p = p / tot
        dmax = ds.max(axis=1) + 2.0 ** -21 * (np.abs(s).max(axis=1) + 1)
        acc = (n + 64) * 2.0 ** -23
        lb[t] = dmax + acc + 2.0 ** -22 * np.abs(lse[t])
        w = p[:, :n]
        if n == 0:
            continue
        o[t] = w @ x
        mass = w @ np.abs(x)
        unit = w.max(axis=1) * 4 * sc.max() * 2.0 ** -18
        ob[t] = (2.0 ** -8 * np.abs(o[t]) + (2.0 ** -7 + 2 * dmax[:, None] + 2 * acc) * mass
                 + unit[:, None] * np.abs(val).sum(axis=0)[None, :] + 1e-30) * 1.01
    return o, lse, ob, lb


def alloc(refcount, table, lens, page):
    """In place; False (nothing changed) with too few pages."""
    want = [(b, j) for b in range(len(lens)) for j in range(-(-int(lens[b]) // page)) if table[b, j] == -1]
    free = [i for i, c in enumerate(refcount) if c == 0]
    if len(want) > len(free):
        return False
    for (b, j), i in zip(want, free):
        table[b, j] = i
        refcount[i] = 1
    return True


def fork(codes, scales, refcount, table, lens, parents, page):
    """child table, or None (nothing changed) with too few pages. In place on the rest."""
    free = [i for i, c in enumerate(refcount) if c == 0]
    if sum(int(lens[p]) % page > 0 for p in parents) > len(free):
        return None
    child = np.full((len(parents), table.shape[1]), -1, dtype=np.int32)
    for i, p in enumerate(parents):
        whole, rest = divmod(int(lens[p]), page)
        for j in range(whole):
            child[i, j] = table[p, j]
            refcount[table[p, j]] += 1
        if rest:
            new = free.pop(0)
            child[i, whole] = new
            refcount[new] = 1
            codes[new], scales[new] = codes[table[p, whole]], scales[table[p, whole]]
    return child


def free_rows(refcount, table, rows):
    for b in rows:
        for j in range(table.shape[1]):
            if table[b, j] >= 0:
                refcount[table[b, j]] -= 1
                table[b, j] = -1


def compact(codes, scales, refcount, table):
    """(new_table, new_refcount); in place on codes and scales."""
    n = int((refcount > 0).sum())
    src = [i for i in range(len(refcount)) if refcount[i] > 0 and i >= n]
    dst = [i for i in range(len(refcount)) if refcount[i] == 0 and i < n]
    count, to = refcount.copy(), {}
    for a, b in zip(src, dst):
        codes[b], scales[b] = codes[a], scales[a]
        count[b], count[a] = refcount[a], 0
        to[a] = b
    new = np.array([[to.get(int(v), int(v)) for v in row] for row in table], dtype=np.int32).reshape(table.shape)
    return new, count
