"""Oracle of the target's side of a cycle: appending to the paged 8-bit
cache, attention over it, and sampling with filters.  Plain loops over
sequences, heads and tokens in float64 (float32 only where a result is
defined by float32 roundings)."""
from __future__ import annotations

import numpy as np

from .dflash_oracle import e4m3_decode, e4m3_encode

MIN_SCALE_EXP = -64
WEIGHT_ONE = 2 ** 44


def block_scale(amax) -> np.float32:
    """The least power of two s >= 2^-64 with amax <= 448 s."""
    amax = float(amax)
    e = MIN_SCALE_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, p, cos, sin, interleaved=False):
    """x [..., D] float32 at position p: the first 2 * cos.shape[1]
    dimensions turned in pairs, every product and sum rounded to float32."""
    x = np.asarray(x, np.float32)
    h = cos.shape[1]
    a_ix = np.arange(0, 2 * h, 2) if interleaved else np.arange(h)
    b_ix = a_ix + (1 if interleaved else h)
    a, b = x[..., a_ix], x[..., b_ix]
    c, s = cos[p].astype(np.float32), sin[p].astype(np.float32)
    y = x.copy()
    y[..., a_ix] = a * c - b * s
    y[..., b_ix] = b * c + a * s
    return y


def kv_append(q, k, v, cos, sin, pos, n_new, table, page, k_codes, v_codes,
              k_scale, v_scale, interleaved=False):
    """q [B,Q,Hq,D], k and v [B,Q,Hkv,D] float32 values of the storage
    dtype; codes [N,Hkv,page,D] uint8 and scales [N,Hkv] are updated in
    place.  Returns q rotated (float32, rows without a token 0) and the new
    lengths."""
    B, Q = k.shape[:2]
    q_out = None if q is None else np.zeros_like(q, np.float32)
    length = np.zeros(B, np.int64)
    for b in range(B):
        p0, n = int(pos[b]), int(n_new[b])
        length[b] = p0 + n
        kb = np.array(k[b, :n], np.float32)
        vb = np.array(v[b, :n], np.float32)
        for i in range(n):
            if cos is not None:
                kb[i] = rotate(kb[i], p0 + i, cos, sin, interleaved)
            if q is not None:
                q_out[b, i] = (q[b, i] if cos is None else
                               rotate(q[b, i], p0 + i, cos, sin, interleaved))
        for pg in range(p0 // page, -(-(p0 + n) // page) if n else 0):
            lo, hi = max(p0, pg * page), min(p0 + n, (pg + 1) * page)
            pid, old = int(table[b, pg]), lo - pg * page
            for x, codes, scale in ((kb, k_codes, k_scale),
                                    (vb, v_codes, v_scale)):
                for h in range(x.shape[1]):
                    new = x[lo - p0:hi - p0, h]
                    s = block_scale(np.abs(new).max())
                    if old and scale[pid, h] > s:
                        s = scale[pid, h]
                    if old and scale[pid, h] != s:
                        val = (e4m3_decode(codes[pid, h, :old]) *
                               (float(scale[pid, h]) / float(s)))
                        codes[pid, h, :old] = e4m3_encode(
                            val.astype(np.float32))
                    scale[pid, h] = s
                    codes[pid, h, old:old + hi - lo] = e4m3_encode(
                        new / np.float32(s))
    return q_out, length


def cached(codes, scale, table_row, n, h, page):
    """The first n cached vectors of one sequence and head, float64."""
    ids = np.asarray(table_row[:-(-n // page)], np.int64)
    x = e4m3_decode(codes[ids, h]) * scale[ids, h].astype(np.float64)[
        :, None, None]
    return x.reshape(-1, codes.shape[3])[:n]


def paged_attn(q, k_codes, v_codes, k_scale, v_scale, table, kv_len, q_len,
               scale, causal=True):
    """q [B,Q,Hq,D] float64.  Returns out, lse, and the two sums a bound of
    the rounding error is made of: the largest |q| . |k| scale and
    sum p |v| of every row."""
    B, Q, Hq, D = q.shape
    Hkv, page = k_codes.shape[1:3]
    g = Hq // Hkv
    out = np.zeros(q.shape)
    lse = np.full((B, Q, Hq), -np.inf)
    size = np.zeros((B, Q, Hq))
    absv = np.zeros(q.shape)
    for b in range(B):
        n, m = int(kv_len[b]), int(q_len[b])
        if not n or not m:
            continue
        for hk in range(Hkv):
            k = cached(k_codes, k_scale, table[b], n, hk, page)
            v = cached(v_codes, v_scale, table[b], n, hk, page)
            for h in range(hk * g, (hk + 1) * g):
                for i in range(m):
                    lim = max(0, n - m + i + 1) if causal else n
                    if lim == 0:
                        continue
                    s = k[:lim] @ q[b, i, h] * scale
                    w = np.exp(s - s.max())
                    lse[b, i, h] = s.max() + np.log(w.sum())
                    p = w / w.sum()
                    out[b, i, h] = p @ v[:lim]
                    absv[b, i, h] = p @ np.abs(v[:lim])
                    size[b, i, h] = (np.abs(k[:lim]) @ np.abs(
                        q[b, i, h])).max() * abs(scale)
    return out, lse, size, absv


def sample_row(l, T, k=0, p=1.0, m=0.0, u=0.0):
    """One row: token, kept mask, and the margins of its two sums: how near
    the top-p cut and the draw came to another answer, relative to the
    total (infinite where no sum decides, or where every weight is 0 or that
    of the maximum and no rounding enters the sums)."""
    l = np.asarray(l, np.float64)
    V = l.size
    ok = l > -np.inf
    if not ok.any():
        return -1, np.zeros(V, bool), np.inf, np.inf
    order = np.lexsort((np.arange(V), -l))     # descending, ids ascending
    order = order[:ok.sum()]
    kept = np.zeros(V, bool)
    if T == 0:
        kept[order[0]] = True
        return int(order[0]), kept, np.inf, np.inf
    inv = np.float32(1) / np.float32(T)
    # (an infinite maximum weighs 1, everything else beside it 0)
    x = np.exp(np.subtract(l, l.max(), out=np.zeros(V), where=l != l.max()) *
               np.float64(inv))
    if 0 < k < V:
        order = order[:k]
    w = np.floor(x[order] * WEIGHT_ONE)
    plain = bool(np.all((w == 0) | (x[order] == 1)))
    near_p = np.inf
    if p < 1:
        before = np.cumsum(w) - w
        keep = before < np.ceil(np.float64(np.float32(p)) * w.sum())
        keep[0] = True
        edge = np.float64(np.float32(p)) * w.sum()
        near_p = np.abs(before[1:] - edge).min() / w.sum() if (
            w.size > 1 and not plain) else np.inf
        order = order[keep]
    if m > 0:
        order = order[x[order] >= m]
    kept[order] = True
    run = np.cumsum(np.where(kept, np.floor(x * WEIGHT_ONE), 0.0))
    at = np.floor(np.float64(np.float32(u)) * run[-1])
    token = int(np.searchsorted(run, at, side="right"))
    near_u = np.inf if plain else np.abs(
        run - np.float64(np.float32(u)) * run[-1]).min() / run[-1]
    return token, kept, near_p, near_u
