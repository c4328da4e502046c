"""Oracle of the target's operators around a shared prompt and a bounded
cache: appending with positions of several axes, attention under a shared
prefix, gathered attention weight, eviction, log probabilities.  Plain loops
in float64 (float32 only where a result is defined by float32 roundings)."""
from __future__ import annotations

import numpy as np

from . import target_ops as to
from .dflash_oracle import e4m3_decode, e4m3_encode


def kv_append_axes(q, k, v, cos, sin, axis_pos, axis_of, pos, n_new, table,
                   page, k_codes, v_codes, k_scale, v_scale,
                   interleaved=False):
    """to.kv_append with the angles of axis_pos [axes, B*Q], axis_of [rot/2];
    the other arguments and results as there."""
    B, Q = k.shape[:2]
    j = np.arange(cos.shape[1])
    kr, qr = np.array(k, np.float32), None if q is None else np.zeros_like(
        q, np.float32)
    for b in range(B):
        for i in range(int(n_new[b])):
            at = axis_pos[axis_of, b * Q + i]     # a row for each angle
            c, s = cos[at, j][None], sin[at, j][None]
            kr[b, i] = to.rotate(k[b, i], 0, c, s, interleaved)
            if q is not None:
                qr[b, i] = to.rotate(q[b, i], 0, c, s, interleaved)
    _, length = to.kv_append(None, kr, v, None, None, pos, n_new, table, page,
                             k_codes, v_codes, k_scale, v_scale)
    return qr, length


def shared_table(table, shared, page):
    """The page table that dflash_shared_attn reads."""
    t = np.array(table)
    t[:, :shared // page] = t[0, :shared // page]
    return t


def attn_mass(q, k_codes, k_scale, table, kv_len, q_len, lse, fresh, first,
              scale, decay, mass, causal=True):
    """mass [B, Hkv, slots] float64, returned anew; also the sum over the
    rows of |q| . |k| |scale| times the weight, of which a bound of the
    rounding error is made."""
    B, Q, Hq, D = q.shape
    Hkv, page = k_codes.shape[1:3]
    g = Hq // Hkv
    out = np.array(mass, np.float64)
    size = np.zeros(mass.shape)
    for b in range(B):
        n, m = int(kv_len[b]), int(q_len[b])
        for hk in range(Hkv):
            k = to.cached(k_codes, k_scale, table[b], n, hk, page)
            add = np.zeros(n)
            for i in range(m):
                for h in range(hk * g, (hk + 1) * g):
                    lim = max(0, n - m + i + 1) if causal else n
                    if lim == 0 or np.isinf(lse[b, i, h]):
                        continue                  # adds nothing
                    s = k[:lim] @ q[b, i, h] * scale
                    w = np.exp(s - np.float64(lse[b, i, h]))
                    add[:lim] += w
                    size[b, hk, :lim] += w * (
                        np.abs(k[:lim]) @ np.abs(q[b, i, h]) * abs(scale) +
                        abs(lse[b, i, h]))
            for t in range(first, n):
                old = fresh is None or t < fresh[b]
                out[b, hk, t] = add[t] + (decay * out[b, hk, t] if old else 0)
    return out, size


def kv_evict(mass, k_codes, v_codes, k_scale, v_scale, table, kv_len, budget,
             sink, recent):
    """Codes and scales are updated in place; returns the new lengths, the
    kept slots [B, Hkv, budget] (-1 past them) and their mass (a list of
    arrays by [b][h])."""
    B, Hkv = mass.shape[:2]
    page = k_codes.shape[2]
    new_len = np.minimum(np.asarray(kv_len), budget)
    kept = np.full((B, Hkv, budget), -1, np.int64)
    moved = [[None] * Hkv for _ in range(B)]
    for b in range(B):
        n = int(kv_len[b])
        for h in range(Hkv):
            slots = list(range(n))
            if n > budget:
                middle = range(sink, n - recent)
                key = lambda t: (  # noqa: E731
                    -np.inf if np.isnan(mass[b, h, t]) else mass[b, h, t])
                nan = lambda t: bool(np.isnan(mass[b, h, t]))  # noqa: E731
                best = sorted(middle, key=lambda t: (nan(t), -key(t), t))
                slots = sorted([*range(sink), *range(n - recent, n),
                                *best[:budget - sink - recent]])
            kept[b, h, :len(slots)] = slots
            moved[b][h] = mass[b, h, slots]
            if n <= budget:
                continue
            for codes, scale in ((k_codes, k_scale), (v_codes, v_scale)):
                x = e4m3_decode(codes[table[b], h]) * scale[
                    table[b], h].astype(np.float64)[:, None, None]
                x = x.reshape(-1, codes.shape[3])[slots]
                for p in range(-(-len(slots) // page)):
                    lo, hi = p * page, min(len(slots), (p + 1) * page)
                    if slots[lo:hi] == list(range(lo, hi)):
                        continue
                    i = table[b, p]
                    s = to.block_scale(np.abs(x[lo:hi]).max())
                    scale[i, h] = s
                    codes[i, h, :hi - lo] = e4m3_encode(
                        (x[lo:hi] / float(s)).astype(np.float32))
    return new_len, kept, moved


def logprobs_row(l, T, token, K):
    """One row: log probability, rank, logsumexp, entropy, top values and ids
    (no +inf; NaN counts as -inf)."""
    l = np.asarray(l, np.float64)
    raw = l[token] if token >= 0 else np.nan
    l = np.where(np.isnan(l), -np.inf, l)
    x = l / np.float64(np.float32(T))
    m = x.max()
    if m == -np.inf:
        z, p = -np.inf, np.full(l.size, np.nan)
    else:
        z = m + np.log(np.exp(x - m).sum())
        p = np.exp(x - z)
    with np.errstate(divide="ignore", invalid="ignore"):
        ent = -np.where(p > 0, p * np.log(np.where(p > 0, p, 1)),
                        np.where(np.isnan(p), np.nan, 0)).sum()
    order = np.lexsort((np.arange(l.size), -l))
    order = order[l[order] > -np.inf][:K]
    top = np.full(K, -np.inf)
    ids = np.full(K, -1)
    top[:order.size], ids[:order.size] = x[order] - z, order
    if token < 0:
        return 0.0, -1, z, ent, top, ids
    if np.isnan(raw):
        return np.nan, -1, z, ent, top, ids
    before = (l > raw) | ((l == raw) & (np.arange(l.size) < token))
    lp = np.nan if z == -np.inf else x[token] - z
    return lp, int(before.sum()), z, ent, top, ids
