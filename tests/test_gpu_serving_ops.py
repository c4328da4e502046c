"""The target's operators around a shared prompt and a bounded cache on the
GPU against the oracle: append with positions of several axes, attention
under a shared prefix, gathered attention weight, eviction, log
probabilities.

Tolerances are derived, not fitted (U = 2^-24, half a step of fp32):
  append    a function of float32 roundings that the oracle repeats: equal
            bit for bit.
  attention as in test_gpu_target_ops, whose check is used.
  mass      a score is off by at most (D + 3) U |q|.|k| scale (fp32 sums in
            any order); its distance to the logsumexp, in bits, by 4 U of
            both; a weight by 4 U more (two steps of the exponential); the
            sum over the rows by a step for each; the decayed old weight by U.
  evict     comparisons and roundings that the oracle repeats: equal.
  logprobs  a weight's exponent is off by 4 U of itself, the weight by 4 U
            more; a thread adds up to V / 512 of them one by one, then 13
            joins.  The mean of |d| p, d the distance to the maximum, bounds
            what the exponents' errors do: delta = (V / 512 + 40) U +
            4 U mean.  Logarithm, maximum and the last sum: 4 U of their sizes.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving_ops as so
from oracle import target_ops as to
from parity import np_
from test_gpu_target_ops import DT, U, Cache, _check_attn, _tables

pytestmark = pytest.mark.gpu


def _i32(a):
    return None if a is None else torch.tensor(
        np.asarray(a), dtype=torch.int32, device="cuda")


def _status(lib, status):
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_check()
    assert e.value.status == status


# --------------------------------------------------------------------------
# append with positions of several axes
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,B,Q,Hq,Hkv,D,page,rot,inter,axes,order", [
    ("bf16", 1, 1, 4, 1, 64, 16, 64, False, 1, None),
    ("bf16", 3, 9, 8, 2, 128, 32, 128, False, 3, "sections"),
    ("bf16", 2, 17, 5, 5, 80, 16, 40, False, 2, "turns"),
    ("bf16", 2, 40, 4, 2, 128, 16, 64, True, 3, "turns"),
    ("bf16", 2, 40, 4, 2, 128, 16, 96, True, 4, "any"),
    ("fp32", 4, 5, 6, 2, 64, 64, 32, True, 4, "sections"),
    ("fp32", 2, 33, 2, 1, 256, 128, 256, False, 3, "any"),
    ("bf16", 2, 300, 2, 2, 256, 128, 256, False, 3, "sections"),
    ("fp32", 3, 4, 2, 2, 16, 16, 8, False, 1, "sections"),
])
def test_append_axes_matches_the_oracle(lib, dtype, B, Q, Hq, Hkv, D, page,
                                        rot, inter, axes, order):
    rng = np.random.default_rng(B * 100 + Q + D + axes)
    pos = rng.integers(0, 3 * page, B)
    n_new = rng.integers(0, Q + 1, B)
    n_new[0] = Q
    if B > 2:
        n_new[1] = 0
    cache = Cache(pos + n_new, page, Hkv, D, rng)
    width = (Hq + 2 * Hkv) * D
    qkv = rng.standard_normal((B * Q, width)) * np.exp2(
        rng.integers(-6, 6, (B * Q, 1)))
    qkv = torch.tensor(qkv, dtype=torch.float32).to(DT[dtype]).cuda()
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    q, k, v = (q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
               v.unflatten(1, (Hkv, D)))
    # positions have nothing to do with slots; their table is shorter
    most = 37
    cos, sin = _tables(most, rot)
    axis_pos = rng.integers(0, most, (axes, B * Q))
    r2 = rot // 2
    axis_of = {None: np.zeros(r2, int), "turns": np.arange(r2) % axes,
               "sections": np.arange(r2) * axes // r2,
               "any": rng.integers(0, axes, r2)}[order]
    (kc, vc, ks, vs), table = cache.cuda()
    q_out = torch.full((B, Q, Hq, D), 9.0, dtype=DT[dtype], device="cuda")
    kv_len = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    of = None if order is None else torch.tensor(
        axis_of, dtype=torch.uint8, device="cuda")
    lib.dflash_kv_append_axes(q, k, v, cos, sin, _i32(axis_pos), of,
                              _i32(pos), _i32(n_new), table, kc, vc, ks, vs,
                              q_out, kv_len, interleaved=inter)
    lib.dflash_check()
    f32 = lambda t: t.float().cpu().numpy()  # noqa: E731
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    oq, olen = so.kv_append_axes(
        f32(q).reshape(B, Q, Hq, D), f32(k).reshape(B, Q, Hkv, D),
        f32(v).reshape(B, Q, Hkv, D), f32(cos), f32(sin), axis_pos, axis_of,
        pos, n_new, cache.table, page, *o, inter)
    assert np.array_equal(np_(kv_len), olen)
    assert np.array_equal(f32(q_out), f32(torch.from_numpy(oq).to(DT[dtype])))
    for got, want in zip((kc, vc), o[:2]):
        assert np.array_equal(np_(got), want)
    for got, want in zip((ks, vs), o[2:]):
        assert np.array_equal(np_(got), want, equal_nan=True)


def test_append_axes_with_positions_of_the_slots_is_append(lib):
    rng = np.random.default_rng(1)
    B, Q, Hq, Hkv, D, page = 3, 5, 4, 2, 128, 16
    pos = np.array([3, 20, 0])
    cache = Cache(pos + Q, page, Hkv, D, rng)
    x = [torch.randn(B * Q, h, D, device="cuda").bfloat16()
         for h in (Hq, Hkv, Hkv)]
    cos, sin = _tables(64, D)
    got = []
    for axes in (False, True):
        (kc, vc, ks, vs), table = cache.cuda()
        q_out = torch.empty(B, Q, Hq, D, dtype=torch.bfloat16, device="cuda")
        kv_len = _i32([0] * B)
        rest = (_i32(pos), None, table, kc, vc, ks, vs, q_out, kv_len)
        if axes:
            at = np.repeat((pos[:, None] + np.arange(Q)).reshape(1, -1), 3, 0)
            of = torch.arange(D // 2, device="cuda").remainder(3).byte()
            lib.dflash_kv_append_axes(*x, cos, sin, _i32(at), of, *rest)
        else:
            lib.dflash_kv_append(*x, cos, sin, *rest)
        got.append([np_(t) for t in (kc, vc, ks, vs, kv_len)] +
                   [np_(q_out.float())])
    for a, b in zip(*got):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def test_append_axes_flags_positions_and_axes(lib):
    """A position outside the tables and an axis that is not there are
    flagged; the nearest row and axis 0 are taken."""
    B, Q, D, page, most = 1, 4, 16, 16, 10
    cos, sin = _tables(most, D)
    k = torch.randn(Q, 1, D, device="cuda")
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    for bad_pos, bad_axis in (([3, -1, 9, 10], 0), ([3, 4, 5, 6], 7)):
        kc, vc = z(1, 1, page, D), z(1, 1, page, D)
        ks, vs = z(1, 1, dt=torch.float32), z(1, 1, dt=torch.float32)
        at = np.array([bad_pos, [1, 2, 3, 4]])
        of = np.array([0, 1, 0, 1, 0, 1, 0, bad_axis])
        lib.dflash_kv_append_axes(
            None, k, k, cos, sin, _i32(at),
            torch.tensor(of, dtype=torch.uint8, device="cuda"), _i32([0]),
            None, z(1, 1, dt=torch.int32), kc, vc, ks, vs, None, _i32([0]))
        _status(lib, 6)
        o = [np.zeros((1, 1, page, D), np.uint8) for _ in range(2)] + [
            np.zeros((1, 1), np.float32) for _ in range(2)]
        kn = np_(k).reshape(B, Q, 1, D)
        so.kv_append_axes(None, kn, kn, np_(cos), np_(sin),
                          at.clip(0, most - 1), np.where(of > 1, 0, of), [0],
                          [Q], np.array([[0]]), page, *o)
        assert np.array_equal(np_(kc), o[0]) and np.array_equal(np_(ks), o[2])


# --------------------------------------------------------------------------
# attention under a shared prefix
# --------------------------------------------------------------------------
class SharedCache(Cache):
    """A Cache whose sequences begin with the pages of the first; the other
    rows of the page table hold nonsense there."""

    def __init__(self, shared, lengths, page, Hkv, D, rng, spread=3.0):
        lengths = np.asarray(lengths)
        # a sequence of its own for the prefix, at the end
        own = np.maximum(lengths - shared, 0)
        super().__init__([*own, shared], page, Hkv, D, rng, spread)
        first = shared // page
        most = max(-(-int(own.max()) // page), 1)
        t = np.full((len(lengths), first + most), -7, np.int32)
        t[:, first:] = self.table[:-1, :most]
        t[0, :first] = self.table[-1, :first]
        t[1:, :first] = rng.integers(-9, 10 ** 6, (len(lengths) - 1, first))
        self.table = t


def _share(lib, dtype, cache, q, kv_len, q_len, shared, causal, scale,
           want_lse=True, **kw):
    (kc, vc, ks, vs), table = cache.cuda()
    B, Q, Hq, D = q.shape
    out = torch.full(q.shape, 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((B, Q, Hq), 7.0, device="cuda") if want_lse else None
    ws = torch.full((lib.dflash_shared_attn_workspace_bytes(
        B, Q, Hq, kc.shape[1], D),), 0xFF, dtype=torch.uint8, device="cuda")
    lib.dflash_shared_attn(q, kc, vc, ks, vs, table, _i32(kv_len),
                           _i32(q_len), shared, scale, out, lse, ws,
                           causal=causal, **kw)
    return out, lse


SHARED = [
    # dtype, Hq, Hkv, D, page, Q, causal, shared, lengths, query lengths
    ("bf16", 4, 1, 128, 16, 1, True, 16, [17], None),
    ("bf16", 8, 2, 128, 32, 1, True, 64, [65, 70, 100, 64, 200], None),
    ("bf16", 8, 2, 128, 32, 1, True, 64, [65, 0, 30, 64, 1], [1, 0, 1, 1, 1]),
    ("bf16", 8, 1, 128, 64, 9, True, 192, [201, 500, 230, 204], None),
    ("bf16", 8, 1, 128, 64, 9, False, 192, [201, 500, 230, 192],
     [9, 4, 0, 8]),
    # sequences that end inside the prefix, and queries before its end
    ("bf16", 4, 2, 64, 16, 6, True, 160, [163, 100, 160, 3], [6, 6, 2, 5]),
    ("bf16", 16, 1, 128, 128, 17, True, 1024, [1041, 1100, 1300], None),
    ("bf16", 3, 3, 64, 16, 4, True, 288, [300, 292, 400], [4, 1, 4]),
    ("bf16", 10, 2, 80, 32, 6, True, 640, [700, 646], None),
    ("bf16", 4, 4, 16, 16, 3, True, 80, [90, 83], None),
    ("bf16", 4, 2, 256, 32, 3, True, 288, [300, 291], None),
    ("bf16", 4, 2, 112, 64, 40, True, 320, [400, 364], [40, 33]),
    ("bf16", 6, 2, 96, 32, 2, True, 0, [90, 33, 0], [2, 2, 0]),
    ("fp32", 4, 2, 64, 16, 4, True, 320, [333, 324, 0, 350], [4, 4, 0, 2]),
    ("fp32", 6, 1, 128, 128, 5, False, 384, [400, 389, 384], [5, 1, 5]),
    ("fp32", 2, 2, 256, 64, 2, True, 192, [200, 194], None),
    ("fp32", 5, 5, 48, 32, 1, True, 1600, [2000, 1601], None),
    ("fp32", 2, 1, 32, 16, 2, True, 0, [50, 3], None),
]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,Q,causal,shared,kv,ql", SHARED)
def test_shared_attention_matches_the_oracle(lib, dtype, Hq, Hkv, D, page, Q,
                                             causal, shared, kv, ql):
    rng = np.random.default_rng(Hq * 7 + D + Q + shared)
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    B = len(kv)
    q = torch.tensor(rng.standard_normal((B, Q, Hq, D)) * 2,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    scale = 1 / math.sqrt(D)
    out, lse = _share(lib, dtype, cache, q, kv, ql, shared, causal, scale)
    lib.dflash_check()
    nq = [Q] * B if ql is None else ql
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale,
                        so.shared_table(cache.table, shared, page), kv, nq,
                        scale, causal)
    _check_attn(dtype, D, max(kv), out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Q,Hq,Hkv,shared,own", [
    (70, 1, 8, 2, 256, 40), (13, 9, 8, 1, 512, 200), (3, 130, 4, 2, 128, 300),
    (200, 2, 4, 4, 64, 10)])
def test_shared_attention_of_many_rows(lib, dtype, B, Q, Hq, Hkv, shared, own):
    """More rows than a tile has, row tiles that sequences share."""
    rng = np.random.default_rng(B + Q)
    D, page = 64, 16
    kv = [shared + Q + int(rng.integers(0, own + 1)) for _ in range(B)]
    kv[1] = shared + Q
    ql = [int(rng.integers(0, Q + 1)) for _ in range(B)]
    ql[0] = Q
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    q = torch.tensor(rng.standard_normal((B, Q, Hq, D)) * 2,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    out, lse = _share(lib, dtype, cache, q, kv, ql, shared, True, D ** -0.5)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale,
                        so.shared_table(cache.table, shared, page), kv, ql,
                        D ** -0.5, True)
    _check_attn(dtype, D, max(kv), out, lse, ref)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64),
                                     ("bf16", 256)])
def test_shared_attention_scales_far_apart(lib, dtype, D):
    """Key and value scales from 2^-64 to 2^60 side by side, shared and own
    pages of either; a negative and a zero factor of the scores."""
    rng = np.random.default_rng(D)
    page, shared, kv, Hkv, Hq, Q = 16, 96, [150, 98], 2, 4, 2
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    N = cache.scale[1].shape[0]
    cache.scale[1][:] = np.exp2(rng.integers(-64, 61, (N, Hkv)))
    q = torch.tensor(rng.standard_normal((len(kv), Q, Hq, D)),
                     dtype=torch.float32).to(DT[dtype]).cuda()
    # rows of very different sizes (the scores stay moderate: small keys)
    cache.scale[0][:] = np.exp2(rng.integers(-64, -59, (N, Hkv)))
    q[0, 0] *= 2.0 ** 60
    q[1, 1] *= 2.0 ** 54
    for scale in (D ** -0.5, -0.125, 0.0):
        out, lse = _share(lib, dtype, cache, q, kv, None, shared, True, scale)
        lib.dflash_check()
        ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                            *cache.codes, *cache.scale,
                            so.shared_table(cache.table, shared, page), kv,
                            [Q] * 2, scale, True)
        _check_attn(dtype, D, max(kv), out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_shared_attention_large_scores(lib, dtype):
    """Scores of thousands of either sign, growing along the sequence, so that
    the running maximum rises in every tile, and falling."""
    rng = np.random.default_rng(9)
    D, page, Hkv, Hq, Q, shared = 64, 32, 1, 2, 3, 640
    kv = [900, 643]
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    grow = np.exp2(np.linspace(-6, 2, cache.table.shape[1]).round())
    for row, up in ((0, grow), (1, grow[::-1])):
        for p, s in zip(cache.table[row], up):
            if 0 <= p < cache.scale[0].shape[0]:
                cache.scale[0][p] = s
    q = torch.tensor(rng.standard_normal((2, Q, Hq, D)),
                     dtype=torch.float32).to(DT[dtype]).cuda()
    out, lse = _share(lib, dtype, cache, q, kv, None, shared, True, D ** -0.5)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale,
                        so.shared_table(cache.table, shared, page), kv,
                        [Q] * 2, D ** -0.5, True)
    # a score of thousands carries hundreds of steps: the check's bound of
    # the weights is wide there, that of the logsumexp is not
    _check_attn(dtype, D, max(kv), out, lse, ref)


def test_shared_attention_flags_and_survives(lib):
    """A bad page of the prefix and of a sequence count as zeros, lengths are
    clamped; all flagged."""
    rng = np.random.default_rng(4)
    D, page, shared, kv = 64, 16, 64, [100, 90, 70]
    for dtype in ("bf16", "fp32"):
        cache = SharedCache(shared, kv, page, 1, D, rng)
        q = torch.randn(3, 1, 2, D, device="cuda").to(DT[dtype])
        table = so.shared_table(cache.table, shared, page)
        for row, col in ((0, 1), (2, 4)):
            c2 = SharedCache.__new__(SharedCache)
            c2.__dict__ = {k: ([a.copy() for a in v] if isinstance(v, list)
                               else v) for k, v in cache.__dict__.items()}
            c2.table = cache.table.copy()
            c2.table[row, col] = 10 ** 6
            out, lse = _share(lib, dtype, c2, q, kv, None, shared, True, 0.1)
            _status(lib, 6)
            want = so.shared_table(c2.table, shared, page)
            # zeros: a page of its own with codes of 0
            codes = [np.concatenate([c, np.zeros_like(c[:1])])
                     for c in cache.codes]
            scale = [np.concatenate([s, np.ones_like(s[:1])])
                     for s in cache.scale]
            want[want == 10 ** 6] = len(codes[0]) - 1
            ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                                *codes, *scale, want, kv, [1] * 3, 0.1, True)
            _check_attn(dtype, D, max(kv), out, lse, ref)
        most = cache.table.shape[1] * page
        _share(lib, dtype, cache, q, [100, -3, most + 1], None, shared, True,
               0.1)
        _status(lib, 6)
        assert table.shape[1] * page == most


# --------------------------------------------------------------------------
# gathered attention weight
# --------------------------------------------------------------------------
MASS = [
    # dtype, Hq, Hkv, D, page, Q, causal, kv, query lengths, first
    ("bf16", 4, 1, 128, 16, 1, True, [1], None, 0),
    ("bf16", 8, 2, 128, 32, 1, True, [37, 0, 128, 129, 1],
     [1, 0, 1, 1, 1], 0),
    ("bf16", 8, 1, 128, 64, 9, True, [9, 500, 77, 12], None, 5),
    ("bf16", 8, 1, 128, 64, 9, False, [9, 500, 77, 8], [9, 4, 0, 8], 130),
    ("bf16", 16, 1, 128, 128, 17, True, [1000, 17, 127], None, 0),
    ("bf16", 3, 3, 64, 16, 4, True, [300, 33, 2], [4, 1, 4], 1),
    ("bf16", 10, 2, 80, 32, 6, True, [700, 6], None, 256),
    ("bf16", 4, 4, 16, 16, 3, True, [90, 3], None, 0),
    ("bf16", 4, 2, 256, 32, 3, True, [300, 3], None, 17),
    ("bf16", 4, 2, 112, 64, 40, True, [400, 64], [40, 33], 0),
    ("bf16", 64, 1, 64, 16, 11, True, [150, 11], None, 0),
    ("fp32", 4, 2, 64, 16, 4, True, [333, 4, 0, 50], [4, 4, 0, 2], 0),
    ("fp32", 6, 1, 128, 128, 5, False, [400, 1, 5], [5, 1, 5], 129),
    ("fp32", 2, 2, 256, 64, 2, True, [200, 2], None, 0),
]


def _mass_args(rng, dtype, Hq, Hkv, D, page, Q, causal, kv, ql, up=2.0):
    cache = Cache(kv, page, Hkv, D, rng)
    B = len(kv)
    q = torch.tensor(rng.standard_normal((B, Q, Hq, D)) * up,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    nq = [Q] * B if ql is None else ql
    q64 = q.float().cpu().numpy().astype(np.float64)
    _, lse, _, _ = to.paged_attn(q64, *cache.codes, *cache.scale, cache.table,
                                 kv, nq, D ** -0.5, causal)
    return cache, q, q64, nq, lse.astype(np.float32)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,Q,causal,kv,ql,first", MASS)
@pytest.mark.parametrize("with_fresh", [True, False])
def test_mass_matches_the_oracle(lib, dtype, Hq, Hkv, D, page, Q, causal, kv,
                                 ql, first, with_fresh):
    rng = np.random.default_rng(Hq * 7 + D + Q)
    cache, q, q64, nq, lse = _mass_args(rng, dtype, Hq, Hkv, D, page, Q,
                                        causal, kv, ql)
    (kc, _, ks, _), table = cache.cuda()
    slots = max(kv) + 3
    old = rng.random((len(kv), Hkv, slots)).astype(np.float32)
    fresh = np.maximum(np.array(kv) - np.array(nq), 0) if with_fresh else None
    decay = 0.75 if with_fresh else 1.0
    mass = torch.from_numpy(old.copy()).cuda()
    lib.dflash_attn_mass(q, kc, ks, table, _i32(kv), _i32(ql),
                         torch.from_numpy(lse).cuda(), _i32(fresh), first,
                         D ** -0.5, decay, mass, causal=causal)
    lib.dflash_check()
    want, size = so.attn_mass(q64, cache.codes[0], cache.scale[0],
                              cache.table, kv, nq, lse, fresh, first,
                              D ** -0.5, decay, old, causal)
    got = np_(mass).astype(np.float64)
    untouched = want == old
    assert np.array_equal(got[untouched], want[untouched])
    rows = Q * Hq // Hkv
    tol = (D + 12) * U * size + (rows + 16) * U * np.abs(want)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.abs(got - want)[bad].max(), int(bad.sum()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mass_of_odd_rows(lib, dtype):
    """Logsumexps of -inf, +inf and NaN; queries of very different sizes and
    of zeros; a negative scale: nothing but a NaN spreads."""
    rng = np.random.default_rng(3)
    Hq, Hkv, D, page, Q, kv = 8, 2, 64, 16, 3, [100, 20]
    cache, q, _, nq, _ = _mass_args(rng, dtype, Hq, Hkv, D, page, Q, True, kv,
                                    None)
    q[0, 0, 0] = 0
    q[0, 1, 1] *= 16
    q[0, 1, 2] *= 2.0 ** -40
    q64 = q.float().cpu().numpy().astype(np.float64)
    scale = -(D ** -0.5)
    _, lse, _, _ = to.paged_attn(q64, *cache.codes, *cache.scale, cache.table,
                                 kv, nq, scale, True)
    lse = lse.astype(np.float32)
    lse[0, 2, 3] = -np.inf
    lse[1, 1, 0] = np.inf
    (kc, _, ks, _), table = cache.cuda()
    old = np.zeros((2, Hkv, 112), np.float32)
    mass = torch.from_numpy(old.copy()).cuda()
    call = lambda: lib.dflash_attn_mass(  # noqa: E731
        q, kc, ks, table, _i32(kv), None, torch.from_numpy(lse).cuda(), None,
        0, scale, 1.0, mass)
    call()
    lib.dflash_check()
    want, size = so.attn_mass(q64, cache.codes[0], cache.scale[0],
                              cache.table, kv, nq, lse, None, 0, scale, 1.0,
                              old)
    got = np_(mass).astype(np.float64)
    size = np.where(np.isnan(size), 0, size)
    tol = (D + 12) * U * size + (Q * 4 + 16) * U * np.abs(want) + 1e-37
    assert np.all(np.abs(got - want) <= tol)
    lse[1, 2, 7] = np.nan
    call()
    assert np.isnan(np_(mass)[1, 1, :20]).all()
    assert not np.isnan(np_(mass)[1, 0]).any()


def test_mass_flags(lib):
    rng = np.random.default_rng(5)
    for dtype in ("bf16", "fp32"):
        cache, q, q64, nq, lse = _mass_args(rng, dtype, 2, 1, 64, 16, 1, True,
                                            [40, 40], None)
        (kc, _, ks, _), table = cache.cuda()
        t = torch.from_numpy(lse).cuda()
        call = lambda n, tab, m: lib.dflash_attn_mass(  # noqa: E731
            q, kc, ks, tab, _i32(n), None, t, None, 0, 0.125, 1.0, m)
        mass = torch.zeros(2, 1, 30, device="cuda")
        call([20, 40], table, mass)                # beyond the row of mass
        _status(lib, 6)
        bad = table.clone()
        bad[1, 1] = 99
        mass = torch.zeros(2, 1, 48, device="cuda")
        call([40, 40], bad, mass)                  # counts as zero keys
        _status(lib, 6)
        z = np.exp(-lse[1].astype(np.float64)).sum()
        assert np.allclose(np_(mass)[1, 0, 16:32], z, rtol=1e-5)
        call([-1, 40], table, mass)
        _status(lib, 6)


# --------------------------------------------------------------------------
# eviction
# --------------------------------------------------------------------------
EVICT = [
    # Hkv, D, page, budget, sink, recent, lengths
    (2, 64, 16, 33, 4, 8, [100, 33, 0, 34, 12]),
    (1, 128, 32, 64, 0, 0, [65, 400, 64]),
    (3, 16, 16, 48, 16, 32, [200, 49]),            # no free choice
    (2, 256, 128, 200, 1, 0, [700, 201]),
    (2, 80, 64, 1, 0, 1, [5, 1, 300]),
    (2, 80, 64, 1, 0, 0, [5, 1, 300]),
    (4, 32, 16, 500, 64, 100, [501, 517, 3000]),
    (1, 128, 64, 9000, 10, 100, [9001, 9500, 20000]),
    (1, 16, 16, 20, 0, 0, [1500]),
]


def _evict(lib, cache, mass, kv, budget, sink, recent, with_out=True):
    (kc, vc, ks, vs), table = cache.cuda()
    B, Hkv, slots = mass.shape
    m = torch.from_numpy(mass).cuda()
    out = torch.full((B, Hkv, slots), -3.0, device="cuda")
    new_len = _i32([-9] * B)
    kept = torch.full((B, Hkv, budget), -5, dtype=torch.int32, device="cuda")
    ws = torch.full((lib.dflash_kv_evict_workspace_bytes(
        B, Hkv, cache.page, budget),), 0xA5, dtype=torch.uint8, device="cuda")
    lib.dflash_kv_evict(m, kc, vc, ks, vs, table, _i32(kv), budget, sink,
                        recent, out if with_out else None, new_len,
                        kept if with_out else None, ws)
    return kc, vc, ks, vs, out, new_len, kept


def _check_evict(lib, cache, mass, kv, budget, sink, recent, status=None):
    got = _evict(lib, cache, mass, kv, budget, sink, recent)
    if status is None:
        lib.dflash_check()
    else:
        _status(lib, status)
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    new_len, kept, moved = so.kv_evict(mass, *o, cache.table, kv, budget,
                                       sink, recent)
    assert np.array_equal(np_(got[5]), new_len)
    assert np.array_equal(np_(got[6]), kept)
    out = np_(got[4])
    for b in range(mass.shape[0]):
        for h in range(mass.shape[1]):
            n = new_len[b]
            assert np.array_equal(out[b, h, :n], moved[b][h], equal_nan=True)
            assert np.all(out[b, h, n:] == -3.0)
    for g, w in zip(got[:2], o[:2]):
        assert np.array_equal(np_(g), w)
    for g, w in zip(got[2:4], o[2:]):
        assert np.array_equal(np_(g), w, equal_nan=True)
    again = _evict(lib, cache, mass, kv, budget, sink, recent, False)
    for g, w in zip(again[:4], got[:4]):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    if status is None:
        lib.dflash_check()
    else:
        _status(lib, status)


@pytest.mark.parametrize("Hkv,D,page,budget,sink,recent,kv", EVICT)
@pytest.mark.parametrize("kind", ["random", "ties", "front", "back"])
def test_evict_matches_the_oracle(lib, Hkv, D, page, budget, sink, recent, kv,
                                  kind):
    rng = np.random.default_rng(D + budget)
    cache = Cache(kv, page, Hkv, D, rng, spread=20)
    shape = (len(kv), Hkv, max(max(kv), budget) + 5)
    mass = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        mass = rng.integers(0, 3, shape).astype(np.float32) - 1
        mass[mass == 0] = -0.0
    elif kind == "front":        # all move by as much as there is to evict
        mass = np.broadcast_to(np.arange(shape[2], dtype=np.float32),
                               shape).copy()
    elif kind == "back":
        mass = np.broadcast_to(-np.arange(shape[2], dtype=np.float32),
                               shape).copy()
    _check_evict(lib, cache, mass, kv, budget, sink, recent)


def test_evict_special_weights_and_codes(lib):
    """Infinite weights and subnormal ones in order, a NaN last and flagged;
    pages of zeros; scales at both ends of their range."""
    rng = np.random.default_rng(2)
    kv, page = [200, 90], 16
    cache = Cache(kv, page, 2, 32, rng)
    N = cache.scale[0].shape[0]
    cache.scale[0][:] = np.exp2(rng.choice([-64, -60, 0, 100, 120], (N, 2)))
    cache.codes[0][::3] = 0
    cache.codes[1][::2] &= 0x83                    # zeros and subnormals
    mass = rng.choice(np.array([0, 1e-45, -1e-45, 1, np.inf, -np.inf, 3],
                               np.float32), (2, 2, 208))
    _check_evict(lib, cache, mass, kv, 77, 3, 5)
    mass[0, 1, 50:150] = np.nan
    _check_evict(lib, cache, mass, kv, 77, 3, 5, status=4)


def test_evict_long_chains_of_pages(lib):
    """Every page waits for the one below it, over thousands of pages and a
    hundred at a time."""
    rng = np.random.default_rng(8)
    for shift in (1, 1600):
        kv = [40000]
        cache = Cache(kv, 16, 1, 16, rng)
        mass = np.ones((1, 1, kv[0]), np.float32)
        mass[0, 0, 5:5 + shift] = 0
        _check_evict(lib, cache, mass, kv, kv[0] - shift, 0, 0)


def test_evict_leaves_shared_pages(lib):
    """Sequences that share their first pages, covered by sink."""
    rng = np.random.default_rng(6)
    kv, page, shared = [150, 130, 97], 16, 48
    cache = Cache(kv, page, 2, 64, rng)
    cache.table[1:, :3] = cache.table[0, :3]
    mass = rng.random((3, 2, 160)).astype(np.float32)
    _check_evict(lib, cache, mass, kv, 96, shared, 10)


def test_evict_flags(lib):
    rng = np.random.default_rng(7)
    kv, page = [60, 60], 16
    cache = Cache(kv, page, 1, 16, rng)
    mass = rng.random((2, 1, 64)).astype(np.float32)
    full = [np_(t) for t in _evict(lib, cache, mass, [60, 60], 40, 0, 0)]
    lib.dflash_check()
    got = [np_(t) for t in _evict(lib, cache, mass, [65, 60], 40, 0, 0)]
    _status(lib, 6)                       # clamped to the table's 64 slots
    assert got[5].tolist() == [40, 40]
    got = [np_(t) for t in _evict(lib, cache, mass, [-1, 60], 40, 0, 0)]
    _status(lib, 6)
    assert got[5].tolist() == [0, 40]
    mine = cache.table[1, :4]
    for a, b in zip(got[:2], full[:2]):
        assert np.array_equal(a[mine], b[mine])
    others = np.setdiff1d(np.arange(len(got[0])), mine)
    assert np.array_equal(got[0][others], cache.codes[0][others])
    bad = Cache.__new__(Cache)
    bad.__dict__ = dict(cache.__dict__)
    bad.table = cache.table.copy()
    bad.table[0, 1] = -2
    got = [np_(t) for t in _evict(lib, bad, mass, kv, 40, 0, 0)]
    _status(lib, 6)
    for a, b in zip(got[:2], full[:2]):   # the other sequence is unharmed
        assert np.array_equal(a[mine], b[mine])


# --------------------------------------------------------------------------
# log probabilities
# --------------------------------------------------------------------------
def _logprobs(lib, l, T, token, K, parts=None):
    R = l.shape[0]
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    got = dict(logprob=f(R), rank=i(R), lse=f(R), entropy=f(R),
               top=f(R, K) if K else None, top_id=i(R, K) if K else None)
    if parts is not None:
        got = {k: v if k in parts else None for k, v in got.items()}
    t = None if T is None else torch.tensor(T, dtype=torch.float32,
                                            device="cuda")
    lib.dflash_logprobs(l, t, _i32(token), *got.values())
    return {k: None if v is None else np_(v) for k, v in got.items()}


def _check_logprobs(l, T, token, K, got):
    l = l.float().cpu().numpy()
    R, V = l.shape
    for r in range(R):
        t = 1.0 if T is None else float(np.float32(T[r]))
        lp, rank, z, ent, top, ids = so.logprobs_row(l[r], t, token[r], K)
        x = np.where(np.isnan(l[r]), -np.inf, l[r].astype(np.float64)) / t
        m = x.max()
        assert got["rank"][r] == rank
        if K:
            assert np.array_equal(got["top_id"][r], ids)
        if m == -np.inf:
            assert got["lse"][r] == -np.inf
            assert np.isnan(got["entropy"][r])
            continue
        p = np.exp(x - z)
        d = np.where(p > 0, x - m, 0)
        mean = -(p * d).sum()
        delta = (V / 512 + 40) * U + 4 * U * mean
        assert abs(got["lse"][r] - z) <= delta + 4 * U * (abs(m) + abs(z))
        assert abs(got["entropy"][r] - ent) <= (
            delta * (1 + 2 * mean) + 8 * U * (1 + ent))

        def near(a, b):
            a, b = np.float64(a), np.float64(b)
            if not np.isfinite(b):
                assert a == b or (np.isnan(a) and np.isnan(b))
            else:
                assert abs(a - b) <= delta + 8 * U * (abs(b) + (z - m)), (
                    a, b, delta)
        near(got["logprob"][r], lp)
        for k in range(K):
            near(got["top"][r, k], top[k])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,V,K,temper", [
    (1, 1, 1, False), (3, 5, 8, True), (2, 100, 32, False), (7, 4099, 5, True),
    (1, 151936, 20, False), (40, 20011, 32, True), (700, 1000, 1, False),
    (1, 40000, 0, True)])
def test_logprobs_match_the_oracle(lib, dtype, R, V, K, temper):
    rng = np.random.default_rng(V + R)
    x = 3 * rng.standard_normal((R, V))
    x[:, rng.integers(0, V, min(V, 30))] += 8
    # rows apart by an odd number: they start anywhere in a 16-byte word
    wide = torch.full((R, V + 3), float("nan"))
    wide[:, 1:V + 1] = torch.from_numpy(x)
    l = wide.to(DT[dtype]).cuda()[:, 1:V + 1]
    T = rng.uniform(0.3, 2, R).astype(np.float32) if temper else None
    token = rng.integers(0, V, R)
    token[0] = int(x[0].argmax())
    if R > 2:
        token[1], token[2] = -1, V - 1
    got = _logprobs(lib, l, T, token, K)
    lib.dflash_check()
    _check_logprobs(l, T, token, K, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_of_ties(lib, dtype):
    """Equal logits by the ten thousand: the lowest ids, and every rank."""
    V, K = 60000, 32
    rng = np.random.default_rng(0)
    x = np.zeros((5, V), np.float32)
    x[1] = rng.integers(0, 3, V)                   # three values
    x[2, :20000] = 4                               # in one CTA's slice
    x[3] = np.where(np.arange(V) % 2048 < 1500, 2, 1)
    x[4] = -np.inf
    x[4, [7, 59999, 8]] = 1, 1, 0
    l = torch.from_numpy(x).to(DT[dtype]).cuda()
    token = [59999, 30000, 40000, 5, 6]
    got = _logprobs(lib, l, None, token, K)
    lib.dflash_check()
    _check_logprobs(l, None, token, K, got)
    assert got["rank"][4] == 3 + 6                 # -inf: by id


def test_logprobs_of_the_filtered_row_are_those_of_what_is_kept(lib):
    """Logits that dflash_sample filtered: -inf is no token."""
    R, V, K = 4, 5000, 8
    l = 3 * torch.randn(R, V, device="cuda")
    full = lambda v, t: torch.full((R,), v, dtype=t, device="cuda")  # noqa: E731
    filtered = torch.empty_like(l)
    token, n = full(0, torch.int32), full(0, torch.int32)
    ws = torch.empty(lib.dflash_sample_workspace_bytes(R, V),
                     dtype=torch.uint8, device="cuda")
    lib.dflash_sample(l, full(1.0, torch.float32), full(5, torch.int32), None,
                      None, torch.rand(R, device="cuda"), token, n, filtered,
                      ws)
    got = _logprobs(lib, filtered, None, np_(token), K)
    lib.dflash_check()
    _check_logprobs(filtered, None, np_(token), K, got)
    assert np.all(got["top_id"][:, 5:] == -1)
    assert np.all(got["rank"] < 5)


def test_logprobs_non_finite(lib):
    V = 3000
    x = torch.randn(7, V)
    x[0, 100] = float("nan")
    x[1, 5] = float("inf")
    x[2] = float("-inf")
    x[3, 9] = float("nan")
    l = x.cuda()
    token = [7, 5, 3, 9, V, -2, 4]
    T = [1, 1, 1, 1, 1, 1, 0.0]
    got = _logprobs(lib, l, T, token, 2)
    # NaN logits, an infinite one, an empty row and T = 0 set one bit, bad
    # tokens another; the lower one is reported
    with pytest.raises(lib.DFlashError):
        lib.dflash_check()
    ok = [0]
    _check_logprobs(l[ok], None, [7], 2, {k: v[ok] for k, v in got.items()})
    assert got["lse"][1] == np.inf and np.isnan(got["logprob"][1])
    assert got["rank"][1] == 0 and got["top_id"][1, 0] == 5
    assert np.isnan(got["top"][1]).all() and np.isnan(got["entropy"][1])
    assert got["lse"][2] == -np.inf and np.isnan(got["logprob"][2])
    assert got["top_id"][2].tolist() == [-1, -1]
    assert np.isnan(got["logprob"][3]) and got["rank"][3] == -1
    assert np.isnan(got["logprob"][4]) and got["rank"][4] == -1
    assert np.isnan(got["logprob"][5]) and got["rank"][5] == -1
    _check_logprobs(l[6:], None, [4], 2, {k: v[6:] for k, v in got.items()})
    for rows, t, status in (([0], [7], 4), ([1], [5], 4), ([2], [3], 4),
                            ([5], [-2], 6), ([4], [V], 6)):
        _logprobs(lib, l[rows], None, t, 0)
        _status(lib, status)
    _logprobs(lib, l[6:], [float("inf")], [4], 0)
    _status(lib, 4)


def test_logprobs_outputs_are_optional(lib):
    l = torch.randn(3, 777, device="cuda").bfloat16()
    full = _logprobs(lib, l, None, [1, 2, 3], 4)
    for parts in (["lse"], ["entropy"], ["rank"], ["logprob"],
                  ["top", "top_id"], ["lse", "rank", "top", "top_id"]):
        got = _logprobs(lib, l, None, [1, 2, 3], 4, parts)
        for k in parts:
            assert np.array_equal(got[k], full[k])
    got = {k: torch.empty(3, device="cuda") for k in ("lse", "entropy")}
    lib.dflash_logprobs(l, None, None, None, None, got["lse"],
                        got["entropy"], None, None)
    lib.dflash_check()
    assert np.array_equal(np_(got["lse"]), full["lse"])
