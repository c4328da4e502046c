"""The operators around a shared prompt and a bounded cache at calls that their
documentation allows and the other tests do not make.  Oracle and tolerances as
in test_gpu_serving_ops, whose derivations stand there."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_ops as so
from oracle import target_ops as to
from parity import np_
from test_gpu_serving_ops import (SharedCache, _check_evict, _evict, _i32,
                                  _logprobs, _mass_args, _share)
from test_gpu_target_ops import DT, U, Cache, _check_attn

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# log probabilities
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,far", [(1e-32, 3.0), (1.0, 1e33), (1.0, 3e37),
                                   (0.25, 1e31)])
@pytest.mark.parametrize("given", ["none", "masked", "far"])
def test_masked_tokens_before_a_far_logit_count_nothing(lib, dtype, T, far,
                                                        given):
    """A thread whose first words are all at the type's lowest value and that
    meets a logit of 1e31 bits or more only then: a step that passes fp32's
    range.  Every slice of the row is masked but for its end.

    A product l log2(e) / T is rounded (U of itself), and so is its logarithm:
    alternatives are off by 4 U of the largest x."""
    V, K = 70001, 4
    low = torch.finfo(DT[dtype]).min
    x = torch.full((3, V), low, dtype=torch.float64)
    x[0, V - 5:] = far * torch.tensor([0.5, 0.25, 1.0, 0.125, -0.5])
    x[1, 8700] = far                      # the last words of a slice
    x[1, V - 1] = far / 2
    x[2, 40000] = -far                    # nothing above 0
    l = x.to(DT[dtype]).cuda()
    token = {"none": None, "masked": [3, 5, 7],
             "far": [V - 3, 8700, 40000]}[given]
    got = _logprobs(lib, l, [T] * 3, token, K,
                    None if token else ["lse", "entropy", "top", "top_id"])
    lib.dflash_check()
    l = l.double().cpu().numpy()
    for r, n in ((0, 4), (1, 2), (2, 1)):
        lp, rank, z, ent, top, ids = so.logprobs_row(
            l[r], T, token[r] if token else -1, K)
        assert ent == 0
        assert abs(got["entropy"][r]) <= 40 * U
        assert abs(got["lse"][r] - z) <= 4 * U * abs(z) + 40 * U
        assert np.array_equal(got["top_id"][r, :n], ids[:n])
        tol = 4 * U * abs(z) + 40 * U
        assert np.all(np.abs(got["top"][r, :n] - top[:n]) <=
                      tol + 8 * U * np.abs(top[:n]))
        assert abs(got["top"][r, 0]) <= 40 * U
        if token:
            assert got["rank"][r] == rank
        if given == "far":
            assert abs(got["logprob"][r]) <= 40 * U


# --------------------------------------------------------------------------
# attention under a shared prefix
# --------------------------------------------------------------------------
def _ends_inside(dtype, B, Q, Hq, Hkv, D, page, shared, most, numbers, rng):
    """A SharedCache all of whose sequences end at `most` or before, within
    the prefix; what lies behind holds NaN codes and scales or, without page
    `numbers`, is in no page."""
    kv = [int(rng.integers(0, most + 1)) for _ in range(B)]
    kv[0] = most
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    row = cache.table[0]
    if most % page:
        for c in cache.codes:
            c[row[most // page], :, most % page:] = 0x7F
    behind = row[-(-most // page):shared // page].copy()
    for c, s in zip(cache.codes, cache.scale):
        c[behind] = 0x7F
        s[behind] = np.nan
    if not numbers:
        row[-(-most // page):] = rng.choice([-9, 10 ** 6],
                                            row.size - -(-most // page))
    q = torch.tensor(rng.standard_normal((B, Q, Hq, D)) * 2,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    return cache, q, kv


# dtype, B, Q, Hq, Hkv, D, page, shared, the longest
INSIDE = [
    ("bf16", 2, 40, 32, 2, 64, 32, 7040, 7001),       # together
    ("bf16", 2, 40, 32, 2, 128, 16, 7040, 150),
    ("bf16", 320, 1, 8, 2, 64, 32, 3840, 3300),       # apart
    ("bf16", 320, 2, 8, 2, 80, 64, 3840, 64),
    ("bf16", 3, 1, 8, 2, 64, 16, 320, 100),           # unshared
    ("fp32", 3, 5, 4, 2, 64, 16, 1600, 777),
    ("bf16", 3, 5, 4, 2, 256, 64, 640, 129),
]


@pytest.mark.parametrize("dtype,B,Q,Hq,Hkv,D,page,shared,most", INSIDE)
@pytest.mark.parametrize("causal,numbers", [(True, True), (False, False)])
def test_prefix_that_no_sequence_has_to_its_end(lib, dtype, B, Q, Hq, Hkv, D,
                                                page, shared, most, causal,
                                                numbers):
    """Slots past every length may hold anything, entries of the page table
    that no token needs too."""
    rng = np.random.default_rng(B + most)
    cache, q, kv = _ends_inside(dtype, B, Q, Hq, Hkv, D, page, shared, most,
                                numbers, rng)
    ql = [int(rng.integers(0, Q + 1)) for _ in range(B)]
    ql[0] = Q
    out, lse = _share(lib, dtype, cache, q, kv, ql, shared, causal, D ** -0.5)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale,
                        so.shared_table(cache.table, shared, page), kv, ql,
                        D ** -0.5, causal)
    _check_attn(dtype, D, max(kv), out, lse, ref)


# --------------------------------------------------------------------------
# gathered attention weight
# --------------------------------------------------------------------------
def _check_mass(lib, dtype, cache, q, kv, ql, lse, first, scale=None):
    Q, Hq, D = q.shape[1:]
    Hkv = cache.codes[0].shape[1]
    scale = D ** -0.5 if scale is None else scale
    (kc, _, ks, _), table = cache.cuda()
    old = np.zeros((len(kv), Hkv, max(max(kv), 1) + 5), np.float32)
    mass = torch.from_numpy(old.copy()).cuda()
    lib.dflash_attn_mass(q, kc, ks, table, _i32(kv), _i32(ql),
                         torch.from_numpy(lse).cuda(), None, first, scale,
                         1.0, mass)
    lib.dflash_check()
    # (keys past a length are not numbers, and not read)
    want, size = so.attn_mass(q.float().cpu().numpy().astype(np.float64),
                              cache.codes[0], cache.scale[0], cache.table, kv,
                              [Q] * len(kv) if ql is None else ql, lse, None,
                              first, scale, 1.0, old)
    tol = (D + 12) * U * size + (Q * Hq // Hkv + 16) * U * np.abs(want)
    bad = ~(np.abs(np_(mass) - want) <= tol)
    assert not bad.any(), (np.abs(np_(mass) - want)[bad].max(), bad.sum())


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,Q,first", [
    ("bf16", 8, 2, 64, 16, 3, 80), ("bf16", 8, 1, 128, 64, 9, 192),
    ("bf16", 32, 1, 64, 32, 5, 32), ("bf16", 4, 2, 64, 32, 1, 1003),
    ("bf16", 4, 2, 256, 16, 2, 80), ("fp32", 4, 2, 64, 16, 2, 80)])
def test_mass_below_first_reads_no_pages(lib, dtype, Hq, Hkv, D, page, Q,
                                         first):
    """The page numbers of a shared prefix in rows other than the first may be
    anything, as in dflash_shared_attn; those of the first slot's own page are
    needed."""
    rng = np.random.default_rng(first + D)
    kv = [first + Q, first + 200, max(first - 7, Q)]
    cache, q, _, nq, lse = _mass_args(rng, dtype, Hq, Hkv, D, page, Q, True,
                                      kv, None)
    want_table = cache.table.copy()
    cache.table[1:, :first // page] = rng.choice(
        [-9, 10 ** 6], (2, first // page))
    rest = cache.cuda
    seen = cache.table

    def cuda():
        pool, _ = rest()
        return pool, torch.from_numpy(seen.copy()).cuda()
    cache.cuda, cache.table = cuda, want_table
    _check_mass(lib, dtype, cache, q, kv, None, lse, first)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128),
                                     ("bf16", 256), ("fp32", 64)])
@pytest.mark.parametrize("up,down", [(112, -110), (118, -116), (-60, 62)])
def test_mass_of_keys_and_queries_far_from_one(lib, dtype, D, up, down):
    """Key scales up to 2^118 with queries as small, and the other way round:
    scores of ordinary size, of which no intermediate may overflow."""
    rng = np.random.default_rng(up + D)
    Hq, Hkv, page, Q, kv = 8, 2, 32, 3, [300, 77]
    cache, q, *_ = _mass_args(rng, dtype, Hq, Hkv, D, page, Q, True, kv, None)
    # (codes below 256: with those above a value may pass fp32's range)
    cache.codes[0] = np.where((cache.codes[0] & 0x7F) > 0x77,
                              cache.codes[0] & 0x87, cache.codes[0])
    N = cache.scale[0].shape[0]
    cache.scale[0][:] = np.exp2(up - rng.integers(0, 4, (N, Hkv)))
    q = (q.float() * 2.0 ** (down - 6)).to(DT[dtype])
    q64 = q.float().cpu().numpy().astype(np.float64)
    _, lse, _, _ = to.paged_attn(q64, cache.codes[0], cache.codes[0],
                                 cache.scale[0], cache.scale[0], cache.table,
                                 kv, [Q] * 2, D ** -0.5, True)
    _check_mass(lib, dtype, cache, q, kv, None, lse.astype(np.float32), 0)


def test_mass_of_a_key_of_zeros_under_large_scores(lib):
    """Its score is 0, whatever its page's scale and the query's size: a weight
    of exp(0 - lse)."""
    rng = np.random.default_rng(17)
    for dtype in ("bf16", "fp32"):
        cache, q, _, _, lse = _mass_args(rng, dtype, 8, 2, 64, 16, 1, True,
                                         [200], None)
        cache.codes[0][:] = 0
        cache.scale[0][:] = 2.0 ** 60
        q *= 2.0 ** 100
        lse[:] = 3.0
        _check_mass(lib, dtype, cache, q, [200], None, lse, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mass_of_rows_with_an_infinite_logsumexp_adds_nothing(lib, dtype):
    """Whatever those rows hold: queries that are not numbers, infinite ones,
    ones whose scores pass fp32's range."""
    rng = np.random.default_rng(31)
    Hq, Hkv, D, page, Q, kv = 8, 2, 64, 16, 3, [200, 40]
    cache, q, _, nq, lse = _mass_args(rng, dtype, Hq, Hkv, D, page, Q, True,
                                      kv, None)
    cache.scale[0][:] = 2.0 ** 100
    q *= 2.0 ** -106
    q64 = q.float().cpu().numpy().astype(np.float64)
    _, lse, _, _ = to.paged_attn(q64, cache.codes[0], cache.codes[0],
                                 cache.scale[0], cache.scale[0], cache.table,
                                 kv, nq, D ** -0.5, True)
    lse = lse.astype(np.float32)
    for i, x in enumerate((math.nan, math.inf, -math.inf, 2.0 ** 100)):
        for b, z in ((0, -np.inf), (1, np.inf)):
            q[b, i % 3, 2 * i] = x
            lse[b, i % 3, 2 * i] = z
    _check_mass(lib, dtype, cache, q, kv, None, lse, 0)


@pytest.mark.parametrize("Hkv,page,shared,budget", [(2, 16, 80, 100),
                                                    (1, 64, 192, 210)])
def test_eviction_reads_no_pages_of_a_kept_prefix(lib, Hkv, page, shared,
                                                  budget):
    """Nor does dflash_kv_evict with a sink that covers them."""
    rng = np.random.default_rng(page)
    kv = [shared + 150, shared + 90, shared + 5]
    cache = Cache(kv, page, Hkv, 64, rng)
    mass = rng.random((3, Hkv, max(kv))).astype(np.float32)
    got = []
    for nonsense in (False, True):
        if nonsense:
            cache.table[1:, :shared // page] = rng.choice(
                [-9, 10 ** 6], (2, shared // page))
        got.append(_evict(lib, cache, mass, kv, budget, shared, 10))
        lib.dflash_check()
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("Hkv,D,page,shift", [(1, 128, 16, 1), (4, 64, 32, 40),
                                              (2, 16, 128, 300)])
def test_rounds_of_a_cluster_read_before_they_write(lib, Hkv, D, page, shift):
    """Every page takes tokens of the next ones, which other CTAs of the
    cluster write in the same round; many rounds, over and over."""
    rng = np.random.default_rng(shift)
    kv = [20000, 9000]
    cache = Cache(kv, page, Hkv, D, rng, spread=20)
    mass = np.ones((2, Hkv, kv[0]), np.float32)
    for b in range(2):
        mass[b, :, 3 + b:3 + b + shift] = 0
    budget = kv[1] - shift
    _check_evict(lib, cache, mass, kv, budget, 0, 0)
    first = _evict(lib, cache, mass, kv, budget, 0, 0)
    for _ in range(10):
        again = _evict(lib, cache, mass, kv, budget, 0, 0)
        for a, b in zip(again, first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    lib.dflash_check()
