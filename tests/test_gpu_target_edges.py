"""The target's calls at the ends of their stated ranges.  Tolerances are those
of test_gpu_target_ops; where a test has its own, its docstring derives it.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import target_ops as to
from test_gpu_target_ops import (DT, U, Cache, _attend, _check_attn,
                                 _check_sample, _run_sample)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# sampling
# --------------------------------------------------------------------------
@pytest.mark.parametrize("R", [1, 300])
@pytest.mark.parametrize("V,first", [(2047, 0), (4000, 1000),
                                     (151936, 40000)])
@pytest.mark.parametrize("n", [1600, 1800, 1999])
@pytest.mark.parametrize("p,m", [(0.9, 0.0), (0.9, 0.001), (1.0, 0.01)])
def test_sample_fewer_unmasked_tokens_than_k(lib, R, V, first, n, p, m):
    """A masked vocabulary (constrained decoding) with a top-k above the
    number of tokens left, which lie side by side: too many for one CTA's
    list, but no k-th token, so that top-p and min-p alone decide."""
    rng = np.random.default_rng(n + V)
    l = np.full((1, V), -np.inf, np.float32)
    at = first + rng.permutation(min(V - first, n + 40))[:n]
    l[0, at] = 2.5 * rng.standard_normal(n)
    l[0, rng.choice(at, 20)] += 5
    l = np.repeat(l, R, 0)
    u = rng.random(R).astype(np.float32)
    got = _run_sample(lib, torch.from_numpy(l).cuda(), [1.0] * R, [2000] * R,
                      [p] * R, [m] * R, u)
    lib.dflash_check()
    rows = [0] if R == 1 else [0, 1, 150, R - 1]
    _check_sample(l[rows], [1.0] * len(rows), [2000] * len(rows),
                  [p] * len(rows), [m] * len(rows), u[rows],
                  [g[rows] for g in got])
    assert np.all(np.isin(got[0], at)) and np.all(got[1] == got[1][0])


@pytest.mark.parametrize("R", [1, 300])
@pytest.mark.parametrize("count", [1, 2])
@pytest.mark.parametrize("V", [300, 50000])
@pytest.mark.parametrize("k,p,m", [
    (0, 1.0, 0.0), (1, 1.0, 0.0), (5, 1.0, 0.0), (1000, 1.0, 0.0),
    (0, 0.9, 0.0), (0, 0.4, 0.0), (0, 1.0, 0.1), (0, 1.0, 1.0),
    (5, 0.9, 0.1), (0, 0.9, 0.1)])
def test_sample_infinite_logit(lib, R, count, V, k, p, m):
    """An infinite logit weighs 1, every other token 0: flagged, and the
    definition's token, kept set and filtered logits all the same."""
    rng = np.random.default_rng(V + count)
    l = (2.5 * rng.standard_normal((1, V))).astype(np.float32)
    at = rng.choice(V, count, replace=False)
    l[0, at] = np.inf
    l = np.repeat(l, R, 0)
    for T in (0.7, 0.0):
        u = rng.random(R).astype(np.float32)
        got = _run_sample(lib, torch.from_numpy(l).cuda(), [T] * R, [k] * R,
                          [p] * R, [m] * R, u)
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_check()
        assert e.value.status == 4
        assert np.all(np.isin(got[0], at))
        rows = [0] if R == 1 else [0, 1, 150, R - 1]
        _check_sample(l[rows], [T] * len(rows), [k] * len(rows),
                      [p] * len(rows), [m] * len(rows), u[rows],
                      [g[rows] for g in got])


def _ones_below():
    """A logit whose weight against a maximum of 0 ends in (nearly) 23 ones,
    and that weight: 513 of its low halves exceed 32 bits."""
    d = torch.linspace(-6.0, -4.5, 1 << 18, device="cuda")
    w = (torch.exp(d).double() * 2.0 ** 44).long()
    low = w & ((1 << 23) - 1)
    i = int(low.argmax())
    assert 513 * int(low[i]) >= 1 << 32
    return float(d[i]), int(w[i])


def test_sample_sums_of_full_low_halves(lib):
    """All tokens but the first tie at a weight whose low half is nearly all
    ones, in rows of one CTA whose last block is one token short: sums of 512
    and one tokens to a thread.  Integer sums are exact, so uniforms and
    nuclei next to a boundary decide as the integers do."""
    R, V = 609, (1 << 18) - 1                  # one CTA to a row
    d, w = _ones_below()
    big = torch.full((R, V + 1), d, device="cuda")
    big[:, 0] = 0.0
    x = big[:, :V]                             # rows aligned to 16 bytes
    one, total = 1 << 44, (1 << 44) + (V - 1) * w
    # uniforms (and nuclei) whose target lies less than 2^32 above the first
    # weight of a token, so that a lost carry would show
    f = np.arange(1 << 23, 1 << 24).astype(np.float64) / (1 << 24)
    t = np.floor(f * float(total)).astype(np.int64)
    near = f[(t - one) % w < 1 << 32]
    assert near.size >= 2 * R
    pick = near[np.linspace(0, near.size - 1, R).astype(int)]
    u = pick.astype(np.float32)
    tok, nk, _ = _run_sample(lib, x, [1.0] * R, None, None, None, u, False)
    lib.dflash_check()
    t = np.floor(pick * float(total)).astype(np.int64)
    assert np.array_equal(tok, 1 + (t - one) // w)
    assert np.all(nk == V)
    tok, nk, _ = _run_sample(lib, x, [1.0] * R, None, u, None, [0.0] * R,
                             False)
    lib.dflash_check()
    need = np.ceil(pick * float(total)).astype(np.int64)
    # the first token, then as many as have less than `need` before them
    assert np.array_equal(nk, 1 + -(-(need - one) // w))
    assert np.all(tok == 0)


def test_sample_gives_up_on_a_copy_and_recovers(lib):
    """So many slices are copied at once that some outlast a limit of a
    nanosecond: flagged, no token for their rows, and the next call is
    right."""
    R, V = 4000, 9000
    rng = np.random.default_rng(3)
    l = np.repeat((2.5 * rng.standard_normal((1, V))).astype(np.float32), R, 0)
    x = torch.from_numpy(l).cuda()
    u = rng.random(R).astype(np.float32)
    args = ([1.0] * R, [50] * R, [0.9] * R, None, u)
    lib.dflash_check()                         # nothing pending
    try:
        lib.dflash_set_wait_limit_ns(1)
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()
        tok, nk, _ = _run_sample(lib, x, *args, filtered=False)
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_check()
        assert e.value.status == 5             # DFLASH_ERR_DEVICE_TIMEOUT
    finally:
        lib.dflash_set_wait_limit_ns(0)        # back to the default (2 s)
    late = tok == -1
    assert late.any() and np.all(nk[late] == 0)
    got = _run_sample(lib, x, *args, filtered=False)
    lib.dflash_check()
    rows = [0, 1, R // 2, R - 1]
    _check_sample(l[rows], *([a[0]] * 4 for a in args[:3]), None, u[rows],
                  [None if g is None else g[rows] for g in got])


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
def test_append_infinite_key_is_turned(lib, dtype, inter):
    """At position 0 (cosine 1, sine 0) an infinite key stays infinite, stored
    as the largest code, and makes a NaN of its partner, stored as 0; at
    position 1 both are infinite."""
    D, page = 16, 16
    k = torch.ones(2, 1, D, dtype=DT[dtype], device="cuda")
    k[:, 0, 0] = float("inf")
    v = torch.ones_like(k)
    ang = torch.arange(2, device="cuda")[:, None] * torch.ones(
        D // 2, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (torch.zeros(1, 1, page, D, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    ks, vs = (torch.zeros(1, 1, device="cuda") for _ in range(2))
    lib.dflash_kv_append(None, k, v, ang.cos(), ang.sin(), i32(0), None,
                         i32(0).view(1, 1), kc, vc, ks, vs, None, i32(0),
                         interleaved=inter)
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_check()
    assert e.value.status == 4
    other = 1 if inter else D // 2
    got = kc[0, 0, :2].cpu().numpy()
    assert got[:, [0, other]].tolist() == [[0x7E, 0], [0x7E, 0x7E]]
    rest = np.delete(got, [0, other], 1)
    assert np.all(rest != 0x7E) and np.all(rest[0] == 0x78)   # 1 = 256 / 256
    assert float(ks) == 2.0 ** -8


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
SCALES = [(-64, 63), (-64, 120), (63, -64), (120, -64), (100, -20),
          (-10, 90), (2, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("first,rest", SCALES)
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("g,n,B", [(4, 500, 1), (36, 700, 1), (4, 20000, 1),
                                   (20, 1500, 90)])
@pytest.mark.parametrize("scale", [0.02, 3.0])
def test_attention_value_scales_over_their_range(lib, dtype, first, rest,
                                                 zero, g, n, B, scale):
    """Pages whose values lie up to 2^184 apart, among them pages of zeros
    (which carry the smallest scale), first or later, in runs that hold
    whole sequences and in parts that are joined: a token's share of the
    softmax's sum does not depend on its value."""
    rng = np.random.default_rng(g + n)
    D, page = 64, 32
    cache = Cache([n], page, 1, D, rng, spread=0)
    ids = cache.table[0]
    # values of at most 2^7 times a scale of 2^120: bf16 holds them
    cache.codes[1][:] = oracle.e4m3_encode(
        (rng.standard_normal(cache.codes[1].shape) * 8).astype(np.float32))
    cut = len(ids) // 3
    cache.scale[1][ids[:cut]] = 2.0 ** first
    cache.scale[1][ids[cut:]] = 2.0 ** rest
    cache.scale[1][ids[-2]] = 2.0 ** first     # and a late one
    if zero:
        small = ids[cache.scale[1][ids, 0] == 2.0 ** min(first, rest)]
        cache.codes[1][small] = 0
    q = torch.tensor(rng.standard_normal((1, 1, g, D)) * 2,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale, cache.table, [n], [1],
                        scale)
    cache.table = np.repeat(cache.table, B, 0)
    out, lse = _attend(lib, dtype, cache, q.repeat(B, 1, 1, 1), [n] * B,
                       None, True, scale)
    lib.dflash_check()
    for b in {0, B // 2, B - 1}:
        _check_attn(dtype, D, n, out[b:b + 1], lse[b:b + 1], ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("below", [1, 2, 3, 5, 6, 7, 12])
@pytest.mark.parametrize("g", [4, 20])
def test_attention_small_row_beside_a_large_one(lib, dtype, below, g):
    """A row 2^below under the largest of its unit, most of it 2^11 under its
    own largest value: every query value keeps 2^-17 of its own row's largest,
    so that a score is off by that times the sum of |k| at most (fp32: by the
    sum's roundings)."""
    n, D, page, Q = 300, 128, 32, 4
    rng = np.random.default_rng(below)
    cache = Cache([n], page, 1, D, rng, spread=0)
    ids = cache.table[0]
    sign = rng.integers(0, 2, (len(ids), 1, page, 1))
    cache.codes[0][ids] = np.where(sign, 0x38, 0xB8)   # 1 or -1 throughout
    cache.codes[0][ids, :, :, 0] = 0
    cache.scale[0][ids] = 1.0
    for c, s in zip(cache.codes, cache.scale):
        c[ids[-1], :, n % page:] = 0x7F
    x = rng.standard_normal((1, Q, g, D))
    x *= 200 / np.abs(x).max(-1, keepdims=True)        # in [128, 256)
    low = 2.0 ** -below
    x[0, 1, 2] = 0.99 * 2.0 ** -11 * 128 * low
    x[0, 1, 2, 0] = 128 * low
    q = torch.tensor(x, dtype=torch.float32).to(DT[dtype])
    scale = 5 / (127 * float(q[0, 1, 2, 1]))           # scores of 5 and -5
    out, lse = _attend(lib, dtype, cache, q.cuda(), [n], None, True, scale)
    lib.dflash_check()
    ref = to.paged_attn(q.float().numpy().astype(np.float64), *cache.codes,
                        *cache.scale, cache.table, [n], [Q], scale)
    o, z = ref[0][0, 1, 2], ref[1][0, 1, 2]
    part = 2.0 ** -17 if dtype == "bf16" else (D + 3) * U
    d = part * 128 * low * 127 * scale
    assert abs(float(lse[0, 1, 2]) - z) <= d + (n + 16) * U
    tol = (2 * d + (n + 8) * U + (2.0 ** -14 if dtype == "bf16" else 0)
           ) * ref[3][0, 1, 2]
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(o)
    assert np.all(np.abs(out[0, 1, 2].double().cpu().numpy() - o) <= tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bits", [12, 16, 20, 24, 26, 30])
def test_attention_small_weights_of_a_long_run(lib, dtype, bits):
    """One token of weight 1 and value 0, thousands of weight 2^-bits behind
    it in the same run (enough sequences that none is cut more than once).
    With bf16 a weight w keeps 2^-13 of itself and 2^-25 of the largest, so
    that n of them sum to within n (2^-13 w + 2^-25)."""
    n, D, page, B = 6000, 64, 32, 304
    rng = np.random.default_rng(bits)
    cache = Cache([n], page, 1, D, rng, spread=0)
    kc, vc = cache.codes
    ids = cache.table[0]
    kc[ids] = 0
    kc[ids[0], 0, 0, 0] = 0x38                # 1.0: only token 0 scores
    vc[ids] = 0x78                            # 256
    vc[ids[0], 0, 0] = 0
    cache.scale[0][:] = 1
    cache.scale[1][:] = 2.0 ** -8             # every value is 1
    s = bits * math.log(2)
    q = torch.full((B, 1, 1, D), 1.0, dtype=DT[dtype], device="cuda")
    ref = to.paged_attn(np.ones((1, 1, 1, D)), *cache.codes, *cache.scale,
                        cache.table, [n], [1], s)
    cache.table = np.repeat(cache.table, B, 0)
    out, lse = _attend(lib, dtype, cache, q, [n] * B, None, True, s)
    lib.dflash_check()
    o, z = ref[0][0, 0, 0], float(ref[1][0, 0, 0])
    w = 2.0 ** -bits
    tol = (4 * (D + 3) * U * s + 2 * n * U) * o    # scores, sums
    if dtype == "bf16":
        tol = tol + n * (2.0 ** -13 * w + 2.0 ** -25) + 2.0 ** -9 * o
    for b in (0, 1, 150, B - 1):
        assert np.all(np.abs(out[b, 0, 0].double().cpu().numpy() - o) <= tol)
        assert abs(float(lse[b]) - z) <= 4 * (D + 3) * U * s + 2 * n * U


def test_attention_gives_up_on_a_wait_and_recovers(lib):
    """Every CTA has three sequences of 200 tiles, so that the warps that lay
    out q wait a hundred microseconds and more for the softmax: with a limit
    of a nanosecond they give up, the kernel drains, and the next call is
    right."""
    rng = np.random.default_rng(31)
    n, B, Q, Hq, D = 200 * 128, 456, 9, 8, 128
    cache = Cache([n], 128, 1, D, rng)
    q = torch.tensor(rng.standard_normal((1, Q, Hq, D)),
                     dtype=torch.float32).to(torch.bfloat16)
    ref = to.paged_attn(q.float().numpy().astype(np.float64), *cache.codes,
                        *cache.scale, cache.table, [n], [Q], 0.1)
    cache.table = np.repeat(cache.table, B, 0)
    q = q.cuda().repeat(B, 1, 1, 1)
    lib.dflash_check()                         # nothing pending
    try:
        lib.dflash_set_wait_limit_ns(1)
        _attend(lib, "bf16", cache, q, [n] * B, None, True, 0.1)
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_check()
        assert e.value.status == 5             # DFLASH_ERR_DEVICE_TIMEOUT
    finally:
        lib.dflash_set_wait_limit_ns(0)        # back to the default (2 s)
    out, lse = _attend(lib, "bf16", cache, q, [n] * B, None, True, 0.1)
    lib.dflash_check()
    for b in (0, 200, B - 1):
        _check_attn("bf16", D, n, out[b:b + 1], lse[b:b + 1], ref)


@pytest.mark.parametrize("Q,kv,g,Hkv,B", [(700, 700, 8, 1, 1),
                                          (1000, 1900, 3, 2, 2),
                                          (4096, 4096, 8, 2, 1)])
def test_attention_of_a_prompt_chunk(lib, Q, kv, g, Hkv, B):
    """Prompts of many row tiles, most of them whole in one CTA, some cut:
    rows at every place against the oracle's."""
    rng = np.random.default_rng(Q)
    D = 64
    cache = Cache([kv] * B, 64, Hkv, D, rng)
    q = torch.tensor(rng.standard_normal((B, Q, g * Hkv, D)),
                     dtype=torch.float32).to(torch.bfloat16)
    out, lse = _attend(lib, "bf16", cache, q.cuda(), [kv] * B, None, True,
                       0.125)
    lib.dflash_check()
    assert torch.isfinite(lse).all()
    at = rng.choice(Q, 40, replace=False)
    for i in at:                               # one query's rows each
        n = kv - Q + int(i) + 1
        ref = to.paged_attn(q[:, i:i + 1].float().numpy().astype(np.float64),
                            *cache.codes, *cache.scale, cache.table, [n] * B,
                            [1] * B, 0.125)
        _check_attn("bf16", D, n, out[:, i:i + 1], lse[:, i:i + 1], ref)


@pytest.mark.parametrize("dtype,g", [("bf16", 2), ("bf16", 30), ("fp32", 2)])
def test_attention_counts_a_bad_page_as_zeros(lib, dtype, g):
    """A page id outside the pool: flagged, and its tokens have keys and
    values of 0 (a score of 0, a share of the sum)."""
    rng = np.random.default_rng(41)
    n, D, page = 200, 64, 16
    cache = Cache([n], page, 1, D, rng)
    q = torch.tensor(rng.standard_normal((1, 2, g, D)),
                     dtype=torch.float32).to(DT[dtype])
    ids = cache.table[0]
    for c, s in zip(cache.codes, cache.scale):
        c[ids[3]] = 0
        s[ids[3]] = 1.0
    ref = to.paged_attn(q.float().numpy().astype(np.float64), *cache.codes,
                        *cache.scale, cache.table, [n], [2], 0.1)
    for bad in (-1, len(cache.scale[0]), 1 << 30):
        cache.table = cache.table.copy()
        cache.table[0, 3] = bad
        out, lse = _attend(lib, dtype, cache, q.cuda(), [n], None, True, 0.1)
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_check()
        assert e.value.status == 6             # DFLASH_ERR_BAD_INDEX
        _check_attn(dtype, D, n, out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g,n,B", [(4, 1, 1), (4, 300, 1), (20, 300, 3),
                                   (4, 20000, 1), (40, 900, 2)])
@pytest.mark.parametrize("size", [-5000.0, -300.0, -85.0, 85.0, 300.0, 5000.0])
def test_attention_far_scores(lib, dtype, g, n, B, size):
    """Rows whose scores all lie far below 0, or far above: 2^-score and
    2^score pass fp32's range, the softmax does not."""
    rng = np.random.default_rng(n + g)
    D, page = 64, 32
    cache = Cache([n] * B, page, 1, D, rng, spread=0)
    keys = cache.table[:, :-(-n // page)].ravel()
    x = np.full(cache.codes[0][keys].shape, 100.0)     # all keys alike but
    x[..., 0] += 8 * rng.integers(-3, 4, x.shape[:-1])  # for one dimension
    bits = oracle.e4m3_encode(x.astype(np.float32))
    tail = cache.codes[0][keys] == 0x7F                # past the lengths
    cache.codes[0][keys] = np.where(tail, 0x7F, bits)
    cache.scale[0][keys] = 2.0 ** -6
    q = torch.tensor(rng.uniform(1, 2, (B, 1, g, D)), dtype=torch.float32).to(
        DT[dtype])
    scale = size / float(q[0, 0, 0].double().sum() * 100 / 64)
    out, lse = _attend(lib, dtype, cache, q.cuda(), [n] * B, None, True, scale)
    lib.dflash_check()
    ref = to.paged_attn(q.float().numpy().astype(np.float64), *cache.codes,
                        *cache.scale, cache.table, [n] * B, [1] * B, scale)
    assert np.all(np.isfinite(ref[1])) and np.abs(ref[1]).max() > 60
    _check_attn(dtype, D, n, out, lse, ref)
