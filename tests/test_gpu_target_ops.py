"""The target's side of a cycle on the GPU against the oracle: cache append
with rotation, attention over the paged 8-bit cache, filtered sampling.

Tolerances are derived, not fitted:
  append   codes, scales and rotated q are functions of float32 roundings
           that the oracle repeats: equal bit for bit.
  attention  u = 2^-24.  A score is off by at most (D + 3) u |q|.|k| scale =:
           d (fp32 sums in any order; on the tensor cores the products are
           exact and the parts of q sum to q within 2^-18 of its largest
           value); a weight by 2 d + 4 u more; the sum over n tokens by n u.
           bf16: the weights are rounded to 12 bits or more (2^-12), the result to 8
           (2^-9 of its size).
  sample   kept sets and tokens are equal unless the oracle's own sums lie
           within 2^-20 of the decision (float32 exp against float64: 2 ulp).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import target_ops as to
from parity import np_

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _tables(n, rot, seed=0):
    f = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(n)[:, None] * f
    return (torch.tensor(np.cos(a), dtype=torch.float32, device="cuda"),
            torch.tensor(np.sin(a), dtype=torch.float32, device="cuda"))


def _table(lengths, page, rng, extra=1):
    need = [-(-int(n) // page) for n in lengths]
    total = sum(need) + extra
    order = rng.permutation(total)
    t = np.full((len(need), max(max(need), 1)), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


class Cache:
    """A cache with codes of normal values; slots that no token fills hold
    NaN codes, so that reading them shows."""

    def __init__(self, lengths, page, Hkv, D, rng, spread=3.0):
        self.page = page
        self.table, N = _table(lengths, page, rng)
        shape = (N, Hkv, page, D)
        self.codes, self.scale = [], []
        for _ in range(2):
            s = np.exp2(rng.integers(-8, -8 + int(spread) + 1, (N, Hkv)))
            x = rng.standard_normal(shape) * 100
            c = oracle.e4m3_encode(x.astype(np.float32))
            self.codes.append(c)
            self.scale.append(s.astype(np.float32))
        for b, n in enumerate(lengths):
            if n % page:
                last = self.table[b, n // page]
                for c in self.codes:
                    c[last, :, n % page:] = 0x7F
        free = np.setdiff1d(np.arange(N), self.table)
        for c, s in zip(self.codes, self.scale):
            c[free] = 0x7F
            s[free] = np.nan

    def cuda(self):
        d = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        return [d(self.codes[0]), d(self.codes[1]), d(self.scale[0]),
                d(self.scale[1])], d(self.table)


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,B,Q,Hq,Hkv,D,page,rot,inter", [
    ("bf16", 1, 1, 4, 1, 64, 16, 64, False),
    ("bf16", 3, 9, 8, 2, 128, 32, 128, False),
    ("bf16", 2, 17, 5, 5, 80, 16, 40, False),
    ("bf16", 2, 40, 4, 2, 128, 16, 64, True),
    ("fp32", 4, 5, 6, 2, 64, 64, 32, True),
    ("fp32", 2, 33, 2, 1, 256, 128, 256, False),
    ("bf16", 2, 300, 2, 2, 256, 128, 256, False),
    ("fp32", 3, 4, 2, 2, 16, 16, 8, False),
    ("bf16", 3, 6, 2, 2, 48, 32, 0, False),
])
def test_append_matches_the_oracle(lib, dtype, B, Q, Hq, Hkv, D, page, rot,
                                   inter):
    rng = np.random.default_rng(B * 100 + Q + D)
    pos = rng.integers(0, 3 * page, B)
    pos[0] = page - 1 if B > 1 else 0
    n_new = rng.integers(0, Q + 1, B)
    n_new[0] = Q
    if B > 2:
        n_new[1] = 0
    cache = Cache(pos + n_new, page, Hkv, D, rng)
    # rows of one projection's output: q, k, v side by side, odd loudness
    width = (Hq + 2 * Hkv) * D
    qkv = rng.standard_normal((B * Q, width)) * np.exp2(
        rng.integers(-6, 6, (B * Q, 1)))
    qkv = torch.tensor(qkv, dtype=torch.float32).to(DT[dtype]).cuda()
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    q, k, v = (q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
               v.unflatten(1, (Hkv, D)))
    cos, sin = _tables(3 * page + Q, rot) if rot else (None, None)
    (kc, vc, ks, vs), table = cache.cuda()
    q_out = torch.full((B, Q, Hq, D), 9.0, dtype=DT[dtype], device="cuda")
    kv_len = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q, k, v, cos, sin, i32(pos), i32(n_new), table, kc, vc, ks, vs,
            q_out, kv_len)
    lib.dflash_kv_append(*args, interleaved=inter)
    lib.dflash_check()
    f32 = lambda t: t.float().cpu().numpy()  # noqa: E731
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    oq, olen = to.kv_append(
        f32(q).reshape(B, Q, Hq, D), f32(k).reshape(B, Q, Hkv, D),
        f32(v).reshape(B, Q, Hkv, D), None if cos is None else f32(cos),
        None if sin is None else f32(sin), pos, n_new, cache.table, page,
        o[0], o[1], o[2], o[3], inter)
    assert np.array_equal(np_(kv_len), olen)
    assert np.array_equal(f32(q_out), f32(torch.from_numpy(oq).to(DT[dtype])))
    # slots that no token fills may be touched by no one
    for got, want in zip((kc, vc), o[:2]):
        assert np.array_equal(np_(got), want)
    for got, want in zip((ks, vs), o[2:]):
        assert np.array_equal(np_(got), want, equal_nan=True)
    # the same tokens again: nothing changes
    lib.dflash_kv_append(*args, interleaved=inter)
    lib.dflash_check()
    for got, want in zip((kc, vc), o[:2]):
        assert np.array_equal(np_(got), want)


def test_append_without_q_and_counts(lib):
    """q = None rotates keys only; n_new = None appends Q tokens each."""
    rng = np.random.default_rng(5)
    B, Q, Hkv, D, page = 2, 3, 2, 64, 16
    pos = np.array([14, 0])
    cache = Cache(pos + Q, page, Hkv, D, rng)
    k = torch.randn(B * Q, Hkv, D, device="cuda")
    v = torch.randn(B * Q, Hkv, D, device="cuda")
    cos, sin = _tables(32, D)
    (kc, vc, ks, vs), table = cache.cuda()
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    lib.dflash_kv_append(None, k, v, cos, sin, torch.tensor(
        pos, dtype=torch.int32, device="cuda"), None, table, kc, vc, ks, vs,
        None, kv_len)
    lib.dflash_check()
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    to.kv_append(None, np_(k).reshape(B, Q, Hkv, D),
                 np_(v).reshape(B, Q, Hkv, D), np_(cos), np_(sin), pos,
                 [Q, Q], cache.table, page, *o)
    assert np.array_equal(np_(kc), o[0]) and np.array_equal(np_(vc), o[1])
    assert np_(kv_len).tolist() == [17, 3]


def test_append_flags_what_does_not_fit(lib):
    """Tokens past the page table, a page id outside the pool, counts outside
    [0, Q], a negative position: flagged, left out, nothing else harmed."""
    rng = np.random.default_rng(6)
    B, Q, Hkv, D, page = 4, 5, 1, 16, 16
    cache = Cache(np.array([32, 32, 32, 32]), page, Hkv, D, rng)
    (kc, vc, ks, vs), table = cache.cuda()
    table[1, 1] = 10 ** 6
    k = torch.ones(B * Q, Hkv, D, device="cuda")
    pos = torch.tensor([30, 14, 3, -2], dtype=torch.int32, device="cuda")
    n = torch.tensor([5, 5, 6, 1], dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    lib.dflash_kv_append(None, k, k, None, None, pos, n, table, kc, vc, ks,
                         vs, None, kv_len)
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_check()
    assert e.value.status == 6
    assert np_(kv_len).tolist() == [32, 19, 3, -2]
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    x = np.ones((B, Q, Hkv, D), np.float32)
    t = cache.table.copy()
    to.kv_append(None, x, x, None, None, [30, 14, 3, 0], [2, 2, 0, 0], t,
                 page, *o)
    assert np.array_equal(np_(kc), o[0])
    assert np.array_equal(np_(vs), o[3], equal_nan=True)


def test_append_non_finite_inputs(lib):
    B, Q, Hkv, D, page = 1, 2, 1, 16, 16
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    kc, vc = z(1, 1, page, D), z(1, 1, page, D)
    ks, vs = z(1, 1, dt=torch.float32), z(1, 1, dt=torch.float32)
    k = torch.ones(B * Q, Hkv, D, device="cuda")
    v = k.clone()
    k[0, 0, 3] = float("nan")
    v[1, 0, 5] = float("-inf")
    lib.dflash_kv_append(None, k, v, None, None, z(1, dt=torch.int32), None,
                         z(1, 1, dt=torch.int32), kc, vc, ks, vs, None,
                         z(1, dt=torch.int32))
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_check()
    assert e.value.status == 4
    assert int(kc[0, 0, 0, 3]) == 0 and int(vc[0, 0, 1, 5]) == 0xFE
    assert float(ks) == 2.0 ** -8 and float(vs) == 2.0 ** -8
    rest = kc[0, 0, :2].cpu().numpy()
    rest[0, 3] = 0x78
    assert np.all(rest == 0x78)


@pytest.mark.parametrize("dtype,D,page,Q", [
    ("fp32", 256, 128, 200), ("bf16", 256, 128, 131), ("bf16", 64, 16, 3)])
def test_append_non_finite_anywhere(lib, dtype, D, page, Q):
    """NaN and infinities at any token of a page, those a thread reads twice
    among them: stored as 0 and the largest codes, no part of the scale."""
    rng = np.random.default_rng(Q)
    Hkv = 2
    cache = Cache(np.array([Q]), page, Hkv, D, rng)
    (kc, vc, ks, vs), table = cache.cuda()
    x = [torch.from_numpy(rng.standard_normal((Q, Hkv, D)).astype(
        np.float32)).to(DT[dtype]).float().numpy() for _ in range(2)]
    clean, top = [a.copy() for a in x], []
    for a, c in zip(x, clean):
        for bad in (np.nan, np.inf, -np.inf):
            a[rng.random(a.shape) < 0.003] = bad
        a[-1, 0, -1] = np.nan
        c[~np.isfinite(a)] = 0
        top.append(np.isinf(a))
    k, v = (torch.from_numpy(a).to(DT[dtype]).cuda() for a in x)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lib.dflash_kv_append(None, k, v, None, None, i32(0), None, table, kc, vc,
                         ks, vs, None, i32(0))
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_check()
    assert e.value.status == 4
    o = [c.copy() for c in cache.codes] + [s.copy() for s in cache.scale]
    to.kv_append(None, clean[0][None], clean[1][None], None, None, [0], [Q],
                 cache.table, page, *o)
    for a, hit, want in zip(x, top, o[:2]):
        for t, h, d in zip(*np.nonzero(hit)):
            want[cache.table[0, t // page], h, t % page, d] = (
                0x7E if a[t, h, d] > 0 else 0xFE)
    assert np.array_equal(np_(kc), o[0]) and np.array_equal(np_(vc), o[1])
    assert np.array_equal(np_(ks), o[2], equal_nan=True)
    assert np.array_equal(np_(vs), o[3], equal_nan=True)


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
def _attend(lib, dtype, cache, q, kv_len, q_len, causal, scale, want_lse=True,
            **kw):
    (kc, vc, ks, vs), table = cache.cuda()
    B, Q, Hq, D = q.shape
    Hkv = kc.shape[1]
    out = torch.full(q.shape, 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((B, Q, Hq), 7.0, device="cuda") if want_lse else None
    ws = torch.full((lib.dflash_paged_attn_workspace_bytes(
        B, Q, Hq, Hkv, D),), 0xFF, dtype=torch.uint8, device="cuda")
    i32 = lambda a: None if a is None else torch.tensor(  # noqa: E731
        np.asarray(a), dtype=torch.int32, device="cuda")
    lib.dflash_paged_attn(q, kc, vc, ks, vs, table, i32(kv_len), i32(q_len),
                          scale, out, lse, ws, causal=causal, **kw)
    return out, lse


def _check_attn(dtype, D, n, out, lse, ref):
    o, z, size, absv = ref
    got = out.float().cpu().numpy().astype(np.float64)
    live = np.isfinite(z)
    assert np.all(got[~live] == 0.0)
    d = (D + 3) * U * size
    extra = 0.0
    if dtype == "bf16":
        d = d + 2.0 ** -17 * size       # q in two E4M3 parts
        extra = 2.0 ** -12
    tol = (2 * d + 8 * U + n * U + extra)[..., None] * absv + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(o)
    bad = ~(np.abs(got - o) <= tol)          # a NaN is bad
    assert not bad.any(), (np.abs(got - o)[bad].max(), int(bad.sum()))
    if lse is not None:
        g = np_(lse).astype(np.float64)
        assert np.array_equal(np.isfinite(g), live)
        assert np.all(g[~live] == -np.inf)
        lt = d + (n + 8) * U + 4 * U * np.abs(np.where(live, z, 0))
        assert np.all(np.abs(g[live] - z[live]) <= lt[live])


ATTN = [
    # dtype, Hq, Hkv, D, page, Q, causal, kv lengths, query lengths
    ("bf16", 4, 1, 128, 16, 1, True, [1], None),
    ("bf16", 8, 2, 128, 32, 1, True, [37, 0, 128, 129, 1], [1, 0, 1, 1, 1]),
    ("bf16", 8, 1, 128, 64, 9, True, [9, 500, 77, 12], None),
    ("bf16", 8, 1, 128, 64, 9, False, [9, 500, 77, 8], [9, 4, 0, 8]),
    ("bf16", 16, 1, 128, 128, 17, True, [1000, 17, 127], None),
    ("bf16", 3, 3, 64, 16, 4, True, [300, 33, 4], [4, 1, 4]),
    ("bf16", 10, 2, 80, 32, 6, True, [700, 6], None),
    ("bf16", 4, 4, 16, 16, 3, True, [90, 3], None),
    ("bf16", 4, 2, 256, 32, 3, True, [300, 3], None),
    ("bf16", 4, 2, 112, 64, 40, True, [400, 64], [40, 33]),
    ("fp32", 4, 2, 64, 16, 4, True, [333, 4, 0, 50], [4, 4, 0, 2]),
    ("fp32", 6, 1, 128, 128, 5, False, [400, 1, 5], [5, 1, 5]),
    ("fp32", 2, 2, 256, 64, 2, True, [200, 2], None),
    ("fp32", 5, 5, 48, 32, 1, True, [2000, 1], None),
]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,Q,causal,kv,ql", ATTN)
def test_attention_matches_the_oracle(lib, dtype, Hq, Hkv, D, page, Q, causal,
                                      kv, ql):
    rng = np.random.default_rng(Hq * 7 + D + Q)
    cache = Cache(kv, page, Hkv, D, rng)
    B = len(kv)
    q = torch.tensor(rng.standard_normal((B, Q, Hq, D)) * 2,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    scale = 1 / math.sqrt(D)
    out, lse = _attend(lib, dtype, cache, q, kv, ql, causal, scale)
    lib.dflash_check()
    nq = [Q] * B if ql is None else ql
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale, cache.table, kv, nq,
                        scale, causal)
    _check_attn(dtype, D, max(kv), out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_long_cache_is_split_and_joined(lib, dtype):
    """One sequence long enough for many parts, and a very uneven batch."""
    rng = np.random.default_rng(11)
    kv = [30000, 5, 9000]
    cache = Cache(kv, 64, 1, 64, rng)
    q = torch.tensor(rng.standard_normal((3, 2, 2, 64)),
                     dtype=torch.float32).to(DT[dtype]).cuda()
    out, lse = _attend(lib, dtype, cache, q, kv, None, True, 0.125)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale, cache.table, kv,
                        [2, 2, 2], 0.125, True)
    _check_attn(dtype, 64, 30000, out, lse, ref)
    again, _ = _attend(lib, dtype, cache, q, kv, None, True, 0.125)
    assert torch.equal(out, again)            # the same bits every time


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_sink_and_flat_tail(lib, dtype):
    """A token that takes half of the weight while thousands share the other
    half: small weights must keep their share."""
    n, D, page = 6000, 64, 32
    rng = np.random.default_rng(12)
    cache = Cache([n], page, 1, D, rng, spread=0)
    kc, vc = cache.codes
    ks, vs = cache.scale
    ids = cache.table[0]
    kc[ids] = 0
    kc[ids[0], 0, 0] = 0x38                   # 1.0: only token 0 scores
    ks[:] = 1
    vs[:] = 2.0 ** -8
    s = math.log(n)                           # weight of token 0: a half
    q = torch.full((1, 1, 1, D), 1.0, dtype=DT[dtype], device="cuda")
    out, lse = _attend(lib, dtype, cache, q, [n], None, True, s / D)
    lib.dflash_check()
    ref = to.paged_attn(np.ones((1, 1, 1, D)), *cache.codes, *cache.scale,
                        cache.table, [n], [1], s / D)
    _check_attn(dtype, D, n, out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_uneven_scales_and_zero_pages(lib, dtype):
    """Pages of all zeros carry the smallest scale, others a large one; keys
    loud enough that one token takes nearly all."""
    rng = np.random.default_rng(13)
    n, D, page = 200, 64, 16
    cache = Cache([n], page, 2, D, rng)
    ids = cache.table[0]
    for c, s in zip(cache.codes, cache.scale):
        c[ids[3], 0] = 0
        s[ids[3], 0] = 2.0 ** -64
        s[ids[5], 1] = 2.0 ** 10
        s[ids[6], 1] = 2.0 ** -30
    q = torch.tensor(rng.standard_normal((1, 3, 4, D)),
                     dtype=torch.float32).to(DT[dtype]).cuda()
    out, lse = _attend(lib, dtype, cache, q, [n], None, True, 0.05)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale, cache.table, [n], [3],
                        0.05)
    _check_attn(dtype, D, n, out, lse, ref)


def test_attention_bad_lengths_and_pages_are_flagged(lib):
    rng = np.random.default_rng(14)
    for dtype in ("bf16", "fp32"):
        for what in ("kv", "q", "page"):
            cache = Cache([40, 40], 16, 1, 64, rng)
            kv, ql = [40, 40], [1, 1]
            if what == "kv":
                kv = [49, -1]                 # three pages hold 48
            elif what == "q":
                ql = [3, -1]
            else:
                cache.table[1, 1] = 1 << 20
            q = torch.zeros(2, 2, 2, 64, dtype=DT[dtype], device="cuda")
            _attend(lib, dtype, cache, q, kv, ql, True, 1.0)
            with pytest.raises(lib.DFlashError) as e:
                lib.dflash_check()
            assert e.value.status == 6, (dtype, what)


def test_attention_on_another_stream_and_without_lse(lib):
    rng = np.random.default_rng(15)
    cache = Cache([300, 20], 32, 2, 128, rng)
    q = torch.tensor(rng.standard_normal((2, 3, 8, 128)),
                     dtype=torch.float32).to(torch.bfloat16).cuda()
    want, _ = _attend(lib, "bf16", cache, q, [300, 20], None, True, 0.1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = _attend(lib, "bf16", cache, q, [300, 20], None, True, 0.1,
                     want_lse=False, stream=s)
    torch.cuda.synchronize()
    lib.dflash_check()
    assert torch.equal(got, want)


@pytest.mark.parametrize("Q,g", [(5, 4), (10, 4), (12, 5), (25, 3), (18, 5),
                                 (67, 3), (130, 4)])
def test_attention_every_row_count(lib, Q, g):
    """20 to 520 rows to a key head: every number of row columns of the
    tensor-core kernel, and several row tiles."""
    rng = np.random.default_rng(Q * g)
    kv = [Q + 300, Q, Q + 129]
    ql = [Q, Q, max(1, Q // 2)]
    cache = Cache(kv, 32, 2, 64, rng)
    q = torch.tensor(rng.standard_normal((3, Q, 2 * g, 64)),
                     dtype=torch.float32).to(torch.bfloat16).cuda()
    for causal in (True, False):
        out, lse = _attend(lib, "bf16", cache, q, kv, ql, causal, 0.125)
        lib.dflash_check()
        ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                            *cache.codes, *cache.scale, cache.table, kv, ql,
                            0.125, causal)
        _check_attn("bf16", 64, max(kv), out, lse, ref)


@pytest.mark.parametrize("B", [33, 70, 200])
def test_attention_many_sequences(lib, B):
    """More sequences than a warp has lanes, lengths from zero to several
    tiles: runs that start and end anywhere."""
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 700, B)
    kv[rng.integers(0, B, B // 5)] = 0
    kv[rng.integers(0, B, B // 5)] = 1
    ql = np.minimum(kv, rng.integers(0, 4, B))
    cache = Cache(kv, 16, 2, 32, rng)
    q = torch.tensor(rng.standard_normal((B, 3, 4, 32)),
                     dtype=torch.float32).to(torch.bfloat16).cuda()
    out, lse = _attend(lib, "bf16", cache, q, kv, ql, True, 0.2)
    lib.dflash_check()
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *cache.codes, *cache.scale, cache.table, kv, ql, 0.2)
    _check_attn("bf16", 32, 700, out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_rows_of_uneven_size_and_bad_rows(lib, dtype):
    """Heads whose queries differ a thousandfold share a key head; a row with
    a NaN or an infinity spoils only itself; the scale may be negative."""
    rng = np.random.default_rng(21)
    kv = [200]
    cache = Cache(kv, 32, 1, 64, rng)
    x = rng.standard_normal((1, 4, 4, 64))
    x *= np.array([1.0, 1e-3, 30.0, 1.0])[None, None, :, None]
    x[0, 1, 1] = 0.0
    clean = torch.tensor(x, dtype=torch.float32).to(DT[dtype])
    q = clean.clone()
    q[0, 2, 0, 5] = float("nan")
    q[0, 3, 2, 7] = float("inf")
    for scale in (0.05, -0.05):
        out, lse = _attend(lib, dtype, cache, q.cuda(), kv, None, True, scale)
        lib.dflash_check()
        ref = list(to.paged_attn(clean.float().numpy().astype(np.float64),
                                 *cache.codes, *cache.scale, cache.table, kv,
                                 [4], scale))
        for i, h in ((2, 0), (3, 2)):
            assert torch.isnan(out[0, i, h]).all()
            out[0, i, h] = torch.from_numpy(ref[0][0, i, h]).to(
                DT[dtype]).cuda()
            lse[0, i, h] = ref[1][0, i, h]
        _check_attn(dtype, 64, 200, out, lse, ref)


def test_cache_beyond_32_bit_offsets(lib):
    """Pages past the fourth gigabyte of the codes: append to them, attend
    over them."""
    N, Hkv, page, D = 40000, 8, 128, 128       # 5.2 GB of codes each
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    kc = torch.zeros(N, Hkv, page, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.ones(N, Hkv, device="cuda")
    vs = torch.ones(N, Hkv, device="cuda")
    rng = np.random.default_rng(22)
    ids = np.array([N - 1, N - 3, 2])
    table = torch.tensor(ids[None], dtype=torch.int32, device="cuda")
    n = 300
    k = torch.tensor(rng.standard_normal((n, Hkv, D)),
                     dtype=torch.float32).to(torch.bfloat16).cuda()
    v = torch.tensor(rng.standard_normal((n, Hkv, D)),
                     dtype=torch.float32).to(torch.bfloat16).cuda()
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_len = torch.empty_like(pos)
    lib.dflash_kv_append(None, k, v, None, None, pos, None, table, kc, vc, ks,
                         vs, None, kv_len)
    lib.dflash_check()
    small = [np.zeros((3, Hkv, page, D), np.uint8) for _ in range(2)] + [
        np.ones((3, Hkv), np.float32) for _ in range(2)]
    f32 = lambda t: t.float().cpu().numpy()  # noqa: E731
    to.kv_append(None, f32(k)[None], f32(v)[None], None, None, [0], [n],
                 np.array([[0, 1, 2]]), page, *small)
    for got, want in zip((kc, vc, ks, vs), small):
        assert np.array_equal(np_(got[torch.tensor(ids)]), want)
    for dtype in ("bf16", "fp32"):
        q = torch.tensor(rng.standard_normal((1, 2, 16, D)),
                         dtype=torch.float32).to(DT[dtype]).cuda()
        out = torch.empty_like(q)
        lse = torch.empty(1, 2, 16, device="cuda")
        ws = torch.empty(lib.dflash_paged_attn_workspace_bytes(
            1, 2, 16, Hkv, D), dtype=torch.uint8, device="cuda")
        lib.dflash_paged_attn(q, kc, vc, ks, vs, table, kv_len, None, 0.1,
                              out, lse, ws)
        lib.dflash_check()
        ref = to.paged_attn(f32(q).astype(np.float64), *small,
                            np.array([[0, 1, 2]]), [n], [2], 0.1)
        _check_attn(dtype, D, n, out, lse, ref)


def test_calls_replay_from_a_graph(lib):
    """The three calls captured once and replayed on new inputs."""
    rng = np.random.default_rng(23)
    B, Q, Hq, Hkv, D, page = 3, 5, 8, 2, 64, 16
    pos = np.array([20, 0, 47])
    cache = Cache(pos + Q, page, Hkv, D, rng)
    (kc, vc, ks, vs), table = cache.cuda()
    start = [t.clone() for t in (kc, vc, ks, vs)]
    x = torch.randn(B * Q, (Hq + 2 * Hkv) * D, device="cuda").to(
        torch.bfloat16)
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
    args = (q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)),
            v.unflatten(1, (Hkv, D)))
    cos, sin = _tables(64, D)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    qo = torch.empty(B, Q, Hq, D, dtype=torch.bfloat16, device="cuda")
    kl = torch.empty(B, dtype=torch.int32, device="cuda")
    out = torch.empty_like(qo)
    ws = torch.empty(lib.dflash_paged_attn_workspace_bytes(B, Q, Hq, Hkv, D),
                     dtype=torch.uint8, device="cuda")
    logits = torch.randn(B, 500, device="cuda")
    T, u = torch.ones(B, device="cuda"), torch.rand(B, device="cuda")
    kk = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    tok = torch.empty(B, dtype=torch.int32, device="cuda")
    ws2 = torch.empty(256, dtype=torch.uint8, device="cuda")

    def calls():
        lib.dflash_kv_append(*args, cos, sin, p, None, table, kc, vc, ks, vs,
                             qo, kl)
        lib.dflash_paged_attn(qo, kc, vc, ks, vs, table, kl, None, 0.125, out,
                              None, ws)
        lib.dflash_sample(logits, T, kk, None, None, u, tok, None, None, ws2)

    def reset():
        for t, s0 in zip((kc, vc, ks, vs), start):
            t.copy_(s0)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            calls()
    torch.cuda.synchronize()
    x.normal_()
    logits.normal_()
    reset()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (qo, out, tok, kc, vc, ks, vs)]
    reset()
    calls()
    torch.cuda.synchronize()
    lib.dflash_check()
    for a, b in zip(got, (qo, out, tok, kc, vc, ks, vs)):
        assert torch.equal(a.nan_to_num(7) if a.is_floating_point() else a,
                           b.nan_to_num(7) if b.is_floating_point() else b)


# --------------------------------------------------------------------------
# sampling
# --------------------------------------------------------------------------
NEAR = 2.0 ** -20


def _run_sample(lib, logits, T, k, p, m, u, filtered=True):
    R, V = logits.shape
    f = lambda a, dt: None if a is None else torch.tensor(  # noqa: E731
        np.asarray(a), dtype=dt, device="cuda")
    tok = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    nk = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((R, V), 5.0, device="cuda") if filtered else None
    ws = torch.empty(lib.dflash_sample_workspace_bytes(R, V),
                     dtype=torch.uint8, device="cuda")
    lib.dflash_sample(logits, f(T, torch.float32), f(k, torch.int32),
                      f(p, torch.float32), f(m, torch.float32),
                      f(u, torch.float32), tok, nk, out, ws)
    return np_(tok), np_(nk), None if out is None else np_(out)


def _check_sample(l, T, k, p, m, u, got):
    tok, nk, out = got
    R = l.shape[0]
    ties = 0
    for r in range(R):
        t, kept, near_p, near_u = to.sample_row(
            l[r], T[r], 0 if k is None else k[r], 1.0 if p is None else p[r],
            0.0 if m is None else m[r], u[r])
        if near_p < NEAR:
            ties += 1
            continue
        assert nk[r] == kept.sum(), (r, nk[r], kept.sum())
        if out is not None:
            want = np.where(kept, l[r], -np.inf)
            assert np.array_equal(out[r], want.astype(np.float32)), r
        if near_u < NEAR:
            ties += 1
            continue
        assert tok[r] == t, (r, tok[r], t)
    assert ties <= max(2, R // 8)


@pytest.mark.parametrize("dtype,R,V", [
    ("fp32", 1, 1), ("fp32", 3, 7), ("bf16", 5, 40), ("fp32", 40, 1000),
    ("bf16", 17, 4099), ("fp32", 12, 33001), ("fp32", 6, 151936),
    ("bf16", 4, 262144), ("bf16", 3, 45003)])
@pytest.mark.parametrize("mode", ["T", "k", "p", "m", "all"])
def test_sample_matches_the_oracle(lib, dtype, R, V, mode):
    rng = np.random.default_rng(V + len(mode))
    l = rng.standard_normal((R, V)) * 2.5
    l[:, rng.integers(0, V, 12)] += 5
    x = torch.tensor(l, dtype=torch.float32).to(DT[dtype]).cuda()
    l = x.float().cpu().numpy()
    pick = lambda a: np.asarray(a)[rng.integers(0, len(a), R)]  # noqa: E731
    T = pick([0.0, 0.5, 1.0, 1.7] if mode == "all" else [0.7, 1.0])
    k = pick([0, 1, 20, 50, 1000]) if mode in ("k", "all") else None
    p = pick([1.0, 0.95, 0.5, 0.0]) if mode in ("p", "all") else None
    m = pick([0.0, 0.02, 0.2, 1.0]) if mode in ("m", "all") else None
    u = rng.random(R).astype(np.float32)
    got = _run_sample(lib, x, T, k, p, m, u)
    lib.dflash_check()
    _check_sample(l, T, k, p, m, u, got)


def test_sample_ties_and_flat_rows(lib):
    """Equal logits by the thousand (no list holds them), top-k and top-p
    through the middle of a tie, and a top-k that reaches into the tail of
    weightless tokens."""
    V = 20000
    rng = np.random.default_rng(8)
    l = np.zeros((6, V), np.float32)
    l[1] = np.round(rng.standard_normal(V)).astype(np.float32)
    l[2] = -100.0 - (np.arange(V) % 3)
    l[2, 77] = 0.0
    l[3] = np.where(np.arange(V) % 2, -np.inf, 1.0)
    l[4] = -0.0
    l[4, ::2] = 0.0
    l[5] = np.round(rng.standard_normal(V)).astype(np.float32)
    x = torch.from_numpy(l).cuda()
    u = np.array([0.3, 0.9, 0.5, 0.7, 0.0, 0.123], np.float32)
    T = np.array([1, 0.5, 1, 1, 2, 0.7], np.float32)
    for k, p in (([1234, 3000, 5000, 700, 9, 6000], None),
                 (None, [0.3, 0.6, 0.9, 0.25, 0.51, 0.77]),
                 ([1234, 3000, 5000, 700, 9, 6000],
                  [0.3, 0.6, 0.9, 0.25, 0.51, 0.77])):
        got = _run_sample(lib, x, T, k, p, None, u)
        lib.dflash_check()
        _check_sample(l, T, k, p, None, u, got)


def test_sample_beyond_32_bit_offsets(lib):
    """Logits and filtered logits past the 2^31st element."""
    R, V = 8200, 262144
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    x = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    rows = [0, 4096, R - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in rows:
        x[r] = (3 * torch.randn(V, generator=g, device="cuda")).to(x.dtype)
    T = torch.full((R,), 0.8, device="cuda")
    k = torch.full((R,), 30, dtype=torch.int32, device="cuda")
    u = torch.rand(R, generator=g, device="cuda")
    tok = torch.empty(R, dtype=torch.int32, device="cuda")
    nk = torch.empty_like(tok)
    out = torch.empty(R, V, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lib.dflash_sample(x, T, k, None, None, u, tok, nk, out, ws)
    lib.dflash_check()
    l = x[rows].float().cpu().numpy()
    _check_sample(l, [0.8] * 3, [30] * 3, None, None, np_(u[rows]),
                  (np_(tok[rows]), np_(nk[rows]), np_(out[rows])))
    assert int(nk.min()) == 30 and int(nk.max()) == 30


def test_sample_rows_apart_and_misaligned(lib):
    """Rows of a wider matrix, at odd offsets."""
    rng = np.random.default_rng(9)
    for dtype in ("fp32", "bf16"):
        big = torch.tensor(rng.standard_normal((4, 5003)) * 3,
                           dtype=torch.float32).to(DT[dtype]).cuda()
        x = big[:, 1:5000]
        l = x.float().cpu().numpy()
        T = np.full(4, 0.9, np.float32)
        u = rng.random(4).astype(np.float32)
        got = _run_sample(lib, x, T, [40] * 4, [0.9] * 4, None, u)
        lib.dflash_check()
        _check_sample(l, T, [40] * 4, [0.9] * 4, None, u, got)


def test_sample_flags_and_empty_rows(lib):
    l = np.zeros((5, 64), np.float32)
    l[0] = -np.inf                            # nothing to draw from
    l[1, 9] = np.nan
    l[2, 5] = 4.0
    x = torch.from_numpy(l).cuda()
    u = [0.5] * 5
    for rows, T in (([0], [1.0]), ([1], [1.0]), ([2], [-1.0]),
                    ([2], [float("nan")]), ([2], [float("inf")])):
        tok, nk, out = _run_sample(lib, x[rows], T, None, None, None,
                                   [u[r] for r in rows])
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_check()
        assert e.value.status == 4
        if rows == [0]:
            assert tok[0] == -1 and nk[0] == 0 and np.all(out == -np.inf)
        elif rows == [1]:
            assert nk[0] == 63 and out[0, 9] == -np.inf and tok[0] != 9
        else:
            assert tok[0] == 5 and nk[0] == 1
    # u at and outside its ends stays within the kept tokens
    tok, _, _ = _run_sample(lib, x[[2, 2, 2]], [1.0] * 3, [3] * 3, None, None,
                            [0.0, 1.0, -3.0])
    lib.dflash_check()
    assert tok.tolist() == [0, 5, 0]


def test_sample_does_not_depend_on_the_split(lib):
    """The same row as one of many, alone, and inside a wider vocabulary of
    masked tokens (another cluster size): one token, one kept set."""
    rng = np.random.default_rng(10)
    V = 9000
    l = (rng.standard_normal((1, V)) * 2).astype(np.float32)
    wide = np.full((1, 200000), -np.inf, np.float32)
    wide[:, :V] = l
    for u in rng.random(20):
        a = [_run_sample(lib, torch.from_numpy(x).cuda(), [0.8] * x.shape[0],
                         None, [0.97] * x.shape[0], None, [u] * x.shape[0])
             for x in (l, np.repeat(l, 9, 0), wide)]
        assert len({int(t) for g in a for t in g[0]}) == 1
        assert len({int(n) for g in a for n in g[1]}) == 1
    lib.dflash_check()


def _wide_row(V, kind):
    rng = np.random.default_rng(V)
    l = (2.5 * rng.standard_normal(V)).astype(np.float32)
    l[rng.integers(0, V, 30)] += 6
    if kind == "bf16 values":      # values tie by the hundred
        l = torch.from_numpy(l).bfloat16().float().numpy()
    elif kind == "eighths":        # and by the thousand
        l = np.round(l * 8) / 8
    elif kind == "flat":
        l = (l * 0.02).astype(np.float32)
    elif kind == "one tie":        # 700 equal tokens around the cuts
        l[rng.permutation(V)[:700]] = np.partition(l, -650)[-650]
    elif kind == "masked":
        l[rng.random(V) < 0.7] = -np.inf
    return l[None]


@pytest.mark.parametrize("kind", ["spread", "bf16 values", "eighths", "flat",
                                  "one tie", "masked"])
@pytest.mark.parametrize("T,k,p,m", [
    (1.3, 0, 0.95, 0.0), (0.6, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.001),
    (1.0, 0, 0.999, 0.05), (1.0, 900, 1.0, 0.0), (1.0, 1200, 0.8, 0.01),
    (0.02, 1500, 0.9, 0.0), (1.0, 2040, 1.0, 0.0), (1.0, 9000, 0.97, 0.0),
    (40.0, 0, 0.3, 0.0), (1.0, 0, 1.0, 0.0004)])
def test_sample_large_kept_sets(lib, kind, T, k, p, m):
    """Kept sets of a hundred to tens of thousands, ties inside and across
    every list's size, from one row (eight CTAs) and among many (one to four
    CTAs, other registers, logits not held): the oracle's, and all the same."""
    V = 60001 if kind == "masked" else 131072
    l = _wide_row(V, kind)
    x = torch.from_numpy(l).cuda()
    if kind == "bf16 values":
        y = x.bfloat16()
    us = np.array([0.0, 0.37, 0.9999], np.float32)
    for u in us:
        a = _run_sample(lib, x, [T], [k], [p], [m], [u])
        _check_sample(l, [T], [k], [p], [m], [u], a)
        for n in (3, 300, 1300):
            wide = (y if kind == "bf16 values" and n == 3 else x).repeat(n, 1)
            b = _run_sample(lib, wide, [T] * n, [k] * n, [p] * n, [m] * n,
                            [u] * n, filtered=n == 3)
            assert np.all(b[0] == a[0]) and np.all(b[1] == a[1])
            if n == 3:
                assert np.array_equal(b[2], np.repeat(a[2], n, 0))
            del wide
    lib.dflash_check()


def test_sample_largest_vocabulary(lib):
    """Weights of 2^20 - 1 equal tokens add up in 64 bits; one more token is
    refused."""
    V = (1 << 20) - 1
    l = np.full((2, V), -3.25, np.float32)
    x = torch.from_numpy(l).cuda()
    for k, p in ((None, None), (None, [0.75, 0.125]), ([1000, 700000], None)):
        u = np.array([0.6, 0.3], np.float32)
        got = _run_sample(lib, x, [1.0, 0.5], k, p, None, u)
        lib.dflash_check()
        _check_sample(l, [1.0, 0.5], k, p, None, u, got)
    assert lib.dflash_sample_workspace_bytes(2, V + 1) == 0


def test_filtered_logits_make_the_verify_lossless(lib):
    """dflash_verify on the filtered logits draws from the filtered target
    distribution: with no draft accepted by design, the emitted token's
    frequencies over many sequences follow it (chi-square, 8 tokens)."""
    B, K, V = 4096, 1, 8
    rng = np.random.default_rng(16)
    l = np.tile((rng.standard_normal((1, 1, V)) * 1.5).astype(np.float32),
                (B, K + 1, 1))
    x = torch.from_numpy(l).cuda()
    R = B * (K + 1)
    _, _, out = _run_sample(lib, x.view(R, V), [0.9] * R, [5] * R,
                            [0.95] * R, None, [0.5] * R)
    topi = torch.full((B, K, 16), -1, dtype=torch.int32, device="cuda")
    topi[..., :V] = torch.arange(V, device="cuda", dtype=torch.int32)
    q = torch.zeros(B, K, 16, device="cuda")
    q[..., :V] = 1 / V                        # a flat draft distribution
    draft = torch.from_numpy(rng.integers(0, V, (B, K)).astype(
        np.int32)).cuda()
    n = torch.empty(B, dtype=torch.int32, device="cuda")
    tok = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.dflash_workspace_bytes(1, B, K, 0, V),
                     dtype=torch.uint8, device="cuda")
    lib.dflash_verify(torch.from_numpy(out).cuda().view(B, K + 1, V), draft,
                      topi, q, 0.9, 3, 1, n, tok, ws)
    lib.dflash_check()
    got = np.bincount(np_(tok)[:, 0], minlength=V).astype(np.float64)
    _, kept, _, _ = to.sample_row(l[0, 0], 0.9, 5, 0.95)
    p = np.where(kept, np.exp(l[0, 0].astype(np.float64) / 0.9), 0)
    p /= p.sum()
    assert np.all(got[~kept] == 0)
    chi = ((got - B * p)[kept] ** 2 / (B * p[kept])).sum()
    assert chi < 30                           # 4 degrees of freedom: 5e-6
