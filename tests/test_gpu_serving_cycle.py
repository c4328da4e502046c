"""The operators around a shared prompt and a bounded cache together: two
rounds of append, attention, gathered weight and eviction against the oracle,
captured and replayed, on streams side by side, in a pool beyond 32 bits; the
waits' limits; and examples/shared_prompt.py.

Tolerances: those of test_gpu_serving_ops and test_gpu_target_ops, whose
derivations stand there; everything else is equal bit for bit."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from oracle import serving_ops as so
from oracle import target_ops as to
from parity import np_
from test_gpu_serving_ops import (U, _check_evict, _check_logprobs, _i32,
                                  _logprobs, _mass_args, _status)
from test_gpu_target_ops import DT, Cache, _check_attn, _tables

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


class Chain:
    """B sequences with `shared` tokens in common that a first append fills,
    then two rounds: append, attend, count, evict.  Pages are numbered apart by
    `stride` in a pool that large."""

    def __init__(self, lib, dtype="bf16", B=3, Q=5, Hq=8, Hkv=2, D=64,
                 page=16, shared=64, budget=85, seed=0, stride=1):
        self.lib, self.dtype = lib, dtype
        self.B, self.Q, self.Hq, self.Hkv, self.D = B, Q, Hq, Hkv, D
        self.page, self.shared, self.budget = page, shared, budget
        self.recent = 4
        rng = np.random.default_rng(seed)
        first = shared // page
        most = -(-(budget + Q) // page)
        pages = first + B * (most - first)
        order = rng.permutation(pages).astype(np.int32) * stride
        table = np.full((B, most), -1, np.int32)
        table[:, :first] = order[:first]
        table[:, first:] = order[first:].reshape(B, -1)
        self.pages = order
        self.table_np, self.table = table, _i32(table)
        N = pages * stride
        self.pool = [torch.empty(N, Hkv, page, D, dtype=torch.uint8,
                                 device="cuda") for _ in range(2)]
        self.pool += [torch.empty(N, Hkv, device="cuda") for _ in range(2)]
        r = lambda *s: torch.tensor(  # noqa: E731
            rng.standard_normal(s), dtype=torch.float32).to(DT[dtype]).cuda()
        self.prompt = [r(shared, Hkv, D) for _ in range(2)]
        # own tokens up to the budget, then a block in each round
        self.own = budget - shared - 3
        self.fill = [r(B * self.own, Hkv, D) for _ in range(2)]
        self.blocks = [(2 * r(B * Q, Hq, D), r(B * Q, Hkv, D),
                        r(B * Q, Hkv, D)) for _ in range(2)]
        self.n_new = [np.array([Q, 0, Q - 2]), np.array([1, Q, Q])]
        self.cos, self.sin = _tables(500, D)
        self.at = [rng.integers(0, 500, (2, B * Q)) for _ in range(2)]
        self.of = np.arange(D // 2) % 2
        self.at_gpu = [_i32(a) for a in self.at]
        self.of_gpu = torch.tensor(self.of, dtype=torch.uint8, device="cuda")
        self.new_gpu = [_i32(n) for n in self.n_new]
        slots = most * page
        f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.mass, self.mass2 = f(B, Hkv, slots), f(B, Hkv, slots)
        self.start = torch.tensor(rng.random((B, Hkv, slots)),
                                  dtype=torch.float32, device="cuda")
        i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.len, self.kv_len, self.first_len = i(B), i(B), i(1)
        self.kept = i(B, Hkv, budget)
        self.lens0, self.pre_len = _i32([shared] * B), _i32([0])
        self.q_out, self.out = (torch.empty(
            B, Q, Hq, D, dtype=DT[dtype], device="cuda") for _ in range(2))
        self.lse = f(B, Q, Hq)
        u8 = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = u8(lib.dflash_shared_attn_workspace_bytes(B, Q, Hq, Hkv, D))
        self.ws2 = u8(lib.dflash_kv_evict_workspace_bytes(B, Hkv, page,
                                                          budget))

    def run(self):
        """Everything, on the current stream; returns clones of what each
        step left."""
        lib, scale = self.lib, self.D ** -0.5
        said = []

        def keep(**kw):
            said.append({k: v.clone() for k, v in kw.items()})
        for p in self.pool:
            if p.shape[0] == self.pages.size:  # (others are zeroed once)
                p.zero_()
        self.mass.copy_(self.start)
        self.mass2.zero_()
        if self.shared:
            lib.dflash_kv_append(None, *self.prompt, None, None, self.pre_len,
                                 None, self.table[:1], *self.pool, None,
                                 self.first_len)
        lib.dflash_kv_append(None, *self.fill, None, None, self.lens0, None,
                             self.table, *self.pool, None, self.len)
        mass, other = self.mass, self.mass2
        for r in range(2):
            q, k, v = self.blocks[r]
            lib.dflash_kv_append_axes(
                q, k, v, self.cos, self.sin, self.at_gpu[r], self.of_gpu,
                self.len, self.new_gpu[r], self.table, *self.pool, self.q_out,
                self.kv_len)
            keep(q=self.q_out, kv_len=self.kv_len)
            lib.dflash_shared_attn(
                self.q_out, *self.pool, self.table, self.kv_len,
                self.new_gpu[r], self.shared, scale, self.out, self.lse,
                self.ws)
            keep(out=self.out, lse=self.lse)
            lib.dflash_attn_mass(
                self.q_out, self.pool[0], self.pool[2], self.table,
                self.kv_len, self.new_gpu[r], self.lse, self.len, self.shared,
                scale, 0.5, mass)
            keep(mass=mass)
            lib.dflash_kv_evict(
                mass, *self.pool, self.table, self.kv_len, self.budget,
                self.shared, self.recent, other, self.len, self.kept,
                self.ws2)
            keep(mass=other, len=self.len, kept=self.kept)
            mass, other = other, mass
        return said

    def cache(self):
        at = torch.as_tensor(self.pages.astype(np.int64), device="cuda")
        return [np_(p[at]) for p in self.pool]

    def check(self, said):
        """Every step against the oracle's, from what the step before left."""
        f32 = lambda t: t.float().cpu().numpy()  # noqa: E731
        B, Q, Hq, Hkv, D = self.B, self.Q, self.Hq, self.Hkv, self.D
        N = self.pages.size
        o = [np.zeros((N, Hkv, self.page, D), np.uint8) for _ in range(2)] + [
            np.zeros((N, Hkv), np.float32) for _ in range(2)]
        if self.shared:
            k, v = (f32(t).reshape(1, -1, Hkv, D) for t in self.prompt)
            to.kv_append(None, k, v, None, None, [0], [self.shared],
                         self.table_np[:1], self.page, *o)
        k, v = (f32(t).reshape(B, -1, Hkv, D) for t in self.fill)
        _, n = to.kv_append(None, k, v, None, None, [self.shared] * B,
                            [self.own] * B, self.table_np, self.page, *o)
        mass = np_(self.start)
        for r in range(2):
            new = self.n_new[r]
            q, k, v = (f32(t).reshape(B, Q, -1, D) for t in self.blocks[r])
            oq, kv = so.kv_append_axes(
                q, k, v, np_(self.cos), np_(self.sin), self.at[r], self.of, n,
                new, self.table_np, self.page, *o)
            got = said[4 * r]
            assert np.array_equal(np_(got["kv_len"]), kv)
            assert np.array_equal(
                f32(got["q"]), f32(torch.from_numpy(oq).to(DT[self.dtype])))
            q64 = f32(got["q"]).astype(np.float64)
            att = said[4 * r + 1]
            _check_attn(self.dtype, D, int(kv.max()), att["out"], att["lse"],
                        to.paged_attn(q64, *o, self.table_np, kv, new,
                                      D ** -0.5, True))
            want, size = so.attn_mass(
                q64, o[0], o[2], self.table_np, kv, new, np_(att["lse"]), n,
                self.shared, D ** -0.5, 0.5, mass)
            now = np_(said[4 * r + 2]["mass"])
            tol = ((D + 12) * U * size +
                   (Q * Hq // Hkv + 16) * U * np.abs(want))
            assert np.all(np.abs(now - want) <= tol)
            n, kept, moved = so.kv_evict(now, *o, self.table_np, kv,
                                         self.budget, self.shared,
                                         self.recent)
            got = said[4 * r + 3]
            assert np.array_equal(np_(got["len"]), n)
            assert np.array_equal(np_(got["kept"]), kept)
            # past the new lengths the buffer holds what it held before
            mass = np_(got["mass"])
            for b in range(B):
                for h in range(Hkv):
                    assert np.array_equal(mass[b, h, :n[b]], moved[b][h])
        at = self.pages
        for got, want in zip(self.cache(), o):
            assert np.array_equal(got, want[at])


def _same(a, b):
    for x, y in zip(a, b):
        for k in x:
            assert torch.equal(x[k], y[k]), k


def _same_cache(a, b):
    for x, y in zip(a, b):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("dtype,kw", [
    ("bf16", {}), ("fp32", {}),
    ("bf16", dict(Hq=16, Hkv=1, D=128, page=32, Q=9, shared=128, budget=200)),
    ("bf16", dict(B=40, Q=3, Hq=4, Hkv=4, D=32, shared=32, budget=60)),
    ("bf16", dict(Hq=2, Hkv=1, D=256, page=16, Q=4, shared=0, budget=40))])
def test_two_rounds_match_the_oracle(lib, dtype, kw):
    c = Chain(lib, dtype, **kw)
    if c.B != 3:
        rng = np.random.default_rng(1)
        c.n_new = [rng.integers(0, c.Q + 1, c.B) for _ in range(2)]
        c.new_gpu = [_i32(n) for n in c.n_new]
    said = c.run()
    lib.dflash_check()
    c.check(said)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rounds_captured_and_replayed(lib, dtype):
    """A captured chain replayed twice gives the same bits as the calls."""
    c = Chain(lib, dtype)
    plain = c.run()
    cache = c.cache()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        said = c.run()
    for _ in range(2):
        for t in (c.out, c.lse, c.q_out, c.ws, c.ws2, c.len, c.kept):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(plain, said)
        _same_cache(cache, c.cache())
    lib.dflash_check()


def test_two_captured_graphs_share_workspaces(lib):
    """Graphs with one workspace between them, replayed by turns."""
    a, b = Chain(lib, seed=1), Chain(lib, seed=2)
    b.ws, b.ws2 = a.ws, a.ws2
    want, graphs = [], []
    for x in (a, b):
        x.run()
        want.append(x.cache())
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    lib.dflash_check()
    for x, w in zip((a, b), want):
        _same_cache(w, x.cache())


def test_rounds_on_streams_side_by_side(lib):
    chains = [Chain(lib, seed=s) for s in range(4)]
    want = [(c.run(), c.cache()) for c in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(3):
        got = []
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                got.append(c.run())
        torch.cuda.synchronize()
        for c, g, (w, cache) in zip(chains, got, want):
            _same(w, g)
            _same_cache(cache, c.cache())
    lib.dflash_check()


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 64),
                                          ("fp32", 128, 64)])
def test_pool_beyond_32_bits(lib, dtype, D, page):
    """Pages far apart in pools of 5 GB each: the same bits as in small ones."""
    kw = dict(Hq=16, Hkv=8, D=D, page=page, shared=128, budget=300)
    a = Chain(lib, dtype, **kw)
    stride = -(-(5 << 30) // (a.pool[0].numel()))
    assert (int(a.pages.max()) * stride + 1) * 8 * page * D > 1 << 32
    b = Chain(lib, dtype, stride=stride, **kw)
    at = torch.as_tensor(b.pages.astype(np.int64), device="cuda")
    for p in b.pool:
        p[at] = 0
    x, y = a.run(), b.run()
    torch.cuda.synchronize()
    lib.dflash_check()
    _same(x, y)
    _same_cache(a.cache(), b.cache())


def test_mass_of_many_rows_over_many_tiles(lib):
    """More rows than a pass takes and more tiles than it keeps sums of."""
    rng = np.random.default_rng(8)
    Hq, Hkv, D, page, Q, kv, ql = 32, 2, 64, 32, 20, [9001, 130], [20, 9]
    cache, q, q64, nq, lse = _mass_args(rng, "bf16", Hq, Hkv, D, page, Q, True,
                                        kv, ql)
    (kc, _, ks, _), table = cache.cuda()
    old = rng.random((2, Hkv, 9001)).astype(np.float32)
    mass = torch.from_numpy(old.copy()).cuda()
    lib.dflash_attn_mass(q, kc, ks, table, _i32(kv), _i32(ql),
                         torch.from_numpy(lse).cuda(), None, 70, D ** -0.5,
                         1.0, mass)
    lib.dflash_check()
    want, size = so.attn_mass(q64, cache.codes[0], cache.scale[0],
                              cache.table, kv, nq, lse, None, 70, D ** -0.5,
                              1.0, old)
    tol = (D + 12) * U * size + (Q * 16 + 16) * U * np.abs(want)
    assert np.all(np.abs(np_(mass) - want) <= tol)


def test_attention_with_nothing_shared_is_paged_attention(lib):
    """Up to the orders of sums and the roundings of either."""
    rng = np.random.default_rng(12)
    D, page, kv = 128, 32, [700, 64, 1]
    cache, q, q64, nq, _ = _mass_args(rng, "bf16", 8, 2, D, page, 1, True, kv,
                                      None)
    pool, table = cache.cuda()
    ref = to.paged_attn(q64, *cache.codes, *cache.scale, cache.table, kv, nq,
                        0.1, True)
    for name, extra in (("paged", ()), ("shared", (0,))):
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:3], device="cuda")
        ws = torch.empty(getattr(lib, f"dflash_{name}_attn_workspace_bytes")(
            3, 1, 8, 2, D), dtype=torch.uint8, device="cuda")
        getattr(lib, f"dflash_{name}_attn")(q, *pool, table, _i32(kv), None,
                                            *extra, 0.1, out, lse, ws)
        lib.dflash_check()
        _check_attn("bf16", D, 700, out, lse, ref)


@pytest.mark.parametrize("Hkv,D,page,budget,sink,recent,kv", [
    # clusters of eight, whose slots do not fit their registers
    (1, 16, 128, 100001, 5, 1000, [150003]),
    (1, 32, 16, 66000, 0, 0, [70001, 3]),
    # many heads: small CTAs, the same for one sequence
    (8, 16, 64, 12000, 100, 50, [20001] + [90] * 19),
    # nothing to choose in clusters of several CTAs
    (2, 64, 32, 2500, 1500, 1000, [3000, 2501, 2500, 7777]),
    (8, 64, 16, 700, 0, 700, [3000] * 3),
])
@pytest.mark.parametrize("ties", [False, True])
def test_eviction_by_clusters(lib, Hkv, D, page, budget, sink, recent, kv,
                              ties):
    rng = np.random.default_rng(budget + ties)
    cache = Cache(kv, page, Hkv, D, rng)
    mass = rng.random((len(kv), Hkv, max(kv) + 5)).astype(np.float32)
    if ties:
        mass = np.floor(mass * 4) / 4
    _check_evict(lib, cache, mass, kv, budget, sink, recent)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0, 7.0])
def test_log_probabilities_of_masked_rows(lib, dtype, T):
    """Rows masked by the type's lowest value, in whole stretches: as if those
    tokens were not there, also if one of them is the given token, whose own log
    probability is what its logit says."""
    rng = np.random.default_rng(21)
    V, K, low = 30011, 8, torch.finfo(DT[dtype]).min
    l = torch.tensor(rng.standard_normal((4, V)) * 3,
                     dtype=torch.float32).to(DT[dtype]).cuda()
    l[0, 100:] = low
    l[1, :V - 3] = low
    l[2, ::2] = low
    l[3, 5:29000] = low
    token = [3, V - 1, 7, 9]
    got = _logprobs(lib, l, [T] * 4, token, K)
    lib.dflash_check()
    want = l.clone()
    want[want == low] = -torch.inf
    # (the oracle's weights of them are 0 either way)
    seen = {k: v[:3] for k, v in got.items()}
    seen["top"], seen["top_id"] = got["top"][:3, :3], got["top_id"][:3, :3]
    _check_logprobs(want[:3], [T] * 3, token[:3], 3, seen)
    _check_logprobs(want[3:], [T], [0], 4,
                    {k: v[3:] for k, v in _logprobs(
                        lib, l, [T] * 4, [0] * 4, 4).items()})
    # (l / T may pass fp32's range)
    own = low / T if low / T > -3.5e38 else -np.inf
    assert got["logprob"][3] == own or abs(
        got["logprob"][3] / own - 1) <= 4 * U
    # three tokens only: the others follow in the order of their ids
    assert got["top_id"][1, 3:].tolist() == list(range(K - 3))
    assert np.all(got["top"][1, 3:] <= -1e37)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_log_probabilities_of_rows_all_at_one_far_value(lib, dtype, T):
    """All tokens at the type's lowest value, at a large one of either sign,
    some at -inf: uniform over what is not -inf."""
    V = 4099
    for value in (torch.finfo(DT[dtype]).min, -1e30, 1e30, 3e9, -3e9):
        l = torch.full((2, V), value, dtype=torch.float32).to(
            DT[dtype]).cuda()
        l[1, 10:] = -torch.inf
        got = _logprobs(lib, l, [T] * 2, [5, 5], 4)
        lib.dflash_check()
        for r, n in ((0, V), (1, 10)):
            x = float(l[0, 0].float()) / T
            z = -np.inf if x < -3.5e38 else np.float32(x + math.log(n))
            assert got["lse"][r] == z or abs(got["lse"][r] / z - 1) <= 4 * U
            tol = (V / 512 + 40) * U + 8 * U * math.log(n)
            assert abs(got["logprob"][r] + math.log(n)) <= tol
            assert abs(got["entropy"][r] - math.log(n)) <= tol
            assert got["rank"][r] == 5
            assert got["top_id"][r].tolist() == [0, 1, 2, 3]
            assert np.all(np.abs(got["top"][r] + math.log(n)) <= tol)


def _limited(lib, call):
    """call() with a limit of a nanosecond: flagged, and over."""
    lib.dflash_check()                         # nothing pending
    try:
        lib.dflash_set_wait_limit_ns(1)
        call()
        _status(lib, 5)                        # DFLASH_ERR_DEVICE_TIMEOUT
    finally:
        lib.dflash_set_wait_limit_ns(0)        # back to the default (2 s)


def test_shared_attention_gives_up_on_a_wait_and_recovers(lib):
    """A prefix of 60 tiles and rows for several units: the roles wait for one
    another microseconds at least."""
    c = Chain(lib, B=40, Q=9, Hq=8, Hkv=1, D=128, page=64, shared=7680,
              budget=7700)
    c.n_new = [np.full(40, 9)] * 2
    c.new_gpu = [_i32(n) for n in c.n_new]
    want = c.run()
    q = want[0]["q"]
    kv = torch.full_like(c.len, c.shared + 9)
    out, lse = torch.empty_like(q), torch.empty_like(want[1]["lse"])

    def call():
        c.lib.dflash_shared_attn(q, *c.pool, c.table, kv, None, c.shared, 0.1,
                                 out, lse, c.ws)
    call()
    lib.dflash_check()
    good, good_lse = out.clone(), lse.clone()
    c.ws.fill_(0xFF)
    _limited(lib, call)
    call()
    lib.dflash_check()
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_mass_gives_up_on_a_wait_and_recovers(lib):
    """512 rows and 63 tiles for each of 152 sequences or more: a CTA goes
    through 48 tiles four times, and the third time's queries wait for a buffer
    until the first is done, 48 tiles of a microsecond and more.  (Two sequences
    only: three tiles a CTA, none waits that long.)"""
    rng = np.random.default_rng(13)
    B, n = 160, 8000
    cache = _mass_args(rng, "bf16", 8, 1, 128, 64, 1, True, [n], None)[0]
    cache.table = np.repeat(cache.table, B, 0)
    q = torch.randn(B, 64, 8, 128, device="cuda").bfloat16()
    lse = torch.full((B, 64, 8), 60.0, device="cuda")
    (kc, _, ks, _), table = cache.cuda()
    mass = torch.zeros(B, 1, n, device="cuda")
    kv, fresh = _i32([n] * B), _i32([0] * B)

    def call():
        lib.dflash_attn_mass(q, kc, ks, table, kv, None, lse, fresh, 0,
                             0.05, 1.0, mass)
    call()
    lib.dflash_check()
    good = mass.clone()
    _limited(lib, call)
    call()
    lib.dflash_check()
    assert torch.equal(mass, good)


# --------------------------------------------------------------------------
def _prompt(n, V):
    g = torch.Generator().manual_seed(1)
    return torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()


def test_example_without_pressure_is_greedy_decoding(lib):
    """Every emitted token is the target's own choice and its log probability
    the target's, both recomputed over a cache without shared pages.  A logit is
    rounded to bf16 on either side, as is the one it is compared with: four
    times 2^-8 of the largest, and 0.1 for the attention's outputs (bf16) and
    the scales of pages that rejected tokens were in."""
    import shared_prompt as ex
    B, K, P = 4, 4, 48
    target = ex.SharedTarget(B, K, shared=P, budget=300, recent=8)
    prompt = _prompt(P, target.V)
    assert target.prompt_logits(prompt).isfinite().all()
    anchor = torch.tensor([3, 70, 200, 411], dtype=torch.int32, device="cuda")
    tokens, length, said = ex.generate(target, prompt, anchor, 8,
                                       ex.Filters(T=0.0))
    assert torch.equal(target.slots, P + length - 1)
    alone = ex.ToyTarget(B, K)
    where = torch.full((B,), P, dtype=torch.int32, device="cuda")
    alone.logits(prompt.repeat(B, 1), torch.zeros_like(where), where)
    n = int(length.max())
    l = alone.logits(tokens[:, :n].clamp(min=0).contiguous(), where)
    lp = torch.log_softmax(l, -1)
    for b in range(B):
        m = int(length[b])
        tol = 4 * 2.0 ** -8 * float(l[b, :m].abs().max()) + 0.1
        took = l[b, torch.arange(m - 1), tokens[b, 1:m].long()]
        assert (took >= l[b, :m - 1].max(-1).values - tol).all()
        mine = torch.cat([p[b, :int(k[b]) + 1] for k, p, *_ in said])
        theirs = lp[b, torch.arange(m - 1), tokens[b, 1:m].long()]
        assert (mine - theirs).abs().max() < tol
        assert all((r[b, :int(k[b]) + 1] == 0).all() and
                   (r[b, int(k[b]) + 1:] == -1).all() for k, _, r, *_ in said)
    lib.dflash_check()


def test_example_under_pressure_keeps_its_budget(lib):
    import shared_prompt as ex
    target = ex.SharedTarget(4, 4, shared=32, budget=56, recent=8)
    prompt = _prompt(32, target.V)
    anchor = ex.first_tokens(target, prompt, ex.Filters(T=1.0))
    at = target.table[0, :2].long()
    before = [p[at].clone() for p in target.pool]
    tokens, length, _ = ex.generate(target, prompt, anchor, 20,
                                    ex.Filters(T=1.0, top_k=20))
    assert (target.slots <= 56).all() and (length > 24).all()
    assert (target.slots == (32 + length - 1).clamp(max=56)).all()
    for p, was in zip(target.pool, before):
        assert torch.equal(p[at], was)
    for b in range(4):
        n = int(target.slots[b])
        m = target.mass[b, :, 32:n]
        assert m.isfinite().all() and (m >= 0).all() and (m > 0).any()
        t = tokens[b, :int(length[b])]
        assert ((t >= 0) & (t < target.V)).all()
    lib.dflash_check()


def test_example_runs(lib, capsys):
    import shared_prompt as ex
    ex.main()
    assert capsys.readouterr().out.count("nats a token") == 2
