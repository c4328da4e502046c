"""dflash_shared_attn over the sizes at which its work is split differently: a
prefix short enough to be read for each sequence, prefix and own tokens
together, and own tokens in a launch of their own.  Oracle and tolerances as
in test_gpu_serving_ops."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_ops as so
from oracle import target_ops as to
from test_gpu_serving_ops import SharedCache, _i32, _share, _status
from test_gpu_target_ops import DT, _check_attn

pytestmark = pytest.mark.gpu


def _check(lib, cache, q, kv, ql, shared, causal, scale, want_lse=True,
           table=None, codes=None, scales=None, status=None):
    out, lse = _share(lib, "bf16", cache, q, kv, ql, shared, causal, scale,
                      want_lse)
    if status is None:
        lib.dflash_check()
    else:
        _status(lib, status)
    B, Q, _, D = q.shape
    nq = [Q] * B if ql is None else ql
    if table is None:
        table = so.shared_table(cache.table, shared, cache.page)
    ref = to.paged_attn(q.float().cpu().numpy().astype(np.float64),
                        *(codes or cache.codes), *(scales or cache.scale),
                        table, kv, nq, scale, causal)
    _check_attn("bf16", D, max(kv), out, lse, ref)


def _q(rng, B, Q, Hq, D, up=2.0):
    return torch.tensor(rng.standard_normal((B, Q, Hq, D)) * up,
                        dtype=torch.float32).to(DT["bf16"]).cuda()


# B, Q, Hq, Hkv, D, page, shared, longest own, causal
TOGETHER = [                       # few units, much to read again
    (6, 1, 8, 2, 16, 128, 46080, 300, True),
    (3, 9, 8, 1, 64, 64, 36480, 200, True),
    (3, 9, 8, 1, 64, 64, 36480, 200, False),
    (2, 40, 32, 2, 80, 32, 3392, 500, True),
    (3, 130, 4, 2, 128, 16, 5136, 700, True),
    (30, 9, 8, 2, 112, 64, 3328, 100, True),
    (2, 300, 16, 1, 64, 128, 4096, 40, True),
]
APART = [                          # many units of few rows
    (160, 1, 8, 2, 64, 64, 1792, 300, True),
    (160, 4, 8, 2, 80, 32, 1824, 100, True),
    (80, 7, 16, 4, 32, 16, 3600, 1500, True),
    (320, 1, 32, 1, 128, 128, 1664, 40, False),
    (90, 2, 24, 4, 96, 64, 2304, 500, False),
]


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,page,shared,own,causal",
                         TOGETHER + APART)
def test_sizes_match_the_oracle(lib, B, Q, Hq, Hkv, D, page, shared, own,
                                causal):
    rng = np.random.default_rng(B + Q + D)
    kv = [shared + int(rng.integers(0, own + 1)) for _ in range(B)]
    ql = [int(rng.integers(0, Q + 1)) for _ in range(B)]
    kv[0], ql[0] = shared + own, Q
    kv[1], ql[1] = shared + 1, Q          # queries that see the prefix only
    if B > 4:
        kv[2], ql[2] = 0, 0
        kv[3] = shared // 2 + 5           # ends inside the prefix
        ql[4] = 0
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    _check(lib, cache, _q(rng, B, Q, Hq, D), kv, ql, shared, causal,
           1 / math.sqrt(D), want_lse=B % 2 == 0)


FAR = [(2, 40, 32, 2, 64, 32, 3392), (160, 1, 8, 2, 64, 32, 1792)]


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,page,shared", FAR)
def test_scales_far_apart(lib, B, Q, Hq, Hkv, D, page, shared):
    """Value scales from 2^-64 to 2^60, queries of very different sizes; a
    negative and a zero factor of the scores."""
    rng = np.random.default_rng(B)
    kv = [shared + Q + int(rng.integers(0, 90)) for _ in range(B)]
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    N = cache.scale[1].shape[0]
    cache.scale[1][:] = np.exp2(rng.integers(-64, 61, (N, Hkv)))
    cache.scale[0][:] = np.exp2(rng.integers(-64, -59, (N, Hkv)))
    q = _q(rng, B, Q, Hq, D, 1.0)
    q[0, 0] *= 2.0 ** 60
    q[1] *= 2.0 ** 54
    for scale in (D ** -0.5, -0.125, 0.0):
        _check(lib, cache, q, kv, None, shared, True, scale)


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,page,shared", FAR)
@pytest.mark.parametrize("grows", [True, False])
def test_large_scores(lib, B, Q, Hq, Hkv, D, page, shared, grows):
    """Scores of thousands of either sign, their sizes growing or falling
    along the prefix and again along a sequence's own tokens."""
    rng = np.random.default_rng(B + grows)
    kv = [shared + Q + int(rng.integers(0, 200)) for _ in range(B)]
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    table = so.shared_table(cache.table, shared, page)
    step = np.exp2(np.linspace(-6, 2, table.shape[1]).round())
    if not grows:
        step = step[::-1]
    for b in range(B):
        for p in range(-(-kv[b] // page)):
            cache.scale[0][table[b, p]] = step[p]
    _check(lib, cache, _q(rng, B, Q, Hq, D, 1.0), kv, None, shared, True,
           D ** -0.5)


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,page,shared", FAR)
def test_bad_pages_count_as_zeros(lib, B, Q, Hq, Hkv, D, page, shared):
    """A bad page of the prefix, one of a sequence's own, and lengths out of
    range; all flagged."""
    rng = np.random.default_rng(B)
    kv = [shared + Q + 40] * B
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    q = _q(rng, B, Q, Hq, D)
    good = cache.table.copy()
    for row, col in ((0, 1), (1, shared // page)):
        cache.table = good.copy()
        cache.table[row, col] = 10 ** 6
        want = so.shared_table(cache.table, shared, page)
        codes = [np.concatenate([c, np.zeros_like(c[:1])])
                 for c in cache.codes]
        scales = [np.concatenate([s, np.ones_like(s[:1])])
                  for s in cache.scale]
        want[want == 10 ** 6] = len(codes[0]) - 1
        _check(lib, cache, q, kv, None, shared, True, 0.1, table=want,
               codes=codes, scales=scales, status=6)
    cache.table = good
    most = good.shape[1] * page
    _share(lib, "bf16", cache, q, [most + 1, -3] + kv[2:], None, shared, True,
           0.1)
    _status(lib, 6)


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,page,shared", FAR)
def test_calls_repeat_bit_for_bit(lib, B, Q, Hq, Hkv, D, page, shared):
    """Whatever the workspace held, and in a graph."""
    rng = np.random.default_rng(7)
    kv = [shared + Q + int(rng.integers(0, 300)) for _ in range(B)]
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    (kc, vc, ks, vs), table = cache.cuda()
    q, n = _q(rng, B, Q, Hq, D), _i32(kv)
    out = torch.empty_like(q)
    lse = torch.empty(B, Q, Hq, device="cuda")
    ws = torch.empty(lib.dflash_shared_attn_workspace_bytes(
        B, Q, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def call():
        lib.dflash_shared_attn(q, kc, vc, ks, vs, table, n, None, shared, 0.1,
                               out, lse, ws)
    graph = torch.cuda.CUDAGraph()
    got = []
    for fill in (0, 0xFF, 0x55):
        ws.fill_(fill)
        call()
        got.append((out.clone(), lse.clone()))
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got.append((out, lse))
    lib.dflash_check()
    for o, z in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(z, got[0][1])
