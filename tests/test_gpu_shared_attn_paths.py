"""dflash_shared_attn's tensor-core kernels at sizes that are theirs with a
margin of two on any SM count, shown by the kernels' names: row tiles that
sequences share, streams side by side, graphs with one workspace, pools beyond
32 bits.  Oracle and tolerances as in test_gpu_serving_ops."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_gpu_serving_cycle import Chain, _same, _same_cache
from test_gpu_serving_ops import SharedCache, _i32
from test_gpu_shared_attn_sizes import _check, _q

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _tokens(B, Q, Hq, Hkv, page):
    """Shared tokens with which twice as many tiles would be read again as the
    kernel that reads them for each sequence takes: more than 448 an SM, counted
    with the rows (a multiple of 16, 96 at most) of each unit."""
    rows = Q * Hq // Hkv
    tiles = -(-rows // 96)
    N = -(-(-(-rows // tiles)) // 16) * 16
    again = -(-2 * 448 * _sms() // (B * Hkv * tiles * N))
    return -(-again * 128 // page) * page


class _KernelNode(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS_v2."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _kernels(call):
    """Names of the kernels that call() launches, from a graph of it."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu = ctypes.CDLL("libcuda.so.1")

    def run(name, *args):
        status = getattr(cu, name)(*args)
        assert status == 0, (name, status)
    handle, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    run("cuGraphGetNodes", handle, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    run("cuGraphGetNodes", handle, nodes, ctypes.byref(n))
    names = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        run("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:                   # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        k, name = _KernelNode(), ctypes.c_char_p()
        run("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node),
            ctypes.byref(k))
        if k.func:
            run("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(k.func))
        else:
            run("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(k.kern))
        names.append(name.value.decode())
    return names


def _takes(names, kind):
    """kind: together, apart (own tokens by the kernel for few rows)."""
    def has(part):
        return any(part in n for n in names)
    assert has("shared_attn_tc_kernel"), names
    assert has("shared_attn_tc_join_kernel"), names
    assert has("paged_attn_tc_kernel") == (kind == "apart"), names


def _chain(lib, kind, seed=0, **kw):
    if kind == "together":
        size = dict(B=3, Q=40, Hq=32, Hkv=2, D=64, page=32)
    else:
        size = dict(B=_sms(), Q=3, Hq=8, Hkv=4, D=64, page=16)
    size.update(kw)
    shared = _tokens(*(size[k] for k in ("B", "Q", "Hq", "Hkv", "page")))
    c = Chain(lib, seed=seed, shared=shared, budget=shared + 50, **size)
    rng = np.random.default_rng(seed)
    c.n_new = [rng.integers(0, c.Q + 1, c.B) for _ in range(2)]
    c.new_gpu = [_i32(n) for n in c.n_new]
    return c


KINDS = ["together", "apart"]


@pytest.mark.parametrize("kind", KINDS)
def test_sizes_of_the_chains_take_the_kernels_that_they_are_for(lib, kind):
    c = _chain(lib, kind)
    c.run()
    _takes(_kernels(c.run), kind)
    lib.dflash_check()


# kind, B, Q, Hq, Hkv, D, page, longest own
@pytest.mark.parametrize("kind,B,Q,Hq,Hkv,D,page,own", [
    ("together", 5, 9, 8, 1, 128, 64, 200),    # 72 rows each, units of 256
    ("together", 40, 3, 4, 1, 64, 64, 300),    # 12 rows each
    ("together", 3, 130, 4, 2, 80, 16, 70),    # 260 rows each: units of 256
    ("apart", 2, 2, 8, 2, 96, 32, 90),         # (times the SM count)
])
def test_row_tiles_that_sequences_share(lib, kind, B, Q, Hq, Hkv, D, page,
                                        own):
    rng = np.random.default_rng(B + Q)
    if kind == "apart":
        B *= _sms()
    shared = _tokens(B, Q, Hq, Hkv, page)
    kv = [shared + Q + int(rng.integers(0, own + 1)) for _ in range(B)]
    ql = [int(rng.integers(0, Q + 1)) for _ in range(B)]
    kv[0], ql[0], kv[1], ql[1] = shared + Q + own, Q, shared + 1, Q
    cache = SharedCache(shared, kv, page, Hkv, D, rng)
    q = _q(rng, B, Q, Hq, D)
    _check(lib, cache, q, kv, ql, shared, True, 1 / math.sqrt(D))
    pool, table = cache.cuda()
    n, out = _i32(kv), torch.empty_like(q)
    ws = torch.empty(lib.dflash_shared_attn_workspace_bytes(
        B, Q, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    _takes(_kernels(lambda: lib.dflash_shared_attn(
        q, *pool, table, n, None, shared, 1.0, out, None, ws)), kind)


def test_kernels_on_streams_side_by_side(lib):
    chains = [_chain(lib, KINDS[s % 2], seed=s) for s in range(4)]
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


def test_graphs_of_both_kinds_share_a_workspace(lib):
    """Replayed by turns: what one leaves is the other's to overwrite."""
    chains = [_chain(lib, kind, seed=s) for s, kind in enumerate(KINDS * 2)]
    ws = max((c.ws for c in chains), key=torch.Tensor.numel)
    ws2 = max((c.ws2 for c in chains), key=torch.Tensor.numel)
    want, graphs = [], []
    for c in chains:
        c.ws, c.ws2 = ws, ws2
        want.append((c.run(), c.cache()))
    for c in chains:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            said = c.run()
        graphs.append((g, said))
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    lib.dflash_check()
    for c, (_, said), (w, cache) in zip(chains, graphs, want):
        _same(w, said)
        _same_cache(cache, c.cache())


@pytest.mark.parametrize("kind", KINDS)
def test_kernels_in_pools_beyond_32_bits(lib, kind):
    """Pages far apart in pools of 5 GB each: the same bits as in small ones."""
    a = _chain(lib, kind)
    stride = -(-(5 << 30) // a.pool[0].numel())
    assert a.pages.size * stride * a.Hkv * a.page < 1 << 31
    b = _chain(lib, kind, stride=stride)
    assert b.pool[0].numel() > 1 << 32
    at = torch.as_tensor(b.pages.astype(np.int64), device="cuda")
    for p in b.pool:
        p[at] = 0
    x, y = a.run(), b.run()
    torch.cuda.synchronize()
    lib.dflash_check()
    _same(x, y)
    _same_cache(a.cache(), b.cache())
