"""Pins of the oracle of the operators around a shared prompt and a bounded
cache, and the refusals of their entry points: no GPU needed."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import serving_ops as so
from oracle import target_ops as to


def _cache(N, Hkv, page, D, rng):
    codes = [oracle.e4m3_encode((100 * rng.standard_normal(
        (N, Hkv, page, D))).astype(np.float32)) for _ in range(2)]
    scale = [np.exp2(rng.integers(-8, -4, (N, Hkv))).astype(np.float32)
             for _ in range(2)]
    return codes, scale


def test_axes_that_agree_with_the_slots_are_an_append():
    rng = np.random.default_rng(0)
    B, Q, Hq, Hkv, D, page = 2, 3, 4, 2, 16, 16
    ang = np.arange(64)[:, None] * 10.0 ** (-np.arange(D // 2) / 4)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    q = rng.standard_normal((B, Q, Hq, D)).astype(np.float32)
    k, v = rng.standard_normal((2, B, Q, Hkv, D)).astype(np.float32)
    pos, table = np.array([4, 15]), np.array([[0, 1], [2, 3]])
    got = []
    for axes in (False, True):
        codes, scale = _cache(4, Hkv, page, D, np.random.default_rng(1))
        rest = (pos, [Q] * B, table, page, *codes, *scale)
        if axes:
            at = np.stack([(pos[:, None] + np.arange(Q)).ravel()] * 2)
            out = so.kv_append_axes(q, k, v, cos, sin, at,
                                    np.arange(D // 2) % 2, *rest)
        else:
            out = to.kv_append(q, k, v, cos, sin, *rest)
        got.append([*out, *codes, *scale])
    for a, b in zip(*got):
        assert np.array_equal(a, b)


def test_one_axis_turns_only_its_angles():
    D = 16
    ang = np.arange(9)[:, None] * 10.0 ** (-np.arange(D // 2) / 4)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    q = np.ones((1, 1, 1, D), np.float32)
    codes, scale = _cache(1, 1, 16, D, np.random.default_rng(2))
    of = np.array([0, 0, 0, 1, 1, 0, 1, 1])
    out, _ = so.kv_append_axes(q, q, q, cos, sin, np.array([[0], [8]]), of,
                               [0], [1], np.array([[0]]), 16, *codes, *scale)
    turned = out[0, 0, 0] != 1.0
    assert np.array_equal(turned, np.tile(of == 1, 2))


def test_weight_gathered_is_the_softmax():
    """With decay 0 the heads' and queries' weights add up to the queries that
    see a token, and weights times values are the attention's output."""
    rng = np.random.default_rng(3)
    B, Q, Hq, Hkv, D, page = 2, 3, 4, 2, 16, 16
    codes, scale = _cache(5, Hkv, page, D, rng)
    table, kv, nq = np.array([[0, 1, 2], [3, 4, -1]]), [40, 20], [3, 0]
    q = rng.standard_normal((B, Q, Hq, D))
    out, lse, _, _ = to.paged_attn(q, *codes, *scale, table, kv, nq, 0.25)
    old = rng.random((B, Hkv, 48))
    m, _ = so.attn_mass(q, codes[0], scale[0], table, kv, nq, lse, None, 0,
                        0.25, 0.0, old)
    np.testing.assert_allclose(m[0, :, :40].sum(1), 3 * 2)
    assert np.all(m[1, :, :20] == 0) and np.array_equal(m[1, :, 20:],
                                                        old[1, :, 20:])
    one, _ = so.attn_mass(q[:1, 2:, :1], codes[0][:, :1], scale[0][:, :1],
                          table, [40], [1], lse[:1, 2:, :1], None, 0, 0.25,
                          0.0, old[:1, :1])
    v = to.cached(codes[1], scale[1], table[0], 40, 0, page)
    np.testing.assert_allclose(one[0, 0, :40] @ v, out[0, 2, 0])


def test_fresh_and_decay_and_first():
    codes, scale = _cache(1, 1, 16, 16, np.random.default_rng(4))
    m, _ = so.attn_mass(np.zeros((1, 1, 1, 16)), codes[0], scale[0],
                        np.array([[0]]), [4], [1], np.log([[[4.0]]]), [3], 1,
                        1.0, 0.5, np.full((1, 1, 5), 8.0))
    assert m[0, 0].tolist() == [8.0, 4.25, 4.25, 0.25, 8.0]


def test_eviction_by_hand():
    mass = np.array([[[9, 1, 5, 5, np.nan, 2, 5, 0, 0]]], np.float32)
    codes, scale = _cache(1, 1, 16, 16, np.random.default_rng(5))
    before, s0 = codes[0].copy(), float(scale[0][0, 0])
    n, kept, moved = so.kv_evict(mass, *codes, *scale, np.array([[0]]), [9],
                                 5, 1, 2)
    assert n.tolist() == [5] and kept[0, 0].tolist() == [0, 2, 3, 7, 8]
    assert moved[0][0].tolist() == [9, 5, 5, 0, 0]
    s = float(scale[0][0, 0])
    np.testing.assert_array_equal(
        oracle.e4m3_decode(codes[0][0, 0, :5]) * s,
        oracle.e4m3_decode(before[0, 0, kept[0, 0]]) * s0)
    assert np.array_equal(codes[0][0, 0, 5:], before[0, 0, 5:])
    # not above its budget: nothing moves
    n, kept, _ = so.kv_evict(mass, *codes, *scale, np.array([[0]]), [4], 5, 1,
                             2)
    assert n.tolist() == [4] and kept[0, 0].tolist() == [0, 1, 2, 3, -1]


def test_log_probabilities_by_hand():
    p = np.array([0.1, 0.4, 0.1, 0.25, 0.15])
    l = np.log(p).astype(np.float32)
    lp, rank, z, ent, top, ids = so.logprobs_row(l, 1.0, 2, 3)
    assert abs(lp - np.log(0.1)) < 1e-6 and rank == 4 and abs(z) < 1e-6
    assert abs(ent + (p * np.log(p)).sum()) < 1e-6
    assert ids.tolist() == [1, 3, 4]
    np.testing.assert_allclose(np.exp(top), [0.4, 0.25, 0.15], rtol=1e-6)
    assert so.logprobs_row(l, 1.0, 0, 0)[1] == 3       # ties: the lower id
    assert so.logprobs_row(l, 0.5, -1, 1)[:2] == (0.0, -1)
    _, _, z, ent, top, ids = so.logprobs_row([-np.inf, 2.0], 1.0, -1, 2)
    assert z == 2 and ent == 0 and ids.tolist() == [1, -1]
    assert so.logprobs_row(np.full(3, -np.inf), 1.0, 1, 0)[2] == -np.inf


# --------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from block_drafter_verify_gb300 import build
    import block_drafter_verify_gb300 as pkg
    return pkg.load(build.build()) or pkg.load()


P = ctypes.c_void_p(0x100000)
P2 = ctypes.c_void_p(0x200000)
ODD = ctypes.c_void_p(0x100002)
HALF = ctypes.c_void_p(0x100008)


def _refused(lib, name, ok, bad):
    """Each argument error is refused (DFLASH_ERR_INVALID_ARG) before the
    library looks for a device."""
    f = getattr(lib, name)
    for change in bad:
        assert set(change) <= set(ok), change
        assert f(*{**ok, **change}.values()) == 1, (name, change)


def test_append_axes_refuses_on_the_host(lib):
    ok = dict(q=P, k=P, v=P, ld_q=256, ld_k=128, ld_v=128, cos=P, sin=P,
              axis_pos=P, axis_of=P, axes=3, pos=P, n_new=None, table=P, B=2,
              Q=3, Hq=4, Hkv=2, D=64, rot=64, inter=0, max_pos=100, page=16,
              num_pages=8, max_pages=4, dt=0, q_out=P, kc=P, vc=P, ks=P, vs=P,
              kv_len=P2, stream=None)
    _refused(lib, "dflash_kv_append_axes", ok, [
        {"axis_pos": None}, {"axis_of": None}, {"axes": 0}, {"axes": 5},
        {"axis_of": ODD}, {"rot": 0}, {"rot": 4}, {"rot": 72}, {"cos": None},
        {"k": None}, {"q_out": None}, {"max_pos": 0}, {"page": 48},
        {"ld_v": 130}, {"dt": 2}, {"kv_len": P}])


def test_shared_attention_refuses_on_the_host(lib):
    size = lib.dflash_shared_attn_workspace_bytes(2, 3, 4, 2, 64)
    assert size > 0 and size % 256 == 0
    ok = dict(q=P, kc=P, vc=P, ks=P, vs=P, table=P, kv_len=P, q_len=None,
              shared=32, B=2, Q=3, Hq=4, Hkv=2, D=64, page=16, num_pages=8,
              max_pages=4, causal=1, scale=0.125, dt=0, out=P, lse=None, ws=P,
              ws_bytes=size, stream=None)
    _refused(lib, "dflash_shared_attn", ok, [
        {"q": None}, {"kc": None}, {"vc": None}, {"ks": None}, {"vs": None},
        {"table": None}, {"kv_len": None}, {"out": None}, {"ws": None},
        {"shared": -16}, {"shared": 24}, {"shared": 80}, {"B": 0}, {"Q": 0},
        {"Hkv": 3}, {"D": 72}, {"D": 272}, {"page": 8}, {"num_pages": 0},
        {"max_pages": 0}, {"dt": 2}, {"scale": float("nan")},
        {"scale": float("inf")}, {"q": HALF}, {"out": HALF}, {"kc": HALF},
        {"vc": HALF}, {"ws": HALF}, {"ws_bytes": size - 1}])
    for D in (64, 256):
        for bad in ((0, 1, 4, 2), (1, 0, 4, 2), (1, 1, 4, 3),
                    (1, 1, 130, 2), (1 << 24, 1, 128, 2)):
            assert lib.dflash_shared_attn_workspace_bytes(*bad, D) == 0


def test_mass_refuses_on_the_host(lib):
    ok = dict(q=P, kc=P, ks=P, table=P, kv_len=P, q_len=None, lse=P,
              fresh=None, first=0, B=2, Q=3, Hq=4, Hkv=2, D=64, page=16,
              num_pages=8, max_pages=4, causal=1, scale=0.125, decay=1.0,
              dt=0, mass=P, ld=64, stream=None)
    _refused(lib, "dflash_attn_mass", ok, [
        {"q": None}, {"kc": None}, {"ks": None}, {"table": None},
        {"kv_len": None}, {"lse": None}, {"mass": None}, {"first": -1},
        {"ld": 0}, {"B": 0}, {"Q": 0}, {"Hkv": 3}, {"Hq": 130}, {"D": 24},
        {"D": 288}, {"page": 20}, {"num_pages": 0}, {"max_pages": 0},
        {"dt": 2}, {"scale": float("inf")}, {"decay": float("nan")},
        {"q": HALF}, {"kc": HALF}])


def test_evict_refuses_on_the_host(lib):
    size = lib.dflash_kv_evict_workspace_bytes(2, 2, 16, 40)
    assert size > 0 and size % 256 == 0
    ok = dict(mass=P, ld=64, kc=P, vc=P, ks=P, vs=P, table=P, kv_len=P, B=2,
              Hkv=2, D=64, page=16, num_pages=8, max_pages=4, budget=40,
              sink=4, recent=8, mass_out=P2, ld_out=40, new_len=P2, kept=None,
              ws=P, ws_bytes=size, stream=None)
    _refused(lib, "dflash_kv_evict", ok, [
        {"mass": None}, {"kc": None}, {"vc": None}, {"ks": None},
        {"vs": None}, {"table": None}, {"kv_len": None}, {"new_len": None},
        {"ws": None}, {"new_len": P}, {"mass_out": P}, {"ld": 0},
        {"ld_out": 0}, {"ld_out": 39}, {"sink": -1}, {"recent": -1},
        {"sink": 33}, {"recent": 37}, {"sink": 2 ** 31 - 1}, {"budget": 0},
        {"B": 0}, {"Hkv": 0}, {"D": 40}, {"page": 17}, {"num_pages": 0},
        {"max_pages": 0}, {"kc": HALF}, {"vc": HALF}, {"ws": HALF},
        {"ws_bytes": size - 1}])
    for bad in ((0, 2, 16, 4), (2, 0, 16, 4), (2, 2, 24, 4), (2, 2, 16, 0),
                (2, 2, 16, (1 << 30) + 1), (1 << 20, 1 << 12, 16, 4)):
        assert lib.dflash_kv_evict_workspace_bytes(*bad) == 0


def test_logprobs_refuse_on_the_host(lib):
    ok = dict(logits=P, ld=100, dt=0, T=None, token=P, R=3, V=100, K=5,
              logprob=P, rank=P, lse=P, entropy=P, top=P, top_id=P,
              stream=None)
    _refused(lib, "dflash_logprobs", ok, [
        {"logits": None}, {"ld": 99}, {"dt": 2}, {"token": None}, {"R": 0},
        {"V": 0}, {"V": 2 ** 31 - 1, "ld": 2 ** 31}, {"K": -1}, {"K": 33},
        {"K": 0}, {"top": None}, {"top_id": None},
        {"logits": ctypes.c_void_p(0x100001)}, {"dt": 1, "logits": ODD},
        {"logprob": None, "token": None}])


def test_binding_refuses_shapes():
    """What the binding checks, on tensors of the CPU: a ValueError before any
    call."""
    import torch
    import block_drafter_verify_gb300 as dv
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = torch.zeros
    codes, scale, table = u8(4, 2, 16, 32), f32(4, 2), i32(3, 2)
    q, n, lse = f32(3, 1, 4, 32), i32(3), f32(3, 1, 4)
    pool = (codes, codes, scale, scale)
    for change in (dict(q=f32(3, 1, 4, 16)), dict(kv_len=i32(2)),
                   dict(out=f32(3, 4, 32)), dict(lse=f32(3, 1, 2)),
                   dict(q_len=i32(4)), dict(page_table=i32(2, 2)), {}):
        a = dict(q=q, k_codes=codes, v_codes=codes, k_scale=scale,
                 v_scale=scale, page_table=table, kv_len=n, q_len=None,
                 shared=16, scale=1.0, out=q, lse=lse, ws=u8(1 << 20))
        with pytest.raises(ValueError):
            dv.dflash_shared_attn(**{**a, **change})
    for change in (dict(mass=f32(3, 1, 32)), dict(mass=f32(6, 32)),
                   dict(lse=f32(3, 1, 3)), dict(fresh=i32(2)),
                   dict(k_scale=f32(4)), dict(kv_len=i32(1)), {}):
        a = dict(q=q, k_codes=codes, k_scale=scale, page_table=table,
                 kv_len=n, q_len=None, lse=lse, fresh=None, first=0,
                 scale=1.0, decay=1.0, mass=f32(3, 2, 32))
        with pytest.raises(ValueError):
            dv.dflash_attn_mass(**{**a, **change})
    for change in (dict(new_len=i32(2)), dict(kept=i32(3, 2, 7)),
                   dict(mass_out=f32(3, 32)), dict(kv_len=i32(4)), {}):
        a = dict(mass=f32(3, 2, 32), kv_len=n, budget=8, sink=1, recent=1,
                 mass_out=None, new_len=i32(3), kept=None, ws=u8(4096))
        a = {**a, **change}
        with pytest.raises(ValueError):
            dv.dflash_kv_evict(a["mass"], *pool, table, *list(a.values())[1:])
    for change in (dict(axis_pos=i32(2, 4)), dict(axis_of=u8(8)), {}):
        a = {**dict(axis_pos=i32(2, 3), axis_of=u8(16)), **change}
        kv = f32(3, 2, 32)
        with pytest.raises(ValueError):
            dv.dflash_kv_append_axes(
                None, kv, kv, f32(9, 16), f32(9, 16), a["axis_pos"],
                a["axis_of"], n, None, table, *pool, None, n)
    l = f32(3, 50)
    for change in (dict(token=i32(2)), dict(top=f32(3, 4)),
                   dict(top=f32(3, 4), top_id=i32(3, 5)),
                   dict(top=f32(2, 4), top_id=i32(2, 4)), {}):
        a = dict(logits=l, temperature=None, token=n, logprob=f32(3),
                 rank=None, lse=None, entropy=None, top=None, top_id=None)
        with pytest.raises(ValueError):
            dv.dflash_logprobs(**{**a, **change})


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The calls run on the current device; a tensor of another one would be
    read from it."""
    import torch
    from block_drafter_verify_gb300 import binding

    class Elsewhere:
        is_cuda = True

        def get_device(self):
            return 1
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError):
        binding._here(Elsewhere(), "q")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    binding._here(Elsewhere(), "q")
