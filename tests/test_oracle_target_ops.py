"""Pins of the target-side oracle (append, attention, sampling) and the
refusals of the three entry points: no GPU needed."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import target_ops as to


def test_block_scale_is_the_least_power_of_two():
    assert to.block_scale(448.0) == 1.0
    assert to.block_scale(np.nextafter(np.float32(448), np.float32(1e9))) == 2
    assert to.block_scale(3.5) == 2.0 ** -7
    assert to.block_scale(0.0) == 2.0 ** -64
    assert to.block_scale(1e-30) == 2.0 ** -64
    for a in np.exp2(np.random.default_rng(0).uniform(-50, 100, 200)):
        s = float(to.block_scale(a))
        assert a <= 448 * s and (a > 224 * s)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(inter):
    rng = np.random.default_rng(1)
    D, n = 16, 40
    ang = np.arange(n)[:, None] * 10.0 ** (-np.arange(D // 2) / 4)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    a, b = rng.standard_normal((2, D)).astype(np.float32)
    assert np.array_equal(to.rotate(a, 0, cos, sin, inter), a)

    def dot(i, j):
        return float(to.rotate(a, i, cos, sin, inter).astype(np.float64) @
                     to.rotate(b, j, cos, sin, inter))
    assert abs(dot(7, 3) - dot(29, 25)) < 1e-5   # depends on i - j only
    assert abs(np.linalg.norm(to.rotate(a, 33, cos, sin, inter)) -
               np.linalg.norm(a)) < 1e-5


def test_append_requantises_only_what_grew():
    page, D = 16, 16
    kc = np.zeros((2, 1, page, D), np.uint8)
    ks = np.zeros((2, 1), np.float32)
    vc, vs = kc.copy(), ks.copy()
    x = np.ones((1, 3, 1, D), np.float32)
    to.kv_append(None, x, x, None, None, [0], [3], np.array([[1, 0]]), page,
                 kc, vc, ks, vs)
    assert ks[1, 0] == 2.0 ** -8 and np.all(kc[1, 0, :3] == 0x78)  # 256
    big = 100 * x
    to.kv_append(None, big, x, None, None, [3], [1], np.array([[1, 0]]),
                 page, kc, vc, ks, vs)
    assert ks[1, 0] == 0.25 and vs[1, 0] == 2.0 ** -8
    assert np.all(oracle.e4m3_decode(kc[1, 0, :3]) * 0.25 == 1.0)  # exact
    assert np.all(vc[1, 0, :4] == 0x78)
    assert ks[0, 0] == 0                       # the other page is untouched


def test_attention_of_equal_keys_is_the_mean():
    page, D = 16, 16
    kc = np.zeros((3, 1, page, D), np.uint8)
    vc = oracle.e4m3_encode(np.random.default_rng(2).standard_normal(
        kc.shape).astype(np.float32))
    one = np.ones((3, 1), np.float32)
    q = np.ones((1, 2, 1, D))
    out, lse, _, _ = to.paged_attn(q, kc, vc, one, one, np.array([[2, 0]]),
                                   [20], [2], 0.3)
    v = np.concatenate([oracle.e4m3_decode(vc[2, 0]),
                        oracle.e4m3_decode(vc[0, 0])])
    np.testing.assert_allclose(out[0, 0, 0], v[:19].mean(0))
    np.testing.assert_allclose(out[0, 1, 0], v[:20].mean(0))
    np.testing.assert_allclose(lse[0, :, 0], np.log([19, 20]))


def test_sample_filters_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.1, 0.25, 0.15]))
    t, kept, _, _ = to.sample_row(l, 1.0, k=3, u=0.0)
    assert kept.tolist() == [False, True, False, True, True] and t == 1
    t, kept, _, _ = to.sample_row(l, 1.0, p=0.5, u=0.999)
    assert kept.tolist() == [False, True, False, True, False] and t == 3
    _, kept, _, _ = to.sample_row(l, 1.0, m=0.3, u=0.5)
    assert kept.tolist() == [False, True, False, True, True]
    _, kept, _, _ = to.sample_row(l, 1.0, k=4, u=0.5)
    assert kept.tolist() == [True, True, False, True, True]  # ties: lower id
    t, kept, _, _ = to.sample_row(l, 0.0)
    assert t == 1 and kept.sum() == 1
    assert to.sample_row(np.full(4, -np.inf), 1.0)[0] == -1


def test_sampled_frequencies_follow_the_filtered_distribution():
    rng = np.random.default_rng(3)
    l = rng.standard_normal(12) * 1.5
    u = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([to.sample_row(l, 0.8, k=6, u=x)[0] for x in u],
                      minlength=12) / u.size
    p = np.exp(l / 0.8)
    p[np.argsort(-l)[6:]] = 0
    np.testing.assert_allclose(got, p / p.sum(), atol=2e-4)


# --------------------------------------------------------------------------
@pytest.fixture(scope="module")
def so():
    from block_drafter_verify_gb300 import build
    import block_drafter_verify_gb300 as pkg
    return pkg.load(build.build()) or pkg.load()


def _refused(so, name, names, ok, bad):
    f = getattr(so, name)
    for change in bad:
        a = dict(zip(names, ok))
        assert set(change) <= set(names), change
        a.update(change)
        assert f(*[a[n] for n in names]) == 1, (name, change)


def test_append_refuses_on_the_host(so):
    """Each argument error is refused before the library looks for a
    device."""
    p = ctypes.c_void_p(0x100000)
    odd = ctypes.c_void_p(0x100002)
    names = ["q", "k", "v", "ld_q", "ld_k", "ld_v", "cos", "sin", "pos",
             "n_new", "table", "B", "Q", "Hq", "Hkv", "D", "rot", "inter",
             "max_pos", "page", "num_pages", "max_pages", "dt", "q_out",
             "kc", "vc", "ks", "vs", "kv_len", "stream"]
    other = ctypes.c_void_p(0x200000)
    ok = [p, p, p, 256, 128, 128, p, p, p, None, p, 2, 3, 4, 2, 64, 64, 0,
          100, 16, 8, 4, 0, p, p, p, p, p, other, None]
    _refused(so, "dflash_kv_append", names, ok, [
        {"k": None}, {"v": None}, {"pos": None}, {"table": None},
        {"kc": None}, {"vs": None}, {"kv_len": None}, {"q_out": None},
        {"cos": None}, {"B": 0}, {"Q": 0}, {"Hkv": 3}, {"D": 72},
        {"D": 272}, {"rot": 4}, {"rot": 72}, {"page": 48}, {"page": 8},
        {"num_pages": 0}, {"max_pages": 0}, {"dt": 2}, {"ld_k": 64},
        {"ld_q": 255}, {"ld_v": 130}, {"k": odd}, {"q": odd}, {"kc": odd},
        {"max_pos": 0}, {"kv_len": p, "pos": p}])


def test_attention_refuses_on_the_host(so):
    p = ctypes.c_void_p(0x100000)
    odd = ctypes.c_void_p(0x100008)
    names = ["q", "kc", "vc", "ks", "vs", "table", "kv_len", "q_len", "B",
             "Q", "Hq", "Hkv", "D", "page", "num_pages", "max_pages",
             "causal", "scale", "dt", "out", "lse", "ws", "ws_bytes",
             "stream"]
    size = so.dflash_paged_attn_workspace_bytes(2, 3, 4, 2, 64)
    assert size > 0 and size % 256 == 0
    ok = [p, p, p, p, p, p, p, None, 2, 3, 4, 2, 64, 16, 8, 4, 1, 0.125, 0,
          p, None, p, size, None]
    _refused(so, "dflash_paged_attn", names, ok, [
        {"q": None}, {"kc": None}, {"ks": None}, {"table": None},
        {"kv_len": None}, {"out": None}, {"ws": None}, {"B": 0}, {"Q": 0},
        {"Hq": 5}, {"Hq": 130}, {"D": 40}, {"D": 512}, {"page": 24},
        {"scale": float("nan")}, {"scale": float("inf")}, {"dt": 7},
        {"ws": odd}, {"q": odd}, {"vc": odd}, {"ws_bytes": size - 1}])
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 3, 2, 64),
                (1, 1, 65, 1, 64), (1, 1, 1, 1, 8)):
        assert so.dflash_paged_attn_workspace_bytes(*bad) == 0


def test_sample_refuses_on_the_host(so):
    p = ctypes.c_void_p(0x100000)
    names = ["logits", "ld", "dt", "T", "k", "p", "m", "u", "R", "V",
             "token", "n", "filtered", "ws", "ws_bytes", "stream"]
    size = so.dflash_sample_workspace_bytes(4, 100)
    ok = [p, 100, 1, p, None, None, None, p, 4, 100, p, None, None, p, size,
          None]
    _refused(so, "dflash_sample", names, ok, [
        {"logits": None}, {"T": None}, {"u": None}, {"token": None},
        {"ws": None}, {"R": 0}, {"V": 0}, {"ld": 99}, {"dt": 3},
        {"ws": ctypes.c_void_p(0x100010)}, {"ws_bytes": size - 1}])
    assert so.dflash_sample_workspace_bytes(0, 100) == 0
    assert so.dflash_sample_workspace_bytes(4, 0) == 0
    assert so.dflash_sample_workspace_bytes(4, (1 << 20) - 1) > 0
    assert so.dflash_sample_workspace_bytes(4, 1 << 20) == 0


def test_binding_refuses_wrong_tensors():
    """The binding's own checks: dtypes, devices, shapes."""
    import torch

    import block_drafter_verify_gb300 as dv
    t = torch.zeros(2, 4)
    r = torch.zeros(2)
    with pytest.raises(ValueError):
        dv.dflash_sample(t, r, None, None, None, r, r.int(), None, None, r)
    with pytest.raises(ValueError):
        dv.dflash_sample(t.half(), r, None, None, None, r, r.int(), None,
                         None, r)
    c = torch.zeros(3, 1, 16, 16, dtype=torch.uint8)
    s = torch.zeros(3, 1)
    with pytest.raises(ValueError):
        dv.dflash_paged_attn(torch.zeros(1, 1, 1, 32), c, c, s, s,
                             torch.zeros(1, 1).int(), r[:1].int(), None, 1.0,
                             torch.zeros(1, 1, 1, 32), None, r)
    with pytest.raises(ValueError):
        dv.dflash_kv_append(None, torch.zeros(3, 1, 16),
                            torch.zeros(3, 1, 16), None, None, r.int(), None,
                            torch.zeros(2, 1).int(), c, c, s, s, None,
                            r.int())
