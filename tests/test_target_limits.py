"""Sizes at which the target's calls start to refuse: no GPU needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def so():
    from block_drafter_verify_gb300 import build
    import block_drafter_verify_gb300 as pkg
    return pkg.load(build.build()) or pkg.load()


@pytest.mark.parametrize("B,Q,Hq,Hkv", [
    (1 << 24, 1, 128, 2), (1 << 12, 1 << 12, 128, 128), (1, 1 << 19, 4096, 64)])
def test_attention_refuses_rows_beyond_32_bits(so, B, Q, Hq, Hkv):
    """B * Q * Hq rows of q and out are counted in 32 bits: 2^31 and more are
    refused, one token less is not."""
    D = 16
    size = so.dflash_paged_attn_workspace_bytes
    assert size(B, Q, Hq, Hkv, D) == 0
    less = (B - 1, Q) if Q == 1 else (B, Q - 1)
    ok = size(*less, Hq, Hkv, D)
    assert ok > 0
    p = ctypes.c_void_p(0x100000)

    def call(B, Q):
        return so.dflash_paged_attn(p, p, p, p, p, p, p, None, B, Q, Hq, Hkv,
                                    D, 16, 8, 4, 1, 0.125, 0, p, None, p,
                                    1 << 40, None)
    assert call(B, Q) == 1                     # DFLASH_ERR_INVALID_ARG
