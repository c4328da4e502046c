"""The target's calls at the ends of their stated ranges.  Tolerances are those
of test_gpu_target_ops; where a test has its own, its docstring derives it.
"""
import numpy as np
import pytest
import torch

from test_gpu_target_ops import _check_sample, _run_sample

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
