"""The gated delta rule over prompts at the ends of fp32's range: small and large values, decays that hide them, factors that grow
(needs a B200).

Tolerances are those of test_gpu_gdn_scan.py.  Where tokens are looked at one by one, 4 of them: an output is one product of
the state with a query, in which errors of the state, spread evenly over its 128 columns, count more or less than on average;
of 128 columns four standard deviations do not happen.
"""

import numpy as np
import pytest
import torch

from oracle.prompts import gdn_scan as oracle_scan
from test_gpu_gdn_scan import BF, F32, SCALE, make, on_gpu, scan, tol
from synth import round_to_dtype

pytestmark = pytest.mark.gpu


def run(d, dtype, resume):
    g = on_gpu(d, dtype)
    y = scan(g, [0, len(d["v"])], resume=[resume])
    return y.double().cpu().numpy(), g["S"][0].double().cpu().numpy()


def near(got, want, bound):
    """Along the last axis: errors within the bound of the values' norm."""
    err, size = np.linalg.norm(got - want, axis=-1), np.linalg.norm(want, axis=-1)
    assert (err <= bound * size).all(), np.max(err / np.maximum(size, 1e-300))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e-20, 1e-25, 1e-4, 1e25, 1e30])
@pytest.mark.parametrize("alpha", [0.5, 0.78, 0.999])
def test_values_of_any_size(cuda_ok, dtype, size, alpha):
    """Values and a state of 1e-25 to 1e30 under decays of 2^-64, 2^-23 and 2^-0.1 a chunk: each token's output and the state
    are as exact as for values of 1.  Every row is scaled alike, so the oracle's values are those for values of 1."""
    d = make(71, dtype, 150, 2, 1, 64, 1)
    d["alpha"][:] = np.float32(alpha)
    d["v"] = round_to_dtype((d["v"] * size).astype(np.float32), "bf16" if dtype == BF else "f32")
    d["S"] = (d["S"] * size).astype(np.float32)
    S, y = oracle_scan(**d, offsets=[0, 150], resume=[1], q_scale=SCALE)
    y_got, S_got = run(d, dtype, 1)
    near(y_got, y, 4 * tol(150))
    near(S_got.reshape(2, -1), S[0].reshape(2, -1), tol(150))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("resume", [0, 1])
def test_factors_that_grow(cuda_ok, dtype, resume):
    """alpha = 2 on values of 1e30: tokens keep their outputs as long as the state is far from fp32's end, and a state that
    has passed it is not finite."""
    n = 64
    d = make(72, dtype, n, 2, 1, 64, 1)
    d["alpha"][:] = 2.0
    d["v"] = round_to_dtype((d["v"] * 1e30).astype(np.float32), "bf16" if dtype == BF else "f32")
    d["S"] = (d["S"] * 1e30).astype(np.float32)
    y_got, S_got = run(d, dtype, resume)
    assert not np.isfinite(S_got).any()
    few = 0
    while few < n:
        head = {k: v if k == "S" else v[:few + 1] for k, v in d.items()}
        S, y = oracle_scan(**head, offsets=[0, few + 1], resume=[resume], q_scale=SCALE)
        if np.abs(S).max() > 1e36:
            break
        few += 1
    assert 5 < few < 40
    near(y_got[:few], y[:few], 4 * tol(n))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_of_factors_past_the_range(cuda_ok, dtype):
    """Three factors of 1e25 in one head: its state passes fp32's end at the second of them; tokens before it keep their
    outputs, from it on none is finite, and the other head keeps its bits."""
    d = make(73, dtype, 100, 2, 2, 64, 1)
    clean = run(d, dtype, 1)
    d["alpha"][20:23, 0] = 1e25
    y_got, S_got = run(d, dtype, 1)
    head = {k: v if k == "S" else v[:21] for k, v in d.items()}
    S, y = oracle_scan(**head, offsets=[0, 21], resume=[1], q_scale=SCALE)
    near(y_got[:21, 0], y[:, 0], 4 * tol(100))
    assert not np.isfinite(y_got[21:, 0]).any() and not np.isfinite(S_got[0]).any()
    np.testing.assert_array_equal(y_got[:, 1], clean[0][:, 1])
    np.testing.assert_array_equal(S_got[1], clean[1][1])
