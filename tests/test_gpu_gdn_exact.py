"""How exact the gated delta rule over prompts is, by how alike its keys are (needs a B200).

Tolerances, on the 2-norm of the error over that of the result, for a prompt and head.

bf16, a chunk of 64 tokens: a value passes four products (K S^T, T R, U^T K, and Q S^T with M U), each a sum of at most 24 steps
of the tensor core (8 blocks of 16 terms in three pieces), each step off by at most 2^-24 of the running sum and independent of
the others: sqrt(96) 2^-24; operands are held to 2^-24 and formed from fp32 products, six times 2^-24 beside it: 2^-20 in all.
Tokens do not amplify an error (unit keys, beta and alpha up to 1), chunks are independent: sqrt(chunks) of it.  Where keys are
alike their errors add up along the common direction instead of across directions, which doubles the bound at most (the sum of a
row of (I + A)^-1 is then up to 2).
fp32, token by token: two sums and two updates a token, 2^-23 together, of values that no token amplifies; sqrt(tokens) of it.
"""

import math

import numpy as np
import pytest

from oracle.prompts import gdn_scan as oracle_scan
from synth import round_to_dtype
from test_gpu_gdn_scan import BF, F32, SCALE, make, on_gpu, packed, scan

pytestmark = pytest.mark.gpu


def bound(dtype, n, cosine):
    if dtype == F32:
        return 2.0 ** -23 * n ** 0.5
    return (2.0 ** -19 if cosine else 2.0 ** -20) * (-(-n // 64)) ** 0.5


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cosine", [0.0, 0.5, 0.8, 0.95])
@pytest.mark.parametrize("decay", [0.02, 0.3, 1.4])
@pytest.mark.parametrize("lens", [(64,), (512,), (90, 700)])
def test_keys_alike(cuda_ok, dtype, cosine, decay, lens):
    """Keys with the mean cosine given, strong writes, decays of up to exp(-decay) a token (the forms of a chunk without and
    with decays in its matrices)."""
    r = np.random.default_rng(81)
    total, n = sum(lens), len(lens)
    d = make(80, dtype, total, 4, 2, 128, n)
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
    k = unit(math.sqrt(cosine) * unit(r.standard_normal((1, 2, 128))) +
             math.sqrt(1 - cosine) * unit(r.standard_normal((total, 2, 128)))) * 0.999
    d["k"] = round_to_dtype(k.astype(np.float32), "bf16" if dtype == BF else "f32")
    d["alpha"] = np.exp(-r.uniform(0, decay, (total, 4))).astype(np.float32)
    d["beta"] = r.uniform(0.5, 1, (total, 4)).astype(np.float32)
    offsets = packed(lens)
    S, y = oracle_scan(**d, offsets=offsets, resume=[1] * n, q_scale=SCALE)
    g = on_gpu(d, dtype)
    y_got = scan(g, offsets, resume=[1] * n).double().cpu().numpy()
    S_got = g["S"].double().cpu().numpy()
    for i, m in enumerate(lens):
        part = slice(offsets[i], offsets[i + 1])
        for h in range(4):
            for what, got, want in (("y", y_got[part, h], y[part, h]), ("S", S_got[i, h], S[i, h])):
                off = np.linalg.norm(got - want) / np.linalg.norm(want)
                assert off <= bound(dtype, m, cosine), f"{what} of prompt {i}, head {h}: {off:.2e}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [64, 128])
def test_outputs_of_a_held_state(cuda_ok, dtype, n):
    """A state that prompts hardly change, under weak writes of small values: outputs are its products with the queries, so that
    they are as exact as the form in which it is read."""
    r = np.random.default_rng(82)
    d = make(83, dtype, n, 2, 1, 128, 1, slow=100.0)
    d["S"] = r.standard_normal(d["S"].shape).astype(np.float32)
    d["v"] = round_to_dtype((d["v"] * 1e-3).astype(np.float32), "bf16" if dtype == BF else "f32")
    d["beta"] = r.uniform(0, 0.01, (n, 2)).astype(np.float32)
    S, y = oracle_scan(**d, offsets=[0, n], resume=[1], q_scale=SCALE)
    g = on_gpu(d, dtype)
    y_got = scan(g, [0, n], resume=[1]).double().cpu().numpy()
    for h in range(2):
        assert np.linalg.norm(y_got[:, h] - y[:, h]) <= bound(dtype, n, 0.0) * np.linalg.norm(y[:, h])
        assert np.linalg.norm(g["S"].double().cpu().numpy()[0, h] - S[0, h]) <= bound(dtype, n, 0.0) * np.linalg.norm(S[0, h])
