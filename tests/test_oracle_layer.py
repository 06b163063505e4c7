"""Pins of the oracle's packed gated delta rule and of what stands between a layer's projections (no GPU)."""

import numpy as np
import torch

from oracle.layer import e4m3_scaled, gated, gdn_inputs, rmsnorm
from oracle.prompts import gdn_scan


def test_gdn_scan_is_the_product_of_its_factors():
    """S_t from the matrices alpha (I - beta k k^T) multiplied out, heads shared, prompts independent and split anywhere."""
    r = np.random.default_rng(0)
    total, H, Hk, P, N = 9, 4, 2, 3, 5
    q, k = r.standard_normal((2, total, Hk, N))
    v, alpha, beta = r.standard_normal((total, H, P)), r.uniform(0.5, 1, (total, H)), r.uniform(0, 1, (total, H))
    S0 = r.standard_normal((3, H, P, N))
    S, y = gdn_scan(S0, q, k, v, alpha, beta, [0, 5, 9], slots=[2, 0], resume=[1, 0], q_scale=0.5)
    np.testing.assert_array_equal(S[1], S0[1])
    for h in range(H):
        for lo, hi, start, slot in ((0, 5, S0[2, h], 2), (5, 9, np.zeros((P, N)), 0)):
            for t in range(lo, hi):
                s = start
                for i in range(lo, t + 1):
                    kk = k[i, h // 2]
                    s = alpha[i, h] * s @ (np.eye(N) - beta[i, h] * np.outer(kk, kk)) + beta[i, h] * np.outer(v[i, h], kk)
                np.testing.assert_allclose(y[t, h], 0.5 * s @ q[t, h // 2], rtol=1e-11, atol=1e-13)
            np.testing.assert_allclose(S[slot, h], s, rtol=1e-11, atol=1e-13)
    Sa, ya = gdn_scan(S0, q, k, v, alpha, beta, [0, 2], slots=[2], resume=[1], q_scale=0.5)
    Sb, yb = gdn_scan(Sa, q, k, v, alpha, beta, [2, 5], slots=[2], resume=[1], q_scale=0.5)
    np.testing.assert_array_equal(Sb[2], S[2])
    np.testing.assert_array_equal(np.concatenate([ya[:2], yb[2:5]]), y[:5])


def test_layer_functions_equal_torch_in_64_bits():
    r = np.random.default_rng(1)
    q, k = r.standard_normal((2, 5, 2, 8))
    a, b, A_log, bias = r.standard_normal((5, 6)) * 9, r.standard_normal((5, 6)), r.standard_normal(6), r.standard_normal(6)
    qn, kn, alpha, beta = gdn_inputs(q, k, a, b, A_log, bias, 0.0, repeat=3)
    np.testing.assert_allclose(np.linalg.norm(qn, axis=-1), 1.0, rtol=1e-14)
    np.testing.assert_array_equal(kn[:, 0], kn[:, 2])
    t = torch.from_numpy
    np.testing.assert_allclose(alpha, torch.exp(-t(A_log).exp() * torch.nn.functional.softplus(t(a + bias), threshold=700)),
                               rtol=1e-12)
    np.testing.assert_allclose(beta, torch.sigmoid(t(b)), rtol=1e-13)
    h, w, z = r.standard_normal((4, 24)), r.standard_normal(24), r.standard_normal((4, 24))
    want = torch.nn.functional.rms_norm(t(h), (24,), t(1 + w), 1e-3)
    np.testing.assert_allclose(rmsnorm(h, w, 24, 1e-3, offset=1.0), want, rtol=1e-13)
    silu = torch.nn.functional.silu(t(z))
    per = torch.nn.functional.rms_norm(t(h).view(4, 3, 8), (8,), t(w[:8]), 1e-3).view(4, 24)
    np.testing.assert_allclose(gated(h, z, w[:8], 8, 1e-3, 0.0, True), per * silu, rtol=1e-12)
    first = torch.nn.functional.rms_norm(t(h) * silu, (24,), t(w), 1e-3)
    np.testing.assert_allclose(gated(h, z, w, 24, 1e-3, 0.0, False), first, rtol=1e-12)
    v, s = e4m3_scaled(h, 16)
    assert s.shape == (4, 2) and np.allclose(np.abs(v[:, :16]).max(1), 448) and np.allclose(np.abs(v[:, 16:]).max(1), 448)
    np.testing.assert_allclose(v[:, 16:] * s[:, 1:], h[:, 16:], rtol=1e-14)
    v, s = e4m3_scaled(np.zeros((2, 8)))
    assert (v == 0).all() and (s == 2.0 ** -126).all()
