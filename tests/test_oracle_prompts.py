"""Pins of the oracle's prompt, short-convolution and draft-verification functions (no GPU)."""

import itertools

import numpy as np
import pytest

from oracle.prompts import ShortConvRing, accept_drafts, mamba2_scan, shortconv


def _layer(r, total, H=4, G=2, P=3, N=5):
    return dict(x=r.standard_normal((total, H, P)), B=r.standard_normal((total, G, N)),
                C=r.standard_normal((total, G, N)), dt=r.uniform(0.01, 0.3, (total, H)), A=-r.uniform(0.5, 2, H),
                D=r.standard_normal(H))


def test_scan_equals_the_unrolled_sum():
    """y_t = exp(A sum dt) S0 C_t + sum_i exp(A sum_{j>i} dt_j) dt_i (B_i . C_t) x_i + D x_t, written out."""
    r = np.random.default_rng(0)
    d = _layer(r, 7)
    S0 = r.standard_normal((1, 4, 3, 5))
    S, y = mamba2_scan(S0, **d, offsets=[0, 7], resume=[1])
    for h in range(4):
        g = h // 2
        cum = np.cumsum(d["dt"][:, h])
        for t in range(7):
            want = np.exp(d["A"][h] * cum[t]) * S0[0, h] @ d["C"][t, g] + d["D"][h] * d["x"][t, h]
            for i in range(t + 1):
                want += (np.exp(d["A"][h] * (cum[t] - cum[i])) * d["dt"][i, h] * (d["B"][i, g] @ d["C"][t, g])
                         * d["x"][i, h])
            np.testing.assert_allclose(y[t, h], want, rtol=1e-12)


def test_prompts_are_independent_and_split_anywhere():
    r = np.random.default_rng(1)
    d = _layer(r, 12)
    S0 = r.standard_normal((3, 4, 3, 5))
    S, y = mamba2_scan(S0, **d, offsets=[1, 5, 5, 11], slots=[2, 0, 1], resume=[0, 1, 1])
    assert np.isnan(y[[0, 11]]).all() and np.isfinite(y[1:11]).all()
    np.testing.assert_array_equal(S[0], S0[0])  # an empty prompt that resumes changes nothing
    # the last prompt in two calls
    Sa, ya = mamba2_scan(S0, **d, offsets=[5, 8], slots=[1], resume=[1])
    Sb, yb = mamba2_scan(Sa, **d, offsets=[8, 11], slots=[1], resume=[1])
    np.testing.assert_array_equal(Sb[1], S[1])
    np.testing.assert_array_equal(np.concatenate([ya[5:8], yb[8:11]]), y[5:11])


def test_shortconv_is_numpy_convolve():
    r = np.random.default_rng(2)
    for K in (2, 3, 4):
        rows, w = r.standard_normal((K - 1 + 9, 6)), r.standard_normal((6, K))
        out = shortconv(rows, w, None, False)
        for c in range(6):
            np.testing.assert_allclose(out[:, c], np.convolve(rows[:, c], w[c, ::-1], "valid"), rtol=1e-12)
        b = r.standard_normal(6)
        v = out + b
        np.testing.assert_allclose(shortconv(rows, w, b, True), v * 0.5 * (1 + np.tanh(v / 2)), rtol=1e-11)


def test_ring_decoding_equals_the_whole_sequence():
    """Prompt, steps, and drafts of which a prefix is committed give the same outputs as one long sequence."""
    r = np.random.default_rng(3)
    K, ch, T = 4, 5, 3
    w, b = r.standard_normal((ch, K)), r.standard_normal(ch)
    ring = ShortConvRing(r.standard_normal((2, K - 1 + T, ch)), [4, 1], w, b, True)
    seq = [list(r.standard_normal((6, ch))), list(r.standard_normal((1, ch)))]
    out = ring.prefill(np.concatenate([np.array(s) for s in seq]), [0, 6, 7])
    got = [list(out[:6]), list(out[6:])]
    for rnd in range(5):
        x = r.standard_normal((2, T, ch))
        o, acc = ring.verify(x), r.integers(0, T + 1, 2)
        ring.commit(acc)
        for s in range(2):
            seq[s] += list(x[s, :acc[s]])
            got[s] += list(o[s, :acc[s]])
        x = r.standard_normal((2, ch))
        o = ring.step(x)
        for s in range(2):
            seq[s].append(x[s])
            got[s].append(o[s])
    for s in range(2):
        rows = np.concatenate([np.zeros((K - 1, ch)), np.array(seq[s])])
        np.testing.assert_allclose(np.array(got[s]), shortconv(rows, w, b, True), rtol=1e-12)


def test_accepted_tokens_follow_the_target():
    """Over a fine grid of u, the first token out (draft if it stands, else the drawn one) has the target's
    distribution: the defining property of the rule."""
    p = np.array([0.5, 0.1, 0.25, 0.15])
    q = np.array([0.2, 0.5, 0.05, 0.25])
    M = 400
    grid = (np.arange(M) + 0.5) / M
    freq = np.zeros(4)
    for d in range(4):
        target = np.tile(np.stack([p, p])[None], (M, 1, 1))
        draft = np.tile(q[None, None], (M, 1, 1))
        for u1 in (np.arange(20) + 0.5) / 20:
            u = np.stack([grid, np.full(M, u1)], 1)
            acc, nxt = accept_drafts(target, np.full((M, 1), d), u, draft)
            first = np.where(acc == 1, d, nxt)
            freq += q[d] * np.bincount(first, minlength=4) / (M * 20)
    np.testing.assert_allclose(freq, p, atol=0.02)  # 20 draws of the residual: steps of q - p shares of 1/20


@pytest.mark.parametrize("probs", [True, False])
def test_accept_special_rows(probs):
    V = 5
    one = np.eye(V)
    # drafts that the target is sure of all stand, the bonus comes from the last row
    target = np.stack([one[2], one[4], np.array([0, .5, 0, .5, 0])])[None]
    draft = np.stack([one[2], one[4]])[None] if probs else None
    for u, want in ((0.0, 1), (0.49, 1), (0.5, 3), (0.999, 3)):
        acc, nxt = accept_drafts(target, np.array([[2, 4]]), np.array([[0.9, 0.9, u]]), draft)
        assert (acc[0], nxt[0]) == (2, want)
    # a draft the target rules out falls, and is not drawn
    acc, nxt = accept_drafts(target, np.array([[0, 4]]), np.array([[0.0, 0.9, 0.5]]),
                             None if draft is None else np.stack([one[0], one[4]])[None])
    assert (acc[0], nxt[0]) == (0, 2)
    # no mass anywhere
    acc, nxt = accept_drafts(np.zeros((1, 1, V)), np.zeros((1, 0), int), np.array([[0.3]]))
    assert (acc[0], nxt[0]) == (0, -1)


def test_accept_draw_by_enumeration():
    """next against a loop over the sums, for every u on a grid and every rejected place."""
    r = np.random.default_rng(5)
    for V, T in itertools.product((1, 2, 7), (0, 1, 3)):
        target = r.dirichlet(np.ones(V), size=(1, T + 1))
        draft = r.dirichlet(np.ones(V), size=(1, T))
        tokens = r.integers(0, V, (1, T))
        for uu in np.linspace(0, 0.99, 12):
            u = np.concatenate([r.random((1, T)), [[uu]]], 1)
            acc, nxt = accept_drafts(target, tokens, u, draft)
            n = acc[0]
            m = np.maximum(target[0, n] - draft[0, n], 0) if n < T else target[0, n]
            if m.sum() == 0:
                m = target[0, n]
            run, want = 0.0, None
            for v in range(V):
                run += m[v]
                if want is None and run > uu * m.sum() * (1 + 1e-15) and m[v] > 0:
                    want = v
            assert nxt[0] == want


def test_accept_needs_mass_at_the_draft():
    """A draft whose target entry is not a positive finite number falls, whatever its own probability."""
    for p in (np.inf, np.nan, 0.0, -1.0):
        target, draft = np.full((1, 2, 4), 0.25), np.full((1, 1, 4), 0.25)
        target[0, 0, 2], draft[0, 0, 2] = p, -0.5
        for u in (0.0, 0.5):
            assert accept_drafts(target, np.array([[2]]), np.array([[u, 0.5]]), draft)[0][0] == 0
