"""Verification of drafted tokens against the float64 oracle: whole numbers, equal (needs a B200)."""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import accept_drafts
from oracle.prompts import accept_drafts as oracle_accept

pytestmark = pytest.mark.gpu


def rows(r, *shape, scale=2.0):
    z = r.standard_normal(shape) * scale
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def check(target, tokens, u, draft=None, count=None, strided=False):
    def dev(a, t):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t)

    def prob(a):
        t = dev(a, torch.float32)
        if t is None or not strided:
            return t
        wide = torch.full((*a.shape[:2], a.shape[2] + 3), float("nan"), device="cuda")
        wide[..., :a.shape[2]] = t
        return wide[..., :a.shape[2]]

    acc, com, nxt = accept_drafts(prob(target), dev(tokens, torch.int32), dev(u, torch.float32), draft=prob(draft),
                                  count=dev(count, torch.int32))
    want_acc, want_next = oracle_accept(target, tokens, u, draft, count)
    np.testing.assert_array_equal(acc.cpu().numpy(), want_acc)
    np.testing.assert_array_equal(com.cpu().numpy(), want_acc + 1)
    np.testing.assert_array_equal(nxt.cpu().numpy(), want_next)
    return want_acc


def case(seed, batch, T, V, noise=0.5):
    r = np.random.default_rng(seed)
    draft = rows(r, batch, T, V)
    mix = np.exp(noise * r.standard_normal((batch, T + 1, V)))
    base = np.concatenate([draft, rows(r, batch, 1, V)], 1)
    target = (base * mix / (base * mix).sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.zeros((batch, T), np.int64)
    for b in range(batch):
        for j in range(T):
            tokens[b, j] = r.choice(V, p=draft[b, j].astype(np.float64) / draft[b, j].astype(np.float64).sum())
    u = r.random((batch, T + 1)).astype(np.float32)
    return r, target, tokens, u, draft


@pytest.mark.parametrize("batch,T,V", [(1, 0, 1), (1, 4, 32000), (3, 1, 2), (7, 8, 257), (200, 2, 1000), (5, 16, 50257),
                                       (40, 3, 9000), (2, 2, 262144), (160, 1, 33000)])
def test_random_rows(cuda_ok, batch, T, V):
    r, target, tokens, u, draft = case(V + T, batch, T, V)
    check(target, tokens, u, draft)
    check(target, tokens, u, draft, r.integers(-1, T + 2, batch))
    check(target, tokens, u, None)
    check(target, tokens, u, None, r.integers(0, T + 1, batch), strided=True)
    acc = check(target, tokens, u, draft, strided=True)
    if T >= 2 and batch >= 40:
        assert 0 < acc.mean() < T


def test_borders(cuda_ok):
    """u on the borders of the sums (powers of two: exact), at 0, at the largest float below 1; equal distributions
    (nothing is left to draw from a rejection that cannot happen); one-hot rows."""
    V = 4096
    flat = np.full((1, 1, V), 1.0 / V, np.float32)
    for k in (0, 1, 31, 32, 33, 1023, 1024, 4095):
        check(flat, np.zeros((1, 0), int), np.array([[k / V]]))
    check(flat, np.zeros((1, 0), int), np.array([[np.float32(1) - np.float32(2.0 ** -24)]]))
    for v in (0, 5, 4095):
        one = np.zeros((1, 1, V), np.float32)
        one[..., v] = 0.75
        for u in (0.0, 0.5, 0.9999):
            check(one, np.zeros((1, 0), int), np.array([[u]]))
    r, target, tokens, u, draft = case(1, 8, 4, 512)
    target[:, :4] = draft
    assert (check(target, tokens, u, draft) == 4).all()
    # p = q / 2 everywhere: drafts fall and max(p - q, 0) is empty, so p is drawn from
    target[:, :4] = draft / 2
    u[:, :4] = 0.75
    assert (check(target, tokens, u, draft) == 0).all()


def test_entries_without_mass(cuda_ok):
    """NaN, infinities and negative entries carry none; rows without any give -1; drafts outside the vocabulary fall."""
    r, target, tokens, u, draft = case(2, 12, 3, 700)
    for a in (target, draft):
        a[:, :, 10:20] = np.nan
        a[:, :, 30:40] = np.inf
        a[:, :, 50:60] = -1.0
    target[0, :, 60] = 3e38  # with the -3e38 below beyond fp32's range, but finite in 64 bits
    draft[0, :, 60] = -3e38
    target[3:5] = 0.0
    target[5] = np.nan
    tokens[6:8, 0] = (-3, 700)
    tokens[8, 1] = 2 ** 31 - 1
    check(target, tokens, u, draft)
    check(target, tokens, u, None)


def test_long_rows_few_sequences(cuda_ok):
    """A vocabulary whose chunks are searched in two levels, with the draw in its first, middle and last part."""
    r = np.random.default_rng(4)
    V = 262144
    for batch in (1, 300):
        target = torch.rand(batch, 1, V, device="cuda")
        t = target.cpu().numpy()
        u = r.random((batch, 1)).astype(np.float32)
        u[0] = 0.999999
        _, _, nxt = accept_drafts(target, torch.zeros(batch, 0, dtype=torch.int32, device="cuda"),
                                  torch.from_numpy(u).cuda())
        for b in (0, batch - 1):
            assert int(nxt[b]) == oracle_accept(t[b:b + 1], np.zeros((1, 0), int), u[b:b + 1])[1][0]


def test_rows_past_32_bits(cuda_ok):
    """Rows that lie so far apart that the last ones start past 2^31 elements."""
    V, apart = 1000, 2 ** 30 + 8
    r, target, tokens, u, draft = case(9, 2, 1, V)
    wide = torch.empty(3 * apart + V, device="cuda").as_strided((2, 2, V), (2 * apart, apart, 1))
    wide.copy_(torch.from_numpy(target))
    for q in (draft, None):
        got = accept_drafts(wide, torch.from_numpy(tokens).int().cuda(), torch.from_numpy(u).cuda(),
                            draft=None if q is None else torch.from_numpy(q).cuda())
        want = oracle_accept(target, tokens, u, q, None)
        np.testing.assert_array_equal(got[0].cpu().numpy(), want[0])
        np.testing.assert_array_equal(got[2].cpu().numpy(), want[1])


@pytest.mark.parametrize("probs", [True, False])
def test_drafts_that_the_target_gives_no_mass_fall(cuda_ok, probs):
    """An entry that is not a positive finite number carries no mass, so a draft of it never stands, whatever the draft's
    own probability: target inf, NaN, 0 and negative against q = -1, 0, 0.25 and u = 0 and 0.5."""
    V = 64
    cases = [(p, q, u) for p in (np.inf, np.nan, 0.0, -0.5) for q in (-1.0, 0.0, 0.25) for u in (0.0, 0.5)]
    n = len(cases)
    target = np.full((n, 2, V), 1.0 / V, np.float32)
    draft = np.full((n, 1, V), 1.0 / (2 * V), np.float32)
    tokens, us = np.full((n, 1), 7), np.full((n, 2), 0.25)
    for i, (p, q, u) in enumerate(cases):
        target[i, 0, 7], draft[i, 0, 7], us[i, 0] = p, q, u
    acc = check(target, tokens, us, draft if probs else None)
    assert (acc == 0).all()
