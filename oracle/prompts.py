"""Prompts, the short convolution and draft verification in float64 (oracle; test infrastructure only).

* ``mamba2_scan``, ``gdn_scan`` -- the recurrences of ``recurrence`` token by token over packed prompts.
* ``shortconv`` -- the causal depthwise filter over one sequence of rows, with its history as leading rows.
* ``ShortConvRing`` -- the history ring and its cursor: prompts, steps, tentative rows and their commit.
* ``accept_drafts`` -- the rejection rule of speculative sampling (Leviathan, Kalman & Matias, "Fast inference from
  transformers via speculative decoding", 2023) with given random numbers and an inverse-CDF draw.
"""

from __future__ import annotations

import numpy as np

from .recurrence import gdn_step, mamba2_step

f64 = np.float64


def mamba2_scan(S, x, B, C, dt, A, D, offsets, slots=None, resume=None):
    """S [batch][H][P][N]; x [total][H][P]; B, C [total][G][N]; dt [total][H]: (new S, y [total][H][P]).

    Rows of no prompt are NaN in y."""
    S = np.array(S, f64)
    H, G = x.shape[1], B.shape[1]
    groups = [h // (H // G) for h in range(H)]
    y = np.full(x.shape, np.nan)
    for i in range(len(offsets) - 1):
        slot = i if slots is None else int(slots[i])
        s = S[slot] if resume is not None and resume[i] else np.zeros_like(S[slot])
        for t in range(int(offsets[i]), int(offsets[i + 1])):
            s, y[t] = mamba2_step(s, x[t], B[t], C[t], dt[t], A, D, groups)
        S[slot] = s
    return S, y


def shortconv(rows, weight, bias, silu):
    """rows [K-1+n][channels] (history first) -> outputs [n][channels] in float64, unrounded."""
    rows, weight = np.asarray(rows, f64), np.asarray(weight, f64)
    K = weight.shape[1]
    n = rows.shape[0] - (K - 1)
    out = np.zeros((n, rows.shape[1]))
    for t in range(n):
        for k in range(K):
            out[t] += weight[:, k] * rows[t + k]
    if bias is not None:
        out += np.asarray(bias, f64)
    with np.errstate(over="ignore"):
        return out / (1.0 + np.exp(-out)) if silu else out


class ShortConvRing:
    """hist [batch][ring][channels], cur [batch]: the slot of the next token."""

    def __init__(self, hist, cur, weight, bias, silu):
        self.hist, self.cur = np.array(hist, f64), np.array(cur, np.int64)
        self.weight, self.bias, self.silu = weight, bias, silu
        self.K, self.ring = weight.shape[1], self.hist.shape[1]

    def _old(self, b):
        return [(self.cur[b] - (self.K - 1) + k) % self.ring for k in range(self.K - 1)]

    def prefill(self, x, offsets, slots=None, resume=None):
        out = np.full(x.shape, np.nan)
        for i in range(len(offsets) - 1):
            b = i if slots is None else int(slots[i])
            lo, hi = int(offsets[i]), int(offsets[i + 1])
            held = self.hist[b, self._old(b)]
            if resume is None or not resume[i]:
                held = np.zeros_like(held)
            rows = np.concatenate([held, np.asarray(x[lo:hi], f64)])
            out[lo:hi] = shortconv(rows, self.weight, self.bias, self.silu)
            self.hist[b, self._old(b)] = rows[len(rows) - (self.K - 1):]
        return out

    def verify(self, x):
        """x [batch][T][channels]: outputs; the rows are stored and the cursor stays."""
        out = np.empty(x.shape)
        for b in range(x.shape[0]):
            rows = np.concatenate([self.hist[b, self._old(b)], np.asarray(x[b], f64)])
            out[b] = shortconv(rows, self.weight, self.bias, self.silu)
            for t in range(x.shape[1]):
                self.hist[b, (self.cur[b] + t) % self.ring] = x[b, t]
        return out

    def commit(self, accepted):
        acc = np.clip(np.asarray(accepted), 0, self.ring - (self.K - 1))
        self.cur = (self.cur + acc) % self.ring

    def step(self, x):
        out = self.verify(x[:, None])[:, 0]
        self.cur = (self.cur + 1) % self.ring
        return out


def _mass(v):
    v = np.asarray(v, f64)
    return np.where((v > 0) & np.isfinite(v), v, 0.0)


def accept_drafts(target, tokens, u, draft=None, count=None):
    """(accepted, next) per sequence; arrays as the library's call takes them."""
    batch, T1, V = target.shape
    T = T1 - 1
    acc, nxt = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        c = T if count is None else min(max(int(count[b]), 0), T)
        n = 0
        while n < c:
            d = int(tokens[b, n])
            if not 0 <= d < V:
                break
            q = 1.0 if draft is None else f64(draft[b, n, d])
            if not _mass(target[b, n, d]) > 0 or not f64(u[b, n]) * q < f64(target[b, n, d]):
                break
            n += 1
        p = _mass(target[b, n])
        m = p
        if n < c:
            if draft is not None:
                with np.errstate(invalid="ignore"):
                    m = _mass(np.asarray(target[b, n], f64) - np.asarray(draft[b, n], f64))
            elif 0 <= int(tokens[b, n]) < V:
                m = p.copy()
                m[int(tokens[b, n])] = 0.0
        if not m.sum() > 0:
            m = p
        acc[b] = n
        if not m.sum() > 0:
            nxt[b] = -1
            continue
        cdf = np.cumsum(m)
        over = np.nonzero((cdf > f64(u[b, T]) * cdf[-1]) & (m > 0))[0]
        nxt[b] = over[0] if len(over) else np.nonzero(m)[0][-1]
    return acc, nxt


def gdn_scan(S, q, k, v, alpha, beta, offsets, slots=None, resume=None, q_scale=1.0):
    """S [batch][H][dv][dk]; q, k [total][Hk][dk]; v [total][H][dv]; alpha, beta [total][H]: (new S, y [total][H][dv]).

    Value head h takes query and key head h // (H / Hk).  Rows of no prompt are NaN in y."""
    S = np.array(S, f64)
    heads = np.arange(v.shape[1]) // (v.shape[1] // q.shape[1])
    y = np.full(v.shape, np.nan)
    for i in range(len(offsets) - 1):
        slot = i if slots is None else int(slots[i])
        s = S[slot] if resume is not None and resume[i] else np.zeros_like(S[slot])
        for t in range(int(offsets[i]), int(offsets[i + 1])):
            s, y[t] = gdn_step(s, q[t][heads], k[t][heads], v[t], alpha[t], beta[t], q_scale)
        S[slot] = s
    return S, y
