"""What stands between a layer's projections, in float64 (oracle; test infrastructure only).

* ``gdn_inputs`` -- normalised queries and keys, decays and write strengths of the gated delta rule (Yang, Kautz &
  Hatamizadeh, "Gated Delta Networks", 2024).
* ``rmsnorm``, ``gated`` -- the root-mean-square norm (Zhang & Sennrich, 2019) over groups of columns, and its gated forms.
* ``e4m3_scaled`` -- values in units of a scale for each row or block of columns.
"""

from __future__ import annotations

import numpy as np

f64 = np.float64


def gdn_inputs(q, k, a, b, A_log, bias, eps, repeat=1):
    def unit(t):
        t = np.asarray(t, f64)
        with np.errstate(invalid="ignore", divide="ignore"):
            t = t / np.sqrt((t * t).sum(-1, keepdims=True) + eps)
        return np.repeat(t, repeat, -2)

    with np.errstate(over="ignore"):
        z = np.asarray(a, f64) + np.asarray(bias, f64)
        return (unit(q), unit(k), np.exp(-np.exp(np.asarray(A_log, f64)) * np.logaddexp(0.0, z)),
                1.0 / (1.0 + np.exp(-np.asarray(b, f64))))


def rmsnorm(h, weight, group, eps, offset=0.0):
    """h [rows][n] over groups of columns; weight [n] or [group]."""
    h = np.asarray(h, f64)
    rows, n = h.shape
    parts = h.reshape(rows, n // group, group)
    unit = parts / np.sqrt((parts * parts).mean(-1, keepdims=True) + eps)
    w = offset + np.asarray(weight, f64)
    return (unit * (w.reshape(-1, group))).reshape(rows, n)


def gated(y, gate, weight, group, eps, offset, norm_first):
    z = np.asarray(gate, f64)
    with np.errstate(over="ignore"):
        s = z / (1.0 + np.exp(-z))
    if norm_first:
        return rmsnorm(y, weight, group, eps, offset) * s
    return rmsnorm(np.asarray(y, f64) * s, weight, group, eps, offset)


def e4m3_scaled(v, block=None):
    """(v / scale unrounded, scales): the largest magnitude of a row, or of each ``block`` columns, becomes 448."""
    rows, n = v.shape
    size = block or n
    edges = range(0, n, size)
    scales = np.stack([np.abs(v[:, c:c + size]).max(1) / 448.0 for c in edges], 1)
    scales = np.maximum(scales, 2.0 ** -126)
    return v / np.repeat(scales, size, 1)[:, :n], scales if block else scales[:, 0]
