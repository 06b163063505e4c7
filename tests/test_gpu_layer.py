"""What stands between a layer's projections against the float64 oracle (needs a B200).

Tolerances.  fp32 results: sums of n squares are formed in chains of at most 32 and trees of at most 15 levels, 2^-24 of
the (positive) sum each, of which the root keeps half: 24 units of 2^-24; a dozen more operations and exp and log1p (2 units
each) add 20: 2^-18 holds them all.  A result in bf16 adds half a step, 2^-8 of its value, and one in E4M3 2^-4 or half the
spacing of its subnormal numbers, 2^-10, in units of the scale.
"""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import (ReplaySSM, add_rmsnorm, gated_rmsnorm, gdn_inputs, shortconv_prefill, shortconv_step)
from oracle import layer as ref
from oracle.prompts import gdn_scan as oracle_scan, shortconv as oracle_conv
from synth import round_to_dtype

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FINE = 2.0 ** -18
HALF = {BF: 2.0 ** -8, F32: 0.0}


def values(r, dtype, *shape, std=1.0):
    return round_to_dtype((std * r.standard_normal(shape)).astype(np.float32), "bf16" if dtype == BF else "f32")


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def close(got, want, dtype, floor=0.0):
    assert got.dtype == dtype
    got = got.double().cpu().numpy()
    bound = (HALF[dtype] + FINE) * np.abs(want) + floor
    assert got.shape == want.shape and (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / (bound + 1e-300))


def close_e4m3(got, scales, want, block):
    v, s = ref.e4m3_scaled(want.reshape(-1, want.shape[-1]), block)
    v, s = v.reshape(want.shape), s.reshape(scales.shape)
    assert got.dtype == E4M3 and scales.dtype == F32
    assert (np.abs(scales.double().cpu().numpy() - s) <= FINE * s).all()
    err = np.abs(got.double().cpu().numpy() - v)
    assert (err <= (2.0 ** -4 + 2 * FINE) * np.abs(v) + 2.0 ** -10).all()


# ------------------------------------------------------------------------------------------ inputs of the gated delta rule


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H,Hk,expand", [(1, 32, 16, True), (1, 1, 1, False), (7, 6, 2, True), (7, 6, 2, False),
                                              (333, 8, 8, True), (2500, 5, 5, False), (3000, 12, 4, True)])
def test_gdn_inputs(cuda_ok, dtype, rows, H, Hk, expand):
    r = np.random.default_rng(rows + H)
    q, k = values(r, dtype, rows, Hk, 128, std=2.0), values(r, dtype, rows, Hk, 128, std=1e-3)
    k[0, 0] = 0.0
    a, b = values(r, dtype, rows, H, std=3.0), values(r, dtype, rows, H, std=3.0)
    A_log, bias = r.uniform(-1, 3, H).astype(np.float32), r.uniform(-7, 2, H).astype(np.float32)
    got = gdn_inputs(*(dev(t, dtype) for t in (q, k, a, b)), dev(A_log), dev(bias), expand=expand)
    want = ref.gdn_inputs(q, k, a, b, A_log, bias, 1e-6, H // Hk if expand else 1)
    for g, w, t in zip(got[:2], want[:2], (dtype, dtype)):
        close(g, w, t)
    # alpha = exp(-x): x is relatively off by FINE, so alpha by x FINE of itself (and fp32's underflow)
    x = -np.log(np.maximum(want[2], 1e-300))
    err = np.abs(got[2].double().cpu().numpy() - want[2])
    assert (err <= FINE * (1 + x) * want[2] + 2.0 ** -149).all()
    close(got[3], want[3], F32)


def test_gdn_inputs_extremes(cuda_ok):
    """Gates far out on both sides stay in their ranges; NaN and infinities go where the formulas take them, and keep to
    their own vectors and gates."""
    H = 8
    a = torch.tensor([[-300.0, 300.0, np.nan, np.inf, -np.inf, 0.0, 88.0, -88.0]], device="cuda")
    b = torch.tensor([[-300.0, 300.0, 0.0, np.inf, -np.inf, np.nan, 88.0, -88.0]], device="cuda")
    q = torch.ones(1, H, 128, device="cuda")
    q[0, 1, 5], q[0, 2, 6], q[0, 3] = np.nan, np.inf, 3e38
    qn, kn, alpha, beta = gdn_inputs(q, torch.ones_like(q), a, b, torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda"))
    alpha, beta = alpha[0].cpu().numpy(), beta[0].cpu().numpy()
    assert alpha[0] == 1 and alpha[1] == 0 and np.isnan(alpha[2]) and alpha[3] == 0 and alpha[4] == 1
    assert abs(alpha[5] - 0.5) < 1e-6 and 0 < alpha[6] < 1e-37 and alpha[7] == 1
    assert beta[0] == 0 and beta[1] == 1 and beta[3] == 1 and beta[4] == 0 and np.isnan(beta[5]) and beta[6] == 1
    assert torch.isnan(qn[0, 1]).all() and torch.isnan(qn[0, 2, 6]) and (qn[0, 3] == 0).all()
    assert (qn[0, [0, 4, 5, 6, 7]] == qn[0, 0, 0]).all() and (kn == kn[0, 0, 0]).all()


@pytest.mark.parametrize("lead", [(5,), (3, 4), (1, 6), (6, 1), (2, 3, 2), ()])
def test_gdn_inputs_of_slices(cuda_ok, lead):
    """Slices of wider projections with any leading dimensions, and outputs of the caller."""
    r = np.random.default_rng(3)
    Hk, H = 2, 4
    wide = dev(values(r, BF, *lead, 2 * Hk * 128 + 8 + 2 * H), BF)
    q = wide[..., :Hk * 128].unflatten(-1, (Hk, 128))
    k = wide[..., Hk * 128:2 * Hk * 128].unflatten(-1, (Hk, 128))
    a, b = wide[..., -2 * H:-H], wide[..., -H:]
    A_log, bias = dev(r.uniform(0, 1, H)), dev(r.uniform(-1, 1, H))
    want = gdn_inputs(q.contiguous(), k.contiguous(), a.contiguous(), b.contiguous(), A_log, bias, expand=True)
    out = tuple(torch.empty_like(t) for t in want)
    got = gdn_inputs(q, k, a, b, A_log, bias, expand=True, out=out)
    assert all(g is o and torch.equal(g, w) for g, o, w in zip(got, out, want))
    assert got[0].shape == (*lead, H, 128) and got[2].shape == (*lead, H)


# ------------------------------------------------------------------------------------------ norms

COLUMNS = [8, 24, 128, 256, 264, 512, 1000, 1024, 1032, 2048, 4096, 5000, 8192, 16384, 16392, 32768]


@pytest.mark.parametrize("n", COLUMNS)
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (F32, F32), (BF, F32)])
def test_add_rmsnorm(cuda_ok, n, dtype, wdtype):
    r = np.random.default_rng(n)
    rows = 5 if n > 2000 else 37
    x, res, w = values(r, dtype, rows, n), values(r, dtype, rows, n, std=3.0), values(r, wdtype, n)
    h = x.astype(np.float64) + res
    for residual in (True, False):
        for scale, out_dtype in ((None, None), (None, F32), ("row", None), ("block", None)):
            rt = dev(res, dtype) if residual else None
            got = add_rmsnorm(dev(x, dtype), dev(w, wdtype), rt, eps=1e-5, offset=0.5, out_dtype=out_dtype, scale=scale)
            want = ref.rmsnorm(h if residual else x, w, n, 1e-5, 0.5)
            floor = FINE * np.abs(want).max()  # offset + w is rounded: 2^-24 of the larger of the two
            if scale:
                close_e4m3(*got, want, 128 if scale == "block" else None)
            else:
                close(got, want, out_dtype or dtype, floor)
            if residual:
                close(rt, h, dtype)


@pytest.mark.parametrize("n,group,shared", [(128, 128, True), (4096, 128, True), (4096, 128, False), (8192, 1024, False),
                                            (512, 512, False), (48, 24, True), (640, 320, False), (1024, 8, True),
                                            (1536, 256, True), (2000, 1000, False), (1280, 40, True), (32768, 4096, True),
                                            (16384, 64, False), (256, 32, False)])
@pytest.mark.parametrize("gate_dtype", [BF, F32])
def test_gated_rmsnorm(cuda_ok, n, group, shared, gate_dtype):
    r = np.random.default_rng(n + group)
    rows = 4 if n > 2000 else 19
    w = values(r, gate_dtype, group if shared else n)
    z = values(r, gate_dtype, rows, n, std=3.0)
    for y_dtype in (F32, BF):
        y = values(r, y_dtype, rows, n, std=0.2)
        for norm_first in (True, False):
            want = ref.gated(y, z, w, group, 1e-6, 0.0, norm_first)
            args = dict(group=group, norm_first=norm_first)
            close(gated_rmsnorm(dev(y, y_dtype), dev(z, gate_dtype), dev(w, gate_dtype), **args), want, gate_dtype)
            for scale in ("row", "block"):
                got = gated_rmsnorm(dev(y, y_dtype), dev(z, gate_dtype), dev(w, gate_dtype), scale=scale, **args)
                close_e4m3(*got, want, 128 if scale == "block" else None)


def test_rows_side_by_side_and_in_place(cuda_ok):
    """Input, residual and gate as slices of one wide matrix; x as its own residual; outputs over inputs are refused."""
    r = np.random.default_rng(44)
    wide = dev(values(r, BF, 9, 640), BF)
    w = dev(values(r, BF, 200), BF)
    x, res, z = wide[:, :200], wide[:, 200:400], wide[:, 400:600]
    apart = [t.contiguous() for t in (x, res, z)]
    want = add_rmsnorm(apart[0], w, apart[1])
    assert torch.equal(add_rmsnorm(x, w, res), want) and torch.equal(wide[:, 200:400], apart[1])
    assert torch.equal(wide[:, :200], apart[0]) and torch.equal(wide[:, 400:600], apart[2])
    assert torch.equal(gated_rmsnorm(x, z, w, group=40), gated_rmsnorm(apart[0], apart[2], w, group=40))
    twice = apart[0].clone()
    want = add_rmsnorm(apart[0], w, res2 := apart[0].clone())
    assert torch.equal(add_rmsnorm(twice, w, twice), want) and torch.equal(twice, res2)
    for call in (lambda: add_rmsnorm(twice, w, out=twice), lambda: gated_rmsnorm(apart[0], twice, w, out=twice),
                 lambda: add_rmsnorm(twice, w, res2, out=res2), lambda: add_rmsnorm(wide[:, :200], w, wide[:, 8:208])):
        with pytest.raises(RuntimeError, match="RSSM_ERR_ARG"):
            call()
    q, a = dev(values(r, BF, 9, 2, 128), BF), dev(values(r, BF, 9, 4), BF)
    A = torch.zeros(4, device="cuda")
    out = (q, torch.empty_like(q), torch.empty(9, 4, device="cuda"), torch.empty(9, 4, device="cuda"))
    with pytest.raises(RuntimeError, match="RSSM_ERR_ARG"):
        gdn_inputs(q, q, a, a, A, A, out=out)


@pytest.mark.parametrize("rows,n", [(2 ** 19 + 5, 8192), (2 ** 17 + 3, 32768)])
def test_rows_past_32_bits(cuda_ok, rows, n):
    """Matrices with more than 2^32 elements: the last rows are what they are in a small one."""
    r = np.random.default_rng(45)
    x, z, w = (dev(values(r, BF, *s), BF) for s in ((5, n), (5, n), (n,)))
    big, gate = torch.empty(rows, n, dtype=BF, device="cuda"), torch.empty(rows, n, dtype=BF, device="cuda")
    big[-5:], gate[-5:] = x, z
    res, small = gate.clone(), z.clone()
    out, scales = add_rmsnorm(big, w, res, scale="block")
    want, s = add_rmsnorm(x, w, small, scale="block")
    assert torch.equal(out[-5:].view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales[-5:], s)
    assert torch.equal(res[-5:], small)
    del out, res
    assert torch.equal(gated_rmsnorm(big, gate, w, group=64)[-5:], gated_rmsnorm(x, z, w, group=64))


def test_inputs_past_32_bits(cuda_ok):
    r = np.random.default_rng(46)
    rows, H, Hk = 2 ** 21 + 77, 32, 16
    q, a = dev(values(r, BF, 77, Hk, 128), BF), dev(values(r, BF, 77, H), BF)
    A, bias = (torch.from_numpy(r.uniform(-1, 1, H).astype(np.float32)).cuda() for _ in range(2))
    big, gates = torch.empty(rows, Hk, 128, dtype=BF, device="cuda"), torch.empty(rows, H, dtype=BF, device="cuda")
    big[-77:], gates[-77:] = q, a
    for got, want in zip(gdn_inputs(big, big, gates, gates, A, bias), gdn_inputs(q, q, a, a, A, bias)):
        assert torch.equal(got[-77:], want)


def test_norms_of_slices_and_own_outputs(cuda_ok):
    """Rows that lie apart, any leading dimensions, outputs of the caller, no rows at all."""
    r = np.random.default_rng(4)
    for lead in ((6,), (2, 3), (1, 4), (4, 1), ()):
        wide = dev(values(r, BF, *lead, 640), BF)
        x, z, w = wide[..., :256], wide[..., 384:], dev(values(r, BF, 256), BF)
        res = dev(values(r, BF, *lead, 300), BF)[..., :256].contiguous()
        res2 = torch.cat([res, res], -1)[..., :256]
        want = add_rmsnorm(x.contiguous(), w, res, scale="block")
        out = tuple(torch.empty_like(t) for t in want)
        got = add_rmsnorm(x, w, res2, scale="block", out=out)
        assert got is out and torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
        assert torch.equal(res, res2) and got[1].shape == (*lead, 2)
        o = torch.empty(*lead, 256, dtype=BF, device="cuda")
        assert gated_rmsnorm(x, z, w, group=64, out=o) is o
        assert torch.equal(o, gated_rmsnorm(x.contiguous(), z.contiguous(), w, group=64))
    e = torch.empty(0, 256, dtype=BF, device="cuda")
    assert add_rmsnorm(e, w, e.clone()).shape == (0, 256) and gated_rmsnorm(e, e, w, scale="row")[1].shape == (0,)


def test_norm_extremes(cuda_ok):
    """Rows of zeros, of values whose 8-bit scale would leave the normal numbers, with NaN or infinities: each keeps to its
    own row (groups to theirs), and codes hold no NaN but theirs."""
    n = 512
    x = torch.randn(8, n, device="cuda")
    x[0] = 0.0
    x[2, 3], x[3, 4] = np.nan, np.inf
    x[4] *= 1e-30
    w = torch.ones(n, device="cuda")
    tiny = torch.full((n,), 1e-38, device="cuda")
    y = add_rmsnorm(x, w)
    assert (y[0] == 0).all() and torch.isnan(y[2]).all() and torch.isnan(y[3, 4]) and (y[3, 5:] == 0).all()
    for scale in ("row", "block"):
        q, s = add_rmsnorm(x, w, scale=scale)
        f = q.float()
        assert (f[0] == 0).all() and (s[0] == 2.0 ** -126).all()
        assert torch.isnan(f[2]).all() and torch.isnan(s[2]).all()
        assert torch.isfinite(f[[0, 1, 4, 5, 6, 7]]).all() and torch.isnan(f[3, 4])
        q, s = add_rmsnorm(x, tiny, scale=scale)
        assert torch.isfinite(q.float()[[0, 1, 5, 6, 7]]).all() and (s[[1, 5, 6, 7]] >= 2.0 ** -126).all()
    z = torch.ones_like(x)
    z[5, 0], z[6, 200] = np.nan, -np.inf
    g = gated_rmsnorm(x, z, w[:128], group=128, norm_first=False)
    assert torch.isnan(g[5, :128]).all() and torch.isfinite(g[5, 128:]).all()
    assert torch.isfinite(g[6, :128]).all() and torch.isnan(g[6, 200]) and torch.isfinite(g[6, 256:]).all()
    assert torch.isfinite(g[[0, 1, 4, 7]]).all()


def test_refusals_on_the_device(cuda_ok):
    x, w = torch.zeros(4, 256, device="cuda"), torch.zeros(256, device="cuda")
    with pytest.raises(ValueError, match="scale"):
        add_rmsnorm(x, w, scale="column")
    with pytest.raises(ValueError, match="weight"):
        add_rmsnorm(x, w[:128])
    with pytest.raises(ValueError, match="group"):
        gated_rmsnorm(x, x, w, group=100)
    with pytest.raises(ValueError, match="residual"):
        add_rmsnorm(x, w, x.bfloat16())
    with pytest.raises(ValueError, match="rows overlap"):
        add_rmsnorm(x[:1].expand(4, 256), w)
    with pytest.raises(ValueError, match="contiguous rows"):
        add_rmsnorm(torch.zeros(256, 4, device="cuda").t(), w)
    with pytest.raises(ValueError, match="evenly apart"):
        add_rmsnorm(torch.zeros(3, 5, 256, device="cuda")[:, :4], w)
    with pytest.raises(RuntimeError, match="RSSM_ERR_SHAPE"):
        add_rmsnorm(torch.zeros(4, 260, device="cuda")[:, :256], torch.zeros(256, device="cuda"))
    with pytest.raises(RuntimeError, match="RSSM_ERR_SHAPE"):
        add_rmsnorm(torch.zeros(4, 100, device="cuda"), torch.zeros(100, device="cuda"))
    q, a = torch.zeros(4, 2, 128, device="cuda"), torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError, match="A_log"):
        gdn_inputs(q, q, a, a, w, w)
    with pytest.raises(ValueError, match="k"):
        gdn_inputs(q, q[:, :1], a, a, w[:4], w[:4])


# ------------------------------------------------------------------------------------------ together

H, HK, P, K, BATCH = 4, 2, 128, 4, 3
SPLITS = (HK * 128, HK * 128, H * P)
CH, HID = sum(SPLITS), 512


class Layer:
    """A GDN layer between its projections, as a serving loop runs it: norm, (projection,) convolution, inputs, prompts or
    steps, gated norm."""

    def __init__(self, r):
        self.norm_w, self.out_w = dev(values(r, BF, HID), BF), dev(values(r, BF, P), BF)
        self.w, self.b = dev(values(r, BF, CH, K, std=0.5), BF), dev(values(r, BF, CH, std=0.3), BF)
        self.proj = dev(values(r, BF, HID, CH + 2 * H + H * P, std=HID ** -0.5), BF)
        self.A_log, self.bias = dev(r.uniform(0, 1, H)), dev(r.uniform(-4, -1, H))
        self.hist = torch.zeros(BATCH, K, CH, dtype=BF, device="cuda")
        self.cur = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
        self.state = ReplaySSM("gdn", BATCH, H, P, 128, 1, 8, 0, BF, q_scale=128 ** -0.5)
        self.state.load_checkpoint(torch.zeros(BATCH, H, P, 128, device="cuda"))

    def run(self, x, residual, offsets=None):
        h = add_rmsnorm(x, self.norm_w, residual)
        z = h @ self.proj
        a, b, gate = z[:, CH:CH + H], z[:, CH + H:CH + 2 * H], z[:, CH + 2 * H:]
        if offsets is None:
            q, k, v = shortconv_step(self.hist, self.cur, z[:, :CH], self.w, self.b, splits=SPLITS)
        else:
            q, k, v = shortconv_prefill(self.hist, self.cur, z[:, :CH], self.w, self.b, offsets, splits=SPLITS)
        n = x.shape[0]
        tok = gdn_inputs(q.view(n, HK, 128), k.view(n, HK, 128), a, b, self.A_log, self.bias, expand=offsets is None)
        v = v.view(n, H, P)
        if offsets is None:
            y = self.state.gdn_step(*tok[:2], v, *tok[2:])
        else:
            y = self.state.gdn_prefill(*tok[:2], v, *tok[2:], offsets)
        return z, tok, v, y, gated_rmsnorm(y.view(n, H * P), gate, self.out_w, group=P, scale="block")


def test_a_layer_from_prompt_to_decoding(cuda_ok):
    """Prompts and then single tokens through the whole layer, each call against the oracle on the call's own inputs."""
    r = np.random.default_rng(5)
    layer = Layer(r)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    bounds = [0, 70, 75, 160]
    x, res = dev(values(r, BF, 160, HID), BF), dev(values(r, BF, 160, HID), BF)
    want = ref.rmsnorm(f(x) + f(res), f(layer.norm_w), HID, 1e-6)
    close(add_rmsnorm(x, layer.norm_w, res.clone()), want, BF)
    z, tok, v, y, (codes, scales) = layer.run(x, res, dev(np.array(bounds), torch.int32))
    w, b = f(layer.w), f(layer.b)
    lines = []
    for lo, hi in zip(bounds, bounds[1:]):
        rows = np.concatenate([np.zeros((K - 1, CH)), f(z[lo:hi, :CH])])
        out = oracle_conv(rows, w, b, True)
        assert (np.abs(f(v[lo:hi]).reshape(hi - lo, -1) - out[:, -H * P:]) <= 2.0 ** -8 * np.abs(out[:, -H * P:]) + 2.0 ** -17).all()
        lines.append(rows)
    S, y_ref = oracle_scan(np.zeros((BATCH, H, P, 128)), *(f(t) for t in (*tok[:2], v, *tok[2:])), bounds, q_scale=128 ** -0.5)
    assert np.linalg.norm(f(y) - y_ref) <= 2.0 ** -14 * np.linalg.norm(y_ref)
    gate = f(z[:, CH + 2 * H:])
    close_e4m3(codes, scales, ref.gated(f(y).reshape(160, -1), gate, f(layer.out_w), P, 1e-6, 0.0, True), 128)
    for _ in range(10):  # more than a window
        x, res = dev(values(r, BF, BATCH, HID), BF), dev(values(r, BF, BATCH, HID), BF)
        z, tok, v, y, (codes, scales) = layer.run(x, res)
        for i in range(BATCH):
            lines[i] = np.concatenate([lines[i], f(z[i:i + 1, :CH])])
            out = oracle_conv(lines[i][-K:], w, b, True)[0, -H * P:]
            assert (np.abs(f(v[i]).ravel() - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -17).all()
        for i in range(BATCH):
            S[i:i + 1], y_ref = oracle_scan(S[i:i + 1], *(f(t[i:i + 1]) for t in (*tok[:2], v, *tok[2:])), [0, 1], resume=[1],
                                            q_scale=128 ** -0.5)
            assert np.linalg.norm(f(y[i]) - y_ref[0]) <= 1e-4 * np.linalg.norm(y_ref)
        gate = f(z[:, CH + 2 * H:])
        close_e4m3(codes, scales, ref.gated(f(y).reshape(BATCH, -1), gate, f(layer.out_w), P, 1e-6, 0.0, True), 128)
    assert layer.state.get_error() == (0, -1)


def test_a_decode_step_in_a_graph(cuda_ok):
    """Two steps of the whole layer (an even number of calls of the context) captured, replayed, against eager ones.  A
    context that knows all counts picks a step's kernel by them, and a captured one would keep its choice; prompts between
    steps make the counts unknown, so that both sides run the same kernels and give the same bits."""
    eager, graphed = Layer(np.random.default_rng(6)), Layer(np.random.default_rng(6))
    r = np.random.default_rng(7)
    feed = [tuple(dev(values(r, BF, BATCH, HID), BF) for _ in range(4)) for _ in range(5)]
    fixed = tuple(t.clone() for t in feed[0])
    prompt, offsets = dev(values(r, BF, 40, HID), BF), dev(np.array([0, 20, 21, 40]), torch.int32)
    for side in (eager, graphed):  # (the projection's library handle is made before the capture, too)
        side.run(*(t.clone() for t in fixed[:2]))
        side.run(prompt, prompt.clone(), offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = [graphed.run(fixed[0], fixed[1]), graphed.run(fixed[2], fixed[3])]
    for d in feed:
        for t, new in zip(fixed, d):
            t.copy_(new)
        graph.replay()
        d = tuple(t.clone() for t in d)
        want = [eager.run(d[0], d[1]), eager.run(d[2], d[3])]
        for g, w in zip(out, want):
            assert torch.equal(g[3], w[3]) and torch.equal(g[4][0].view(torch.uint8), w[4][0].view(torch.uint8))
            assert torch.equal(g[4][1], w[4][1])
        assert torch.equal(fixed[1], d[1]) and torch.equal(fixed[3], d[3])
    del graph
