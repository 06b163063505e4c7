"""Argument checks of the gated-delta-rule prompts and of the calls between a layer's projections, before any device work
(no GPU)."""

import ctypes as C

import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi, add_rmsnorm, gated_rmsnorm, gdn_inputs, gdn_scan
from hybrid_model_ssm_gdn_b200.build import build

ARG, SHAPE, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build()
    return abi.load()


def cfg(**kw):
    base = dict(kind=abi.GDN, batch=4, nheads=4, headdim=128, dstate=128, ngroups=1, window=1, in_dtype=abi.BF16,
                q_scale=1.0)
    base.update(kw)
    return abi.Config(**base)


def test_gdn_scan_refusals(lib):
    tok, p16 = abi.Tokens(q=16, k=16, v=16, alpha=16, beta=16), C.c_void_p(16)
    ok = dict(total=8, nseq=2, offsets=16)

    def scan(c=None, hk=4, pr=None, tok=tok, S=p16, y=p16):
        pr = abi.Prompts(**{**ok, **(pr or {})})
        return lib.rssm_gdn_scan(C.byref(c or cfg()), hk, C.byref(pr), None if tok is None else C.byref(tok), S, y, None, 0,
                                 None)

    assert lib.rssm_gdn_scan(None, 4, None, None, None, None, None, 0, None) == ARG
    assert lib.rssm_gdn_scan(C.byref(cfg()), 4, None, C.byref(tok), p16, p16, None, 0, None) == ARG
    assert scan(c=cfg(kind=abi.MAMBA2, headdim=64, A=16, D=16)) == UNSUPPORTED
    for bad in (dict(dstate=64), dict(headdim=136), dict(headdim=20), dict(ngroups=2), dict(batch=0), dict(nheads=65536)):
        assert scan(c=cfg(**bad), hk=1) == SHAPE, bad
    for hk in (0, -1, 3, 8):
        assert scan(hk=hk) == SHAPE
    assert scan(pr=dict(offsets=None)) == ARG
    for bad in (dict(nseq=0), dict(nseq=5), dict(total=-1), dict(total=2 ** 30 + 1)):
        assert scan(pr=bad) == SHAPE, bad
    assert scan(c=cfg(batch=2 ** 20, nheads=4096), pr=dict(nseq=2 ** 20)) == SHAPE
    assert scan(tok=None) == ARG
    for name in ("q", "k", "v", "alpha", "beta"):
        assert scan(tok=abi.Tokens(**{**dict(q=16, k=16, v=16, alpha=16, beta=16), name: None})) == ARG
    for name in ("q", "k", "v"):
        assert scan(tok=abi.Tokens(**{**dict(q=16, k=16, v=16, alpha=16, beta=16), name: 24})) == ARG
    assert scan(S=C.c_void_p(8)) == ARG
    assert scan(y=None) == ARG
    n = C.c_size_t()
    assert lib.rssm_gdn_scan_workspace(C.byref(cfg()), 8, 5, C.byref(n)) == SHAPE
    assert lib.rssm_gdn_scan_workspace(C.byref(cfg()), 8, 2, None) == ARG
    assert lib.rssm_gdn_scan_workspace(C.byref(cfg(kind=abi.MAMBA2, headdim=64, A=16, D=16)), 8, 2, C.byref(n)) == UNSUPPORTED
    assert lib.rssm_gdn_prefill(None, 4, None, None, None, None, 0, None) == ARG


def test_gdn_inputs_refusals(lib):
    p = C.c_void_p(16)
    base = dict(rows=3, nheads=4, qk_heads=2, out_heads=2, in_dtype=abi.BF16, eps=1e-6, q=16, k=16, a=2, b=2, q_stride=256,
                k_stride=256, a_stride=4, b_stride=4, A_log=4, bias=4)

    def call(q_out=p, alpha=p, **kw):
        return lib.rssm_gdn_inputs(C.byref(abi.GdnInputsConfig(**{**base, **kw})), q_out, p, alpha, p, None)

    assert lib.rssm_gdn_inputs(None, p, p, p, p, None) == ARG
    for bad in (dict(in_dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None), dict(k=None), dict(a=None),
                dict(b=None), dict(A_log=None), dict(bias=None), dict(q=24), dict(k=8), dict(q_out=None),
                dict(q_out=C.c_void_p(8)), dict(alpha=None)):
        assert call(**bad) == ARG, bad
    for bad in (dict(rows=-1), dict(nheads=0), dict(qk_heads=0), dict(qk_heads=3), dict(out_heads=3), dict(out_heads=1),
                dict(q_stride=248), dict(k_stride=260), dict(a_stride=3), dict(b_stride=0),
                dict(rows=1 << 30, qk_heads=64, out_heads=64, nheads=64)):
        assert call(**bad) == SHAPE, bad
    assert call(rows=0, q=None, q_out=None) == 0


def test_norm_refusals(lib):
    p = C.c_void_p(16)
    base = dict(rows=3, columns=64, group=64, weight_columns=64, x_dtype=1, gate_dtype=1, weight_dtype=1, out_dtype=1,
                scale=0, norm_first=1, eps=1e-6, offset=0.0)

    def add(x=p, xs=64, r=p, rs=64, w=p, out=p, s=None, **kw):
        return lib.rssm_add_rmsnorm(C.byref(abi.NormConfig(**{**base, **kw})), x, xs, r, rs, w, out, s, None)

    def gate(x=p, xs=64, z=p, zs=64, w=p, out=p, s=None, **kw):
        return lib.rssm_gated_rmsnorm(C.byref(abi.NormConfig(**{**base, **kw})), x, xs, z, zs, w, out, s, None)

    assert lib.rssm_add_rmsnorm(None, p, 64, p, 64, p, p, None, None) == ARG
    assert lib.rssm_gated_rmsnorm(None, p, 64, p, 64, p, p, None, None) == ARG
    for f in (add, gate):
        for bad in (dict(x_dtype=2), dict(weight_dtype=-1), dict(out_dtype=2), dict(scale=3), dict(eps=-1e-9), dict(x=None),
                    dict(w=None), dict(out=None), dict(x=C.c_void_p(8)), dict(w=C.c_void_p(4)), dict(out=C.c_void_p(24)),
                    dict(scale=1), dict(scale=2)):
            assert f(**bad) == ARG, bad
        for bad in (dict(rows=-1), dict(columns=60, group=60, weight_columns=60), dict(columns=0), dict(columns=32776),
                    dict(group=24), dict(group=4), dict(group=0), dict(weight_columns=32), dict(xs=56), dict(xs=68)):
            assert f(**bad) == SHAPE, bad
        assert f(rows=0, x=None, out=None) == 0
    assert add(group=32) == SHAPE
    assert add(rs=60) == SHAPE and add(r=C.c_void_p(8)) == ARG
    assert gate(gate_dtype=2) == ARG and gate(z=None) == ARG and gate(z=C.c_void_p(8)) == ARG and gate(zs=63) == SHAPE


def test_outputs_that_meet_inputs_are_refused(lib):
    """Rows are read ahead of the outputs before them: no output may lie over an input or another output.  Every call here is
    one that is refused, at addresses that nobody reads."""
    M = 1 << 24
    at = dict(x=M, r=2 * M, w=3 * M, out=4 * M, s=5 * M)
    base = dict(rows=3, columns=64, group=64, weight_columns=64, x_dtype=1, gate_dtype=1, weight_dtype=1, out_dtype=1,
                scale=0, norm_first=1, eps=1e-6, offset=0.0)

    def call(f, xs=64, rs=64, scale=0, **kw):
        p = {k: C.c_void_p(v) for k, v in {**at, **kw}.items()}
        return f(C.byref(abi.NormConfig(**{**base, "scale": scale})), p["x"], xs, p["r"], rs, p["w"], p["out"], p["s"], None)

    for f in (lib.rssm_add_rmsnorm, lib.rssm_gated_rmsnorm):
        for name in ("x", "r", "w"):
            assert call(f, out=at[name]) == ARG and call(f, out=at[name] - 3 * 128 + 16) == ARG
        assert call(f, out=M + 2 * 128) == ARG  # the last row of x
        assert call(f, xs=1024, out=M + 2 * 2048 + 112) == ARG
        assert call(f, scale=1, s=M) == ARG and call(f, scale=2, s=4 * M + 128) == ARG and call(f, scale=1, out=2 * M + 256) == ARG
    for r, xs, rs in ((M + 128, 64, 64), (M - 16, 64, 64), (M + 64, 128, 128), (M, 64, 128), (M - 64, 128, 128), (M + 256, 64, 72)):
        assert call(lib.rssm_add_rmsnorm, r=r, xs=xs, rs=rs) == ARG, (r, xs, rs)

    cfg_ = dict(rows=3, nheads=4, qk_heads=2, out_heads=2, in_dtype=abi.BF16, eps=1e-6, q=M, k=2 * M, a=3 * M, b=4 * M,
                q_stride=256, k_stride=256, a_stride=4, b_stride=4, A_log=9 * M, bias=10 * M)
    for i in range(4):
        for where in (M, M + 2 * 512, 2 * M, 2 * M + 3 * 512 - 16, 3 * M + 16, 4 * M, *(m * M for m in (5, 6, 7, 8) if m != 5 + i)):
            outs = [5 * M, 6 * M, 7 * M, 8 * M]
            outs[i] = where
            assert lib.rssm_gdn_inputs(C.byref(abi.GdnInputsConfig(**cfg_)), *map(C.c_void_p, outs), None) == ARG, (i, where)


def test_inputs_of_more_blocks_than_a_launch_has_are_refused(lib):
    """Rows and heads whose blocks, as the launch is cut (64 / qk_heads rows of vectors, 1024 / nheads of gates, at least one),
    pass 2^31 - 1."""
    p, most = C.c_void_p(16), 1 << 30
    for hk, h in ((64, 64), (33, 33), (40, 1200), (50, 65500)):
        blocks = 2 * -(-most // max(1, 64 // hk)) + -(-most // max(1, 1024 // h))
        c = abi.GdnInputsConfig(rows=most, nheads=h, qk_heads=hk, out_heads=hk, in_dtype=abi.BF16, eps=1e-6, q=16, k=16, a=2, b=2,
                                q_stride=128 * hk, k_stride=128 * hk, a_stride=h, b_stride=h, A_log=4, bias=4)
        assert blocks > 2 ** 31 - 1 and lib.rssm_gdn_inputs(C.byref(c), p, p, p, p, None) == SHAPE, (hk, h)


def test_outputs_over_parameters_are_refused(lib):
    """A_log and bias under each output of the inputs, and the weight under the residual, whose h goes back while other rows
    read it; at addresses that nobody reads, as above."""
    M = 1 << 24
    cfg_ = dict(rows=3, nheads=4, qk_heads=2, out_heads=2, in_dtype=abi.BF16, eps=1e-6, q=M, k=2 * M, a=3 * M, b=4 * M,
                q_stride=256, k_stride=256, a_stride=4, b_stride=4, A_log=9 * M, bias=10 * M)
    for i in range(4):
        size = 3 * 512 if i < 2 else 48  # bytes of the output
        for at in (9 * M, 10 * M):
            for where in (at, at - size + 16):
                outs = [5 * M, 6 * M, 7 * M, 8 * M]
                outs[i] = where
                assert lib.rssm_gdn_inputs(C.byref(abi.GdnInputsConfig(**cfg_)), *map(C.c_void_p, outs), None) == ARG, (i, where)

    for dtype, esz in ((abi.BF16, 2), (abi.F32, 4)):
        base = dict(rows=3, columns=64, group=64, weight_columns=64, x_dtype=abi.BF16, weight_dtype=dtype, out_dtype=abi.BF16,
                    eps=1e-6)

        def add(r, rs, w):
            return lib.rssm_add_rmsnorm(C.byref(abi.NormConfig(**base)), M, 64, r, rs, w, 4 * M, None, None)

        for rs in (64, 72, 1024):
            for w in (2 * M, 2 * M + 2 * rs * 2, 2 * M + 2 * rs * 2 + 112, 2 * M - 64 * esz + 16):
                assert add(2 * M, rs, w) == ARG, (rs, w - 2 * M)


def test_binding_checks_shapes_and_devices():
    """Shapes and types are refused with ValueError, and tensors off the GPU before a pointer is taken from them."""
    t = torch.zeros
    args = dict(S=t(2, 4, 64, 128), q=t(9, 2, 128), k=t(9, 2, 128), v=t(9, 4, 64), alpha=t(9, 4), beta=t(9, 4),
                offsets=t(3, dtype=torch.int32))
    for bad in (dict(), dict(S=t(2, 4, 64)), dict(v=t(9, 64)), dict(v=t(9, 4, 64).half())):
        with pytest.raises(ValueError):
            gdn_scan(**{**args, **bad})
    q, a, w = t(3, 2, 128), t(3, 4), t(4)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        gdn_inputs(q, q, a, a, w, w)
    with pytest.raises(ValueError, match="dimensions"):
        gdn_inputs(w, w, a, a, w, w)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        add_rmsnorm(t(3, 64).half(), t(64))
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        add_rmsnorm(t(3, 64), t(64))
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        gated_rmsnorm(t(3, 64), t(3, 64), t(64))
