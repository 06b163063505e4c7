"""Argument checks of the prompt, short-convolution and draft-verification calls, before any device work (no GPU)."""

import ctypes as C

import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi, accept_drafts, mamba2_scan, shortconv_prefill, shortconv_step, shortconv_verify
from hybrid_model_ssm_gdn_b200.build import build

ARG, SHAPE, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build()
    return abi.load()


def cfg(**kw):
    base = dict(kind=abi.MAMBA2, batch=4, nheads=4, headdim=64, dstate=128, ngroups=2, window=1, in_dtype=abi.BF16,
                A=16, D=16)
    base.update(kw)
    return abi.Config(**base)


def test_scan_refusals(lib):
    tok, p16 = abi.Tokens(x=16, B=16, C=16, dt=16), C.c_void_p(16)
    ok = dict(total=8, nseq=2, offsets=16)

    def scan(c=None, pr=None, tok=tok, S=p16, y=p16):
        pr = abi.Prompts(**{**ok, **(pr or {})})
        return lib.rssm_mamba2_scan(C.byref(c or cfg()), C.byref(pr), None if tok is None else C.byref(tok), S, y, None,
                                    0, None)

    assert lib.rssm_mamba2_scan(None, None, None, None, None, None, 0, None) == ARG
    assert lib.rssm_mamba2_scan(C.byref(cfg()), None, C.byref(tok), p16, p16, None, 0, None) == ARG
    assert scan(c=cfg(kind=abi.GDN, headdim=128, ngroups=1)) == UNSUPPORTED
    assert scan(c=cfg(dstate=64)) == SHAPE
    assert scan(c=cfg(headdim=72)) == SHAPE
    assert scan(c=cfg(ngroups=3)) == SHAPE
    assert scan(pr=dict(offsets=None)) == ARG
    assert scan(pr=dict(nseq=0)) == SHAPE
    assert scan(pr=dict(nseq=5)) == SHAPE           # more prompts than sequences
    assert scan(pr=dict(total=-1)) == SHAPE
    assert scan(pr=dict(total=2 ** 31 - 1)) == SHAPE
    assert scan(tok=None) == ARG
    assert scan(tok=abi.Tokens(x=16, B=16, C=None, dt=16)) == ARG
    assert scan(tok=abi.Tokens(x=24, B=16, C=16, dt=16)) == ARG
    assert scan(S=C.c_void_p(8)) == ARG
    assert scan(y=None) == ARG
    n = C.c_size_t()
    assert lib.rssm_mamba2_scan_workspace(C.byref(cfg()), 8, 9, C.byref(n)) == SHAPE
    assert lib.rssm_mamba2_scan_workspace(C.byref(cfg()), 8, 2, None) == ARG
    assert lib.rssm_mamba2_prefill(None, None, None, None, None, 0, None) == ARG


def conv(**kw):
    base = dict(batch=4, channels=64, width=4, ring=5, in_dtype=abi.BF16, silu=1, split=(C.c_int * 3)(32, 16, 16),
                weight=16, bias=16)
    base.update(kw)
    return abi.ShortConvConfig(**base)


def test_shortconv_refusals(lib):
    p16, out = C.c_void_p(16), (C.c_void_p * 3)(16, 16, 16)

    def step(c, hist=p16, cur=p16, x=p16, stride=64, out=out):
        return lib.rssm_shortconv_step(C.byref(c), hist, cur, x, stride, C.byref(out), None)

    assert lib.rssm_shortconv_step(None, p16, p16, p16, 64, C.byref(out), None) == ARG
    for bad in (dict(batch=0), dict(channels=60), dict(width=1), dict(width=5), dict(ring=3),
                dict(split=(C.c_int * 3)(32, 16, 8)), dict(split=(C.c_int * 3)(64, -8, 8)),
                dict(split=(C.c_int * 3)(0, 32, 32)), dict(split=(C.c_int * 3)(36, 12, 16))):
        assert step(conv(**bad)) == SHAPE, bad
    for bad in (dict(in_dtype=2), dict(weight=None), dict(weight=8), dict(bias=8)):
        assert step(conv(**bad)) == ARG, bad
    assert step(conv(), hist=None) == ARG
    assert step(conv(), cur=None) == ARG
    assert step(conv(), x=C.c_void_p(8)) == ARG
    assert step(conv(), out=(C.c_void_p * 3)(16, None, 16)) == ARG
    assert step(conv(), stride=56) == SHAPE
    assert step(conv(), stride=68) == SHAPE
    ver = lambda T, c: lib.rssm_shortconv_verify(C.byref(c), T, p16, p16, p16, 64, C.byref(out), None)  # noqa: E731
    assert ver(0, conv()) == ARG
    assert ver(3, conv()) == SHAPE                  # ring 5 holds 3 + 2 rows
    pr = abi.Prompts(8, 5, 16)
    assert lib.rssm_shortconv_prefill(C.byref(conv()), C.byref(pr), p16, p16, p16, 64, C.byref(out), None) == SHAPE
    assert lib.rssm_shortconv_prefill(C.byref(conv()), None, p16, p16, p16, 64, C.byref(out), None) == ARG
    assert lib.rssm_shortconv_commit(C.byref(conv()), None, p16, None) == ARG
    assert lib.rssm_shortconv_commit(C.byref(conv(ring=2)), p16, p16, None) == SHAPE


def test_size_and_overlap_refusals(lib):
    """More tokens than positions rounded up to tiles can count; convolution outputs that meet their inputs."""
    n = C.c_size_t()
    for total in (2 ** 30 + 1, 2 ** 31 - 1):
        assert lib.rssm_mamba2_scan_workspace(C.byref(cfg()), total, 1, C.byref(n)) == SHAPE
    base, row, stride = 1 << 20, 64 * 2, 96 * 2  # four rows of 64 bf16, 96 elements apart
    outs = lambda *p: (C.c_void_p * 3)(*p)  # noqa: E731
    far = 1 << 24
    for out in (outs(base, far, far), outs(far, base + 3 * stride, far), outs(far, far, base + 3 * stride + row - 16),
                outs(base - 16, far, far), outs(base + row, far, far)):
        assert lib.rssm_shortconv_step(C.byref(conv()), C.c_void_p(far), C.c_void_p(16), C.c_void_p(base), 96,
                                       C.byref(out), None) == ARG
    pr = abi.Prompts(4, 2, 16)
    assert lib.rssm_shortconv_prefill(C.byref(conv()), C.byref(pr), C.c_void_p(far), C.c_void_p(16), C.c_void_p(base), 96,
                                      C.byref(outs(base, far, far)), None) == ARG
    assert lib.rssm_shortconv_verify(C.byref(conv(ring=8)), 4, C.c_void_p(far), C.c_void_p(16), C.c_void_p(base), 96,
                                     C.byref(outs(far, base + 15 * stride, far)), None) == ARG


def test_accept_refusals(lib):
    p = C.c_void_p(16)

    def acc(batch=2, T=2, V=10, target=p, ldt=10, draft=p, ldd=10, tokens=p, u=p, a=p, nxt=p):
        return lib.rssm_accept_drafts(batch, T, V, target, ldt, draft, ldd, tokens, None, u, a, None, nxt, None)

    for bad in (dict(target=None), dict(tokens=None), dict(u=None), dict(a=None), dict(nxt=None)):
        assert acc(**bad) == ARG, bad
    for bad in (dict(batch=0), dict(T=-1), dict(T=17), dict(V=0), dict(ldt=9), dict(ldd=9)):
        assert acc(**bad) == SHAPE, bad


def test_binding_checks_shapes_and_devices():
    """Shapes and types are refused with ValueError, and tensors off the GPU before a pointer is taken from them."""
    t = torch.zeros
    S, x, B, dt = t(2, 4, 64, 128), t(9, 4, 64), t(9, 2, 128), t(9, 4)
    A, D, off = t(4), t(4), t(3, dtype=torch.int32)
    for bad in (dict(S=t(2, 4, 64, 64)), dict(x=t(9, 64)), dict(A=t(3)), dict(x=x.half())):
        a = dict(S=S, x=x, B=B, C_=B, dt=dt, A=A, D=D, offsets=off)
        a.update(bad)
        with pytest.raises(ValueError):
            mamba2_scan(**a)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        mamba2_scan(S, x, B, B, dt, A, D, off)
    hist, cur, w, xr = t(2, 4, 64), t(2, dtype=torch.int32), t(64, 4), t(2, 64)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        shortconv_step(hist, cur, xr, w)
    with pytest.raises(ValueError, match="dimensions"):
        shortconv_step(hist[0], cur, xr, w)
    with pytest.raises(ValueError, match="3 dimensions"):
        shortconv_verify(hist, cur, xr, w)
    with pytest.raises(ValueError):
        shortconv_prefill(hist, cur, xr, w, None, off)
    with pytest.raises(ValueError, match="target"):
        accept_drafts(t(2, 3, 10), t(2, 2, dtype=torch.int32), t(2, 3))
    with pytest.raises(ValueError, match="3 dimensions"):
        accept_drafts(t(2, 10), t(2, 2, dtype=torch.int32), t(2, 3))
