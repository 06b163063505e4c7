"""The short causal convolution against the float64 oracle (needs a B200).

Tolerance: at most five fp32 terms (below 2^-20 of their magnitudes, through SiLU's slope of at most 1.1 and its own
exp and division), then one rounding to the output type: half a step, finfo.eps / 2 of the value.
"""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import shortconv_commit, shortconv_prefill, shortconv_step, shortconv_verify
from oracle.prompts import ShortConvRing
from synth import round_to_dtype

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, seed, dtype, splits, K, batch, T=1, bias=True, silu=True):
        r = self.r = np.random.default_rng(seed)
        self.dtype, self.splits, self.K, self.silu = dtype, splits, K, silu
        self.ch = sum(splits)
        self.f = lambda a: round_to_dtype(a.astype(np.float32), "bf16" if dtype == BF else "f32")
        w, b = self.f(r.uniform(-.5, .5, (self.ch, K))), self.f(r.uniform(-.5, .5, self.ch)) if bias else None
        hist = self.f(r.standard_normal((batch, K - 1 + T, self.ch)))
        cur = r.integers(0, K - 1 + T, batch)
        self.orc = ShortConvRing(hist, cur, w, b, silu)
        self.mag = ShortConvRing(np.abs(hist), cur, np.abs(w), None if b is None else np.abs(b), False)
        self.hist, self.cur = self.dev(hist), torch.tensor(cur, dtype=torch.int32, device="cuda")
        self.w, self.b = self.dev(w), None if b is None else self.dev(b)
        self.kw = dict(splits=splits, activation="silu" if silu else None)

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(self.dtype)

    def rows(self, *lead):
        return self.f(self.r.standard_normal((*lead, self.ch)))

    def check(self, out, ref, mag):
        got = torch.cat([o.float() for o in out], -1).cpu().numpy()
        inside = np.isfinite(ref)
        bound = torch.finfo(self.dtype).eps / 2 * np.abs(ref) + 2.0 ** -20 * mag + 2.0 ** -126
        err = (np.abs(got - ref) / bound)[inside]
        assert err.max(initial=0.0) <= 1.0, f"{err.max():.2f} of the bound"
        return got

    def check_state(self):
        np.testing.assert_array_equal(self.hist.float().cpu().numpy(), self.orc.hist)
        np.testing.assert_array_equal(self.cur.cpu().numpy(), self.orc.cur)


def idx(v, t=torch.int32):
    return None if v is None else torch.tensor(v, dtype=t, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("splits", [(8,), (512, 128, 128), (1032, 40)])
def test_prompts(cuda_ok, dtype, K, splits):
    """Lengths below, at and above the filter's width and the tiles', empty ones, resumed and not."""
    lens = [1, 0, 2, 33, 32, 3, 100, 64, 0]
    offsets = np.concatenate([[2], 2 + np.cumsum(lens)]).tolist()
    slots, resume = [4, 9, 0, 7, 2, 10, 1, 5, 8], [1, 0, 1, 0, 1, 0, 1, 1, 1]
    c = Case(K, dtype, splits, K, 12, bias=K != 3, silu=K != 2)
    x = c.rows(offsets[-1] + 5)
    x[:2] = x[offsets[-1]:] = np.nan
    out = tuple(torch.full((len(x), n), 7.0, dtype=dtype, device="cuda") for n in splits)
    shortconv_prefill(c.hist, c.cur, c.dev(x), c.w, c.b, idx(offsets), idx(slots), idx(resume, torch.uint8), out=out, **c.kw)
    ref, mag = c.orc.prefill(x, offsets, slots, resume), c.mag.prefill(np.abs(x), offsets, slots, resume)
    got = c.check(out, ref, mag)
    assert (got[:2] == 7.0).all() and (got[offsets[-1]:] == 7.0).all()
    c.check_state()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,T,batch,splits", [(4, 1, 1, (8,)), (4, 8, 3, (512, 128, 128)), (3, 2, 5, (4096, 1024, 1024)),
                                              (2, 5, 2, (24, 16)), (4, 3, 160, (2048,))])
def test_decoding(cuda_ok, dtype, K, T, batch, splits):
    """Steps and committed prefixes of drafts, until the ring has wrapped."""
    c = Case(T, dtype, splits, K, batch, T)
    for rnd in range(4):
        x = c.rows(batch)
        c.check(shortconv_step(c.hist, c.cur, c.dev(x), c.w, c.b, **c.kw), c.orc.step(x), c.mag.step(np.abs(x)))
        x = c.rows(batch, T)
        c.check(shortconv_verify(c.hist, c.cur, c.dev(x), c.w, c.b, **c.kw), c.orc.verify(x), c.mag.verify(np.abs(x)))
        acc = c.r.integers(-1, T + 2, batch)  # clamped to what the ring can hold
        c.orc.commit(acc)
        c.mag.commit(acc)
        shortconv_commit(c.hist, c.cur, idx(acc), K)
        c.check_state()


def test_strided_rows(cuda_ok):
    """Inputs that are slices of a wider projection's rows."""
    c = Case(1, BF, (64, 32), 4, 3, 2)
    wide = c.dev(c.f(c.r.standard_normal((40, 160))))
    x = wide[:, 16:112]
    out = shortconv_prefill(c.hist, c.cur, x, c.w, c.b, idx([0, 10, 40]), **c.kw)
    xn = x.float().cpu().numpy()
    c.check(out, c.orc.prefill(xn, [0, 10, 40]), c.mag.prefill(np.abs(xn), [0, 10, 40]))
    x = wide[:6].view(3, 2, 160)[..., 16:112]
    xn = x.float().cpu().numpy()
    c.check(shortconv_verify(c.hist, c.cur, x, c.w, c.b, **c.kw), c.orc.verify(xn), c.mag.verify(np.abs(xn)))
    c.check_state()


def test_bad_prompts_write_nothing(cuda_ok):
    c = Case(2, BF, (64,), 4, 4)
    x = c.dev(c.rows(60))
    for offsets, slots in (([0, 40, 30, 60], None), ([0, 61], None), ([-2, 60], None), ([0, 30, 60], [1, 4])):
        out = (torch.full((60, 64), 7.0, dtype=BF, device="cuda"),)
        shortconv_prefill(c.hist, c.cur, x, c.w, c.b, idx(offsets), idx(slots), out=out, **c.kw)
        assert (out[0] == 7.0).all()
        c.check_state()
    out = (torch.full((60, 64), 7.0, dtype=BF, device="cuda"),)
    shortconv_prefill(c.hist, c.cur, x, c.w, c.b, idx([0, 20, 40, 60]), idx([3, 1, 3]), out=out, **c.kw)
    assert (out[0][:20] == 7.0).all() and (out[0][40:] == 7.0).all()
    xn = x.float().cpu().numpy()
    ref, mag = c.orc.prefill(xn, [20, 40], [1]), c.mag.prefill(np.abs(xn), [20, 40], [1])
    c.check((out[0],), ref, mag)
    c.check_state()


def test_infinities_stay_in_their_window(cuda_ok):
    """inf and NaN inputs reach the K outputs that see them and no others; silu(-inf side) is -0, not NaN."""
    c = Case(3, F32, (8,), 4, 1, bias=False)
    x = np.ones((20, 8), np.float32)
    x[5] = 3e38
    c.w.fill_(0.0)
    c.w[:, 3] = -1.0
    out, = shortconv_prefill(c.hist, c.cur, c.dev(x), c.w, None, idx([0, 20]), **c.kw)
    assert (out[5] == 0).all() and torch.isfinite(out).all()
    x[5] = np.nan
    c.w.fill_(0.25)
    out, = shortconv_prefill(c.hist, c.cur, c.dev(x), c.w, None, idx([0, 20]), **c.kw)
    assert torch.isnan(out[5:9]).all() and torch.isfinite(out[:5]).all() and torch.isfinite(out[9:]).all()


def test_rows_past_32_bits(cuda_ok):
    """The last rows of inputs with more than 2^32 elements."""
    c = Case(3, BF, (1024,), 4, 3, 2)
    n, total = 300, 2 ** 22 + 1000
    x = c.dev(c.rows(n))
    wide = torch.empty(total, 1024, dtype=BF, device="cuda")
    wide[-n:] = x
    out = (torch.empty(total, 1024, dtype=BF, device="cuda"),)
    shortconv_prefill(c.hist, c.cur, wide, c.w, c.b, idx([total - n, total]), idx([2]), out=out, **c.kw)
    xn = x.float().cpu().numpy()
    c.check((out[0][-n:],), c.orc.prefill(xn, [0, n], [2]), c.mag.prefill(np.abs(xn), [0, n], [2]))
    c.check_state()


def test_outputs_between_the_rows_of_their_input(cuda_ok):
    """Rows that lie apart leave room for outputs; those that meet a row are refused."""
    c = Case(4, BF, (64,), 4, 2, 2)
    wide = torch.zeros(2, 512, dtype=BF, device="cuda")
    x, out = wide[:, :64], wide[0, 64:192].view(2, 64)
    x.copy_(c.dev(c.rows(2)))
    xn = x.float().cpu().numpy()
    shortconv_step(c.hist, c.cur, x, c.w, c.b, out=(out,), **c.kw)
    c.check((out,), c.orc.step(xn), c.mag.step(np.abs(xn)))
    c.check_state()
    for bad in (wide[0, 56:184], wide.view(-1)[448:576]):
        with pytest.raises(RuntimeError, match="RSSM_ERR_ARG"):
            shortconv_step(c.hist, c.cur, x, c.w, c.b, out=(bad.view(2, 64),), **c.kw)
    c.check_state()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_silu_over_its_whole_range(cuda_ok, dtype):
    """act alone (taps 0, 0, 0, 1): to 2^-20 of its value, the rounding to the type apart.  fp32 down to where the result
    leaves the normal numbers (half a step of 2^-149 there, and one before the last product).  bf16 results below 2^-119
    may be 0: exp(-v) is beyond 2^126 only for v < -87.33, where |v| exp(v) <= 87.4 * 2^-126."""
    v = np.linspace(-96, 96, 20 * 8 * 64).astype(np.float32).reshape(-1, 8)
    c = Case(6, dtype, (8,), 4, 1, bias=False)
    v = c.f(v)
    c.w.copy_(torch.tensor([0.0, 0.0, 0.0, 1.0]))
    c.hist.zero_()
    out, = shortconv_prefill(c.hist, c.cur, c.dev(v), c.w, None, idx([0, len(v)]), **c.kw)
    v = v.astype(np.float64)
    ref = np.where(v < 0, v * np.exp(-np.abs(v)), v) / (1 + np.exp(-np.abs(v)))
    err = np.abs(out.double().cpu().numpy() - ref)
    bound = (2.0 ** -20 + (torch.finfo(BF).eps / 2 if dtype == BF else 0)) * np.abs(ref)
    bound += 2.0 ** -119 if dtype == BF else 2.0 ** -148
    assert (err / bound).max() <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_refused_prompts_in_new_outputs_are_nan(cuda_ok, dtype):
    """Where the call makes the outputs: all rows for a bad offset or slot, the prompts' own for a slot named twice."""
    c = Case(5, dtype, (64, 1032), 4, 4)
    x = c.dev(c.rows(300))
    for offsets, slots in (([0, 150, 100, 300], None), ([0, 301], None), ([-1, 300], None), ([0, 300], [4])):
        torch.full((300, 1032), 5.0, dtype=dtype, device="cuda")
        out = shortconv_prefill(c.hist, c.cur, x, c.w, c.b, idx(offsets), idx(slots), **c.kw)
        assert all(torch.isnan(o).all() for o in out), (offsets, slots)
        c.check_state()
    torch.full((300, 1032), 5.0, dtype=dtype, device="cuda")
    out = shortconv_prefill(c.hist, c.cur, x, c.w, c.b, idx([0, 100, 130, 300]), idx([3, 1, 3]), **c.kw)
    for o in out:
        assert torch.isnan(o[:100]).all() and torch.isnan(o[130:]).all()
    xn = x.float().cpu().numpy()
    ref, mag = c.orc.prefill(xn, [100, 130], [1]), c.mag.prefill(np.abs(xn), [100, 130], [1])
    c.check([o[100:130] for o in out], ref[100:130], mag[100:130])
    c.check_state()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_prompts_than_threads_of_a_block(cuda_ok, dtype):
    r = np.random.default_rng(7)
    lens = r.integers(0, 6, 300)
    offsets, slots = np.concatenate([[0], np.cumsum(lens)]).tolist(), r.permutation(310)[:300].tolist()
    resume = r.integers(0, 2, 300).tolist()
    c = Case(8, dtype, (64, 32), 4, 310)
    x = c.rows(offsets[-1])
    out = shortconv_prefill(c.hist, c.cur, c.dev(x), c.w, c.b, idx(offsets), idx(slots), idx(resume, torch.uint8), **c.kw)
    c.check(out, c.orc.prefill(x, offsets, slots, resume), c.mag.prefill(np.abs(x), offsets, slots, resume))
    c.check_state()
