"""The chunk kernel of the gated delta rule: blocks that take heads and prompts in turn against blocks of one, waits that run
out, calls side by side, offsets past 32 bits (needs a B200).  Tolerances as in test_gpu_gdn_scan.py.
"""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi, gdn_scan
from test_gpu_gdn_scan import BF, F32, SCALE, TOK, compare, context, idx, make, on_gpu, packed, scan, tokens

pytestmark = pytest.mark.gpu


def same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), want.cpu().numpy())


@pytest.mark.parametrize("nseq,H,P", [(40, 6, 128), (64, 4, 40), (65, 4, 40)])
def test_units_in_turn_give_what_each_gives_alone(cuda_ok, nseq, H, P):
    """More heads of prompts than SMs: each block takes several, the longest prompts first up to 64 of them.  Among them empty
    prompts (fresh and resumed), a slot named twice, strong decays, values, keys and states that are not finite; everything
    is bit by bit what a call of that prompt alone gives, which has a block for each head."""
    r = np.random.default_rng(nseq)
    lens = r.integers(16, 230, nseq)
    lens[[3, 11, 20]] = 0
    offsets, batch = packed(lens), nseq + 3
    total = offsets[-1]
    assert 16 * nseq <= total <= 256 * nseq and nseq * H > torch.cuda.get_device_properties(0).multi_processor_count
    d = make(nseq, BF, total, H, 2, P, batch)
    slots = r.permutation(batch)[:nseq]
    slots[25] = slots[7]
    resume = r.integers(0, 2, nseq)
    resume[[3, 11, 20]] = [0, 1, 0]
    d["alpha"][offsets[5]:offsets[6], 1] = 1e-9
    for i, value in ((2, np.inf), (8, np.nan), (30, -np.inf)):
        d["v"][offsets[i] + 9, i % H, 3] = value
        d["k"][offsets[i + 1] + 12, 1, 5] = value
    d["alpha"][offsets[15] + 3, 0] = np.nan
    resume[33] = 1
    d["S"][slots[33], 1, 2, 7] = np.nan
    g = on_gpu(d, BF)
    start = g["S"].clone()
    y = torch.full((total, H, P), 7.0, device="cuda")
    scan(g, offsets, slots.tolist(), resume.tolist(), y)
    states = g["S"]
    named = set()
    for i in range(nseq):
        lo, hi, b = offsets[i], offsets[i + 1], slots[i]
        if i in (7, 25):  # refused
            assert (y[lo:hi] == 7.0).all()
            same(states[b], start[b])
            continue
        named.add(b)
        if lo == hi:
            same(states[b], start[b] if resume[i] else torch.zeros_like(start[b]))
            continue
        one = start[b:b + 1].clone()
        alone = gdn_scan(one, *(g[k][lo:hi] for k in TOK), idx([0, hi - lo]), None, idx([resume[i]], torch.uint8), q_scale=SCALE)
        same(y[lo:hi], alone)
        same(states[b], one[0])
    for b in set(range(batch)) - named:
        same(states[b], start[b])


def test_thousands_of_prompts_most_of_them_empty(cuda_ok):
    """5000 prompts (a block a head of each) and 4000 (in turn) with tokens in every 40th: states of the others become zero, or
    stay where they resume."""
    for nseq in (5000, 4000):
        lens = [0] * nseq
        for i in range(0, nseq, 40):
            lens[i] = 640 + i % 7
        offsets, some = packed(lens), list(range(0, nseq, 40))
        total = offsets[-1]
        assert 16 * nseq <= total <= 256 * nseq
        d = make(nseq, BF, 647, 2, 1, 8, 1)
        g = on_gpu(d, BF)
        rows = torch.cat([torch.arange(lens[i]) for i in some]).cuda()
        S = g["S"].expand(nseq, -1, -1, -1).clone()
        resume = [(i // 3) % 2 for i in range(nseq)]
        y = gdn_scan(S, *(g[k][rows] for k in TOK), idx(offsets), idx(list(range(nseq))[::-1]), idx(resume, torch.uint8),
                     q_scale=SCALE)
        for i in (some[0], some[1], some[63], some[-1]):
            compare({**d, **{k: d[k][:lens[i]] for k in TOK}}, [0, lens[i]], None, [resume[i]],
                    S[nseq - 1 - i:nseq - i].cpu().numpy(), y[offsets[i]:offsets[i + 1]].cpu().numpy())
        for i in range(1, nseq, 197):
            if lens[i] == 0:
                same(S[nseq - 1 - i], g["S"][0] if resume[i] else torch.zeros_like(g["S"][0]))


@pytest.mark.parametrize("lens,H", [((150, 250), 4), ((100,) * 45, 4)])
def test_a_load_that_never_comes_times_out_and_the_context_recovers(cuda_ok, monkeypatch, lens, H):
    """Every wait of the chunk kernel is bounded: with the second chunk's load withheld (and the bound shortened to about a
    millisecond) the launch ends, outputs and states are NaN, the context reports it, and after a reload it serves prompts
    again; blocks of one unit and of several."""
    offsets, n = packed(lens), len(lens)
    d = make(31, BF, offsets[-1], H, 2, 64, n)
    g = on_gpu(d, BF)
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, BF, n)
    monkeypatch.delenv("RSSM_WITHHOLD_TILE")
    monkeypatch.delenv("RSSM_WAIT_CYCLES")
    y = torch.full((offsets[-1], H, 64), 7.0, device="cuda")
    layer.gdn_prefill(*tokens(g), idx(offsets), y=y)
    code, seq = layer.get_error()
    assert code == abi.DEV_TIMEOUT and 0 <= seq < n
    assert torch.isnan(y).all() and torch.isnan(layer.export(ring=False)["S"]).all()
    layer.load_checkpoint(torch.from_numpy(d["S"]).cuda())
    y.fill_(7.0)
    layer.gdn_prefill(*tokens(g), idx(offsets), y=y)
    compare(d, offsets, None, None, layer.export(ring=False)["S"].cpu().numpy(), y.cpu().numpy())
    assert layer.get_error() == (0, -1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_calls_at_once(cuda_ok, dtype):
    """Calls on two streams, of their own states, with prompts that fill the machine: each is what it is alone."""
    lens = [(300, 40, 1, 77) * 5, (64, 65, 130, 5) * 6]
    work = []
    for i, ls in enumerate(lens):
        d = make(50 + i, dtype, sum(ls), 8, 4, 64, len(ls))
        g = on_gpu(d, dtype)
        want = scan(dict(g, S=(w := g["S"].clone())), packed(ls), resume=[1] * len(ls))
        work.append((g, packed(ls), want, w, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for g, off, _, _, stream in work:
            with torch.cuda.stream(stream):
                S = g["S"].clone()
                got.append((scan(dict(g, S=S), off, resume=[1] * (len(off) - 1)), S))
    torch.cuda.synchronize()
    for i, (y, S) in enumerate(got):
        same(y, work[i % 2][2])
        same(S, work[i % 2][3])


@pytest.mark.parametrize("dtype,H,total,nseq,n", [(BF, 16, 2 ** 21 + 1000, 1, 200), (F32, 16, 2 ** 21 + 1000, 1, 100),
                                                  (BF, 16, 2 ** 21 + 500, 2200, 4), (BF, 64, 40 * 600, 600, 40)])
def test_rows_past_32_bits(cuda_ok, dtype, H, total, nseq, n):
    """The last rows of inputs with more than 2^32 elements (or of states with more than 2^31 bytes), in the last sequence of
    many, in each of the kernels."""
    P = 128
    d = make(23, dtype, n, H, 16, P, 1)
    g = on_gpu(d, dtype)
    big = {k: torch.empty(total, *g[k].shape[1:], dtype=g[k].dtype, device="cuda") for k in TOK}
    if n * nseq == total:  # every prompt has tokens
        for k, t in big.items():
            t.view(nseq, n, *t.shape[1:])[:] = g[k]
        offsets = list(range(0, total + 1, n))
    else:
        for k, t in big.items():
            t[-n:] = g[k]
        offsets = [total - n] * nseq + [total]
    y = torch.empty(total, H, P, device="cuda")
    y[:-n].view(torch.int32)[-1000:] = 7
    S = torch.empty(nseq, H, P, 128, device="cuda")
    S[:] = g["S"][0]
    gdn_scan(S, *(big[k] for k in TOK), idx(offsets), None, idx([1] * nseq, torch.uint8), q_scale=SCALE, y=y)
    if n * nseq != total:
        assert (y[:-n].view(torch.int32)[-1000:] == 7).all()
        assert nseq == 1 or torch.equal(S[-2], g["S"][0])  # an empty prompt that resumes
    else:
        same(y[:n], y[-n:])
        same(S[0], S[-1])
    compare(d, [0, n], None, [1], S[-1:].cpu().numpy(), y[-n:].cpu().numpy())


@pytest.mark.parametrize("long", [5, 40, 99, 180])
def test_a_timeout_names_the_sequence_that_waited(cuda_ok, monkeypatch, long):
    """Blocks that take heads and prompts in turn, of which one prompt alone has a second chunk, which is not loaded: whatever the
    blocks have taken on in the meantime, behind it or to their ends, the context reports the slot of that prompt. Prompts of
    other blocks have their results."""
    n, H = 200, 4
    lens = [20] * n
    lens[long] = 100
    offsets = packed(lens)
    d = make(61, BF, offsets[-1], H, 2, 64, n)
    slots = [(i + n - long + 150) % n for i in range(n)]  # the long one's is 150; lower ones come before and behind it
    assert slots[long] == 150 and min(slots[long + 1:] + slots[:long]) == 0
    assert n * H > 4 * torch.cuda.get_device_properties(0).multi_processor_count and offsets[-1] <= 256 * n
    g = on_gpu(d, BF)
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, BF, n)
    monkeypatch.delenv("RSSM_WITHHOLD_TILE")
    monkeypatch.delenv("RSSM_WAIT_CYCLES")
    y = torch.full((offsets[-1], H, 64), 7.0, device="cuda")
    layer.gdn_prefill(*tokens(g), idx(offsets), idx(slots), y=y)
    assert layer.get_error() == (abi.DEV_TIMEOUT, 150)
    assert torch.isnan(y[offsets[long]:offsets[long + 1]]).all()
    want = scan(dict(g, S=g["S"].clone()), offsets)
    fine = torch.isfinite(y)
    assert fine.float().mean() > 0.9 and torch.equal(y[fine], want[fine])
