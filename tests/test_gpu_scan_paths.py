"""Paths of the prompt scan that depend on lengths, sizes and waits, against the float64 oracle (needs a B200)."""

import ctypes as C

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi, make_config, mamba2_scan
from test_gpu_scan import SHAPES, compare, context, idx, make, on_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def packed(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def workspace(H, P, G, total, nseq):
    """Bytes of scratch for prompts of this size: more than 0 where they are cut into pieces."""
    cfg = make_config("mamba2", nseq, H, P, 128, G, 1, 0, BF, A=torch.empty(H), D=torch.empty(H))
    n = C.c_size_t()
    assert abi.load().rssm_mamba2_scan_workspace(C.byref(cfg), total, nseq, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("withheld", [1, 3])
@pytest.mark.parametrize("H,P,G,lens,cut", [(4, 64, 1, (790, 610), False), (64, 8, 1, (3900,), True)])
def test_a_load_missing_from_long_prompts_ends_and_recovers(cuda_ok, monkeypatch, H, P, G, lens, cut, withheld):
    """One chunk's load withheld with several behind it: the block asks for no more, ends within the bound of its waits
    and leaves NaN, and the launches after it give the oracle's values."""
    offsets = packed(lens)
    total = offsets[-1]
    assert (workspace(H, P, G, total, len(lens)) > 0) == cut
    d = make(31, BF, total, H, P, G, len(lens), decay=0.05)
    g = on_gpu(d, BF)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", str(withheld))
    layer = context(d, BF, len(lens))
    monkeypatch.delenv("RSSM_WITHHOLD_TILE")
    monkeypatch.delenv("RSSM_WAIT_CYCLES")
    y = torch.full((total, H, P), 7.0, device="cuda")
    layer.prefill(*tok, idx(offsets), y=y)
    assert layer.get_error()[0] == abi.DEV_TIMEOUT
    assert torch.isnan(y).all() and torch.isnan(layer.export(ring=False)["S"]).all()
    layer.load_checkpoint(g["S"])
    y.fill_(7.0)
    layer.prefill(*tok, idx(offsets), y=y)
    assert layer.get_error() == (0, -1)
    compare(d, offsets, None, None, layer.export(ring=False)["S"].cpu().numpy(), y.cpu().numpy())


def test_a_timeout_names_the_sequence(cuda_ok, monkeypatch):
    """With slots, the index reported is the slot of a prompt that gave up, as for every other code."""
    d = make(32, BF, 400, 4, 64, 2, 6)
    g = on_gpu(d, BF)
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, BF, 6)
    layer.prefill(g["x"], g["B"], g["C"], g["dt"], idx([0, 150, 400]), idx([5, 3]))
    assert layer.get_error() == (abi.DEV_TIMEOUT, 3)  # both gave up: the lowest
    S = layer.export(ring=False)["S"]
    assert torch.isnan(S[[3, 5]]).all() and torch.equal(S[[0, 1, 2, 4]], g["S"][[0, 1, 2, 4]])


def test_refused_prompts_leave_the_counts_known(cuda_ok):
    """A prefill that the device refuses (prompts that resume on buffered records; a bad offset) changes nothing, so the
    steps after it, the fold among them, give the bits of a context that never saw the call."""
    batch, H, P, G = 3, 4, 64, 2
    d = make(33, BF, 12 * batch, H, P, G, batch)
    g = on_gpu(d, BF)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    plain, refused, bad = (context(d, BF, batch) for _ in range(3))
    for t in range(12):  # a window of 8: one fold
        if t == 5:
            refused.prefill(*tok, idx([0, 9, 10, 36]), resume=idx([1, 1, 1], torch.uint8))
            assert refused.get_error() == (abi.DEV_BUFFERED, 0)
            bad.prefill(*tok, idx([0, 9, 10, 37]))
            assert bad.get_error() == (abi.DEV_PROMPT, 2)
        now = tuple(v[t * batch:(t + 1) * batch].contiguous() for v in tok)
        ys = [layer.mamba2_step(*now) for layer in (plain, refused, bad)]
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2]), t
    a, b, c = (layer.export(ring=False) for layer in (plain, refused, bad))
    for e in (b, c):
        assert torch.equal(a["S"], e["S"]) and torch.equal(a["meta"], e["meta"])


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("H,P,G,lens,cut", [(4, 64, 2, (40, 1, 23), False), (3, 24, 1, (33, 16), False),
                                            (4, 64, 2, (300, 1, 260), False), (3, 40, 1, (128, 400), False),
                                            (2, 64, 1, (1900,), True), (64, 8, 1, (3900,), True)])
def test_values_that_are_not_finite_reach_no_earlier_token(cuda_ok, H, P, G, lens, cut, value):
    """From a value of x that is not finite on, its head's row p has no finite outputs and no finite state; everything
    else, the same row before it above all, keeps its bits."""
    offsets = packed(lens)
    total, n = offsets[-1], len(lens)
    assert (workspace(H, P, G, total, n) > 0) == cut
    d = make(34, BF, total, H, P, G, n, decay=0.2)
    g = on_gpu(d, BF)
    r = np.random.default_rng(35)
    at = {(total - 1, 0, 1), (offsets[1] - 1, H - 1, P - 1), (0, 0, 0)}
    at |= {(int(r.integers(total)), int(r.integers(H)), int(r.integers(P))) for _ in range(6)}
    hit_y = torch.zeros(total, H, P, dtype=torch.bool, device="cuda")
    hit_S = torch.zeros(n, H, P, dtype=torch.bool, device="cuda")
    x = g["x"].clone()
    for t, h, p in at:
        i = int(np.searchsorted(offsets, t, side="right")) - 1
        x[t, h, p] = value
        hit_y[t:offsets[i + 1], h, p] = True
        hit_S[i, h, p] = True
    got = []
    for xs in (g["x"], x):
        S = g["S"].clone()
        y = mamba2_scan(S, xs, g["B"], g["C"], g["dt"], g["A"], g["D"], idx(offsets), resume=idx([1] * n, torch.uint8))
        got.append((S, y))
    (S0, y0), (S1, y1) = got
    assert torch.isfinite(y0).all() and torch.isfinite(S0).all()
    assert torch.equal(y0[~hit_y], y1[~hit_y]) and torch.equal(S0[~hit_S], S1[~hit_S])
    assert not torch.isfinite(y1[hit_y]).any() and not torch.isfinite(S1[hit_S]).any()


@pytest.mark.parametrize("key", ["B", "C", "dt"])
@pytest.mark.parametrize("lens", [(40, 1, 23), (300, 1, 260)])
def test_other_inputs_that_are_not_finite_reach_no_earlier_token(cuda_ok, lens, key):
    """NaN and infinities in B, C or dt: tokens before theirs and other prompts keep their bits, with C all others do."""
    offsets = packed(lens)
    total, n = offsets[-1], len(lens)
    d = make(38, BF, total, 4, 64, 2, n)
    g = on_gpu(d, BF)
    for value in (np.nan, np.inf):
        for t in (offsets[1] - 10, offsets[1], total - 1, offsets[2] + 17):
            bad = {k: v.clone() for k, v in g.items()}
            bad[key][t, 0, ...] = value  # the first group's heads, or the first head
            got = []
            for e in (g, bad):
                S = e["S"].clone()
                y = mamba2_scan(S, e["x"], e["B"], e["C"], e["dt"], e["A"], e["D"], idx(offsets),
                                resume=idx([1] * n, torch.uint8))
                got.append((S, y))
            (S0, y0), (S1, y1) = got
            i = int(np.searchsorted(offsets, t, side="right")) - 1
            heads = 1 if key == "dt" else 2
            hit = torch.zeros_like(y0, dtype=torch.bool)
            hit[t:(t + 1 if key == "C" else offsets[i + 1]), :heads] = True
            assert torch.equal(y0[~hit], y1[~hit])
            assert not torch.isfinite(y1[t, :heads]).any()
            others = [s for s in range(n) if s != i]
            assert torch.equal(S0[others], S1[others])
            assert torch.equal(S0, S1) if key == "C" else not torch.isfinite(S1[i, :heads]).any()


def stale(*shape, dtype=torch.float32):
    """Leave memory that looks like results where the next tensor of this size will lie."""
    torch.full(shape, 5.0, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("H,total", [(2, 90), (3, 260), (2, 2100)])
def test_refused_prompts_in_new_outputs_are_nan(cuda_ok, dtype, H, total):
    """Where the call makes the outputs, rows of prompts that it refuses are NaN: all of them for a bad offset or slot,
    those of the prompts themselves for a slot named twice.  Each kernel, prompts cut into pieces among them."""
    P, a, b = 40, total // 3, total // 2
    d = make(36, dtype, total, H, P, 1, 4, decay=0.1)
    g = on_gpu(d, dtype)
    args = (g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"])
    for offsets, slots in (([0, b, a, total], None), ([0, total + 1], None), ([-1, total], None), ([0, total], [4]),
                           ([0, a, total], [0, -1])):
        stale(total, H, P)
        y = mamba2_scan(g["S"], *args, idx(offsets), idx(slots))
        assert torch.isnan(y).all(), (offsets, slots)
        assert np.array_equal(g["S"].cpu().numpy(), d["S"])
    stale(total, H, P)
    y = mamba2_scan(g["S"], *args, idx([0, a, b, total]), idx([2, 1, 2]))
    assert torch.isnan(y[:a]).all() and torch.isfinite(y[a:b]).all() and torch.isnan(y[b:]).all()
    S = g["S"].cpu().numpy()
    assert all(np.array_equal(S[i], d["S"][i]) for i in (0, 2, 3))


def test_refused_prompts_of_a_context_are_nan(cuda_ok):
    """Prompts that resume on buffered records, and a slot named twice, in outputs that the call makes."""
    d = make(37, BF, 300, 4, 64, 2, 4)
    g = on_gpu(d, BF)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    layer = context(d, BF, 4)
    layer.mamba2_step(*(v[:4].contiguous() for v in tok))
    stale(300, 4, 64)
    y = layer.prefill(*tok, idx([0, 100, 120, 300]), idx([3, 0, 1]), idx([1, 0, 1], torch.uint8))
    assert layer.get_error() == (abi.DEV_BUFFERED, 1)
    assert torch.isnan(y[:100]).all() and torch.isfinite(y[100:120]).all() and torch.isnan(y[120:]).all()
    stale(300, 4, 64)
    y = layer.prefill(*tok, idx([0, 100, 120, 300]), idx([2, 0, 2]))
    assert torch.isnan(y[:100]).all() and torch.isfinite(y[100:120]).all() and torch.isnan(y[120:]).all()


def check_prompts(d, dtype, lens, slots, resume):
    offsets = packed(lens)
    g = on_gpu(d, dtype)
    y = torch.full(d["x"].shape, 7.0, device="cuda")
    mamba2_scan(g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], idx(offsets), idx(slots), idx(resume, torch.uint8),
                y=y)
    compare(d, offsets, slots, resume, g["S"].cpu().numpy(), y.cpu().numpy())


@pytest.mark.parametrize("H,P,G", SHAPES)
def test_mixed_lengths_above_the_short_kernel(cuda_ok, H, P, G):
    """Empty (from zero and resumed), single-token, tile-sized and long prompts that average more than 80 tokens, so that
    chunks of 128 take them: odd heads, several groups, every height of X."""
    lens = [1, 0, 130, 127, 300, 128, 0, 257, 3]
    assert sum(lens) > 80 * len(lens) and workspace(H, P, G, sum(lens), len(lens)) == 0
    d = make(H * 1000 + P, BF, sum(lens), H, P, G, 12)
    check_prompts(d, BF, lens, [4, 9, 0, 7, 2, 10, 1, 5, 11], [0, 0, 1, 0, 1, 1, 1, 0, 1])


@pytest.mark.parametrize("H,P,G,lens", [(3, 40, 1, (700, 0, 1400, 390, 800, 5)), (2, 8, 1, (130, 900))])
def test_uneven_long_prompts_handed_out_by_length(cuda_ok, H, P, G, lens):
    """Whole prompts of 512 tokens or more on average go to the blocks longest first."""
    n = len(lens)
    assert sum(lens) >= 512 * n and workspace(H, P, G, sum(lens), n) == 0
    d = make(41, BF, sum(lens), H, P, G, n + 2, decay=0.1)
    r = np.random.default_rng(42)
    check_prompts(d, BF, lens, r.permutation(n + 2)[:n].tolist(), [i % 3 != 1 for i in range(n)])


@pytest.mark.parametrize("n", [64, 65])
def test_the_number_of_prompts_handed_out_by_length(cuda_ok, n):
    """As many prompts as are sorted, and one more: each repeats one of two, so that two runs of the oracle cover them."""
    lens = [300 + 500 * (i % 2) for i in range(n)]
    d = make(43, BF, 800, 1, 8, 1, 1, decay=0.1)
    g = on_gpu(d, BF)
    x, B, C, dt = (torch.cat([g[k][:m] for m in lens]) for k in ("x", "B", "C", "dt"))
    assert workspace(1, 8, 1, sum(lens), n) == 0
    S = torch.zeros(n, 1, 8, 128, device="cuda")
    y = mamba2_scan(S, x, B, C, dt, g["A"], g["D"], idx(packed(lens)))
    off = packed(lens)
    for i in range(2):
        compare({**d, **{k: d[k][:lens[i]] for k in ("x", "B", "C", "dt")}}, [0, lens[i]], None, None,
                S[i:i + 1].cpu().numpy(), y[off[i]:off[i + 1]].cpu().numpy())
    for i in range(2, n):
        assert torch.equal(y[off[i]:off[i + 1]], y[off[i % 2]:off[i % 2 + 1]]) and torch.equal(S[i], S[i % 2])


@pytest.mark.parametrize("dtype,each,n", [(BF, 85, 700), (BF, 40, 300), (torch.float32, 20, 300)])
def test_more_prompts_than_threads_of_a_block(cuda_ok, dtype, each, n):
    """Every block looks through more prompts than it has threads; all prompts are the same, to slots in reverse."""
    d = make(44, dtype, each, 2, 16, 1, 1)
    g = on_gpu(d, dtype)
    x, B, C, dt = (g[k].repeat(n, *[1] * (g[k].dim() - 1)) for k in ("x", "B", "C", "dt"))
    S = g["S"].repeat(n + 1, 1, 1, 1)
    y = mamba2_scan(S, x, B, C, dt, g["A"], g["D"], idx(packed([each] * n)), idx(list(range(n, 0, -1))),
                    idx([1] * n, torch.uint8)).view(n, each, 2, 16)
    compare(d, [0, each], None, [1], S[1:2].cpu().numpy(), y[0].cpu().numpy())
    assert (y == y[:1]).all() and (S[1:] == S[1:2]).all() and torch.equal(S[0], g["S"][0])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lens", [[700] + [1] * 20, [1] * 9 + [400]])
def test_one_long_prompt_among_single_tokens(cuda_ok, dtype, lens):
    d = make(45, dtype, sum(lens), 4, 64, 2, len(lens), decay=0.2)
    check_prompts(d, dtype, lens, None, [i % 2 for i in range(len(lens))])


def test_prefill_captured(cuda_ok):
    """Two calls of a context's prefill (an even number keeps its bookkeeping in place) in a graph, replayed on new
    prompts while another sequence goes on decoding between the replays."""
    batch, H, P, G = 3, 4, 64, 2
    d = make(46, BF, 300, H, P, G, batch)
    g = on_gpu(d, BF)
    layer, eager = context(d, BF, batch), context(d, BF, batch)
    tok = tuple(g[k].clone() for k in ("x", "B", "C", "dt"))
    first, second = (idx([0, 90]), idx([1])), (idx([90, 300]), idx([1]), idx([1], torch.uint8))
    y = torch.empty(300, H, P, device="cuda")

    def prompt(layer, tok, y):
        layer.prefill(*tok, *first, y=y)
        layer.prefill(*tok, *second, y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        prompt(layer, tok, y)
    for seed in (47, 48, 49):
        new = on_gpu(make(seed, BF, 300, H, P, G, batch), BF)
        for t, k in zip(tok, ("x", "B", "C", "dt")):
            t.copy_(new[k])
        graph.replay()
        y2 = torch.empty_like(y)
        prompt(eager, tok, y2)
        assert torch.equal(y, y2)
        for _ in range(2):
            now = tuple(t[:batch].contiguous() for t in tok)
            assert torch.equal(layer.mamba2_step(*now), eager.mamba2_step(*now))
    a, b = layer.export(ring=False), eager.export(ring=False)
    assert torch.equal(a["S"], b["S"]) and torch.equal(a["meta"], b["meta"])
    assert layer.get_error() == (0, -1)
    del graph


def test_cut_prompts_on_two_streams(cuda_ok):
    """Prompts that are cut into pieces, at once on two streams, each call with scratch of its own."""
    H, P, G, total = 8, 64, 1, 3000
    assert workspace(H, P, G, total, 1) > 0
    gs = [on_gpu(make(50 + i, BF, total, H, P, G, 1, decay=0.1), BF) for i in range(2)]

    def run(g):
        S = g["S"].clone()
        return S, mamba2_scan(S, g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], idx([0, total]),
                              resume=idx([1], torch.uint8))

    want = [run(g) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for g, st in zip(gs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(g))
        torch.cuda.synchronize()
        for (S, y), (S0, y0) in zip(got, want):
            assert torch.equal(S, S0) and torch.equal(y, y0)


@pytest.mark.parametrize("dtype,each", [(BF, 40), (BF, 150), (torch.float32, 40)])
def test_captured_with_outputs_of_its_own(cuda_ok, dtype, each):
    """A captured call that makes its outputs, replayed on good offsets, bad ones and good ones again."""
    total = 3 * each
    d = make(52, dtype, total, 4, 64, 2, 3)
    g = on_gpu(d, dtype)
    offsets = idx([0, each, 2 * each, total])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = mamba2_scan(g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], offsets)
        after = y + 1
    for off in ([0, each, 2 * each, total], [0, each, 2 * each, total + 1], [0, 1, 2 * each + 5, total]):
        offsets.copy_(idx(off))
        graph.replay()
        torch.cuda.synchronize()
        if off[-1] > total:
            assert torch.isnan(y).all() and torch.isnan(after).all()
        else:
            compare(d, off, None, None, g["S"].cpu().numpy(), y.cpu().numpy())
            assert torch.equal(after, y + 1)
    del graph
