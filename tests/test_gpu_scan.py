"""The Mamba-2 scan over packed prompts against the float64 oracle (needs a B200).

Tolerance, per element, against the sum of the magnitudes of the terms (the oracle run on absolute values): a term is
a product of exact inputs and one fp32 weight that reaches the tensor cores in two bf16 pieces (relative error at most
2^-17), its decay exp(A sum dt) carries the rounding of the sum (2^-24 times the exponent, and exp(-c) c <= 0.37), and
sums are fp32 (2^-24 a level): together below 2^-16.
"""

import ctypes as C

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import ReplaySSM, abi, make_config, mamba2_scan
from oracle.prompts import mamba2_scan as oracle_scan
from synth import round_to_dtype

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -16


def make(seed, dtype, total, H, P, G, batch, decay=1.0):
    r = np.random.default_rng(seed)
    f = lambda a: round_to_dtype(a.astype(np.float32), "bf16" if dtype == torch.bfloat16 else "f32")  # noqa: E731
    return dict(
        S=(r.standard_normal((batch, H, P, 128)) * 0.05).astype(np.float32),
        x=f(r.standard_normal((total, H, P))), B=f(r.standard_normal((total, G, 128)) / np.sqrt(128)),
        C=f(r.standard_normal((total, G, 128)) / np.sqrt(128)), dt=f(r.uniform(1e-3, 0.1, (total, H))),
        A=(-np.exp(r.uniform(0, np.log(16), H)) * decay).astype(np.float32),
        D=(0.1 * r.standard_normal(H)).astype(np.float32))


def on_gpu(d, dtype):
    return {k: torch.from_numpy(v).cuda().to(dtype if k in ("x", "B", "C", "dt") else torch.float32) for k, v in d.items()}


def idx(v, t=torch.int32):
    return None if v is None else torch.tensor(v, dtype=t, device="cuda")


def check(d, dtype, offsets, slots=None, resume=None, fill=np.nan):
    """Run the library, compare y and every state (those of no prompt bit for bit)."""
    g = on_gpu(d, dtype)
    y = torch.full(d["x"].shape, 7.0, device="cuda")
    mamba2_scan(g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], idx(offsets), idx(slots),
                idx(resume, torch.uint8), y=y)
    compare(d, offsets, slots, resume, g["S"].cpu().numpy(), y.cpu().numpy())
    return g["S"], y


def compare(d, offsets, slots, resume, S_got, y_got):
    S, y = oracle_scan(**d, offsets=offsets, slots=slots, resume=resume)
    mag = {k: np.abs(v) for k, v in d.items() if k != "A"}
    S_mag, y_mag = oracle_scan(**mag, A=d["A"], offsets=offsets, slots=slots, resume=resume)
    inside = np.isfinite(y)
    assert (y_got[~inside] == 7.0).all(), "rows of no prompt were written"
    err = np.abs(y_got - y)[inside] / (y_mag[inside] + 1e-30)
    assert err.max(initial=0.0) <= TOL, f"y {err.max():.3e}"
    named = set(range(len(offsets) - 1)) if slots is None else set(slots)
    for b in range(S.shape[0]):
        if b not in named:
            np.testing.assert_array_equal(S_got[b], d["S"][b])
    err = np.abs(S_got - S) / (S_mag + 1e-30)
    assert err.max() <= TOL, f"S {err.max():.3e}"


SHAPES = [(8, 64, 1), (4, 64, 2), (3, 64, 1), (5, 24, 5), (1, 8, 1), (6, 40, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,P,G", SHAPES)
def test_mixed_lengths(cuda_ok, dtype, H, P, G):
    """Empty, single-token, tile-sized and long prompts, from zero and resumed, to permuted slots."""
    lens = [1, 0, 130, 127, 128, 200, 0, 3]
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(H * 1000 + P, dtype, offsets[-1], H, P, G, 11)
    check(d, dtype, offsets, slots=[4, 9, 0, 7, 2, 10, 1, 5], resume=[0, 0, 1, 0, 1, 1, 1, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[1], [64], [129], [777], [1], [40, 700, 1]])
def test_few_prompts(cuda_ok, dtype, lens):
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(sum(lens), dtype, offsets[-1], 2, 64, 1, len(lens))
    check(d, dtype, offsets, resume=[1] * len(lens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decay_extremes(cuda_ok, dtype):
    """Decays so fast that exp(A sum dt) underflows within a tile, and dt = 0 (no decay, nothing added)."""
    offsets = [0, 300, 450]
    d = make(5, dtype, 450, 4, 64, 1, 2, decay=60.0)
    d["dt"][100:140] = 0.0
    d["dt"][300:] = 0.0
    check(d, dtype, offsets, resume=[1, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_no_prompt_and_neighbours(cuda_ok, dtype):
    """NaN before the first prompt, behind the last and in a prompt of its own reach nothing else."""
    offsets = [5, 70, 203, 331]
    d = make(6, dtype, 400, 4, 64, 2, 3)
    clean = {k: v.copy() for k, v in d.items()}
    for k in ("x", "B", "C", "dt"):
        d[k][:5] = np.nan
        d[k][331:] = np.nan
        d[k][70:203] = np.nan
    g = on_gpu(d, dtype)
    y = torch.full(d["x"].shape, 7.0, device="cuda")
    mamba2_scan(g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], idx(offsets), y=y)
    S_got, y_got = g["S"].cpu().numpy(), y.cpu().numpy()
    assert np.isnan(y_got[70:203]).all() and np.isnan(S_got[1]).any()
    y_got[70:203] = oracle_scan(**clean, offsets=offsets)[1][70:203]
    S_got[1] = oracle_scan(**clean, offsets=offsets)[0][1]
    compare(clean, offsets, None, None, S_got, y_got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_repeatable_and_piecewise(cuda_ok, dtype):
    """Two runs give the same bits; a prompt in two resumed pieces gives the whole prompt's results."""
    d = make(7, dtype, 400, 4, 64, 2, 1)
    S1, y1 = check(d, dtype, [0, 400])
    S2, y2 = check(d, dtype, [0, 400])
    assert torch.equal(S1, S2) and torch.equal(y1, y2)
    g = on_gpu(d, dtype)
    args = (g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"])
    y = torch.full_like(y1, 7.0)
    mamba2_scan(*args, idx([0, 133]), y=y)
    mamba2_scan(*args, idx([133, 400]), resume=idx([1], torch.uint8), y=y)
    compare(d, [0, 400], None, None, g["S"].cpu().numpy(), y.cpu().numpy())


def test_bad_prompts_write_nothing(cuda_ok):
    """Offsets that fall or leave the tokens, slots out of range: nothing is written; slots named twice: those prompts
    are left out."""
    d = make(8, torch.bfloat16, 100, 2, 64, 1, 4)
    g = on_gpu(d, torch.bfloat16)
    args = (g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"])
    for offsets, slots in (([0, 60, 50, 100], None), ([0, 50, 101], None), ([-1, 50, 100], None),
                           ([0, 50, 100], [0, 4]), ([0, 50, 100], [-1, 2])):
        y = torch.full((100, 2, 64), 7.0, device="cuda")
        mamba2_scan(g["S"], *args, idx(offsets), idx(slots), y=y)
        assert (y == 7.0).all() and np.array_equal(g["S"].cpu().numpy(), d["S"])
    y = torch.full((100, 2, 64), 7.0, device="cuda")
    mamba2_scan(g["S"], *args, idx([0, 30, 60, 100]), idx([2, 1, 2]), y=y)
    assert (y[:30] == 7.0).all() and (y[60:] == 7.0).all() and (y[30:60] != 7.0).all()
    S = g["S"].cpu().numpy()
    for b in (0, 2, 3):
        np.testing.assert_array_equal(S[b], d["S"][b])


def test_no_tokens(cuda_ok):
    """A call without tokens sets the states of prompts that start from zero."""
    S = torch.ones(3, 2, 64, 128, device="cuda")
    e = dict(dtype=torch.bfloat16, device="cuda")
    y = mamba2_scan(S, torch.empty(0, 2, 64, **e), torch.empty(0, 1, 128, **e), torch.empty(0, 1, 128, **e),
                    torch.empty(0, 2, **e), torch.full((2,), -1.0, device="cuda"), torch.ones(2, device="cuda"),
                    idx([0, 0, 0]), resume=idx([0, 1], torch.uint8))
    assert y.shape == (0, 2, 64)
    assert (S[0] == 0).all() and (S[1:] == 1).all()


def context(d, dtype, batch, **kw):
    H, P, G = d["x"].shape[1], d["x"].shape[2], d["B"].shape[1]
    layer = ReplaySSM("mamba2", batch, H, P, 128, G, 8, 4, dtype, A=torch.from_numpy(d["A"]), D=torch.from_numpy(d["D"]),
                      **kw)
    layer.load_checkpoint(torch.from_numpy(d["S"]).cuda())
    return layer


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_of_a_context(cuda_ok, dtype):
    """Checkpoint, bookkeeping and skip flags after a prefill beside sequences that go on; refusals name their
    sequence and leave it alone."""
    batch, H, P, G = 5, 4, 64, 2
    d = make(9, dtype, 260, H, P, G, batch, decay=8.0)
    g = on_gpu(d, dtype)
    layer = context(d, dtype, batch, skip_tau=0.5)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    for t in range(3):
        layer.mamba2_step(*(v[t * batch:(t + 1) * batch].contiguous() for v in tok))
    before = layer.export(ring=False)
    flags = layer.export_skip()
    offsets, slots = [0, 130, 131, 260], [3, 0, 4]
    y = torch.full((260, H, P), 7.0, device="cuda")
    layer.prefill(*tok, idx(offsets), idx(slots), y=y)
    after = layer.export(ring=False)
    assert layer.get_error() == (0, -1)
    held = dict(d, S=before["S"].cpu().numpy())
    compare(held, offsets, slots, None, after["S"].cpu().numpy(), y.cpu().numpy())
    meta, old = after["meta"].cpu().numpy(), before["meta"].cpu().numpy()
    for b in range(batch):
        want = [0, old[b, 1] + 1, 0] if b in slots else list(old[b, :3])
        assert list(meta[b, :3]) == want
    kept = torch.tensor([b not in slots for b in range(batch)], device="cuda")
    assert (layer.export_skip()[~kept] == 0).all() and torch.equal(layer.export_skip()[kept], flags[kept])
    # sequence 1 has three buffered records: it cannot resume, sequence 3 can
    y.fill_(7.0)
    layer.prefill(*tok, idx([0, 50, 90]), idx([1, 3]), idx([1, 1], torch.uint8), y=y)
    assert (y[:50] == 7.0).all() and (y[50:90] != 7.0).all()
    assert layer.get_error() == (6, 1)
    meta2 = layer.export(state=False, ring=False)["meta"].cpu().numpy()
    assert list(meta2[1]) == list(meta[1]) and meta2[3, 1] == meta[3, 1] + 1


def test_prefill_errors_of_a_context(cuda_ok):
    d = make(10, torch.bfloat16, 64, 2, 64, 1, 3)
    g = on_gpu(d, torch.bfloat16)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    layer = context(d, torch.bfloat16, 3)
    layer.prefill(*tok, idx([0, 32, 16]), idx([1, 2]))
    assert layer.get_error() == (5, 1)
    assert np.array_equal(layer.export(ring=False)["S"].cpu().numpy(), d["S"])
    layer = context(d, torch.bfloat16, 3)
    layer.verify(2, **{k: g[k][:6].reshape(3, 2, *g[k].shape[1:]).contiguous() for k in ("x", "B", "C", "dt")})
    layer.prefill(*tok, idx([0, 32, 64]), idx([1, 2]), idx([1, 0], torch.uint8))  # 1 is pending, 2 starts again
    assert layer.get_error() == (1, 1)
    meta = layer.export(state=False, ring=False)["meta"].cpu().numpy()
    assert meta[:, 2].tolist() == [2, 2, 0]
    fresh = ReplaySSM("mamba2", 3, 2, 64, 128, 1, 8, 0, torch.bfloat16, A=g["A"], D=g["D"])
    with pytest.raises(RuntimeError, match="RSSM_ERR_UNSUPPORTED"):
        fresh.prefill(*tok, idx([0, 64]))


def test_prefill_in_a_graph_and_on_a_stream(cuda_ok):
    """Captured on a side stream and replayed on new inputs."""
    d = make(11, torch.bfloat16, 200, 4, 64, 2, 2)
    g = on_gpu(d, torch.bfloat16)
    y = torch.full((200, 4, 64), 7.0, device="cuda")
    offsets = idx([0, 90, 200])
    args = (g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mamba2_scan(*args, y=y)
    for seed in (12, 13):
        d2 = make(seed, torch.bfloat16, 200, 4, 64, 2, 2)
        for k, v in on_gpu(d2, torch.bfloat16).items():
            g[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        compare(d2, [0, 90, 200], None, None, g["S"].cpu().numpy(), y.cpu().numpy())


@pytest.mark.parametrize("H,P,G,lens,resume", [(2, 64, 1, [1900], [1]), (3, 40, 1, [2049], [0]), (4, 64, 4, [1, 2600, 0], [0, 1, 1]),
                                               (2, 64, 2, [1792, 1535], [1, 0])])
def test_long_prompts_in_pieces(cuda_ok, H, P, G, lens, resume):
    """Few heads and long prompts: the prompts are cut into pieces that run side by side."""
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(H + len(lens), torch.bfloat16, offsets[-1], H, P, G, len(lens) + 1, decay=0.05)
    cfg = make_config("mamba2", len(lens) + 1, H, P, 128, G, 1, 0, torch.bfloat16, A=torch.empty(H), D=torch.empty(H))
    n = C.c_size_t()
    assert abi.load().rssm_mamba2_scan_workspace(C.byref(cfg), offsets[-1], len(lens), C.byref(n)) == 0 and n.value > 0
    check(d, torch.bfloat16, offsets, slots=list(range(len(lens), 0, -1)), resume=resume)


def test_workspace_of_the_caller(cuda_ok):
    """Scratch from the caller, with whatever it holds; too small or misplaced scratch is refused before any launch."""
    d = make(20, torch.bfloat16, 2000, 2, 64, 1, 1, decay=0.05)
    g = on_gpu(d, torch.bfloat16)
    args = (g["S"], g["x"], g["B"], g["C"], g["dt"], g["A"], g["D"], idx([0, 2000]))
    y = torch.full((2000, 2, 64), 7.0, device="cuda")
    work = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    mamba2_scan(*args, y=y, workspace=work)
    compare(d, [0, 2000], None, None, g["S"].cpu().numpy(), y.cpu().numpy())
    with pytest.raises(ValueError, match="workspace"):
        mamba2_scan(*args, y=y, workspace=work[:1024])
    with pytest.raises(RuntimeError, match="RSSM_ERR_ARG"):
        mamba2_scan(*args, y=y, workspace=work[16:])


def test_a_load_that_never_comes_times_out_and_the_context_recovers(cuda_ok, monkeypatch):
    """Every wait of the 128-token kernel is bounded: with one chunk's load withheld (and the bound shortened to about a
    millisecond) the launch ends, the context reports it, and after a reload it serves prompts again."""
    d = make(21, torch.bfloat16, 400, 4, 64, 2, 2)
    g = on_gpu(d, torch.bfloat16)
    tok = (g["x"], g["B"], g["C"], g["dt"])
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, torch.bfloat16, 2)
    monkeypatch.delenv("RSSM_WITHHOLD_TILE")
    monkeypatch.delenv("RSSM_WAIT_CYCLES")
    layer.prefill(*tok, idx([0, 150, 400]))
    code, seq = layer.get_error()
    assert code == abi.DEV_TIMEOUT and 0 <= seq < 2
    layer.load_checkpoint(torch.from_numpy(d["S"]).cuda())
    y = torch.full((400, 4, 64), 7.0, device="cuda")
    layer.prefill(*tok, idx([0, 150, 400]), y=y)
    compare(d, [0, 150, 400], None, None, layer.export(ring=False)["S"].cpu().numpy(), y.cpu().numpy())
    assert layer.get_error() == (0, -1)


@pytest.mark.parametrize("H,lens", [(4, (150, 250)), (2, (1900,))])
def test_a_scan_that_timed_out_leaves_nan(cuda_ok, monkeypatch, H, lens):
    """With one chunk's load withheld from every block, whole prompts and pieces: all outputs and states are NaN."""
    offsets = np.concatenate([[0], np.cumsum(lens)]).tolist()
    total = offsets[-1]
    d = make(22, torch.bfloat16, total, H, 64, 1, len(lens), decay=0.05)
    g = on_gpu(d, torch.bfloat16)
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, torch.bfloat16, len(lens))
    y = torch.full((total, H, 64), 7.0, device="cuda")
    layer.prefill(g["x"], g["B"], g["C"], g["dt"], idx(offsets), y=y)
    assert layer.get_error()[0] == abi.DEV_TIMEOUT
    assert torch.isnan(y).all()
    assert torch.isnan(layer.export(ring=False)["S"]).all()


@pytest.mark.parametrize("dtype,H,total,nseq", [(torch.bfloat16, 8, 2 ** 23 + 1000, 1), (torch.float32, 8, 2 ** 23 + 1000, 1),
                                                (torch.bfloat16, 128, 2 ** 19 + 1000, 6700)])
def test_rows_past_32_bits(cuda_ok, dtype, H, total, nseq):
    """The last rows of inputs with more than 2^32 elements, in the last sequence of many, in each of the kernels."""
    n, P = 150 if nseq == 1 else 40, 64
    d = make(23, dtype, n, H, P, 1, 1)
    g = on_gpu(d, dtype)
    big = {k: torch.empty(total, *g[k].shape[1:], dtype=dtype, device="cuda") for k in ("x", "B", "C", "dt")}
    for k, t in big.items():
        t[-n:] = g[k]
    y = torch.empty(total, H, P, device="cuda")
    y[:-n].view(torch.int32)[-1000:] = 7
    S = torch.empty(nseq, H, P, 128, device="cuda")
    S[-1] = g["S"][0]
    offsets = [total - n] * nseq + [total]
    mamba2_scan(S, big["x"], big["B"], big["C"], big["dt"], g["A"], g["D"], idx(offsets), resume=idx([1] * nseq, torch.uint8),
                y=y)
    assert (y[:-n].view(torch.int32)[-1000:] == 7).all()
    compare(d, [0, n], None, [1], S[-1:].cpu().numpy(), y[-n:].cpu().numpy())
