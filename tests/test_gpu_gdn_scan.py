"""The gated delta rule over packed prompts against the float64 oracle (needs a B200).

Tolerance, per prompt and head, on the 2-norm of the error over the 2-norm of the result. With unit keys, 0 <= beta <= 1
and |alpha| <= 1 every token's map of the state is non-expanding, so an error made in one chunk of 64 tokens is carried
on without growth, beside values of the size that it was made on. Within a chunk a value passes the inverse, which
reaches the tensor cores in two bf16 pieces (off by at most 2^-17 of itself), and three operands in three pieces (2^-24
each); fp32 sums of 64 to 128 terms add 2^-24 a level and the blocks of the inverse, products of two-piece operands
themselves, another 2^-17: at most 2^-16. Roundings of different chunks are independent, so that n chunks add up to
sqrt(n) of it. The fp32 kernel lies far below (2^-24 for each of some 24 steps of a token, tokens independent).
"""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import ReplaySSM, abi, gdn_scan
from oracle import lowprec as lp
from oracle.decoder import ReplayOracle
from oracle.philox import sr_words
from oracle.prompts import gdn_scan as oracle_scan
from synth import round_to_dtype

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOK = ("q", "k", "v", "alpha", "beta")
SCALE = 128 ** -0.5


def tol(n):
    return 2.0 ** -16 * max(1, -(-n // 64)) ** 0.5


def make(seed, dtype, total, H, Hk, P, batch, slow=1.0):
    """slow: decays nearer to 1."""
    r = np.random.default_rng(seed)
    f = lambda a: round_to_dtype(a.astype(np.float32), "bf16" if dtype == BF else "f32")  # noqa: E731
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
    return dict(S=(r.standard_normal((batch, H, P, 128)) * 0.05).astype(np.float32),
                q=f(unit(r.standard_normal((total, Hk, 128)))), k=f(unit(r.standard_normal((total, Hk, 128))) * 0.999),
                v=f(r.standard_normal((total, H, P))), alpha=np.exp(-r.uniform(0, 0.3 / slow, (total, H))).astype(np.float32),
                beta=r.uniform(0, 1, (total, H)).astype(np.float32))


def packed(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def on_gpu(d, dtype):
    return {k: torch.from_numpy(np.ascontiguousarray(v)).cuda().to(dtype if k in ("q", "k", "v") else F32)
            for k, v in d.items()}


def idx(v, t=torch.int32):
    return None if v is None else torch.tensor(v, dtype=t, device="cuda")


def scan(g, offsets, slots=None, resume=None, y=None, **kw):
    return gdn_scan(g["S"], *(g[k] for k in TOK), idx(offsets), idx(slots), idx(resume, torch.uint8), q_scale=SCALE, y=y, **kw)


def compare(d, offsets, slots, resume, S_got, y_got):
    S, y = oracle_scan(**d, offsets=offsets, slots=slots, resume=resume, q_scale=SCALE)
    outside = np.isnan(y).all((1, 2))
    assert (y_got[outside] == 7.0).all(), "rows of no prompt were written"
    named = list(range(len(offsets) - 1)) if slots is None else list(slots)
    for b in range(S.shape[0]):
        if b not in named:
            np.testing.assert_array_equal(S_got[b], d["S"][b])
    for i, b in enumerate(named):
        lo, hi = offsets[i], offsets[i + 1]
        for what, got, ref in (("y", y_got[lo:hi].transpose(1, 0, 2), y[lo:hi].transpose(1, 0, 2)), ("S", S_got[b], S[b])):
            for h in range(S.shape[1]):
                err, size = np.linalg.norm(got[h] - ref[h]), np.linalg.norm(ref[h])
                assert err <= tol(hi - lo) * size, f"{what} of prompt {i}, head {h}: {err / max(size, 1e-300):.2e}"


def check(d, dtype, offsets, slots=None, resume=None, **kw):
    g = on_gpu(d, dtype)
    y = torch.full(d["v"].shape, 7.0, device="cuda")
    scan(g, offsets, slots, resume, y, **kw)
    compare(d, offsets, slots, resume, g["S"].cpu().numpy(), y.cpu().numpy())
    return g["S"], y


SHAPES = [(8, 8, 64), (4, 2, 128), (3, 1, 88), (5, 5, 24), (1, 1, 8), (6, 2, 40), (2, 1, 120)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk,P", SHAPES)
def test_mixed_lengths(cuda_ok, dtype, H, Hk, P):
    """Empty, single-token, tile-sized and long prompts, from zero and resumed, to permuted slots."""
    lens = [1, 0, 130, 63, 64, 200, 0, 3, 65]
    d = make(H * 1000 + P, dtype, sum(lens), H, Hk, P, 11)
    check(d, dtype, packed(lens), slots=[4, 9, 0, 7, 2, 10, 1, 5, 3], resume=[0, 0, 1, 0, 1, 1, 1, 1, 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [64], [129], [777], [40, 700, 1], [3] * 9, [700] + [1] * 20])
def test_few_prompts(cuda_ok, dtype, lens):
    d = make(sum(lens), dtype, sum(lens), 2, 1, 128, len(lens), slow=8.0)
    check(d, dtype, packed(lens), resume=[i % 3 != 1 for i in range(len(lens))])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_extremes(cuda_ok, dtype):
    """Decays that underflow within a tile, exact zeros, ones and negative factors; beta 0 and 1; keys alike."""
    offsets = [0, 300, 450, 600]
    d = make(5, dtype, 600, 4, 4, 64, 3, slow=4.0)
    d["alpha"][:100] = np.float32(1e-7)
    d["alpha"][[5, 64, 120, 127, 128, 140, 141, 333]] = 0.0
    d["alpha"][200:260] = 1.0
    d["alpha"][310:330] *= -1
    d["beta"][300:340:2] = 0.0
    d["beta"][301:340:2] = 1.0
    d["k"][450:] = d["k"][450]
    d["alpha"][450:500] = 1.0
    d["beta"][450:500] = 1.0
    d["alpha"][560:] = np.float32(1e-30)
    check(d, dtype, offsets, resume=[1, 1, 1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, 1.3])
def test_keys_that_are_not_unit(cuda_ok, dtype, scale):
    """Keys of length 0, and beyond 1 as long as beta |k|^2 <= 2 keeps each map non-expanding."""
    d = make(6, dtype, 200, 2, 2, 128, 1, slow=4.0)
    d["k"] = round_to_dtype((d["k"] * np.float32(scale)).astype(np.float32), "bf16")
    check(d, dtype, [0, 200], resume=[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_no_prompt_and_neighbours(cuda_ok, dtype):
    """NaN before the first prompt, behind the last and in a prompt of its own reach nothing else."""
    offsets = [5, 70, 203, 331]
    d = make(7, dtype, 400, 4, 2, 64, 3)
    clean = {k: v.copy() for k, v in d.items()}
    for k in TOK:
        d[k][:5] = np.nan
        d[k][331:] = np.nan
        d[k][70:203] = np.nan
    g = on_gpu(d, dtype)
    y = torch.full(d["v"].shape, 7.0, device="cuda")
    scan(g, offsets, y=y)
    S_got, y_got = g["S"].cpu().numpy(), y.cpu().numpy()
    assert np.isnan(y_got[70:203]).all() and np.isnan(S_got[1]).all()
    S, ref = oracle_scan(**clean, offsets=offsets, q_scale=SCALE)
    y_got[70:203], S_got[1] = ref[70:203], S[1]
    compare(clean, offsets, None, None, S_got, y_got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeatable_and_piecewise(cuda_ok, dtype):
    """Two runs give the same bits; a prompt in two resumed pieces gives the whole prompt's results."""
    d = make(8, dtype, 400, 4, 2, 128, 1, slow=4.0)
    S1, y1 = check(d, dtype, [0, 400])
    S2, y2 = check(d, dtype, [0, 400])
    assert torch.equal(S1, S2) and torch.equal(y1, y2)
    g = on_gpu(d, dtype)
    y = torch.full_like(y1, 7.0)
    scan(g, [0, 133], y=y)
    scan(g, [133, 400], resume=[1], y=y)
    compare(d, [0, 400], None, None, g["S"].cpu().numpy(), y.cpu().numpy())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("total", [90, 400])
def test_refused_prompts(cuda_ok, dtype, total):
    """Offsets that fall or leave the tokens, slots out of range: nothing is written; slots named twice: those prompts
    are left out.  In outputs that the call makes, their rows are NaN."""
    a, b = total // 3, total // 2
    d = make(9, dtype, total, 2, 2, 64, 4)
    g = on_gpu(d, dtype)
    for offsets, slots in (([0, b, a, total], None), ([0, a, total + 1], None), ([-1, a, total], None),
                           ([0, a, total], [0, 4]), ([0, a, total], [-1, 2])):
        y = torch.full((total, 2, 64), 7.0, device="cuda")
        scan(g, offsets, slots, y=y)
        assert (y == 7.0).all()
        torch.full((total, 2, 64), 5.0, device="cuda")
        assert torch.isnan(scan(g, offsets, slots)).all()
        assert np.array_equal(g["S"].cpu().numpy(), d["S"])
    y = torch.full((total, 2, 64), 7.0, device="cuda")
    scan(g, [0, a, b, total], [2, 1, 2], y=y)
    assert (y[:a] == 7.0).all() and (y[b:] == 7.0).all() and (y[a:b] != 7.0).all()
    y = scan(g, [0, a, b, total], [2, 1, 2])
    assert torch.isnan(y[:a]).all() and torch.isnan(y[b:]).all() and torch.isfinite(y[a:b]).all()
    S = g["S"].cpu().numpy()
    for i in (0, 2, 3):
        np.testing.assert_array_equal(S[i], d["S"][i])


def test_no_tokens(cuda_ok):
    """A call without tokens sets the states of prompts that start from zero."""
    S, e = torch.ones(3, 2, 64, 128, device="cuda"), dict(dtype=BF, device="cuda")
    f = dict(device="cuda")
    y = gdn_scan(S, torch.empty(0, 1, 128, **e), torch.empty(0, 1, 128, **e), torch.empty(0, 2, 64, **e),
                 torch.empty(0, 2, **f), torch.empty(0, 2, **f), idx([0, 0, 0]), resume=idx([0, 1], torch.uint8))
    assert y.shape == (0, 2, 64)
    assert (S[0] == 0).all() and (S[1:] == 1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("H,Hk,P,lens", [(4, 2, 64, (40, 1, 23)), (3, 3, 24, (9, 4)), (4, 4, 128, (300, 1, 260)),
                                         (3, 1, 40, (128, 400))])
def test_values_that_are_not_finite_reach_no_earlier_token(cuda_ok, dtype, H, Hk, P, lens, value):
    """From a value of v that is not finite on, its head's row has no finite outputs and no finite state; everything else,
    the same row before it above all, keeps its bits."""
    offsets = packed(lens)
    total, n = offsets[-1], len(lens)
    d = make(34, dtype, total, H, Hk, P, n, slow=8.0)
    g = on_gpu(d, dtype)
    r = np.random.default_rng(35)
    at = {(total - 1, 0, 1), (offsets[1] - 1, H - 1, P - 1), (0, 0, 0)}
    at |= {(int(r.integers(total)), int(r.integers(H)), int(r.integers(P))) for _ in range(6)}
    hit_y = torch.zeros(total, H, P, dtype=torch.bool, device="cuda")
    hit_S = torch.zeros(n, H, P, dtype=torch.bool, device="cuda")
    v = g["v"].clone()
    for t, h, p in at:
        i = int(np.searchsorted(offsets, t, side="right")) - 1
        v[t, h, p] = value
        hit_y[t:offsets[i + 1], h, p] = True
        hit_S[i, h, p] = True
    got = []
    for vs in (g["v"], v):
        e = dict(g, S=g["S"].clone(), v=vs)
        got.append((e["S"], scan(e, offsets, resume=[1] * n)))
    (S0, y0), (S1, y1) = got
    assert torch.isfinite(y0).all() and torch.isfinite(S0).all()
    assert torch.equal(y0[~hit_y], y1[~hit_y]) and torch.equal(S0[~hit_S], S1[~hit_S])
    assert not torch.isfinite(y1[hit_y]).any() and not torch.isfinite(S1[hit_S]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("key", ["q", "k", "alpha", "beta"])
@pytest.mark.parametrize("lens", [(40, 1, 23), (300, 1, 260)])
def test_other_inputs_that_are_not_finite_reach_no_earlier_token(cuda_ok, dtype, lens, key):
    """NaN and infinities in k, alpha or beta: tokens before theirs and other prompts keep their bits; in q all others do.
    Chunks may scale their tokens by the product of alpha up to their end, so with alpha the chunk's earlier tokens of that
    head keep their values to the rounding of both runs."""
    offsets = packed(lens)
    total, n = offsets[-1], len(lens)
    g = on_gpu(make(38, dtype, total, 4, 2, 64, n, slow=8.0), dtype)
    for value in (np.nan, np.inf, -np.inf):
        for t in (offsets[1] - 10, offsets[1], total - 1, offsets[2] + 17):
            for where in ((0, 3), (0, slice(None))):
                bad = {k: v.clone() for k, v in g.items()}
                bad[key][(t, *where) if key in ("q", "k") else (t, 0)] = value
                got = []
                for e in (g, bad):
                    e = dict(e, S=e["S"].clone())
                    got.append((e["S"], scan(e, offsets, resume=[1] * n)))
                (S0, y0), (S1, y1) = got
                i = int(np.searchsorted(offsets, t, side="right")) - 1
                heads = 2 if key in ("q", "k") else 1
                hit = torch.zeros_like(y0, dtype=torch.bool)
                end = t + 1 if key == "q" else offsets[i + 1]
                hit[t:end, :heads] = True
                if key == "alpha":
                    near = torch.zeros_like(hit)
                    near[offsets[i]:t, 0] = True
                    assert torch.linalg.vector_norm((y0 - y1)[near]) <= 2 * tol(300) * torch.linalg.vector_norm(y0[near])
                    hit |= near
                    assert torch.isfinite(y1[near]).all()
                assert torch.equal(y0[~hit], y1[~hit])
                hit[:t] = False
                assert not torch.isfinite(y1[hit]).any()
                others = [s for s in range(n) if s != i]
                assert torch.equal(S0[others], S1[others]) and torch.equal(S0[i, heads:], S1[i, heads:])
                assert torch.equal(S0, S1) if key == "q" else not torch.isfinite(S1[i, :heads]).any()


def test_a_state_that_is_not_finite_keeps_to_its_rows(cuda_ok):
    for lens in ((5, 3), (100, 200)):
        g = on_gpu(make(39, BF, sum(lens), 2, 1, 64, 2, slow=8.0), BF)
        bad = dict(g, S=g["S"].clone())
        bad["S"][1, 1, 7, 100] = np.nan
        got = []
        for e in (dict(g, S=g["S"].clone()), bad):
            got.append((e["S"], scan(e, packed(lens), resume=[1, 1])))
        (S0, y0), (S1, y1) = got
        hit = torch.zeros_like(y0, dtype=torch.bool)
        hit[lens[0]:, 1, 7] = True
        assert torch.equal(y0[~hit], y1[~hit]) and not torch.isfinite(y1[hit]).any()
        assert not torch.isfinite(S1[1, 1, 7]).any()
        S1[1, 1, 7] = S0[1, 1, 7]
        assert torch.equal(S0, S1)


def test_in_a_graph_and_on_a_stream(cuda_ok):
    """Captured on a side stream and replayed on new inputs."""
    d = make(11, BF, 300, 4, 2, 64, 2)
    g = on_gpu(d, BF)
    y = torch.full((300, 4, 64), 7.0, device="cuda")
    offsets = idx([0, 90, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn_scan(g["S"], *(g[k] for k in TOK), offsets, q_scale=SCALE, y=y)
    for seed in (12, 13):
        d2 = make(seed, BF, 300, 4, 2, 64, 2)
        for k, v in on_gpu(d2, BF).items():
            g[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        compare(d2, [0, 90, 300], None, None, g["S"].cpu().numpy(), y.cpu().numpy())


@pytest.mark.parametrize("dtype,each,n", [(BF, 3, 700), (BF, 90, 300), (F32, 5, 300)])
def test_more_prompts_than_threads_of_a_block(cuda_ok, dtype, each, n):
    """Every block looks through more prompts than it has threads; all prompts are the same, to slots in reverse."""
    d = make(44, dtype, each, 2, 1, 16, 1)
    g = on_gpu(d, dtype)
    e = {k: g[k].repeat(n, *[1] * (g[k].dim() - 1)) for k in TOK}
    e["S"] = g["S"].repeat(n + 1, 1, 1, 1)
    y = scan(e, packed([each] * n), list(range(n, 0, -1)), [1] * n).view(n, each, 2, 16)
    compare(d, [0, each], None, [1], e["S"][1:2].cpu().numpy(), y[0].cpu().numpy())
    assert (y == y[:1]).all() and (e["S"][1:] == e["S"][1:2]).all() and torch.equal(e["S"][0], g["S"][0])


# ------------------------------------------------------------------------------------------ contexts


def context(d, dtype, batch, **kw):
    H, P = d["v"].shape[1:]
    layer = ReplaySSM("gdn", batch, H, P, 128, 1, 8, 4, dtype, q_scale=SCALE, **kw)
    layer.load_checkpoint(torch.from_numpy(d["S"]).cuda())
    return layer


def tokens(g):
    return tuple(g[k] for k in TOK)


def decode(layer, g, t, batch):
    """One token a sequence, heads of q and k repeated as the decode calls take them."""
    rep = layer.nheads // g["q"].shape[1]
    now = [g[k][t * batch:(t + 1) * batch] for k in TOK]
    now[:2] = [x.repeat_interleave(rep, 1) for x in now[:2]]
    return layer.gdn_step(*(x.contiguous() for x in now))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_of_a_context(cuda_ok, dtype):
    """Checkpoint, bookkeeping and skip flags after a prefill beside sequences that go on; refusals name their sequence and
    leave it alone; decoding goes on from the new checkpoints."""
    batch, H, P = 5, 4, 64
    d = make(9, dtype, 260, H, 2, P, batch)
    d["alpha"][:15] = np.float32(0.5)
    g = on_gpu(d, dtype)
    layer = context(d, dtype, batch, skip_tau=0.2)
    for t in range(3):
        decode(layer, g, t, batch)
    before, flags = layer.export(ring=False), layer.export_skip()
    assert flags.any()
    offsets, slots = [0, 130, 131, 260], [3, 0, 4]
    y = torch.full((260, H, P), 7.0, device="cuda")
    layer.gdn_prefill(*tokens(g), idx(offsets), idx(slots), y=y)
    after = layer.export(ring=False)
    assert layer.get_error() == (0, -1)
    compare(dict(d, S=before["S"].cpu().numpy()), offsets, slots, None, after["S"].cpu().numpy(), y.cpu().numpy())
    meta, old = after["meta"].cpu().numpy(), before["meta"].cpu().numpy()
    for b in range(batch):
        assert list(meta[b, :3]) == ([0, old[b, 1] + 1, 0] if b in slots else list(old[b, :3]))
    kept = torch.tensor([b not in slots for b in range(batch)], device="cuda")
    assert (layer.export_skip()[~kept] == 0).all() and torch.equal(layer.export_skip()[kept], flags[kept])
    y.fill_(7.0)
    layer.gdn_prefill(*tokens(g), idx([0, 50, 90]), idx([1, 3]), idx([1, 1], torch.uint8), y=y)
    assert (y[:50] == 7.0).all() and (y[50:90] != 7.0).all()
    assert layer.get_error() == (abi.DEV_BUFFERED, 1)
    held = layer.export(ring=False)
    assert list(held["meta"][1].tolist()) == list(meta[1]) and held["meta"][3, 1] == meta[3, 1] + 1


def test_decoding_goes_on_after_a_prefill(cuda_ok):
    """A window and more of single tokens on top of prompts, against the oracle that starts from the same checkpoints."""
    batch, H, P, total = 3, 4, 128, 150
    d = make(40, BF, total, H, 2, P, batch)
    g = on_gpu(d, BF)
    layer = context(d, BF, batch)
    layer.gdn_prefill(*tokens(g), idx([0, 70, 71, 150]))
    orc = ReplayOracle("gdn", layer.export(ring=False)["S"].cpu().numpy(), 8, nheads=H, q_scale=SCALE)
    for t in range(19):
        y = decode(layer, g, t, batch)
        inp = {k: d[k][t * batch:(t + 1) * batch] for k in TOK}
        inp["q"], inp["k"] = np.repeat(inp["q"], 2, 1), np.repeat(inp["k"], 2, 1)
        _, ref = orc.step(inp)
        err = np.linalg.norm(y.cpu().numpy() - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert err.max() <= 1e-4, t
    assert layer.get_error() == (0, -1)


@pytest.mark.parametrize("hp,read", [("f32", "nvfp4"), ("f16sr", "same"), ("f16sr", "nvfp4"), ("f8sr", "same"),
                                     ("f8sr", "nvfp4d"), ("f32", "nvfp4d"), ("f32", "shared_nvfp4")])
@pytest.mark.parametrize("P", [128, 40])
def test_prefill_into_checkpoint_formats(cuda_ok, hp, read, P):
    """The stored formats are the oracle's roundings, with the new epoch's random words, of the state that a scan on the
    widened checkpoints leaves; sequences of no prompt keep theirs; a resumed prompt continues from what is stored."""
    batch, H, seed = 4, 3, 0x5EED0123456789AB
    lens, slots, resume = [70, 9, 0, 0], [2, 0, 3, 1], [0, 1, 0, 1]
    d = make(50, BF, sum(lens), H, 1, P, batch)
    g = on_gpu(d, BF)
    layer = context(d, BF, batch, hp=hp, read=read, seed=seed)
    for epoch in (1, 2):
        before = layer.export(ring=False)
        copy = None if read == "same" else layer.export_read_copy()
        y = layer.gdn_prefill(*tokens(g), idx(packed(lens)), idx(slots), idx(resume, torch.uint8))
        e = dict(g, S=before["S"].clone())
        assert torch.equal(y, scan(e, packed(lens), slots, resume))
        want, after = e["S"].cpu().numpy(), layer.export(ring=False)
        got = after["S"].cpu().numpy()
        assert after["meta"][:, :3].tolist() == [[0, epoch, 0], [0, 0, 0], [0, epoch, 0], [0, epoch, 0]]
        np.testing.assert_array_equal(got[1], before["S"][1].cpu().numpy())
        new = [0, 2, 3]
        if read != "same":
            rc = layer.export_read_copy()
            q = (lp.nvfp4d_quantize_state if read == "nvfp4d" else lp.nvfp4_quantize_state)(want)
            for name in ("packed", "scales", "g"):
                np.testing.assert_array_equal(rc[name].cpu().numpy()[new], q[name][new], err_msg=name)
                assert torch.equal(rc[name][1], copy[name][1])
            if read == "nvfp4d":
                np.testing.assert_array_equal(layer.export_column_scales().cpu().numpy()[new], q["colscales"][new])
        for b in new:
            words = sr_words(seed, b * H + np.arange(H), epoch, P * 128).reshape(H, P, 128)
            ref = {"f32": lambda s: s, "f16sr": lambda s: lp.fp16_stochastic_round(s, words),
                   "f8sr": lambda s: lp.fp8_quantize_state(s, words)["values"]}[hp]
            if read == "shared_nvfp4":
                np.testing.assert_array_equal(got[b], lp.nvfp4_roundtrip_state(want[b:b + 1])[0])
            else:
                np.testing.assert_array_equal(got[b], ref(want[b]))
    assert layer.get_error() == (0, -1)


@pytest.mark.parametrize("hp", ["f32", "f16sr"])
def test_prefill_errors_of_a_context(cuda_ok, hp):
    d = make(10, BF, 64, 2, 2, 64, 3)
    g = on_gpu(d, BF)
    layer = context(d, BF, 3, hp=hp)
    S = layer.export(ring=False)["S"]
    layer.gdn_prefill(*tokens(g), idx([0, 32, 16]), idx([1, 2]))
    assert layer.get_error() == (abi.DEV_PROMPT, 1)
    assert torch.equal(layer.export(ring=False)["S"], S)
    layer = context(d, BF, 3, hp=hp)
    layer.verify(2, **{k: g[k][:6].reshape(3, 2, *g[k].shape[1:]).contiguous() for k in TOK})
    y = layer.gdn_prefill(*tokens(g), idx([0, 32, 64]), idx([1, 2]), idx([1, 0], torch.uint8))  # 1 is pending
    assert layer.get_error() == (abi.DEV_PENDING, 1)
    assert torch.isnan(y[:32]).all() and torch.isfinite(y[32:]).all()
    out = layer.export(ring=False)
    assert out["meta"][:, 2].tolist() == [2, 2, 0] and torch.equal(out["S"][:2], S[:2])
    y = layer.gdn_prefill(*tokens(g), idx([0, 10, 20, 64]), idx([1, 0, 1]))
    assert torch.isnan(y[:10]).all() and torch.isfinite(y[10:20]).all() and torch.isnan(y[20:]).all()
    fresh = ReplaySSM("gdn", 3, 2, 64, 128, 1, 8, 0, BF, hp=hp)
    with pytest.raises(RuntimeError, match="RSSM_ERR_UNSUPPORTED"):
        fresh.gdn_prefill(*tokens(g), idx([0, 64]))
    wrong = ReplaySSM("mamba2", 3, 2, 64, 128, 1, 8, 0, BF, A=torch.ones(2), D=torch.ones(2))
    wrong.load_checkpoint(torch.zeros(3, 2, 64, 128, device="cuda"))
    with pytest.raises(RuntimeError, match="RSSM_ERR_UNSUPPORTED"):
        wrong.gdn_prefill(*tokens(g), idx([0, 64]))


def test_scratch_of_the_caller(cuda_ok):
    """A context whose checkpoint is not the fp32 state takes scratch from the caller, with whatever it holds."""
    d = make(51, BF, 100, 2, 2, 64, 2)
    g = on_gpu(d, BF)
    a, b = context(d, BF, 2, hp="f16sr"), context(d, BF, 2, hp="f16sr")
    work = torch.full((2 * 2 * 64 * 128 * 4 + 256,), 255, dtype=torch.uint8, device="cuda")
    args = (*tokens(g), idx([0, 40, 100]), None, idx([1, 0], torch.uint8))
    assert torch.equal(a.gdn_prefill(*args), b.gdn_prefill(*args, workspace=work))
    assert torch.equal(a.export(ring=False)["S"], b.export(ring=False)["S"])
    with pytest.raises(ValueError, match="workspace"):
        b.gdn_prefill(*args, workspace=work[:1024])
    with pytest.raises(RuntimeError, match="RSSM_ERR_ARG"):
        b.gdn_prefill(*args, workspace=work[16:])


@pytest.mark.parametrize("hp", ["f32", "f8sr"])
def test_prefill_captured(cuda_ok, hp):
    """Two prefills (an even number keeps the bookkeeping in place) in a graph, replayed on new prompts while another
    sequence goes on decoding between the replays."""
    batch, H, P = 3, 4, 64
    d = make(46, BF, 300, H, 4, P, batch)
    g = on_gpu(d, BF)
    layer, eager = context(d, BF, batch, hp=hp), context(d, BF, batch, hp=hp)
    tok = tuple(t.clone() for t in tokens(g))
    first, second = (idx([0, 90]), idx([1])), (idx([90, 300]), idx([1]), idx([1], torch.uint8))
    y = torch.empty(300, H, P, device="cuda")

    def prompt(layer, tok, y):
        layer.gdn_prefill(*tok, *first, y=y)
        layer.gdn_prefill(*tok, *second, y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        prompt(layer, tok, y)
    for seed in (47, 48, 49):
        for t, new in zip(tok, tokens(on_gpu(make(seed, BF, 300, H, 4, P, batch), BF))):
            t.copy_(new)
        graph.replay()
        y2 = torch.empty_like(y)
        prompt(eager, tok, y2)
        assert torch.equal(y, y2)
        for _ in range(2):
            now = tuple(t[:batch].contiguous() for t in tok)
            assert torch.equal(layer.gdn_step(*now), eager.gdn_step(*now))
    a, b = layer.export(ring=False), eager.export(ring=False)
    assert torch.equal(a["S"], b["S"]) and torch.equal(a["meta"], b["meta"])
    assert layer.get_error() == (0, -1)
    del graph
