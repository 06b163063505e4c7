"""The prompt and drafting operators with the decode calls they sit between, as a serving loop runs them (needs a B200):
prompts through convolution and scan into a context, then speculative rounds of convolution, verify, draft verification
and the two commits."""

import numpy as np
import pytest
import torch

from gpu_harness import TOL_F32, head_rel_err
from hybrid_model_ssm_gdn_b200 import ReplaySSM, accept_drafts, shortconv_commit, shortconv_prefill, shortconv_verify
from oracle.decoder import ReplayOracle
from oracle.prompts import ShortConvRing, accept_drafts as oracle_accept, mamba2_scan as oracle_scan
from synth import round_to_dtype

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
H, P, G, K, BATCH, T, VOCAB = 4, 64, 2, 4, 5, 4, 300  # T verified tokens a round: the one drawn before and T-1 drafts
SPLITS = (H * P, G * 128, G * 128)
CH = sum(SPLITS)


def bf16(r, *shape, std=1.0):
    return round_to_dtype((std * r.standard_normal(shape)).astype(np.float32), "bf16")


def dev(a, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


class Serving:
    """One layer's convolution history and context."""

    def __init__(self, r):
        self.w, self.b = bf16(r, CH, K, std=0.3), bf16(r, CH, std=0.3)
        self.A, self.D = -np.exp(r.uniform(0, 2, H)).astype(np.float32), r.standard_normal(H).astype(np.float32)
        hist = bf16(r, BATCH, K - 1 + T, CH)
        cur = r.integers(0, K - 1 + T, BATCH)
        self.ring = ShortConvRing(hist, cur, self.w, self.b, True)
        self.hist, self.cur = dev(hist), dev(cur, torch.int32)
        self.layer = ReplaySSM("mamba2", BATCH, H, P, 128, G, 8, T, BF, A=torch.from_numpy(self.A),
                               D=torch.from_numpy(self.D))
        self.layer.load_checkpoint(torch.zeros(BATCH, H, P, 128, device="cuda"))
        self.wt, self.bt = dev(self.w), dev(self.b)

    def split(self, out, *lead):
        return out[0].view(*lead, H, P), out[1].view(*lead, G, 128), out[2].view(*lead, G, 128)

    def prompts(self, raw, dt, offsets):
        off = dev(np.array(offsets), torch.int32)
        out = shortconv_prefill(self.hist, self.cur, raw, self.wt, self.bt, off, splits=SPLITS)
        x, B, C = self.split(out, raw.shape[0])
        return (x, B, C), self.layer.prefill(x, B, C, dt, off)

    def round(self, raw, dt, target, tokens, u, draft):
        out = shortconv_verify(self.hist, self.cur, raw, self.wt, self.bt, splits=SPLITS)
        x, B, C = self.split(out, BATCH, T)
        y = self.layer.verify(T, x=x, B=B, C=C, dt=dt)
        accepted, committed, drawn = accept_drafts(target, tokens, u, draft=draft)
        self.layer.commit(committed)
        shortconv_commit(self.hist, self.cur, committed, K)
        return (x, B, C), y, accepted, committed, drawn


def round_inputs(r):
    logits = 2 * r.standard_normal((BATCH, T, VOCAB))
    draft = np.exp(logits[:, :T - 1])
    target = np.exp(logits + 0.5 * r.standard_normal(logits.shape))
    draft, target = draft / draft.sum(-1, keepdims=True), target / target.sum(-1, keepdims=True)
    tokens = np.array([[r.choice(VOCAB, p=draft[b, j]) for j in range(T - 1)] for b in range(BATCH)])
    return dict(raw=bf16(r, BATCH, T, CH), dt=bf16(r, BATCH, T, H, std=0.02), target=target.astype(np.float32),
                tokens=tokens, u=r.random((BATCH, T)).astype(np.float32), draft=draft.astype(np.float32))


def on_gpu(d):
    d = dict(d, dt=np.abs(d["dt"]) + np.float32(2.0 ** -8))
    kinds = dict(raw=BF, dt=BF, target=torch.float32, tokens=torch.int32, u=torch.float32, draft=torch.float32)
    return {k: dev(v, kinds[k]) for k, v in d.items()}


def conv_close(got, ref):
    got = torch.cat([v.float().reshape(ref.shape[0], -1) for v in got], -1).cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -17).all()  # bf16 rounding; fp32 sums of five terms


def test_prompts_then_speculative_rounds(cuda_ok):
    r = np.random.default_rng(0)
    s = Serving(r)
    offsets = [0, 20, 21, 21, 154, 161]
    raw, dt = bf16(r, 161, CH), np.abs(bf16(r, 161, H, std=0.02)) + np.float32(2.0 ** -8)
    dt = round_to_dtype(dt, "bf16")
    (x, B, C), y = s.prompts(dev(raw), dev(dt), offsets)
    conv_close((x, B, C), s.ring.prefill(raw, offsets))
    xn, Bn, Cn = (v.float().cpu().numpy() for v in (x, B, C))
    S, y_ref = oracle_scan(np.zeros((BATCH, H, P, 128)), xn, Bn, Cn, dt, s.A, s.D, offsets)
    assert head_rel_err(y.cpu().numpy(), y_ref).max() <= TOL_F32
    S_gpu = s.layer.export(ring=False)["S"].cpu().numpy()
    live = [b for b in range(BATCH) if b != 2]  # prompt 2 is empty: its state is zero
    assert (S_gpu[2] == 0).all()
    assert head_rel_err(S_gpu[live].reshape(4, H, -1), S[live].reshape(4, H, -1)).max() <= 1e-5
    orc = ReplayOracle("mamba2", S_gpu, 8, nheads=H, ngroups=G, params={"A": s.A, "D": s.D})
    for rnd in range(6):
        d = round_inputs(r)
        g = on_gpu(d)
        (x, B, C), y, accepted, committed, drawn = s.round(**g)
        conv_close(tuple(v.reshape(BATCH * T, -1) for v in (x, B, C)), s.ring.verify(d["raw"]).reshape(BATCH * T, CH))
        tok = {k: v.float().cpu().numpy() for k, v in zip(("x", "B", "C", "dt"), (x, B, C, g["dt"]))}
        _, y_true = orc.verify(T, tok)
        assert head_rel_err(y.cpu().numpy(), y_true).max() <= TOL_F32, rnd
        acc, nxt = oracle_accept(d["target"], d["tokens"], d["u"], d["draft"])
        np.testing.assert_array_equal(accepted.cpu().numpy(), acc)
        np.testing.assert_array_equal(drawn.cpu().numpy(), nxt)
        orc.commit(acc + 1)
        s.ring.commit(acc + 1)
        np.testing.assert_array_equal(s.hist.float().cpu().numpy(), s.ring.hist)
        np.testing.assert_array_equal(s.cur.cpu().numpy(), s.ring.cur)
        meta = s.layer.export(state=False, ring=False)["meta"].cpu().numpy()
        np.testing.assert_array_equal(meta[:, 0], orc.count)
    assert s.layer.get_error() == (0, -1)
    # a finished sequence's slot takes a new prompt while the others keep their buffers
    before = s.layer.export(ring=False)
    off, slot = dev(np.array([0, 133]), torch.int32), dev(np.array([3]), torch.int32)
    out = shortconv_prefill(s.hist, s.cur, dev(raw[21:154]), s.wt, s.bt, off, slots=slot, splits=SPLITS)
    x, B, C = s.split(out, 133)
    s.layer.prefill(x, B, C, dev(dt[21:154]), off, slots=slot)
    after = s.layer.export(ring=False)
    # the same prompt alone is long enough for the other kernel: both are within 1e-5 of the oracle, so 2e-5 apart
    assert head_rel_err(after["S"][3].cpu().numpy().reshape(H, -1), S_gpu[3].reshape(H, -1)).max() <= 2e-5
    keep = [0, 1, 2, 4]
    assert torch.equal(after["S"][keep], before["S"][keep]) and torch.equal(after["meta"][keep], before["meta"][keep])
    assert after["meta"][3, 0] == 0 and s.layer.get_error() == (0, -1)


def test_round_in_a_graph(cuda_ok):
    """A round captured once and replayed gives the bits of rounds launched one by one."""
    eager, graphed = Serving(np.random.default_rng(1)), Serving(np.random.default_rng(1))
    r = np.random.default_rng(2)
    inputs = [on_gpu(round_inputs(r)) for _ in range(4)]
    fixed = {k: v.clone() for k, v in inputs[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = graphed.round(**fixed)
    for d in inputs:
        want = eager.round(**d)
        for k, v in d.items():
            fixed[k].copy_(v)
        graph.replay()
        for a, b in zip((*want[0], *want[1:]), (*out[0], *out[1:])):
            assert torch.equal(a, b)
        assert torch.equal(eager.hist, graphed.hist) and torch.equal(eager.cur, graphed.cur)
    a, b = eager.layer.export(ring=False), graphed.layer.export(ring=False)
    assert torch.equal(a["S"], b["S"]) and torch.equal(a["meta"], b["meta"])
    del graph


def test_calls_on_two_streams(cuda_ok):
    """Two layers' prompts on two streams at once, each with its own scratch and history."""
    r = np.random.default_rng(3)
    layers = [Serving(np.random.default_rng(4 + i)) for i in range(2)]
    raw, dt = dev(bf16(r, 161, CH)), dev(np.abs(bf16(r, 161, H, std=0.02)))
    offsets = [0, 20, 21, 21, 154, 161]
    want = [Serving(np.random.default_rng(4 + i)).prompts(raw, dt, offsets)[1] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, st in zip(layers, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(s.prompts(raw, dt, offsets)[1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
