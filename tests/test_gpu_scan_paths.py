"""Paths of the prompt scan that depend on lengths, sizes and waits, against the float64 oracle (needs a B200)."""

import ctypes as C

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi, make_config
from test_gpu_scan import compare, context, idx, make, on_gpu

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
