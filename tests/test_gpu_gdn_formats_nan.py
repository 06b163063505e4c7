"""Prefills that leave rows of a state not finite, in every checkpoint format (needs a B200).

Nothing is compared within a tolerance: stored rows beside such a row are the oracle's roundings, bit by bit, of the state with
that row at 0, since tiles' and columns' maxima leave it out.
"""

import numpy as np
import pytest
import torch

from hybrid_model_ssm_gdn_b200 import abi
from oracle import lowprec as lp
from oracle.philox import sr_words
from test_gpu_gdn_scan import BF, F32, context, decode, idx, make, on_gpu, packed, scan, tokens

pytestmark = pytest.mark.gpu

FORMATS = [("f32", "same"), ("f16sr", "same"), ("f8sr", "same"), ("f32", "nvfp4"), ("f16sr", "nvfp4"), ("f8sr", "nvfp4"),
           ("f32", "nvfp4d"), ("f8sr", "nvfp4d"), ("f32", "shared_nvfp4")]


def copy_of(layer, read):
    """The values of the read copy."""
    rc = {k: v.cpu().numpy() for k, v in layer.export_read_copy().items()}
    E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6] * 2) * np.repeat([1, -1], 8)
    e4m3 = lambda t: torch.from_numpy(t).view(torch.float8_e4m3fn).double().numpy()  # noqa: E731
    codes = np.stack([rc["packed"] & 15, rc["packed"] >> 4], -1).reshape(*rc["packed"].shape[:-1], 128)
    R = codes.shape[2]
    g = np.repeat(rc["g"], 64, 2)[:, :, :R, None].astype(np.float64)
    v = E2M1[codes] * np.repeat(e4m3(rc["scales"]), 16, -1)
    if read == "nvfp4d":
        return v * np.repeat(e4m3(layer.export_column_scales().cpu().numpy()), 16, 2)[:, :, :R] * g * 2.0 ** -8
    return v * g


@pytest.mark.parametrize("hp,read", FORMATS)
@pytest.mark.parametrize("P,dtype,lens", [(128, BF, (150, 7)), (40, BF, (150, 7)), (128, BF, (9, 7)), (64, F32, (40, 3))])
def test_rows_that_are_not_finite_stay_so(cuda_ok, hp, read, P, dtype, lens):
    """NaN in v of one row, an infinity in another, from the middle of a prompt: both rows are NaN in the checkpoint, in the
    read copy and in every output of the next steps, over folds; all other rows are what the formats make of the state
    without them."""
    batch, H, seed = 2, 2, 0x1234567
    d = make(90, dtype, sum(lens), H, 1, P, batch, slow=8.0)
    d["v"][4, 1, 3] = np.nan
    d["v"][5, 0, P - 1] = np.inf
    hit = np.zeros((batch, H, P), bool)
    hit[0, 1, 3] = hit[0, 0, P - 1] = True
    g = on_gpu(d, dtype)
    layer = context(d, dtype, batch, hp=hp, read=read, seed=seed)
    layer.gdn_prefill(*tokens(g), idx(packed(lens)))
    e = dict(g, S=g["S"].clone())
    scan(e, packed(lens))
    want = e["S"].cpu().numpy()
    assert not np.isfinite(want[hit]).any() and np.isfinite(want[~hit]).all()
    want[hit] = 0
    got = layer.export(ring=False)["S"].cpu().numpy()
    assert (np.isnan(got[hit]).all() if hp != "f32" else not np.isfinite(got[hit]).any())
    if read != "same":
        copy = copy_of(layer, read)
        assert np.isnan(copy[hit]).all() and np.isfinite(copy[~hit]).all()
        q = (lp.nvfp4d_quantize_state if read == "nvfp4d" else lp.nvfp4_quantize_state)(want)
        rc = layer.export_read_copy()
        np.testing.assert_array_equal(rc["g"].cpu().numpy(), q["g"])
        for name in ("packed", "scales"):
            np.testing.assert_array_equal(rc[name].cpu().numpy()[~hit], q[name][~hit], err_msg=name)
        if read == "nvfp4d":
            np.testing.assert_array_equal(layer.export_column_scales().cpu().numpy(), q["colscales"])
    if read == "shared_nvfp4":
        np.testing.assert_array_equal(got[~hit], lp.nvfp4_roundtrip_state(want)[~hit])
    else:
        words = sr_words(seed, np.arange(batch * H), 1, P * 128).reshape(batch, H, P, 128)
        for b in range(batch):
            ref = {"f32": lambda s, w: s, "f16sr": lp.fp16_stochastic_round,
                   "f8sr": lambda s, w: lp.fp8_quantize_state(s, w)["values"]}[hp](want[b], words[b])
            np.testing.assert_array_equal(got[b][~hit[b]], ref[~hit[b]])
    d = make(91, dtype, 20 * batch, H, 1, P, batch, slow=8.0)
    g = on_gpu(d, dtype)
    for t in range(20):
        y = decode(layer, g, t, batch).cpu().numpy()
        assert not np.isfinite(y[hit]).any() and np.isfinite(y[~hit]).all(), t
    assert layer.export(ring=False)["meta"][:, 1].min() >= 3  # two folds after the prefill
    got = layer.export(ring=False)["S"].cpu().numpy()
    assert not np.isfinite(got[hit]).any() and np.isfinite(got[~hit]).all()
    if read != "same":
        copy = copy_of(layer, read)
        assert np.isnan(copy[hit]).all() and np.isfinite(copy[~hit]).all()


@pytest.mark.parametrize("hp,read", [("f8sr", "same"), ("f32", "nvfp4"), ("f32", "shared_nvfp4")])
def test_a_prefill_whose_wait_ran_out_leaves_nan(cuda_ok, monkeypatch, hp, read):
    """With a load withheld, states of every format are NaN and so are the next steps' outputs."""
    d = make(92, BF, 300, 2, 2, 64, 2)
    g = on_gpu(d, BF)
    monkeypatch.setenv("RSSM_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("RSSM_WITHHOLD_TILE", "1")
    layer = context(d, BF, 2, hp=hp, read=read)
    monkeypatch.delenv("RSSM_WITHHOLD_TILE")
    monkeypatch.delenv("RSSM_WAIT_CYCLES")
    y = layer.gdn_prefill(*tokens(g), idx([0, 150, 300]))
    assert layer.get_error()[0] == abi.DEV_TIMEOUT
    assert torch.isnan(y).all() and torch.isnan(layer.export(ring=False)["S"]).all()
    if read != "same":
        assert np.isnan(copy_of(layer, read)).all()
