"""What a row of the short convolution depends on: the W rows up to its own and nothing else, for
every tap count.  An infinity or a NaN in a row, a state or a gradient makes exactly those outputs
non-finite whose definition reads it, forward, in steps and in the gradients."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, dev
from test_block_conv import draw, reference

BF, F32 = torch.bfloat16, torch.float32


def same_finite(got, ref, mag, steps, what):
    """got is finite exactly where ref is, and as near as block_cases' comparison asks there."""
    fin = np.isfinite(ref)
    g = got.detach().cpu().reshape(ref.shape)
    assert (torch.isfinite(g).numpy() == fin).all(), what
    close(g[torch.from_numpy(fin)], ref[fin], mag[fin], steps, what)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("dtype,D", [(F32, 16), (F32, 13), (BF, 24), (BF, 7)])
@pytest.mark.parametrize("W", range(2, 9))
def test_bad_rows_reach_their_window_only(W, dtype, D, act):
    """NaN and infinities in rows of two sequences, and in the second's state."""
    cu = [0, 45, 75]
    d = draw(1, 75, D, W, dtype, cu, seed=W + D)
    d["x"][0, 20, 3], d["x"][0, 33, 5], d["x"][0, 60, 1] = float("inf"), float("nan"), -float("inf")
    d["state"][1, 0, 2] = float("inf")
    o = dev(d)
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], o["cu"], silu=act)
    with np.errstate(all="ignore"):
        r, m = reference(d, act), reference(d, act, mag=True)
    same_finite(y, r["out"], m["out"], 2 * W + 32, "out")
    assert np.array_equal(fin.cpu().double().numpy(), r["final"], equal_nan=True)
    state = o["state"][1:].clone()   # the second sequence by steps: the same rows, bit for bit
    for t in range(cu[1], cu[2]):
        row = kda.kda_conv_step(o["x"][:, t], o["w"], state, bias=o["bias"], silu=act)
        assert torch.equal(row.nan_to_num(7.0, 8.0, 9.0), y[:, t].nan_to_num(7.0, 8.0, 9.0)), t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(F32, 16), (F32, 13), (BF, 24), (BF, 7)])
@pytest.mark.parametrize("W", range(2, 9))
def test_bad_gradients_reach_their_window_only(W, dtype, D):
    """An infinite or NaN d_out reaches dx of the W rows up to its own and the state's gradient
    where those lie in front of the sequence; dweight and dbias of its channel."""
    cu = [0, 45, 75]
    for act in (True, False):
        d = draw(1, 75, D, W, dtype, cu, seed=W + 2 * D)
        d["dy"][0, 20, 3], d["dy"][0, 33, 5], d["dy"][0, 46, 1] = float("inf"), float("nan"), -float("inf")
        if act:   # dpre of the W rows from this one on has no value
            d["x"][0, 60, 2] = float("inf")
        o = dev(d)
        g = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], o["cu"], silu=act)
        with np.errstate(all="ignore"):
            r, m = reference(d, act, True), reference(d, act, True, True)
        same_finite(g["dx"], r["dx"], m["dx"], 3 * W + 40, "dx")
        same_finite(g["dstate"], r["dstate"], m["dstate"], 3 * W + 40, "dstate")
        same_finite(g["dweight"], r["dw"], m["dw"], 2 * W + 40 + 75, "dweight")
        same_finite(g["dbias"], r["db"], m["db"], 2 * W + 40 + 75, "dbias")


def test_reference_reads_its_window_only():
    for W in range(2, 9):
        d = draw(1, 40, 4, W, F32, seed=W)
        d["x"][0, 20, 1] = float("inf")
        with np.errstate(all="ignore"):
            bad = ~np.isfinite(reference(d, True)["out"])
        want = np.zeros_like(bad)
        want[20:20 + W, 1] = True
        assert (bad == want).all()
