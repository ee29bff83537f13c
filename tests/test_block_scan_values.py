"""One infinity or NaN in the scan's inputs makes exactly those outputs and gradients non-finite that
the definition does, also where the states are padded to the lanes' number, and across segments."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import dev
from test_block_ssm import backward, draw, forward, reference

F32 = torch.float32
WHERE = ("x", "dt", "B", "C", "z", "dy", "h0", "dh")


def poison(d, key, value, t):
    at = dict(h0=(0, 3, 0), dh=(0, 3, 0), B=(0, t, 0, 0), C=(0, t, 0, 0)).get(key, (0, t, 3))
    d[key][at] = value
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("N", [1, 3, 5, 16, 20, 24, 50, 128])
@pytest.mark.parametrize("T", [40, 700])
def test_finite_where_the_definition_is(T, N, value):
    for key in WHERE:
        d = poison(draw(1, T, 16, N, 1, F32, seed=N), key, value, T // 2 + 3)
        o = dev(d)
        out, hT = forward(o)
        got = dict(out=out, hT=hT, **backward(o))
        with np.errstate(all="ignore"):
            r = reference(d, bwd=True)
        for k, v in got.items():
            a, b = torch.isfinite(v).cpu().numpy().reshape(r[k].shape), np.isfinite(r[k])
            assert (a == b).all(), (key, k, int((~a & b).sum()), int((a & ~b).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 3, 5, 16, 20, 24, 50, 128])
def test_step_finite_where_the_definition_is(N):
    for value in (float("inf"), -float("inf"), float("nan")):
        for key in ("x", "dt", "B", "C", "z", "h0"):
            d = poison(draw(1, 1, 16, N, 1, F32, seed=N), key, value, 0)
            o = dev(d)
            h = o["h0"].clone()
            out = kda.kda_ssm_step(o["x"][:, 0], o["dt"][:, 0], o["A"], o["B"][:, 0], o["C"][:, 0], h, D=o["D"], z=o["z"][:, 0],
                                   dt_bias=o["dt_bias"])
            with np.errstate(all="ignore"):
                r = reference(d)
            for v, w in ((out, r["out"]), (h, r["hT"])):
                assert (torch.isfinite(v).cpu().numpy().reshape(w.shape) == np.isfinite(w)).all(), (key, value)
