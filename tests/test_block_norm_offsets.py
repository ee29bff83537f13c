"""Layer norm's gradient on rows whose mean is far above their deviation.  The mean and 1 / deviation
are the call's inputs, so the reference takes them as they are, and the only digits that may be lost
are those of fp32 arithmetic on x - mean, which is exact where the two are within a factor of two.

Steps: xhat two roundings, the products one or two; the two sums in chains of at most 32 per lane
and 12 exchanges, 48; their quotients and the factors of dx six, its two multiply-adds two: 64, each
2^-24 of the terms' absolute values, in which xhat and not x stands."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, rnd
from oracle import block as ob

BF, F32 = torch.bfloat16, torch.float32


def gradient(dy, x, mean, rstd, w, mag=False):
    """dx, dw, db of out = (x - mean) rstd w + b for the given mean and rstd [R, G]."""
    a = np.abs if mag else (lambda v: v)
    r = rstd[..., None]
    xh, gw = a((x - mean[..., None]) * r), a(dy) * a(w)
    c1, c2 = gw.mean(-1, keepdims=True), (gw * xh).mean(-1, keepdims=True)
    return r * (gw + c1 + xh * c2 if mag else gw - c1 - xh * c2), (a(dy) * xh).sum(0), a(dy).sum(0)


# rows, groups, D, type, mean, deviation: every layout with rows ahead, without, and of elements
CASES = [(5, 1, 64, F32, 1e3, 1e-2), (9, 3, 128, F32, -3e4, 1.0), (4, 1, 1000, F32, 1e5, 1.0), (6, 1, 2048, F32, 1e3, 1e-3),
         (3, 1, 4096, F32, 1.0, 1e-5), (5, 1, 250, F32, 1e4, 0.1), (2, 1, 8191, F32, 1e3, 1e-2), (2, 1, 16384, F32, 1e3, 1e-2),
         (2, 1, 32768, F32, -1e4, 1.0), (7, 1, 1024, BF, 100.0, 1.0), (5, 1, 4096, BF, -200.0, 2.0), (3, 1, 4095, BF, 64.0, 1.0),
         (2, 1, 32768, BF, 128.0, 1.0), (40, 16, 64, BF, 50.0, 0.5)]


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,D,dtype,mean,dev", CASES)
def test_gradient(R, G, D, dtype, mean, dev):
    gen = torch.Generator().manual_seed(D + R)
    x = (mean + dev * rnd(gen, R, G, D, dtype=torch.float64)).to(dtype)
    w, dy = 1 + 0.3 * rnd(gen, G, D), rnd(gen, R, G, D, dtype=dtype)
    f = ob.f64
    m = f(x).mean(-1)
    m, s = (torch.from_numpy(v).float() for v in (m, 1 / np.sqrt(f(x).var(-1) + 1e-12)))
    g = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), m.cuda(), s.cuda(), w.cuda())
    r, mag = (gradient(f(dy), f(x), f(m), f(s), f(w), k) for k in (False, True))
    close(g["dx"], r[0], mag[0], 64, "dx")
    close(g["dweight"], r[1], mag[1], 64 + R, "dweight")
    close(g["dbias"], r[2], mag[2], 8 + R, "dbias")


def test_the_reference_is_the_norm_s_gradient():
    """With the row's own mean and deviation: the gradient of the other reference."""
    gen = torch.Generator().manual_seed(1)
    x, w, dy = rnd(gen, 4, 2, 9, dtype=torch.float64), rnd(gen, 2, 9, dtype=torch.float64), rnd(gen, 4, 2, 9, dtype=torch.float64)
    x, w, dy = (t.numpy() for t in (x, w, dy))
    r = ob.norm(x, w, 0 * w, 1e-5, dy)
    for a, b in zip(gradient(dy, x, r["mean"], r["rstd"], w), (r["dx"], r["dw"], r["db"])):
        assert np.abs(a - b).max() < 1e-12
