"""Layer norm: forward and gradients against the float64 reference, for rows of one element
to rows longer than a CTA's registers, odd sizes, groups, strides, missing parameters; constant
rows; refusals; the reference's gradients against differences.

Steps (see block_cases): a mean over D elements is summed in chains of at most 32 per lane and
12 exchanges, 48 steps with the quotient; the deviations, the variance and its root as much again,
the weights two more: 128.  The gradient's two sums add 64; dw and db are sums over the rows."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, rnd, strided_like
from kimi_delta_attention_22_b200 import build as kbuild
from oracle import block as ob
from test_block_conv import _differences

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def draw(R, G, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = rnd(g, R, G, D) * 1.5 + 0.4 * rnd(g, R, G, 1)
    return x.to(dtype), 1 + 0.3 * rnd(g, G, D), 0.2 * rnd(g, G, D), rnd(g, R, G, D, dtype=dtype)


# every layout of a row: lanes per row 8 to 1024, one to many accesses per lane, element accesses
SHAPES = [(1, 1, 1, F32), (3, 1, 1, BF), (5, 1, 7, BF), (9, 2, 8, BF), (300, 1, 32, F32), (17, 1, 33, F32), (40, 16, 64, BF),
          (33, 3, 128, BF), (5, 1, 250, F32), (70, 1, 256, BF), (9, 2, 512, BF), (6, 1, 1000, F32), (5, 1, 1024, BF),
          (4, 1, 1023, BF), (3, 1, 2048, BF), (7, 1, 4096, BF), (3, 1, 4100, F32), (2, 1, 8191, BF), (3, 1, 8192, F32),
          (2, 2, 16384, BF), (2, 1, 16384, F32), (2, 1, 32768, BF), (1, 1, 32768, F32), (1, 1, 32767, F32),
          (5, 3, 313, BF), (4, 1, 700, F32), (3, 1, 2047, BF), (3, 2, 4095, F32), (3, 1, 4097, BF), (2, 1, 12345, BF),
          (9, 2, 200, F32), (6, 1, 400, F32), (4, 1, 1800, F32), (3, 1, 6000, BF), (3, 1, 2052, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,D,dtype", SHAPES)
def test_forward(R, G, D, dtype):
    x, w, b, _ = draw(R, G, D, dtype, seed=R + D)
    out, mean, rstd = kda.kda_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), EPS)
    f = ob.f64
    r, m = ob.norm(f(x), f(w), f(b), EPS), ob.norm(f(x), f(w), f(b), EPS, mag=True)
    close(out, r["out"], m["out"], 128, "out")
    close(mean, r["mean"], m["mean"], 48, "mean")
    if D > 1:   # a relative error of the variance is half as large in rstd
        close(rstd, r["rstd"], r["rstd"] * (1 + m["mean"] ** 2 * r["rstd"] ** 2), 128, "rstd")
    plain, mean2, rstd2 = kda.kda_layer_norm_fwd(x.cuda(), want_stats=False)
    assert mean2 is None and rstd2 is None
    one = np.ones((1, D))
    close(plain, ob.norm(f(x), one, 0 * one, EPS)["out"], ob.norm(f(x), one, 0 * one, EPS, mag=True)["out"], 128, "without parameters")


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,D,dtype", SHAPES)
def test_backward(R, G, D, dtype):
    x, w, b, dy = draw(R, G, D, dtype, seed=R + 2 * D)
    o = [t.cuda() for t in (x, w, dy)]
    _, mean, rstd = kda.kda_layer_norm_fwd(o[0], o[1], None, EPS)
    g = kda.kda_layer_norm_bwd(o[2], o[0], mean, rstd, o[1])
    f = ob.f64
    r, m = (ob.norm(f(x), f(w), f(b), EPS, f(dy), mag=k) for k in (False, True))
    close(g["dx"], r["dx"], m["dx"], 320, "dx")
    close(g["dweight"], r["dw"], m["dw"], 160 + R, "dweight")
    close(g["dbias"], r["db"], m["db"], 8 + R, "dbias")


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,D", [(5000, 1, 96), (3001, 4, 64), (2500, 1, 1536)])
def test_many_rows(R, G, D):
    """More rows than CTAs: the parameter gradients' partial sums and their join."""
    x, w, b, dy = draw(R, G, D, BF, seed=D)
    _, mean, rstd = kda.kda_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), EPS)
    g = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    again = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    f = ob.f64
    r, m = (ob.norm(f(x), f(w), f(b), EPS, f(dy), mag=k) for k in (False, True))
    close(g["dx"], r["dx"], m["dx"], 320, "dx")
    close(g["dweight"], r["dw"], m["dw"], 160 + R, "dweight")
    close(g["dbias"], r["db"], m["db"], 8 + R, "dbias")
    for k in g:
        assert torch.equal(g[k], again[k])
    only = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda(), want_params=False)
    assert only["dweight"] is None and torch.equal(only["dx"], g["dx"])


@pytest.mark.gpu
@pytest.mark.parametrize("shift,pad", [(0, 8), (8, 24), (1, 3)])
def test_row_strided_input(shift, pad):
    x, w, b, dy = (t.cuda() for t in draw(50, 4, 64, BF, seed=2))
    xs = strided_like(x.reshape(50, 256), pad + shift, shift).unflatten(-1, (4, 64))
    assert not xs.is_contiguous()
    a, c = kda.kda_layer_norm_fwd(x, w, b), kda.kda_layer_norm_fwd(xs, w, b)
    for u, v in zip(a, c):
        assert torch.allclose(u.float(), v.float(), rtol=2.0 ** -7, atol=1e-6)   # another order of the sums: one bf16 step
    g, h = kda.kda_layer_norm_bwd(dy, x, a[1], a[2], w), kda.kda_layer_norm_bwd(dy, xs, a[1], a[2], w)
    assert torch.allclose(g["dx"].float(), h["dx"].float(), rtol=2.0 ** -7, atol=1e-6)
    assert torch.allclose(g["dweight"], h["dweight"], rtol=1e-4, atol=1e-4)


@pytest.mark.gpu
def test_constant_and_special_rows():
    """A constant row has variance 0: out = bias; a NaN or an infinity stays in its row."""
    x = torch.randn(6, 256, device="cuda")
    x[1] = 3.0
    x[3, 17] = float("nan")
    x[4, 200] = float("inf")
    b = torch.randn(256, device="cuda")
    out, mean, rstd = kda.kda_layer_norm_fwd(x, None, b, EPS)
    assert torch.equal(out[1], b) and mean[1] == 3.0
    fin = torch.isfinite(out).all(-1).tolist()
    assert fin == [True, True, True, False, False, True]
    big = torch.full((2, 512), 1000.0, device="cuda") + torch.randn(2, 512, device="cuda") * 1e-2   # no cancellation of moments
    out, _, _ = kda.kda_layer_norm_fwd(big)
    d = big.double()
    ref = (d - d.mean(-1, keepdim=True)) / (d.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
    # the mean is off by 48 half steps of 1000 at most: 48 * 2^-24 * 1000 over a deviation of 1e-2
    assert (out.double() - ref).abs().max() < 48 * 2.0 ** -24 * 1000 / 1e-2


@pytest.mark.gpu
def test_empty_and_refusals():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    out, mean, rstd = kda.kda_layer_norm_fwd(x, w)
    assert out.shape == (0, 64) and mean.shape == (0,)
    g = kda.kda_layer_norm_bwd(out, x, mean, rstd, w)
    assert g["dweight"].eq(0).all() and g["dbias"].eq(0).all()
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(TypeError):
        kda.kda_layer_norm_fwd(x.half())
    with pytest.raises(TypeError):
        kda.kda_layer_norm_fwd(x, w.bfloat16())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, torch.ones(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x.t())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x.cpu())
    with pytest.raises(kda.KDAError):
        kda.kda_layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(kda.KDAError):
        kda.kda_layer_norm_fwd(torch.zeros(1, 32769, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_bwd(x, x, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))


def test_validation(lib):
    P = ctypes.c_void_p
    A = P(0x10000)

    def sh(rows=0, G=1, D=64, dt=kda.KDA_BF16, eps=1e-5, xs=0):
        return kda.NormShape(rows, G, D, dt, eps, xs)

    def fwd(s, x=A, out=A, mean=None, rstd=None, w=None):
        return lib.kda_layer_norm_fwd(None if s is None else ctypes.byref(s), x, w, None, out, mean, rstd, None)

    assert fwd(None) == 1 and fwd(sh()) == 0
    assert fwd(sh(rows=-1)) == 1 and fwd(sh(G=0)) == 1 and fwd(sh(D=0)) == 1 and fwd(sh(dt=9)) == 1
    assert fwd(sh(eps=-1e-3)) == 1 and fwd(sh(eps=float("nan"))) == 1 and fwd(sh(xs=63)) == 1 and fwd(sh(xs=64)) == 0
    assert fwd(sh(D=32769)) == 2 and fwd(sh(G=65536)) == 2
    assert fwd(sh(rows=1), x=None) == 1 and fwd(sh(rows=1), mean=A) == 1
    assert fwd(sh(), x=P(0x10001)) == 3 and fwd(sh(), w=P(0x10002)) == 3

    def bwd(s, ws=A, nb=0, dw=A, db=A, mean=A):
        return lib.kda_layer_norm_bwd(ctypes.byref(s), A, A, None, mean, A, A, dw, db, ws, nb, None)

    s = sh(rows=100)
    need = lib.kda_layer_norm_bwd_workspace_size(ctypes.byref(s))
    assert need > 0 and lib.kda_layer_norm_bwd_workspace_size(None) == 0
    assert bwd(s, nb=need - 1) == 1 and bwd(s, ws=P(0x10010), nb=need) == 3 and bwd(s, nb=need, mean=None) == 1
    assert bwd(sh(), dw=None, db=None) == 0


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(2)
    R, G, D = 3, 2, 5
    v = dict(x=rng.standard_normal((R, G, D)), w=rng.standard_normal((G, D)), b=rng.standard_normal((G, D)))
    dy = rng.standard_normal((R, G, D))
    r = ob.norm(v["x"], v["w"], v["b"], EPS, dy)
    for name, grad in (("x", "dx"), ("w", "dw"), ("b", "db")):
        _differences(lambda: (ob.norm(v["x"], v["w"], v["b"], EPS)["out"] * dy).sum(), v[name], r[grad], name)
