"""The short causal convolution: forward, one-row step and gradients against the float64
reference, for every tap count, type and alignment, packed and dense, with and without state,
sequences of zero, one and few rows (shorter than the window), and rows behind the last
sequence; refusals; the reference's gradients against differences.

Steps (see block_cases): the pre-activation is W fused multiply-adds and a bias; SiLU adds an
exponential, a sum, a quotient and a product of a few units each: 2 W + 32.  dx adds W products
over those; dw and db are sums over the rows, in chains of at most the rows themselves."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, dev, lengths, rnd, strided_like
from kimi_delta_attention_22_b200 import build as kbuild
from oracle import block as ob

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def draw(B, T, D, W, dtype, cu=None, state=True, bias=True, grad=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    return dict(x=rnd(g, B, T, D, dtype=dtype), w=rnd(g, D, W, scale=0.6), bias=rnd(g, D, scale=0.3) if bias else None,
                state=rnd(g, n, W - 1, D, dtype=dtype) if state else None, dy=rnd(g, B, T, D, dtype=grad or dtype),
                dfin=rnd(g, n, W - 1, D, dtype=dtype), cu=None if cu is None else torch.tensor(cu, dtype=torch.int32))


def reference(d, act, bwd=False, mag=False):
    B, T, D = d["x"].shape
    cu = None if d["cu"] is None else d["cu"].tolist()
    return ob.conv(ob.f64(d["x"]).reshape(-1, D), ob.f64(d["w"]), ob.f64(d["bias"]), ob.f64(d["state"]),
                   ob.bounds(B, T, cu), act, ob.f64(d["dy"]).reshape(-1, D) if bwd else None,
                   ob.f64(d["dfin"]) if bwd and d["dfin"] is not None else None, mag)


# B, T, D, W, dtype, sequence lengths (None: dense), state, bias, SiLU
CASES = [
    (2, 37, 64, 4, BF, None, True, True, True),
    (1, 1, 8, 4, BF, None, True, True, True),
    (3, 2, 24, 4, F32, None, True, False, True),          # fewer rows than taps
    (2, 65, 13, 3, BF, None, True, True, True),           # odd channels: element accesses
    (1, 130, 40, 2, F32, None, False, True, False),
    (2, 33, 48, 5, BF, None, True, True, True),
    (1, 40, 16, 6, F32, None, True, False, False),
    (1, 50, 12, 7, BF, None, False, True, True),
    (2, 70, 32, 8, BF, None, True, True, True),
    (1, 9, 20, 8, F32, None, True, True, True),
    (1, 0, 16, 4, BF, [0, 0, 0], True, True, True),       # nothing but empty sequences
    (1, 100, 64, 4, BF, [0, 1, 40, 0, 2, 3, 54, 0], True, True, True),
    (1, 90, 136, 4, F32, [33, 31, 1, 1, 20], True, True, True),   # four rows behind the last sequence
    (1, 90, 7, 4, BF, [90], False, False, True),
    (1, 300, 520, 4, BF, [1, 255, 44], True, True, False),
    (2, 0, 16, 4, F32, None, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,W,dtype,lens,state,bias,act", CASES)
def test_forward(B, T, D, W, dtype, lens, state, bias, act):
    cu = None if lens is None else lengths(lens)
    d = draw(B, T, D, W, dtype, cu, state, bias, seed=T + D)
    o = dev(d)
    out = torch.full((B, T, D), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], o["cu"], silu=act, out=out, dev_status=st)
    assert y is out and st.item() == 0
    r, m = reference(d, act), reference(d, act, mag=True)
    used = T if cu is None else cu[-1]
    flat = out.reshape(-1, D) if B * T else out.reshape(0, D)
    n = flat.shape[0] if cu is None else used
    close(flat[:n], r["out"][:n], m["out"][:n], 2 * W + 32, "out")
    assert (flat[n:] == 7.0).all()                                 # rows behind the last sequence
    assert torch.equal(fin.cpu().double(), torch.from_numpy(r["final"]))   # copies, bit for bit


@pytest.mark.gpu
@pytest.mark.parametrize("grad32", [False, True])
@pytest.mark.parametrize("B,T,D,W,dtype,lens,state,bias,act", CASES)
def test_backward(B, T, D, W, dtype, lens, state, bias, act, grad32):
    cu = None if lens is None else lengths(lens)
    d = draw(B, T, D, W, dtype, cu, state, bias, F32 if grad32 else None, seed=T + 3 * D)
    if not state:
        d["dfin"] = None
    o = dev(d)
    dx = torch.full((B, T, D), 7.0, dtype=dtype, device="cuda")
    g = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], o["cu"], silu=act,
                         want_dstate=state, grads=dict(dx=dx))
    r, m = reference(d, act, True), reference(d, act, True, True)
    n = B * T if cu is None else cu[-1]
    flat = g["dx"].reshape(B * T, D)
    close(flat[:n], r["dx"][:n], m["dx"][:n], 3 * W + 40, "dx")
    assert (flat[n:] == 7.0).all()
    close(g["dweight"], r["dw"], m["dw"], 2 * W + 40 + n, "dweight")
    if bias:
        close(g["dbias"], r["db"], m["db"], 2 * W + 40 + n, "dbias")
    else:
        assert g["dbias"] is None
    if state:
        close(g["dstate"], r["dstate"], m["dstate"], 3 * W + 40, "dstate")
    else:
        assert g["dstate"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,W,dtype", [(1, 8, 4, BF), (5, 64, 4, BF), (3, 13, 3, F32), (7, 40, 2, BF), (2, 24, 8, BF),
                                         (3, 20, 6, F32), (33, 257, 4, F32)])
def test_steps_equal_forward(N, D, W, dtype):
    """Steps from a state give the forward's rows and final state, bit for bit."""
    T = 2 * W + 1
    o = dev(draw(N, T, D, W, dtype, seed=N))
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"])
    s = o["state"].clone()
    for t in range(T):
        row = kda.kda_conv_step(o["x"][:, t], o["w"], s, bias=o["bias"])   # strided rows
        assert torch.equal(row, y[:, t]), t
    assert torch.equal(s, fin)


@pytest.mark.gpu
def test_split_prompt_equals_whole():
    """A prompt in two calls, the second from the first's final state."""
    o = dev(draw(2, 41, 48, 4, BF, seed=5))
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"])
    for cut in (1, 2, 17, 40):
        y1, f1 = kda.kda_conv_fwd(o["x"][:, :cut].contiguous(), o["w"], o["bias"], o["state"])
        y2, f2 = kda.kda_conv_fwd(o["x"][:, cut:].contiguous(), o["w"], o["bias"], f1)
        assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(f2, fin)


@pytest.mark.gpu
@pytest.mark.parametrize("shift,pad", [(0, 8), (8, 24), (1, 3)])
def test_row_strided_input(shift, pad):
    o = dev(draw(2, 50, 64, 4, BF, seed=9))
    xs = strided_like(o["x"], pad + shift, shift)
    assert not xs.is_contiguous()
    a, b = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"]), kda.kda_conv_fwd(xs, o["w"], o["bias"], o["state"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"])
    gb = kda.kda_conv_bwd(xs, o["w"], o["dy"], o["bias"], o["state"], o["dfin"])
    for k in ("dx", "dstate"):
        assert torch.equal(ga[k], gb[k])
    assert torch.allclose(ga["dweight"], gb["dweight"], rtol=1e-4, atol=1e-4)   # another order of the same sums


@pytest.mark.gpu
def test_special_values_stay_in_their_window():
    d = draw(1, 40, 16, 4, F32, state=False, seed=3)
    d["x"][0, 10, 3] = float("nan")
    d["x"][0, 20, 5] = float("inf")
    o = dev(d)
    y, _ = kda.kda_conv_fwd(o["x"], o["w"], o["bias"])
    bad = ~torch.isfinite(y[0])
    want = torch.zeros_like(bad)
    want[10:14, 3] = True
    hit = torch.isfinite(y[0, 20:24, 5])   # silu(-inf) has no value, silu(inf) is inf
    assert not hit.any()
    want[20:24, 5] = True
    assert torch.equal(bad, want)


@pytest.mark.gpu
def test_bad_values_stay_in_their_sequence():
    """A NaN sequence, and NaN rows of no sequence, leave the others as they were, bit for bit."""
    lens = [40, 3, 70, 1, 90]
    cu = lengths(lens)
    d = draw(1, cu[-1] + 7, 24, 4, BF, cu, seed=31)
    o = dev(d)
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], o["cu"])
    g = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], o["cu"])
    for bad in range(5):
        p = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in o.items()}
        for k in ("x", "dy"):
            p[k][:, cu[bad]:cu[bad + 1]] = float("nan")
            p[k][:, cu[-1]:] = float("nan")
        p["state"][bad] = p["dfin"][bad] = float("nan")
        y2, fin2 = kda.kda_conv_fwd(p["x"], p["w"], p["bias"], p["state"], p["cu"])
        g2 = kda.kda_conv_bwd(p["x"], p["w"], p["dy"], p["bias"], p["state"], p["dfin"], p["cu"])
        keep = [n for n in range(5) if n != bad]
        rows = torch.cat([torch.arange(cu[n], cu[n + 1]) for n in keep]).cuda()
        assert torch.equal(y2[:, rows], y[:, rows]) and torch.equal(fin2[keep], fin[keep])
        assert torch.equal(g2["dx"][:, rows], g["dx"][:, rows]) and torch.equal(g2["dstate"][keep], g["dstate"][keep])
    p = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in o.items()}
    for k in ("x", "dy"):
        p[k][:, cu[-1]:] = float("nan")
    g2 = kda.kda_conv_bwd(p["x"], p["w"], p["dy"], p["bias"], p["state"], p["dfin"], p["cu"])
    assert torch.equal(g2["dweight"], g["dweight"]) and torch.equal(g2["dbias"], g["dbias"])


@pytest.mark.gpu
def test_inconsistent_cu_seqlens_is_flagged():
    """A broken bound sets the status word; consistent neighbours keep their rows; no row of
    another sequence is written."""
    o = dev(draw(1, 64, 16, 4, BF, [0, 20, 40, 64], seed=8))
    good, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], o["cu"])
    for bad in ([0, 20, 70, 64], [0, 40, 20, 64], [0, 20, -5, 64], [5, 20, 40, 64]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], cu, dev_status=st)
        assert st.item() == kda.KDA_DEV_BAD_SEQLENS, bad
        st.zero_()
        kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], cu, dev_status=st)
        assert st.item() == kda.KDA_DEV_BAD_SEQLENS, bad


@pytest.mark.gpu
def test_binding_refusals():
    o = dev(draw(2, 8, 16, 4, BF, seed=1))
    x, w = o["x"], o["w"]
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(x.half(), w)
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(x, w.bfloat16())
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w[:8])
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x.transpose(1, 2), w)                  # channels not contiguous
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x[:, :1].expand(2, 8, 16), w)          # broadcast rows
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, state=o["state"][:1])
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))   # B = 2
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x.cpu(), w)
    with pytest.raises(kda.KDAError):
        kda.kda_conv_fwd(x, torch.zeros(16, 9, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.kda_conv_fwd(x, w, state=o["state"], final_state=o["state"])
    with pytest.raises(kda.KDAError):
        kda.kda_conv_fwd(x, w, out=x)
    with pytest.raises(ValueError):
        kda.kda_conv_bwd(x, w, o["dy"], grads=dict(dw=w))
    with pytest.raises(TypeError):
        kda.kda_conv_bwd(x.float(), w, o["dy"])                  # bf16 gradient of an fp32 input


def test_validation(lib):
    """Answers of the C entry points before any launch (the addresses are never touched)."""
    P = ctypes.c_void_p
    A = P(0x10000)

    def sh(B=0, T=8, D=16, n=None, W=4, dt=kda.KDA_BF16, gd=kda.KDA_BF16, act=1, xs=0):
        return kda.ConvShape(B, T, D, B if n is None else n, W, dt, gd, act, xs, None)

    def fwd(s, x=A, w=A, st=None, cu=None, out=A, fin=None):
        return lib.kda_conv_fwd(None if s is None else ctypes.byref(s), x, w, None, st, cu, out, fin, None)

    assert fwd(None) == 1 and fwd(sh()) == 0
    assert fwd(sh(n=2)) == 1 and fwd(sh(B=2, n=0), cu=A) == 1 and fwd(sh(D=0)) == 1 and fwd(sh(T=-1)) == 1
    assert fwd(sh(W=0)) == 1 and fwd(sh(W=1)) == 2 and fwd(sh(W=9)) == 2
    assert fwd(sh(dt=5)) == 1 and fwd(sh(act=2)) == 1 and fwd(sh(xs=8)) == 1 and fwd(sh(xs=16)) == 0
    assert fwd(sh(), w=None) == 1 and fwd(sh(B=1), x=None) == 1
    assert fwd(sh(), st=A, fin=A) == 1                            # in place is not possible
    assert fwd(sh(), x=P(0x10001)) == 3 and fwd(sh(), w=P(0x10002)) == 3 and fwd(sh(dt=kda.KDA_F32), x=P(0x10002)) == 3

    def step(s, st=A):
        return lib.kda_conv_step(ctypes.byref(s), A, A, None, st, A, None)

    assert step(sh(T=1)) == 0 and step(sh(T=2)) == 1 and step(sh(B=2, T=1), st=None) == 1

    def bwd(s, ws=A, nb=0, dw=A, dy=A):
        return lib.kda_conv_bwd(ctypes.byref(s), A, A, None, None, None, dy, None, A, dw, None, None, ws, nb, None)

    s = sh(B=2)
    need = lib.kda_conv_bwd_workspace_size(ctypes.byref(s))
    assert need > 0 and lib.kda_conv_bwd_workspace_size(None) == 0
    assert bwd(s, nb=need - 1) == 1 and bwd(s, ws=P(0x10010), nb=need) == 3
    assert bwd(s, dw=None, nb=need) == 1 and bwd(s, dy=None, nb=need) == 1
    assert bwd(sh(B=2, dt=kda.KDA_F32, gd=kda.KDA_BF16), nb=need) == 1


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    M, D, W = 7, 3, 4
    seqs = [(0, 2), (2, 2), (2, 7)]
    v = dict(x=rng.standard_normal((M, D)), w=rng.standard_normal((D, W)), bias=rng.standard_normal(D),
             state=rng.standard_normal((3, W - 1, D)))
    dy, df = rng.standard_normal((M, D)), rng.standard_normal((3, W - 1, D))
    for act in (True, False):
        def loss():
            r = ob.conv(v["x"], v["w"], v["bias"], v["state"], seqs, act)
            return (r["out"] * dy).sum() + (r["final"] * df).sum()

        r = ob.conv(v["x"], v["w"], v["bias"], v["state"], seqs, act, dy, df)
        for name, grad in (("x", "dx"), ("w", "dw"), ("bias", "db"), ("state", "dstate")):
            _differences(loss, v[name], r[grad], name)


def _differences(loss, arr, grad, name, step=1e-5):
    """Central differences of `loss` in every element of arr: off by step^2 of a third
    derivative and the loss' rounding over 2 step, about 1e-9 here."""
    flat, g = arr.reshape(-1), grad.reshape(-1)
    for i in range(flat.size):
        old = flat[i]
        flat[i] = old + step
        up = loss()
        flat[i] = old - step
        down = loss()
        flat[i] = old
        assert abs((up - down) / (2 * step) - g[i]) <= 1e-6 * (1 + abs(g[i])), (name, i)
