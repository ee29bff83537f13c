"""Which outputs may take an input's buffer.  Where a kernel would read what another thread has
overwritten the call is refused before any launch; where every element is read by the thread that
later writes it the result is the same as in a buffer of its own."""
import ctypes

import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import dev
from kimi_delta_attention_22_b200 import build as kbuild
from test_block_conv import draw as draw_conv
from test_block_ssm import backward
from test_block_ssm import draw as draw_ssm

BF, F32 = torch.bfloat16, torch.float32


def at(k):
    """Distinct addresses that nothing reads: the calls of the tests without a GPU end in their checks."""
    return ctypes.c_void_p(0x1000000 * k)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


# ---------------------------------------------------------------- gradients of the states


@pytest.mark.parametrize("dstate", [8, 9])   # state0's buffer, d_stateT's
def test_conv_state_gradient(lib, dstate):
    """The runs of a sequence read its state and its final state's gradient while others store."""
    sh = kda.ConvShape(2, 300, 16, 2, 4, kda.KDA_BF16, kda.KDA_BF16, 1, 0, None)
    need = lib.kda_conv_bwd_workspace_size(ctypes.byref(sh))
    assert lib.kda_conv_bwd(ctypes.byref(sh), at(1), at(2), None, at(8), None, at(3), at(9), at(4), at(5), None, at(dstate),
                            at(6), need, None) == 1


def test_scan_state_gradient(lib):
    """The segment with a sequence's first row stores dh0, the one with its last reads d_hT."""
    sh = kda.SsmShape(1, 600, 16, 16, 1, 1, kda.KDA_BF16, 1, 0, 0, 0, 0, 0, None)
    need = lib.kda_ssm_bwd_workspace_size(ctypes.byref(sh), 0)
    assert lib.kda_ssm_bwd(ctypes.byref(sh), at(1), at(2), at(3), at(4), at(5), None, None, None, at(8), None, at(6), at(9),
                           at(11), at(12), at(13), at(14), at(15), None, None, None, at(9), at(7), need, None) == 1


# ---------------------------------------------------------------- outputs


def other(k, names, given):
    """Addresses by name: each its own (from k on), but for those in `given`."""
    a = {n: at(k + i) for i, n in enumerate(names)}
    a.update({n: a[i] for n, i in given.items()})
    return a


@pytest.mark.parametrize("out,inp", [("out", "x"), ("out", "state0"), ("out", "w"), ("fin", "x"), ("fin", "state0")])
def test_conv_forward(lib, out, inp):
    a = other(1, ("x", "w", "b", "state0", "out", "fin"), {out: inp})
    sh = kda.ConvShape(2, 3, 16, 2, 4, kda.KDA_F32, 0, 1, 0, None)
    assert lib.kda_conv_fwd(ctypes.byref(sh), a["x"], a["w"], a["b"], a["state0"], None, a["out"], a["fin"], None) == 1


@pytest.mark.parametrize("out,inp,stride", [("out", "state", 0), ("out", "w", 0), ("state", "x", 0), ("out", "x", 24)])
def test_conv_step(lib, out, inp, stride):
    a = other(1, ("x", "w", "b", "state", "out"), {out: inp})
    sh = kda.ConvShape(2, 1, 16, 2, 2, kda.KDA_F32, 0, 1, stride, None)
    assert lib.kda_conv_step(ctypes.byref(sh), a["x"], a["w"], a["b"], a["state"], a["out"], None) == 1


@pytest.mark.parametrize("out,inp", [("dx", "x"), ("dx", "dy"), ("dx", "state0"), ("dx", "dfin"), ("dst", "x"), ("dst", "dy")])
def test_conv_gradient(lib, out, inp):
    a = other(1, ("x", "w", "state0", "dy", "dfin", "dx", "dw", "dst", "ws"), {out: inp})
    sh = kda.ConvShape(2, 3, 16, 2, 4, kda.KDA_F32, 0, 1, 0, None)
    need = lib.kda_conv_bwd_workspace_size(ctypes.byref(sh))
    assert lib.kda_conv_bwd(ctypes.byref(sh), a["x"], a["w"], None, a["state0"], None, a["dy"], a["dfin"], a["dx"], a["dw"],
                            None, a["dst"], a["ws"], need, None) == 1


SSM_IN = ("x", "dt", "A", "B", "C", "D", "z", "bias")


@pytest.mark.parametrize("out,inp", [("out", n) for n in SSM_IN + ("h0",)] + [("hT", "x"), ("hT", "A"), ("hT", "h0")])
def test_scan_forward(lib, out, inp):
    a = other(1, SSM_IN + ("h0", "out", "hT"), {out: inp})
    sh = kda.SsmShape(2, 8, 16, 16, 1, 2, kda.KDA_F32, 1, 0, 0, 0, 0, 0, None)
    assert lib.kda_ssm_fwd(ctypes.byref(sh), *(a[n] for n in SSM_IN), a["h0"], None, a["out"], a["hT"], None, 0, None) == 1


@pytest.mark.parametrize("out,inp,strides", [("out", n, (0, 0, 0)) for n in ("A", "B", "C", "D", "bias", "h")] +
                         [("h", "x", (0, 0, 0)), ("h", "A", (0, 0, 0)), ("out", "x", (24, 0, 0)), ("out", "dt", (0, 24, 0)),
                          ("out", "z", (0, 0, 24))])
def test_scan_step(lib, out, inp, strides):
    a = other(1, SSM_IN + ("h", "out"), {out: inp})
    sh = kda.SsmShape(2, 1, 16, 16, 1, 2, kda.KDA_F32, 1, *strides, 0, 0, None)
    assert lib.kda_ssm_step(ctypes.byref(sh), *(a[n] for n in SSM_IN), a["h"], a["out"], None) == 1


@pytest.mark.parametrize("out", ["dx", "ddt", "dB", "dC", "dz", "dh0"])
def test_scan_gradient(lib, out):
    for inp in SSM_IN + ("dy", "h0", "dh"):
        if (out, inp) == ("dh0", "h0"):
            continue
        a = other(1, SSM_IN + ("h0", "dy", "dh", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "ws"), {out: inp})
        sh = kda.SsmShape(2, 8, 16, 16, 1, 2, kda.KDA_F32, 1, 0, 0, 0, 0, 0, None)
        need = lib.kda_ssm_bwd_workspace_size(ctypes.byref(sh), 0)
        assert lib.kda_ssm_bwd(ctypes.byref(sh), *(a[n] for n in SSM_IN), a["h0"], None, a["dy"], a["dh"], a["dx"], a["ddt"],
                               a["dA"], a["dB"], a["dC"], a["dD"], a["dz"], a["db"], a["dh0"], a["ws"], need, None) == 1, inp


@pytest.mark.parametrize("out,inp,stride", [("out", "w", 0), ("out", "b", 0), ("mean", "x", 0), ("rstd", "b", 0), ("out", "x", 72)])
def test_norm_forward(lib, out, inp, stride):
    a = other(1, ("x", "w", "b", "out", "mean", "rstd"), {out: inp})
    sh = kda.NormShape(3, 1, 64, kda.KDA_F32, 1e-5, stride)
    assert lib.kda_layer_norm_fwd(ctypes.byref(sh), *a.values(), None) == 1


@pytest.mark.parametrize("out,inp,stride", [("dx", "w", 0), ("dx", "mean", 0), ("dx", "rstd", 0), ("dx", "x", 72)])
def test_norm_gradient(lib, out, inp, stride):
    a = other(1, ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"), {out: inp})
    sh = kda.NormShape(3, 1, 64, kda.KDA_F32, 1e-5, stride)
    need = lib.kda_layer_norm_bwd_workspace_size(ctypes.byref(sh))
    assert lib.kda_layer_norm_bwd(ctypes.byref(sh), *a.values(), need, None) == 1


def pairs(names):
    return [(a, b) for i, a in enumerate(names) for b in names[i + 1:]]


def test_two_outputs_at_one_address(lib):
    sh = kda.ConvShape(2, 3, 16, 2, 4, kda.KDA_F32, 0, 1, 0, None)
    a = other(1, ("x", "w", "b", "state0", "out", "fin"), dict(fin="out"))
    assert lib.kda_conv_fwd(ctypes.byref(sh), a["x"], a["w"], a["b"], a["state0"], None, a["out"], a["fin"], None) == 1
    need = lib.kda_conv_bwd_workspace_size(ctypes.byref(sh))
    for p, q in pairs(("dx", "dw", "db", "dst")):
        a = other(1, ("x", "w", "b", "dy", "dx", "dw", "db", "dst", "ws"), {q: p})
        assert lib.kda_conv_bwd(ctypes.byref(sh), a["x"], a["w"], a["b"], None, None, a["dy"], None, a["dx"], a["dw"], a["db"],
                                a["dst"], a["ws"], need, None) == 1, (p, q)
    sh = kda.SsmShape(2, 8, 16, 16, 1, 2, kda.KDA_F32, 1, 0, 0, 0, 0, 0, None)
    a = other(1, SSM_IN + ("out", "hT"), dict(hT="out"))
    assert lib.kda_ssm_fwd(ctypes.byref(sh), *(a[n] for n in SSM_IN), None, None, a["out"], a["hT"], None, 0, None) == 1
    need = lib.kda_ssm_bwd_workspace_size(ctypes.byref(sh), 0)
    outs = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0")
    for p, q in pairs(outs):
        a = other(1, SSM_IN + ("dy",) + outs + ("ws",), {q: p})
        assert lib.kda_ssm_bwd(ctypes.byref(sh), *(a[n] for n in SSM_IN), None, None, a["dy"], None, *(a[n] for n in outs), a["ws"],
                               need, None) == 1, (p, q)
    sh = kda.NormShape(3, 1, 64, kda.KDA_F32, 1e-5, 0)
    for p, q in pairs(("out", "mean", "rstd")):
        a = other(1, ("x", "w", "b", "out", "mean", "rstd"), {q: p})
        assert lib.kda_layer_norm_fwd(ctypes.byref(sh), *a.values(), None) == 1, (p, q)
    need = lib.kda_layer_norm_bwd_workspace_size(ctypes.byref(sh))
    for p, q in pairs(("dx", "dw", "db")):
        a = other(1, ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"), {q: p})
        assert lib.kda_layer_norm_bwd(ctypes.byref(sh), *a.values(), need, None) == 1, (p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 64), (F32, 64), (BF, 13), (F32, 300), (BF, 4096)])
def test_what_may_be_in_place(dtype, D):
    """Steps on x, delta or z, norms on x, the norm's gradient on x or d_out: as in a buffer of its own."""
    g = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    n = 37
    x, dt, z, dy = (r(n, D).to(dtype) for _ in range(4))
    w, st = r(D, 4), r(n, 3, D).to(dtype)
    s1, s2, y = st.clone(), st.clone(), x.clone()
    assert torch.equal(kda.kda_conv_step(y, w, s1, out=y), kda.kda_conv_step(x, w, s2)) and torch.equal(s1, s2)
    A, B, C, h = -torch.exp(r(D, 16)), r(n, 16).to(dtype), r(n, 16).to(dtype), r(n, D, 16)
    h2 = h.clone()
    want = kda.kda_ssm_step(x, dt, A, B, C, h2, z=z)
    for k in range(3):
        v, h1 = [t.clone() for t in (x, dt, z)], h.clone()
        assert torch.equal(kda.kda_ssm_step(v[0], v[1], A, B, C, h1, z=v[2], out=v[k]), want) and torch.equal(h1, h2), k
    nw, nb, y = r(D), r(D), x.clone()
    want = kda.kda_layer_norm_fwd(x, nw, nb)
    got = kda.kda_layer_norm_fwd(y, nw, nb, out=y)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    want = kda.kda_layer_norm_bwd(dy, x, *want[1:], nw)
    for k in range(2):
        v = [dy.clone(), x.clone()]
        gr = kda.kda_layer_norm_bwd(v[0], v[1], *got[1:], nw, grads=dict(dx=v[k]))
        assert all(torch.equal(gr[i], want[i]) for i in want), k
    if D >= 64:   # a slice of a wider matrix starts where a smaller, contiguous output would
        wide = r(n, 2 * D).to(dtype)
        part, out = wide[:, :D], wide.view(-1)[:n * D].view(n, D)
        for call in (lambda: kda.kda_conv_step(part, w, s1, out=out), lambda: kda.kda_layer_norm_fwd(part, nw, nb, out=out),
                     lambda: kda.kda_ssm_step(part, dt, A, B, C, h2, out=out),
                     lambda: kda.kda_layer_norm_bwd(dy, part, *got[1:], nw, grads=dict(dx=out))):
            with pytest.raises(kda.KDAError):
                call()


@pytest.mark.gpu
def test_state_gradients_are_refused_by_the_binding():
    c = dev(draw_conv(1, 300, 16, 4, F32, [0, 2, 300]))
    args = c["x"], c["w"], c["dy"], c["bias"], c["state"], c["dfin"], c["cu"]
    for name in ("state", "dfin"):
        with pytest.raises(kda.KDAError):
            kda.kda_conv_bwd(*args, grads=dict(dstate=c[name]))
    s = dev(draw_ssm(1, 600, 16, 16, 1, F32, [0, 2, 600]))
    with pytest.raises(kda.KDAError):
        backward(s, grads=dict(dh0=s["dh"]))


@pytest.mark.gpu
def test_scan_state_gradient_in_place_of_the_state():
    """h0 is read for a sequence's first row by the thread that then stores dh0 there."""
    s = dev(draw_ssm(1, 900, 24, 16, 1, F32, [0, 300, 301, 301, 900]))
    want = backward(s)
    h0 = s["h0"].clone()
    got = backward(dict(s, h0=h0), grads=dict(dh0=h0))
    assert got["dh0"] is h0
    for k in want:
        assert torch.equal(got[k], want[k]), k
