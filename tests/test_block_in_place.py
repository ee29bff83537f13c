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
