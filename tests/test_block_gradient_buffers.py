"""Buffers that the caller gives for gradients are written, or the call is refused."""
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import dev
from test_block_conv import draw as draw_conv
from test_block_ssm import backward
from test_block_ssm import draw as draw_ssm

F32 = torch.float32


def buffers(g):
    return {k: torch.full_like(v, 7.0) for k, v in g.items() if v is not None}


def same(got, want, bufs):
    for k, v in bufs.items():
        assert got[k] is v and torch.equal(v, want[k]), k


@pytest.mark.gpu
def test_every_buffer_is_written():
    c = dev(draw_conv(1, 40, 16, 4, F32))
    args = c["x"], c["w"], c["dy"], c["bias"], c["state"], c["dfin"]
    want = kda.kda_conv_bwd(*args)
    b = buffers(want)
    same(kda.kda_conv_bwd(*args, grads=b), want, b)
    s = dev(draw_ssm(1, 40, 16, 16, 1, F32))
    want = backward(s)
    b = buffers(want)
    assert len(b) == 9
    same(backward(s, grads=b), want, b)
    x, w = torch.randn(9, 64, device="cuda"), torch.randn(64, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x, w)
    want = kda.kda_layer_norm_bwd(x, x, mean, rstd, w)
    b = buffers(want)
    same(kda.kda_layer_norm_bwd(x, x, mean, rstd, w, grads=b), want, b)


@pytest.mark.gpu
def test_a_buffer_that_stays_unwritten_is_refused():
    c = dev(draw_conv(1, 40, 16, 4, F32))
    t = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="dbias"):
        kda.kda_conv_bwd(c["x"], c["w"], c["dy"], grads=dict(dbias=t(16)))
    with pytest.raises(ValueError, match="dstate"):
        kda.kda_conv_bwd(c["x"], c["w"], c["dy"], want_dstate=False, grads=dict(dstate=t(1, 3, 16)))
    kda.kda_conv_bwd(c["x"], c["w"], c["dy"], want_dstate=False, grads=dict(dstate=None, dbias=None))
    s = dev(draw_ssm(1, 40, 16, 16, 1, F32))
    for name, buf, drop in (("dD", t(16), "D"), ("dz", t(1, 40, 16), "z"), ("ddt_bias", t(16), "dt_bias")):
        with pytest.raises(ValueError, match=name):
            backward(dict(s, **{drop: None}), grads={name: buf})
    with pytest.raises(ValueError, match="dh0"):
        backward(s, want_dh0=False, grads=dict(dh0=t(1, 16, 16)))
    x = torch.randn(9, 64, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x)
    for name in ("dweight", "dbias"):
        with pytest.raises(ValueError, match=name):
            kda.kda_layer_norm_bwd(x, x, mean, rstd, want_params=False, grads={name: t(64)})
    with pytest.raises(ValueError, match="unknown"):
        kda.kda_layer_norm_bwd(x, x, mean, rstd, grads=dict(dw=t(64)))
