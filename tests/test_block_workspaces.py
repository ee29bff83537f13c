"""Workspaces: as large as the layouts that a call can take need, and no call writes past the bytes
that the library asked for."""
import ctypes

import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import dev, strided_like
from kimi_delta_attention_22_b200 import build as kbuild
from test_block_conv import draw as draw_conv
from test_block_norm import SHAPES
from test_block_norm import draw as draw_norm
from test_block_ssm import backward, forward
from test_block_ssm import draw as draw_ssm

BF, F32 = torch.bfloat16, torch.float32
SMS = 148


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


@pytest.mark.parametrize("rows,G,D,dtype", [(65536, 1, 4096, BF), (16384, 1, 16384, BF), (8192, 1, 32768, BF), (16384, 1, 32768, F32),
                                            (8192, 1, 4095, F32), (8192, 16, 128, BF), (1, 1, 64, F32), (0, 1, 64, BF)])
def test_norm_workspace_is_that_of_resident_ctas(lib, rows, G, D, dtype):
    """A partial sum of both parameters per CTA; of a group at most 2048 threads per SM in CTAs of a
    row's lanes: above 1024 columns a row takes 128 threads or more of at most 1024 per SM, so eight
    CTAs on each of 148 SMs, above 4096 columns of 256 and more, four, above 8192 of 512, two."""
    sh = kda.NormShape(rows, G, D, kda.KDA_BF16 if dtype == BF else kda.KDA_F32, 0.0, 0)
    need = lib.kda_layer_norm_bwd_workspace_size(ctypes.byref(sh))
    per_sm = 16 if D <= 1024 else 8 if D <= 4096 else 4 if D <= 8192 else 2
    one = 4 * 2 * G * D
    assert one <= need <= one * ((per_sm * SMS + G - 1) // G) and need % one == 0
    assert need <= one * max(1, (rows + 3) // 4)


def guarded(need):
    """A workspace of `need` bytes with 4 KB behind it that have to stay as they are."""
    buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    return buf[:need], buf[need:]


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,D,dtype", SHAPES + [(3000, 1, 96, BF), (2500, 4, 1536, BF), (900, 1, 4095, F32)])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_stays_inside(R, G, D, dtype, shift):
    """Both layouts: rows that start on 16 bytes, and rows shifted by an element."""
    x, w, _, dy = (t.cuda() for t in draw_norm(R, G, D, dtype, seed=D))
    if shift:
        x = strided_like(x.reshape(R, G * D), 3, 1).unflatten(-1, (G, D))
    _, mean, rstd = kda.kda_layer_norm_fwd(x, w)
    sh = kda.NormShape(R, G, D, kda.KDA_BF16 if dtype == BF else kda.KDA_F32, 0.0, 0)
    ws, guard = guarded(kda.load_library().kda_layer_norm_bwd_workspace_size(ctypes.byref(sh)))
    got = kda.kda_layer_norm_bwd(dy, x, mean, rstd, w, workspace=ws)
    want = kda.kda_layer_norm_bwd(dy, x, mean, rstd, w, workspace=None)
    assert (guard == 0x5A).all()
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,W", [(BF, 64, 4), (F32, 13, 7), (BF, 520, 2), (F32, 4096, 8)])
@pytest.mark.parametrize("T", [1, 130, 3000])
def test_convolution_stays_inside(dtype, D, W, T):
    o = dev(draw_conv(1, T, D, W, dtype))
    code = kda.KDA_BF16 if dtype == BF else kda.KDA_F32
    sh = kda.ConvShape(1, T, D, 1, W, code, code, 1, 0, None)
    ws, guard = guarded(kda.load_library().kda_conv_bwd_workspace_size(ctypes.byref(sh)))
    args = o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"]
    got, want = kda.kda_conv_bwd(*args, workspace=ws), kda.kda_conv_bwd(*args, workspace=None)
    assert (guard == 0x5A).all()
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 5, 16, 24, 50, 128])
@pytest.mark.parametrize("T", [1, 130, 3000])
def test_scan_stays_inside(N, T):
    for dtype, D, G in ((BF, 40, 1), (F32, 18, 2)):
        o = dev(draw_ssm(1, T, D, N, G, dtype))
        sh = kda.SsmShape(1, T, D, N, G, 1, kda.KDA_BF16 if dtype == BF else kda.KDA_F32, 1, 0, 0, 0, 0, 0, None)
        lib = kda.load_library()
        ws, guard = guarded(lib.kda_ssm_fwd_workspace_size(ctypes.byref(sh), 0))
        got, want = forward(o, workspace=ws if ws.numel() else None), forward(o, workspace=None)
        assert (guard == 0x5A).all() and all(torch.equal(a, b) for a, b in zip(got, want))
        ws, guard = guarded(lib.kda_ssm_bwd_workspace_size(ctypes.byref(sh), 0))
        got, want = backward(o, workspace=ws), backward(o, workspace=None)
        assert (guard == 0x5A).all() and all(torch.equal(got[k], want[k]) for k in want)
