"""A call whose scratch cannot be had from the stream-ordered pool answers with an error, launches
nothing, and leaves nothing behind that a later call would report as its own."""
import ctypes

import pytest
import torch

import kimi_delta_attention_22_b200 as kda


def norm_works():
    x = torch.randn(8, 256, device="cuda")
    out, mean, _ = kda.kda_layer_norm_fwd(x)
    torch.cuda.synchronize()
    assert torch.allclose(mean, x.mean(-1), atol=1e-5) and torch.isfinite(out).all()


def decode_works():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    out = kda.kda_decode_step(r(2, 4, 128), r(2, 4, 128), r(2, 4, 128), -r(2, 4, 128).abs(), r(2, 4).sigmoid(), r(2, 4, 128, 128))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()


@pytest.mark.gpu
@pytest.mark.parametrize("after", [norm_works, decode_works])
@pytest.mark.parametrize("call", ["ssm_bwd", "chunk_fwd", "chunk_bwd"])
def test_the_next_call_is_its_own(call, after):
    """Shapes whose scratch is above 10 TB: the allocation fails before anything is read or launched."""
    lib = kda.load_library()
    after()
    p = ctypes.c_void_p(torch.empty(1 << 20, dtype=torch.uint8, device="cuda").data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if call == "ssm_bwd":
        q = [ctypes.c_void_p(p.value + 4096 * i) for i in range(11)]
        sh = kda.SsmShape(1, 1 << 27, 1 << 16, 128, 1, 1, kda.KDA_BF16, 1, 0, 0, 0, 0, 0, None)
        assert lib.kda_ssm_bwd_workspace_size(ctypes.byref(sh), 0) > 10 ** 13
        st = lib.kda_ssm_bwd(ctypes.byref(sh), *q[:5], None, None, None, None, None, q[5], None, q[6], q[7], q[8], q[9],
                             q[10], None, None, None, None, None, 0, stream)
    else:
        sh = kda.Shape(B=1, T=(1 << 31) - 64, H=32, d_k=128, d_v=128, num_seqs=1, dtype=kda.KDA_BF16, gate=kda.KDA_GATE_NONE,
                       chunk=64)
        size = lib.kda_chunk_fwd_workspace_size if call == "chunk_fwd" else lib.kda_chunk_bwd_workspace_size
        assert size(ctypes.byref(sh), 0) > 10 ** 13
        if call == "chunk_fwd":
            st = lib.kda_chunk_fwd(ctypes.byref(sh), p, p, p, None, p, None, None, p, None, None, 0, stream)
        else:
            st = lib.kda_chunk_bwd(ctypes.byref(sh), p, p, p, None, p, None, None, p, None, p, p, p, None, p, None, None, 0,
                                   stream)
    assert st == 4   # KDA_ERR_CUDA
    after()
