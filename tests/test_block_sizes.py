"""The block operators' largest sizes, as the C entry points answer them."""
import ctypes

import pytest

import kimi_delta_attention_22_b200 as kda
from kimi_delta_attention_22_b200 import build as kbuild

A = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def padded(N):
    """States per channel in the gradient's checkpoints."""
    return next(n for n in (4, 8, 16, 32, 64, 128) if N <= n)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 16, 17, 33, 65, 128])
def test_scan_strides_fit_32_bits(lib, N):
    """Every accepted number of channels times the padded states stays below 2^31; one more channel
    than the largest is refused (no sequences: nothing is launched)."""
    def fwd(D):
        sh = kda.SsmShape(0, 8, D, N, 1, 0, kda.KDA_BF16, 1, 0, 0, 0, 0, 0, None)
        return lib.kda_ssm_fwd(ctypes.byref(sh), A, A, A, A, A, None, None, None, None, None, A, None, None, 0, None)

    most = ((1 << 29) - 1) // N
    assert fwd(most) == 0 and fwd(most + 1) == 2
    assert most * padded(N) < 1 << 31
