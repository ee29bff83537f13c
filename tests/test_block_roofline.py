"""The block operators' algorithmic byte counts worked out by hand."""
from kimi_delta_attention_22_b200.roofline import conv_bytes, norm_bytes, ssm_bytes, ssm_exponentials


def test_convolution_by_hand():
    # 4 sequences x 2048 rows x 6144 channels, 4 taps, bf16, no states in
    rows, D = 8192, 6144
    params = D * 5 * 4
    assert conv_bytes(rows, D, 4, 4, had=False) == rows * D * 4 + 4 * 3 * D * 2 + params
    assert conv_bytes(rows, D, 4, 4, had=False, backward=True) == rows * D * 6 + 2 * params == 302_235_648
    # one row of 256 sequences: the state of three rows read and written
    assert conv_bytes(256, 4096, 4, 256) == 256 * 4096 * 2 * (2 + 6) + 4096 * 20


def test_scan_by_hand():
    rows, D, N = 8192, 2048, 16
    state, params, bc = 4 * D * N * 4, D * 18 * 4, rows * N * 2 * 2
    assert ssm_bytes(rows, D, N, 4) == rows * D * 8 + bc + 2 * state + params == 135_938_048
    assert ssm_bytes(rows, D, N, 4, backward=True) == rows * D * 14 + 2 * bc + 3 * state + 2 * params == 237_797_376
    assert ssm_bytes(256, 4096, 16, 256) == 256 * 4096 * (8 + 2 * 64) + 256 * 16 * 4 + 4096 * 72
    assert ssm_exponentials(rows, D, N) == 268_435_456 and ssm_exponentials(rows, D, N, True) == 603_979_776


def test_norm_by_hand():
    assert norm_bytes(65536, 4096, backward=True) == 65536 * 4096 * 6 + 3 * 4096 * 4 + 65536 * 8
    assert norm_bytes(8192, 128, 16) == 8192 * 16 * 128 * 4 + 2 * 16 * 128 * 4 + 8192 * 16 * 8
