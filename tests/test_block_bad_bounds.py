"""Inconsistent cu_seqlens: the status word, and what the header says of every sequence.  Those whose
bounds break the order are skipped, with their states and the rows that only they claim as they
were; those with no larger bound in front and no smaller one behind keep their results."""
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import dev
from test_block_conv import draw as draw_conv
from test_block_ssm import backward, forward
from test_block_ssm import draw as draw_ssm

M = 640
GOOD = [0, 200, 400, 640]
BAD = [[0, 200, 700, 640], [0, 400, 200, 640], [0, 200, -5, 640], [5, 200, 400, 640], [0, 400, 200, 400, 640],
       [0, 200, 400, 300, 640], [0, 100, 90, 120, 640], [0, 33, 34, 640, 600, 620], [0, 0, 300, 299, 299, 640],
       [0, 10, 500, 20, 30, 640], [0, 640, 0, 640], [0, 1, 0, 1, 0, 640]]


def sort(cu):
    """The numbers of the sequences that are skipped, and of those that keep their results."""
    n = len(cu) - 1
    skip = [q for q in range(n)
            if not (0 <= cu[max(q - 1, 0)] <= cu[q] <= cu[q + 1] <= M) or (q == 0 and cu[0] != 0)]
    keep = [q for q in range(n) if q not in skip and max(cu[:q + 1]) == cu[q] and min(cu[q + 1:]) == cu[q + 1]]
    return skip, keep


def rows_of(cu, which):
    r = torch.zeros(M, dtype=torch.bool)
    for q in which:
        r[cu[q]:cu[q + 1]] = True
    return r.cuda()


def test_the_arrays_break_something():
    for cu in BAD:
        skip, keep = sort(cu)
        assert skip and not set(skip) & set(keep), cu
    assert sort(GOOD) == ([], [0, 1, 2])
    assert sort([0, 400, 200, 640]) == ([1, 2], []) and sort([5, 200, 400, 640]) == ([0], [1, 2])


def check(cu, call, rows, states):
    """call(cu, outputs) writes into the given buffers: `rows` [1, M, ..] and `states` [n, ..] by name,
    each a shape and a type.  Every kept sequence is compared with a call on it alone, packed at its
    place behind rows of no interest."""
    n = len(cu) - 1
    skip, keep = sort(cu)
    buf = {k: torch.full((1, M, *s), 7.0, dtype=t, device="cuda") for k, (s, t) in rows.items()}
    buf.update({k: torch.full((n, *s), 7.0, dtype=t, device="cuda") for k, (s, t) in states.items()})
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(cu, buf, st, list(range(n)))
    assert st.item() == kda.KDA_DEV_BAD_SEQLENS, cu
    only_skipped = ~rows_of(cu, [q for q in range(n) if q not in skip])
    for k in rows:
        assert (buf[k][0, only_skipped] == 7.0).all(), (cu, k)
    for k in states:
        assert (buf[k][skip] == 7.0).all(), (cu, k)
    for q in keep:
        b, e = cu[q], cu[q + 1]
        one = [0, b, e]   # the rows in front as a sequence of their own, with the state of number 0
        alone = {k: torch.full_like(buf[k], 9.0) for k in rows}
        alone.update({k: torch.full((2, *s), 9.0, dtype=t, device="cuda") for k, (s, t) in states.items()})
        st.zero_()
        call(one, alone, st, [0, q])
        assert st.item() == 0
        for k in rows:
            assert torch.equal(buf[k][:, b:e], alone[k][:, b:e]), (cu, q, k)
        for k in states:
            assert torch.equal(buf[k][q], alone[k][1]), (cu, q, k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", BAD)
def test_convolution(cu, dtype):
    d = draw_conv(1, M, 24, 4, dtype, seed=3)
    o = dev(d)
    g = torch.Generator(device="cuda").manual_seed(4)
    state, dfin = (torch.randn(8, 3, 24, device="cuda", generator=g).to(dtype) for _ in range(2))

    def fwd(cu, buf, st, which):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.kda_conv_fwd(o["x"], o["w"], o["bias"], state[which], t, out=buf["out"], final_state=buf["fin"], dev_status=st)

    def bwd(cu, buf, st, which):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], state[which], dfin[which], t, dev_status=st,
                         grads=dict(dx=buf["dx"], dstate=buf["dstate"]))

    check(cu, fwd, dict(out=((24,), dtype)), dict(fin=((3, 24), dtype)))
    check(cu, bwd, dict(dx=((24,), dtype)), dict(dstate=((3, 24), dtype)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", BAD)
def test_scan(cu, dtype):
    o = dev(draw_ssm(1, M, 24, 16, 1, dtype, seed=5))
    g = torch.Generator(device="cuda").manual_seed(6)
    h0, dh = (torch.randn(8, 24, 16, device="cuda", generator=g) for _ in range(2))

    def args(cu, which):
        return dict(o, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), h0=h0[which], dh=dh[which])

    def fwd(cu, buf, st, which):
        forward(args(cu, which), out=buf["out"], hT=buf["hT"], dev_status=st)

    def bwd(cu, buf, st, which):
        backward(args(cu, which), grads=dict(buf), dev_status=st)

    f32 = torch.float32
    check(cu, fwd, dict(out=((24,), dtype)), dict(hT=((24, 16), f32)))
    check(cu, bwd, dict(dx=((24,), dtype), ddt=((24,), dtype), dz=((24,), dtype), dB=((1, 16), dtype), dC=((1, 16), dtype)),
          dict(dh0=((24, 16), f32)))
