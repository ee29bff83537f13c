"""The block operators at the edges of what their documentation allows: packed batches without
sequences, state gradients without states, offsets past 32 bits, scratch from the pool inside
a captured graph, long sequences of many tiles and segments."""
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, dev
from oracle import block as ob
from test_block_conv import draw as draw_conv
from test_block_conv import reference as reference_conv
from test_block_ssm import backward, forward, reference
from test_block_ssm import draw as draw_ssm

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
def test_packed_batch_without_sequences():
    """cu_seqlens of one entry: no row is covered, nothing is written, parameter gradients are 0."""
    o = dev(draw_conv(1, 40, 16, 4, BF, [0, 40]))
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(o["x"], 7.0)
    _, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], cu_seqlens=cu, out=out)
    assert (out == 7.0).all() and fin.shape == (0, 3, 16)
    dx = torch.full_like(o["x"], 7.0)
    g = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], cu_seqlens=cu, grads=dict(dx=dx))
    assert (dx == 7.0).all() and g["dweight"].eq(0).all() and g["dbias"].eq(0).all()
    o = dev(draw_ssm(1, 40, 16, 16, 1, BF, [0, 40], state=False))
    o["cu"] = cu
    out = torch.full_like(o["x"], 7.0)
    _, h = forward(o, out=out)
    assert (out == 7.0).all() and h.shape == (0, 16, 16)
    dx = torch.full_like(o["x"], 7.0)
    g = backward(o, grads=dict(dx=dx))
    assert (dx == 7.0).all() and g["dA"].eq(0).all() and g["dD"].eq(0).all() and g["ddt_bias"].eq(0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [None, [0, 30, 30, 75]])
def test_state_gradients_without_states(cu):
    """A zero initial state with a gradient of the final one, and the gradient of that zero state;
    a state without a gradient of the final one."""
    T = 75
    d = draw_ssm(1, T, 24, 16, 1, F32, cu, seed=41)
    for drop in ("h0", "dh"):
        e = dict(d)
        e[drop] = None
        g = backward(dev(e))
        r, m = reference(e, bwd=True), reference(e, bwd=True, mag=True)
        for k in ("dh0", "dx", "dA"):
            close(g[k], r[k], m[k], 64 * T + 300, k)
    c = draw_conv(1, T, 24, 4, F32, cu, seed=42)
    for drop in ("state", "dfin"):
        e = dict(c)
        e[drop] = None
        o = dev(e)
        g = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], o["cu"])
        r, m = reference_conv(e, True, True), reference_conv(e, True, True, True)
        for k in ("dx", "dstate"):
            close(g[k], r[k], m[k], 60, k)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows 1.1 billion elements apart (a wide matrix's columns): the third lies past 2^31 elements
    and 2^32 bytes."""
    far, T = 1_100_000_000, 3
    wide = torch.empty(far * (T - 1) + 4096, dtype=BF, device="cuda")

    def columns(t, at):   # t [1, T, n]: a copy of it whose rows are `far` apart
        v = wide.as_strided((1, T, t.shape[-1]), (far * T, far, 1), at)
        v.copy_(t)
        return v

    o = dev(draw_conv(1, T, 64, 4, BF, seed=51))
    x = columns(o["x"], 0)
    a, b = (kda.kda_conv_fwd(v, o["w"], o["bias"], o["state"]) for v in (o["x"], x))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (kda.kda_conv_bwd(v, o["w"], o["dy"], o["bias"], o["state"], o["dfin"]) for v in (o["x"], x))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dstate"], b["dstate"]) and torch.equal(a["dweight"], b["dweight"])
    a, b = (kda.kda_conv_step(v[0], o["w"], torch.zeros(T, 3, 64, dtype=BF, device="cuda")) for v in (o["x"], x))
    assert torch.equal(a, b)
    o = dev(draw_ssm(1, T, 64, 16, 1, BF, seed=52))
    s = dict(o, x=columns(o["x"], 0), dt=columns(o["dt"], 64), z=columns(o["z"], 128),
             B=columns(o["B"][:, :, 0], 192), C=columns(o["C"][:, :, 0], 208))
    a, b = forward(o), forward(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = backward(o), backward(s)
    for k in a:
        assert torch.equal(a[k].reshape(-1), b[k].reshape(-1)), k
    h1, h2 = (torch.zeros(T, 64, 16, device="cuda") for _ in range(2))
    a = kda.kda_ssm_step(o["x"][0], o["dt"][0], o["A"], o["B"][0], o["C"][0], h1, z=o["z"][0])
    b = kda.kda_ssm_step(s["x"][0], s["dt"][0], s["A"], s["B"][0], s["C"][0], h2, z=s["z"][0])
    assert torch.equal(a, b) and torch.equal(h1, h2)
    n = torch.randn(1, T, 256, device="cuda").to(BF)
    v = columns(n, 1024)
    a, b = kda.kda_layer_norm_fwd(n), kda.kda_layer_norm_fwd(v)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dy = torch.randn(1, T, 256, device="cuda").to(BF)
    a, b = kda.kda_layer_norm_bwd(dy, n, a[1], a[2]), kda.kda_layer_norm_bwd(dy, v, a[1], a[2])
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
def test_pool_scratch_inside_a_graph():
    """Calls without a workspace captured: allocation and release are nodes of the graph."""
    o = dev(draw_ssm(1, 700, 24, 16, 1, BF, seed=61))
    c = dev(draw_conv(1, 700, 24, 4, BF, seed=62))
    x = torch.randn(700, 96, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x)

    def calls():
        return (forward(o, workspace=None), backward(o, workspace=None),
                kda.kda_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], workspace=None),
                kda.kda_layer_norm_bwd(x, x, mean, rstd, workspace=None))

    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for p, q in zip(a.values() if isinstance(a, dict) else a, b.values() if isinstance(b, dict) else b):
            assert torch.equal(p, q)


@pytest.mark.gpu
def test_long_sequences_against_pieces():
    """20000 rows in one call equal the same rows in pieces, each from the states of the one before."""
    T, D, N = 20000, 40, 16
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dt, z = r(1, T, D), r(1, T, D) - 3, r(1, T, D)
    A, B, C, w = -torch.exp(r(D, N)), r(1, T, N), r(1, T, N), r(D, 4)
    u, cs = kda.kda_conv_fwd(x, w)
    y, h = kda.kda_ssm_fwd(u, dt, A, B, C, z=z)
    state, hs, at = None, None, 0
    for n in (1, 4095, 7, 9000, 6897):
        s = slice(at, at + n)
        up, state = kda.kda_conv_fwd(x[:, s], w, state=state)
        assert torch.equal(up, u[:, s])
        yp, hs = kda.kda_ssm_fwd(up, dt[:, s], A, B[:, s], C[:, s], z=z[:, s], h0=hs)
        # the cut differs, so the roundings do: 32 steps per row of a state's memory (1 / (dt |A|), some
        # 2000 rows of the slowest channels), 2^-24 each, of terms a few times the output's size
        assert (yp - y[:, s]).abs().max() <= 32 * 2000 * 2.0 ** -24 * y.abs().max()
        at += n
    assert torch.equal(state, cs)
    assert (hs - h).abs().max() <= 32 * 2000 * 2.0 ** -24 * h.abs().max()


@pytest.mark.gpu
def test_many_short_sequences():
    """3000 packed sequences of 0 to 4 rows, and 70000 dense sequences of one row."""
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 5, (3000,), generator=g).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d = draw_ssm(1, cu[-1], 8, 4, 1, F32, cu, seed=71)
    o = dev(d)
    out, hT = forward(o)
    gr = backward(o)
    r, m = reference(d, bwd=True), reference(d, bwd=True, mag=True)
    close(out.reshape(-1, 8), r["out"], m["out"], 32 * 4 + 80, "out")
    close(hT, r["hT"], m["hT"], 32 * 4 + 64, "hT")
    for k in ("dx", "dB", "dh0"):
        close(gr[k], r[k].reshape(gr[k].shape), m[k].reshape(gr[k].shape), 64 * 4 + 160, k)
    c = draw_conv(1, cu[-1], 8, 4, F32, cu, seed=72)
    o = dev(c)
    y, fin = kda.kda_conv_fwd(o["x"], o["w"], o["bias"], o["state"], o["cu"])
    gr = kda.kda_conv_bwd(o["x"], o["w"], o["dy"], o["bias"], o["state"], o["dfin"], o["cu"])
    r, m = reference_conv(c, True, True), reference_conv(c, True, True, True)
    close(y.reshape(-1, 8), r["out"], m["out"], 40, "conv")
    assert torch.equal(fin.cpu().double(), torch.from_numpy(r["final"]))
    close(gr["dx"].reshape(-1, 8), r["dx"], m["dx"], 52, "conv dx")
    close(gr["dstate"], r["dstate"], m["dstate"], 52, "conv dstate")
    n = 70000
    x, w, st = torch.randn(n, 1, 8, device="cuda"), torch.randn(8, 4, device="cuda"), torch.randn(n, 3, 8, device="cuda")
    y, fin = kda.kda_conv_fwd(x, w, state=st)
    s2 = st.clone()
    assert torch.equal(kda.kda_conv_step(x[:, 0], w, s2), y[:, 0]) and torch.equal(s2, fin)
    dt, A, B = torch.randn(n, 1, 8, device="cuda"), -torch.rand(8, 4, device="cuda"), torch.randn(n, 1, 4, device="cuda")
    y, h = kda.kda_ssm_fwd(x, dt, A, B, B)
    h2 = torch.zeros(n, 8, 4, device="cuda")
    ys = kda.kda_ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], h2)
    assert torch.allclose(ys, y[:, 0], rtol=1e-5, atol=1e-5) and torch.allclose(h2, h, rtol=1e-5, atol=1e-5)


def test_references_of_many_sequences_agree():
    """The packed reference of several sequences is each sequence's own."""
    cu = [0, 4, 4, 9]
    d = draw_ssm(1, 9, 4, 3, 1, F32, cu, seed=5)
    whole = reference(d, bwd=True)
    for n, (b, e) in enumerate(ob.bounds(1, 9, cu)):
        p = {k: (v[:, b:e] if k in ("x", "dt", "B", "C", "z", "dy") else v) for k, v in d.items()}
        p["h0"], p["dh"], p["cu"] = d["h0"][n:n + 1], d["dh"][n:n + 1], None
        one = reference(p, bwd=True)
        assert (one["out"] == whole["out"][b:e]).all() and (one["dx"] == whole["dx"][b:e]).all()
        assert (one["dh0"][0] == whole["dh0"][n]).all()
