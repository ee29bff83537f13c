"""The block's operators as they run together: norm, convolution, scan (or the KDA recurrence)
and per-head norm, forward and back, prompt then single tokens, packed; on a side stream, in
CUDA graphs whose replays share no workspace, with scratch from the stream-ordered pool."""
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from kimi_delta_attention_22_b200 import inputs
from oracle import block as ob

BF = torch.bfloat16


def block(seed=0, T=130, D=64, N=16, H=4, cu=None, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k)  # noqa: E731
    n = len(cu) - 1 if cu else 1
    d = dict(x=r(1, T, D).to(dtype), nw=1 + r(D, k=0.1), nb=r(D, k=0.1), cw=r(D, 4, k=0.5), cb=r(D, k=0.1),
             cs=r(n, 3, D).to(dtype), dt=r(1, T, D).to(dtype) - 1, A=-torch.exp(r(D, N, k=0.5)), B=r(1, T, 1, N).to(dtype),
             C=r(1, T, 1, N).to(dtype), Ds=r(D), z=r(1, T, D).to(dtype), db=r(D), h0=r(n, D, N), hw=1 + r(H, D // H, k=0.1),
             hb=r(H, D // H, k=0.1), dy=r(1, T, D).to(dtype))
    d = {k: v.cuda() for k, v in d.items()}
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if cu else None
    d["H"] = H
    return d


def run_forward(d):
    a, mean, rstd = kda.kda_layer_norm_fwd(d["x"], d["nw"], d["nb"])
    u, cs = kda.kda_conv_fwd(a, d["cw"], d["cb"], d["cs"], d["cu"])
    y, hT = kda.kda_ssm_fwd(u, d["dt"], d["A"], d["B"], d["C"], D=d["Ds"], z=d["z"], dt_bias=d["db"], h0=d["h0"],
                            cu_seqlens=d["cu"])
    o, m2, r2 = kda.kda_layer_norm_fwd(y.unflatten(-1, (d["H"], -1)), d["hw"], d["hb"])
    return dict(a=a, mean=mean, rstd=rstd, u=u, cs=cs, y=y, hT=hT, o=o.flatten(-2), m2=m2, r2=r2)


def run_backward(d, f):
    H = d["H"]
    g2 = kda.kda_layer_norm_bwd(d["dy"].unflatten(-1, (H, -1)), f["y"].unflatten(-1, (H, -1)), f["m2"], f["r2"], d["hw"])
    gs = kda.kda_ssm_bwd(f["u"], d["dt"], d["A"], d["B"], d["C"], g2["dx"].flatten(-2), D=d["Ds"], z=d["z"], dt_bias=d["db"],
                         h0=d["h0"], cu_seqlens=d["cu"])
    gc = kda.kda_conv_bwd(f["a"], d["cw"], gs["dx"], d["cb"], d["cs"], cu_seqlens=d["cu"])
    gn = kda.kda_layer_norm_bwd(gc["dx"], d["x"], f["mean"], f["rstd"], d["nw"])
    return dict(x=gn["dx"], nw=gn["dweight"], nb=gn["dbias"], cw=gc["dweight"], cb=gc["dbias"], cs=gc["dstate"], dt=gs["ddt"],
                A=gs["dA"], B=gs["dB"], C=gs["dC"], Ds=gs["dD"], z=gs["dz"], db=gs["ddt_bias"], h0=gs["dh0"],
                hw=g2["dweight"], hb=g2["dbias"])


def plain(p, cu, H):
    """The same block in float64 torch, differentiable."""
    F = torch.nn.functional
    T, D = p["x"].shape[1:]
    a = F.layer_norm(p["x"], (D,), p["nw"], p["nb"])[0]
    seqs = ob.bounds(1, T, cu)
    rows = []
    for q, (b, e) in enumerate(seqs):
        line = torch.cat([p["cs"][q], a[b:e]])
        u = F.silu(sum(p["cw"][:, j] * line[j:j + e - b] for j in range(4)) + p["cb"])
        h = p["h0"][q]
        for t in range(b, e):
            dt = F.softplus(p["dt"][0, t] + p["db"])
            h = torch.exp(dt[:, None] * p["A"]) * h + (dt * u[t - b])[:, None] * p["B"][0, t]
            rows.append(((h * p["C"][0, t]).sum(-1) + p["Ds"] * u[t - b]) * F.silu(p["z"][0, t]))
    y = torch.stack(rows)[None]
    return (F.layer_norm(y.unflatten(-1, (H, -1)), (D // H,)) * p["hw"] + p["hb"]).flatten(-2)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [None, [0, 1, 60, 60, 130]])
def test_block_and_gradients_against_autograd(cu):
    """fp32 through four operators and back: each is good to about 1e-5 of its scale
    (test_block_*.py), and the norms in between amplify by a few units."""
    d = block(cu=cu)
    f = run_forward(d)
    g = run_backward(d, f)
    p = {k: v.detach().cpu().double().requires_grad_(True) for k, v in d.items()
         if isinstance(v, torch.Tensor) and k not in ("cu", "dy")}
    o = plain(p, cu, d["H"])
    (o * d["dy"].cpu().double()).sum().backward()
    assert (f["o"].cpu().double() - o).abs().max() < 2e-4 * o.abs().max()
    for k in g:
        ref = p[k].grad
        err = (g[k].cpu().double().reshape(ref.shape) - ref).norm() / ref.norm()
        assert err < 2e-4, (k, float(err))


@pytest.mark.gpu
def test_prompt_then_tokens_equal_one_prompt():
    """Serving: the prompt's states carry the single-token operators to the same rows."""
    d = block(T=40, dtype=torch.float32)
    f = run_forward(d)
    cut = 33
    h = {k: (v[:, :cut].contiguous() if k in ("x", "dt", "B", "C", "z", "dy") else v) for k, v in d.items()}
    s = run_forward(h)
    conv_state, state = s["cs"].clone(), s["hT"].clone()
    for t in range(cut, 40):
        a, _, _ = kda.kda_layer_norm_fwd(d["x"][:, t], d["nw"], d["nb"], want_stats=False)
        u = kda.kda_conv_step(a, d["cw"], conv_state, bias=d["cb"])
        y = kda.kda_ssm_step(u, d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], state, D=d["Ds"], z=d["z"][:, t],
                             dt_bias=d["db"])
        o, _, _ = kda.kda_layer_norm_fwd(y.unflatten(-1, (4, -1)), d["hw"], d["hb"], want_stats=False)
        assert torch.allclose(o.flatten(-2), f["o"][:, t], rtol=1e-4, atol=1e-4), t
    assert torch.equal(conv_state, f["cs"])
    assert torch.allclose(state, f["hT"], rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
def test_kda_layer_convolution_recurrence_norm():
    """The convolution in front of, and the per-head norm behind, the KDA recurrence: forward
    against the parts' own references, and fp32 gradients of the recurrence into the
    convolution's gradient."""
    T, H, K = 100, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    xq, xk, xv = (r(1, T, H * K).to(BF) for _ in range(3))
    w = [r(H * K, 4) * 0.5 for _ in range(3)]
    q, k, v = (kda.kda_conv_fwd(x, c, want_state=False)[0].unflatten(-1, (H, K)) for x, c in zip((xq, xk, xv), w))
    k = torch.nn.functional.normalize(k.float(), dim=-1).to(BF)
    d = inputs.draw(1, T, H, K, K, dtype=BF, s0_std=0.02, seed=5, device="cuda")
    out, ST = kda.kda_chunk_fwd(q, k, v, d["g"], d["beta"], S0=d["S0"])
    nw, nb = 1 + 0.1 * r(H, K), 0.1 * r(H, K)
    o, mean, rstd = kda.kda_layer_norm_fwd(out, nw, nb)
    ref = torch.nn.functional.layer_norm(out.double(), (K,)) * nw.double() + nb.double()
    assert (o.double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-5
    dy = r(1, T, H, K).to(BF)
    gn = kda.kda_layer_norm_bwd(dy, out, mean, rstd, nw)
    gk = kda.kda_chunk_bwd(q, k, v, d["g"], d["beta"], d["S0"], gn["dx"])
    gc = kda.kda_conv_bwd(xv, w[2], gk["dv"].flatten(-2), want_dstate=False)   # fp32 gradient, bf16 input
    x = xv.double().requires_grad_(True)
    c = w[2].double().requires_grad_(True)
    pre = torch.nn.functional.conv1d(x.transpose(1, 2), c[:, None], padding=3, groups=H * K)[..., :T].transpose(1, 2)
    torch.nn.functional.silu(pre).backward(gk["dv"].flatten(-2).double())
    assert (gc["dx"].double() - x.grad).abs().max() <= 2.0 ** -8 * x.grad.abs().max()
    assert (gc["dweight"].double() - c.grad).norm() <= 1e-5 * c.grad.norm()


@pytest.mark.gpu
def test_side_stream_and_pool_scratch():
    """On a stream of its own, with the scratch from the stream-ordered pool: the same bits."""
    d = block(seed=4, T=700, D=48, H=3)
    f = run_forward(d)
    g = run_backward(d, f)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        f2 = run_forward(d)
        h, _ = kda.kda_ssm_fwd(f2["u"], d["dt"], d["A"], d["B"], d["C"], D=d["Ds"], z=d["z"], dt_bias=d["db"], h0=d["h0"],
                               workspace=None)
        g2 = run_backward(d, f2)
        p = kda.kda_conv_bwd(f2["a"], d["cw"], f2["u"], d["cb"], d["cs"], workspace=None)
        q = kda.kda_conv_bwd(f2["a"], d["cw"], f2["u"], d["cb"], d["cs"])
        s = kda.kda_ssm_bwd(f2["u"], d["dt"], d["A"], d["B"], d["C"], f2["y"], workspace=None)
        s2 = kda.kda_ssm_bwd(f2["u"], d["dt"], d["A"], d["B"], d["C"], f2["y"])
    side.synchronize()
    for k in f:
        assert torch.equal(f[k], f2[k]), k
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    assert torch.equal(h, f["y"])
    for a, b in ((p, q), (s, s2)):
        for k in a:
            assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), k


@pytest.mark.gpu
def test_graph_replay_equals_eager():
    """The whole block, forward and back, in two graphs (workspaces of their own: allocated
    during capture) replayed in turn with changed inputs."""
    d = block(seed=5, T=600, D=32, H=2, dtype=BF)
    graphs, outs = [], []
    warm = run_forward(d)
    run_backward(d, warm)
    torch.cuda.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f = run_forward(d)
            b = run_backward(d, f)
        graphs.append(gr)
        outs.append((f, b))
    for seed in (11, 12):
        new = block(seed=seed, T=600, D=32, H=2, dtype=BF)
        for k in ("x", "dt", "B", "C", "z", "dy", "h0", "cs"):
            d[k].copy_(new[k])
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        f = run_forward(d)
        b = run_backward(d, f)
        torch.cuda.synchronize()
        for fo, bo in outs:
            for k in f:
                assert torch.equal(f[k], fo[k]), k
            for k in b:
                assert torch.equal(b[k], bo[k]), k


@pytest.mark.gpu
def test_step_graph_replays_advance_the_state():
    """The single-token operators captured once and replayed: the states advance in place."""
    N, D, S = 6, 40, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dt, z = (r(N, D).to(BF) for _ in range(3))
    B, C, A = r(N, 1, S).to(BF), r(N, 1, S).to(BF), -torch.exp(r(D, S))
    w, cs, h = r(D, 4), r(N, 3, D).to(BF), r(N, D, S)
    cs1, h1 = cs.clone(), h.clone()
    u, y = torch.empty_like(x), torch.empty_like(x)

    def step(cs, h):
        kda.kda_conv_step(x, w, cs, out=u)
        kda.kda_ssm_step(u, dt, A, B, C, h, z=z, out=y)

    step(cs.clone(), h.clone())
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(cs, h)
    for _ in range(4):
        gr.replay()
    torch.cuda.synchronize()
    got = y.clone()
    for _ in range(4):
        step(cs1, h1)
    torch.cuda.synchronize()
    assert torch.equal(cs, cs1) and torch.equal(h, h1) and torch.equal(got, y)
