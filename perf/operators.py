"""Cases and plain forms of the recurrent block's operators: the short causal
convolution, the selective state space scan and layer norm.

Notation: M token rows (a dense batch [B, T, ..] flattened, or the packed rows of
several sequences), D channels, W taps, N states per channel, G groups of channels
that share the input and output vectors of the scan.

conv   pre[t, d] = bias[d] + sum_j w[d, j] x[t - (W-1) + j, d],  out = silu(pre) or pre.
       Rows before a sequence's first come from its state (its last W-1 inputs).
ssm    dt = softplus(raw + dt_bias),  a[t, d, n] = exp(dt[t, d] A[d, n])
       h[t] = a[t] h[t-1] + dt[t] x[t] B[t],  y[t, d] = sum_n h[t, d, n] C[t, n] + D[d] x[t, d]
       out = y silu(z)
norm   out = (x - mean) rstd w + b over the last axis, weights per group of rows.

`run` computes them in plain torch (own = False) or calls the library (own = True).
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _conv(name, do, dtype, B, T, D, W, silu=True, bias=True, state=True, seqs=0):
    c = dict(op="conv", do=do, dtype=dtype, B=B, T=T, D=D, W=W, silu=silu, bias=bias, state=state, seqs=seqs)
    return dict(c, name=name) if name else c


def _ssm(name, do, dtype, B, T, D, N, G=1, gate=True, state=True, seqs=0):
    c = dict(op="ssm", do=do, dtype=dtype, B=B, T=T, D=D, N=N, G=G, gate=gate, state=state, seqs=seqs)
    return dict(c, name=name) if name else c


def _norm(name, do, dtype, M, G, D):
    c = dict(op="norm", do=do, dtype=dtype, M=M, G=G, D=D)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of 256 sequences, 32 heads of 128 channels: the serving loop's convolution
        _conv("conv_step_n256_d4096", "step", "bf16", 256, 1, 4096, 4),
        # a long packed prompt batch, 32 heads of 128 channels
        _conv("conv_fwd_packed_65536_d4096", "fwd", "bf16", 1, 65536, 4096, 4, seqs=8),
        # an odd fp32 shape without activation, three taps
        _conv("conv_fwd_f32_odd", "fwd", "f32", 3, 1537, 1111, 3, silu=False),
        # training: the q, k and v channels of 16 heads side by side
        _conv("conv_bwd_b4_t2048_d6144", "bwd", "bf16", 4, 2048, 6144, 4, state=False),
        # one token of 256 sequences: the state is read and written once
        _ssm("ssm_step_n256_d4096", "step", "bf16", 256, 1, 4096, 16),
        # a prompt batch of 4 sequences
        _ssm("ssm_fwd_b4_t2048_d2048", "fwd", "bf16", 4, 2048, 2048, 16),
        # few channels, a long packed axis
        _ssm("ssm_fwd_packed_32768_d1024", "fwd", "bf16", 1, 32768, 1024, 16, seqs=5),
        # training on the same batch
        _ssm("ssm_bwd_b4_t2048_d2048", "bwd", "bf16", 4, 2048, 2048, 16),
        # odd sizes in fp32, two groups
        _ssm("ssm_bwd_f32_odd", "bwd", "f32", 2, 777, 500, 24, G=2),
        # the norm before a serving step's projections, 8 sequences
        _norm("norm_fwd_8x4096", "fwd", "bf16", 8, 1, 4096),
        # per-head norm of a recurrence's output, 4 x 2048 tokens of 16 heads
        _norm("norm_fwd_heads_8192x16x128", "fwd", "bf16", 8192, 16, 128),
        # training: a long batch's gradient with the reduction of the weights' gradients
        _norm("norm_bwd_65536x4096", "bwd", "bf16", 65536, 1, 4096),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "ssm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _log(rng, 16, 16384)
        G = rng.choice([1, 1, 2, 5, 16])
        M = _log(rng, 1, max(1, min(65536, (1 << 27) // (D * G))))
        return _norm(None, rng.choice(["fwd", "bwd"]), dtype, M, G, D)
    do = rng.choice(["fwd", "bwd", "step"])
    state = rng.random() < 0.6
    if op == "conv":
        D, W = _log(rng, 8, 8192), rng.choice([2, 3, 4, 4, 4, 5, 8])
        if rng.random() < 0.5:
            D = -(-D // 8) * 8
        kw = dict(silu=rng.random() < 0.8, bias=rng.random() < 0.7, state=state)
        if do == "step":
            return _conv(None, do, dtype, _log(rng, 1, 512), 1, D, W, **dict(kw, state=True))
        B = rng.choice([1, 1, 2, 3, 8])
        T = _log(rng, 1, max(1, min(32768, (1 << 26) // (D * B))))
        seqs = rng.randint(1, 12) if B == 1 and rng.random() < 0.6 else 0
        return _conv(None, do, dtype, B, T, D, W, seqs=seqs, **kw)
    N, G = rng.choice([1, 4, 8, 16, 16, 16, 24, 32, 64]), rng.choice([1, 1, 2, 4])
    D = G * _log(rng, 4, 4096 // G)
    if rng.random() < 0.5:
        D = -(-D // (8 * G)) * 8 * G
    gate = rng.random() < 0.7
    if do == "step":
        return _ssm(None, do, dtype, _log(rng, 1, 256), 1, D, N, G, gate)
    B = rng.choice([1, 1, 2, 3, 8])
    T = _log(rng, 1, max(1, min(16384, (1 << 28) // (D * N * B))))
    seqs = rng.randint(1, 12) if B == 1 and rng.random() < 0.6 else 0
    return _ssm(None, do, dtype, B, T, D, N, G, gate, state, seqs)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dtype = DT[c["dtype"]]

    def normal(*shape, dt=torch.float32, scale=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dt)

    s = {"case": c}
    if c["op"] == "norm":
        M, G, D = c["M"], c["G"], c["D"]
        # rows of a residual stream: a scale and an offset of their own
        x = normal(M, G, D) * (0.5 + torch.rand(M, G, 1, device=DEV, generator=g)) + 0.3 * normal(M, G, 1)
        s["x"] = x.to(dtype)
        s["w"], s["b"] = 1.0 + 0.2 * normal(G, D), 0.1 * normal(G, D)
        if c["do"] == "bwd":
            s["dy"] = normal(M, G, D, dt=dtype)
            x = s["x"].double()
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = (((x - mean[..., None]) ** 2).mean(-1) + EPS).rsqrt().float()
        return s
    B, T, D = c["B"], c["T"], c["D"]
    n = c["seqs"] or B
    s["cu"] = None
    if c["seqs"]:   # cut points anywhere: lengths of zero and one among them
        cut = torch.randint(0, T + 1, (n - 1,), device=DEV, generator=g).sort().values
        s["cu"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).to(torch.int32)
    step = c["do"] == "step"
    lead = (B,) if step else (B, T)
    s["x"] = normal(*lead, D, dt=dtype)
    if c["op"] == "conv":
        W = c["W"]
        s["w"] = normal(D, W, scale=1.0 / math.sqrt(W))
        s["bias"] = normal(D, scale=0.1) if c["bias"] else None
        s["state"] = normal(n, W - 1, D, dt=dtype) if c["state"] else None
        if c["do"] == "bwd":
            s["dy"] = normal(*lead, D, dt=dtype)
            s["dstate"] = normal(n, W - 1, D, dt=dtype) if c["state"] else None
        return s
    N, G = c["N"], c["G"]
    # step sizes between 0.001 and 0.1 through the softplus' inverse, decay rates around 1..N
    want = torch.exp(torch.empty(D, device=DEV).uniform_(math.log(1e-3), math.log(1e-1), generator=g))
    s["dt_bias"] = torch.log(torch.expm1(want))
    s["dt"] = normal(*lead, D, dt=dtype, scale=0.5)
    rates = torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
    s["A"] = -rates * (0.8 + 0.4 * torch.rand(D, N, device=DEV, generator=g))
    s["B"], s["C"] = normal(*lead, G, N, dt=dtype), normal(*lead, G, N, dt=dtype)
    s["D"] = normal(D)
    s["z"] = normal(*lead, D, dt=dtype) if c["gate"] else None
    s["h"] = normal(n, D, N, scale=0.5) if c["state"] else None
    if c["do"] == "bwd":
        s["dy"] = normal(*lead, D, dt=dtype)
        s["dh"] = normal(n, D, N, scale=0.5) if c["state"] else None
    return s


EPS = 1e-5


# ---------------------------------------------------------------- one pass


def run(s):
    op, do = s["case"]["op"], s["case"]["do"]
    if own:
        return _OWN[op, do](s)
    return _PLAIN[op, do](s)


def _own_conv_step(s):
    import kimi_delta_attention_22_b200 as kda

    y = kda.kda_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], silu=s["case"]["silu"])
    return {"out": y, "state": s["state"]}


def _own_conv_fwd(s):
    import kimi_delta_attention_22_b200 as kda

    y, st = kda.kda_conv_fwd(s["x"], s["w"], bias=s["bias"], state=s["state"], cu_seqlens=s["cu"],
                             silu=s["case"]["silu"])
    return {"out": y, "state": st}


def _own_conv_bwd(s):
    import kimi_delta_attention_22_b200 as kda

    g = kda.kda_conv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], state=s["state"], d_final_state=s["dstate"],
                         cu_seqlens=s["cu"], silu=s["case"]["silu"], want_dstate=s["state"] is not None)
    return {"dx": g["dx"], "dw": g["dweight"], "db": g["dbias"], "dstate": g["dstate"]}


def _own_ssm_step(s):
    import kimi_delta_attention_22_b200 as kda

    y = kda.kda_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    return {"out": y, "h": s["h"]}


def _own_ssm_fwd(s):
    import kimi_delta_attention_22_b200 as kda

    y, h = kda.kda_ssm_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                           h0=s["h"], cu_seqlens=s["cu"])
    return {"out": y, "h": h}


def _own_ssm_bwd(s):
    import kimi_delta_attention_22_b200 as kda

    g = kda.kda_ssm_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                        h0=s["h"], d_hT=s["dh"], cu_seqlens=s["cu"], want_dh0=s["h"] is not None)
    return {k: g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")}


def _own_norm_fwd(s):
    import kimi_delta_attention_22_b200 as kda

    y, mean, rstd = kda.kda_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    return {"out": y, "mean": mean, "rstd": rstd}


def _own_norm_bwd(s):
    import kimi_delta_attention_22_b200 as kda

    g = kda.kda_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    return {"dx": g["dx"], "dw": g["dweight"], "db": g["dbias"]}


# ---- plain forms


def _rows(s):
    """(first row, row past the last, sequence) of every token row, and of every sequence its bounds."""
    c, dev = s["case"], s["x"].device
    if s["cu"] is not None:
        cu = s["cu"].long()
    else:
        cu = torch.arange(c["B"] + 1, device=dev) * c["T"]
    t = torch.arange(c["B"] * c["T"], device=dev)
    q = torch.bucketize(t, cu[1:], right=True)   # empty sequences own no row
    return t, q, cu[:-1], cu[1:]


def _taps(pos, q, start, M, W):
    """Row of [x; states] that holds position `pos` of sequence q (negative offsets: its state)."""
    back = pos - start[q]
    return torch.where(back >= 0, pos, M + q * (W - 1) + (W - 1) + back)


def _conv_table(s):
    c = s["case"]
    M, D, W = c["B"] * c["T"], c["D"], c["W"]
    n = c["seqs"] or c["B"]
    x = s["x"].reshape(M, D)
    st = s["state"] if s["state"] is not None else x.new_zeros(n, W - 1, D)
    return torch.cat([x, st.reshape(-1, D)]), M, D, W, n


def _conv_pre(s):
    table, M, D, W, n = _conv_table(s)
    t, q, start, end = _rows(s)
    j = torch.arange(W, device=t.device)
    idx = _taps(t[:, None] - (W - 1) + j, q[:, None], start, M, W)
    win = table[idx].float()                                   # [M, W, D]
    pre = (win * s["w"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    return pre, win, table, q, start, end, M, D, W, n


def _plain_conv_fwd(s):
    pre, _, table, q, start, end, M, D, W, n = _conv_pre(s)
    y = pre * torch.sigmoid(pre) if s["case"]["silu"] else pre
    seq = torch.arange(n, device=q.device)[:, None]
    pos = end[:, None] - (W - 1) + torch.arange(W - 1, device=q.device)
    fin = table[_taps(pos, seq, start, M, W)]
    return {"out": y.to(s["x"].dtype).reshape(s["x"].shape), "state": fin}


def _plain_conv_step(s):
    win = torch.cat([s["state"], s["x"][:, None]], 1)         # [n, W, D]
    pre = (win.float() * s["w"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = pre * torch.sigmoid(pre) if s["case"]["silu"] else pre
    s["state"].copy_(win[:, 1:])
    return {"out": y.to(s["x"].dtype), "state": s["state"]}


def _plain_conv_bwd(s):
    pre, win, table, q, start, end, M, D, W, n = _conv_pre(s)
    dy = s["dy"].reshape(M, D).float()
    if s["case"]["silu"]:
        sg = torch.sigmoid(pre)
        dpre = dy * sg * (1.0 + pre * (1.0 - sg))
    else:
        dpre = dy
    dw = (dpre[:, None] * win).sum(0).t().contiguous()
    db = dpre.sum(0) if s["bias"] is not None else None
    # every row of [x; states] with its position and sequence
    dev = q.device
    seq = torch.arange(n, device=dev)[:, None].expand(n, W - 1)
    pos = torch.cat([torch.arange(M, device=dev), (start[:, None] - (W - 1) + torch.arange(W - 1, device=dev)).reshape(-1)])
    own_seq = torch.cat([q, seq.reshape(-1)])
    to = pos[:, None] + (W - 1) - torch.arange(W, device=dev)  # the output row that tap j of this input feeds
    ok = (to >= start[own_seq][:, None]) & (to < end[own_seq][:, None])
    dpre0 = torch.cat([dpre, dpre.new_zeros(1, D)])
    dtab = (dpre0[torch.where(ok, to, M)] * s["w"].t()).sum(1)
    if s["dstate"] is not None:                                # the final state's rows are inputs themselves
        j = pos - end[own_seq] + (W - 1)
        at = torch.where((j >= 0) & (j < W - 1), own_seq * (W - 1) + j, n * (W - 1))
        df = s["dstate"].float().reshape(-1, D)
        dtab = dtab + torch.cat([df, df.new_zeros(1, D)])[at]
    dtab = dtab.to(s["x"].dtype)
    dst = dtab[M:].reshape(n, W - 1, D) if s["state"] is not None else None
    return {"dx": dtab[:M].reshape(s["x"].shape), "dw": dw, "db": db, "dstate": dst}


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def _silu(v):
    return v * torch.sigmoid(v)


def _scan(a, u):
    """h[t] = a[t] h[t-1] + u[t] along the first axis, by doubling."""
    off = 1
    while off < a.shape[0]:
        u = torch.cat([u[:off], u[off:] + a[off:] * u[:-off]])
        a = torch.cat([a[:off], a[off:] * a[:-off]])
        off *= 2
    return u


def _ssm_terms(s):
    c = s["case"]
    M, D, N, G = c["B"] * c["T"], c["D"], c["N"], c["G"]
    x = s["x"].reshape(M, D).float()
    raw = s["dt"].reshape(M, D).float() + s["dt_bias"]
    dt = _softplus(raw)
    a = torch.exp(dt[..., None] * s["A"])
    Bx = s["B"].reshape(M, G, N).float().repeat_interleave(D // G, 1)
    Cx = s["C"].reshape(M, G, N).float().repeat_interleave(D // G, 1)
    return x, raw, dt, a, Bx, Cx, M, D, N, G


def _ssm_states(s, x, dt, a, Bx, M, D, N):
    """h of every row, h before every row, and where sequences begin and end."""
    t, q, start, end = _rows(s)
    n = start.numel()
    h0 = s["h"] if s["h"] is not None else torch.zeros(n, D, N, device=x.device)
    first = (t == start[q])
    u = (dt * x)[..., None] * Bx
    before = h0[q] * first[:, None, None]                       # the incoming state, at first rows only
    h = _scan(torch.where(first[:, None, None], 0.0, a), u + a * before)
    prev = torch.cat([h[:1], h[:-1]])
    prev = torch.where(first[:, None, None], before, prev)
    return h, prev, h0, t, q, start, end, first


def _plain_ssm_fwd(s):
    x, raw, dt, a, Bx, Cx, M, D, N, G = _ssm_terms(s)
    h, _, h0, t, q, start, end, _ = _ssm_states(s, x, dt, a, Bx, M, D, N)
    y = (h * Cx).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].reshape(M, D).float())
    hT = torch.where((end > start)[:, None, None], h[(end - 1).clamp(min=0)], h0)
    return {"out": y.to(s["x"].dtype).reshape(s["x"].shape), "h": hT}


def _plain_ssm_step(s):
    x, raw, dt, a, Bx, Cx, M, D, N, G = _ssm_terms(s)
    h = a * s["h"] + (dt * x)[..., None] * Bx
    y = (h * Cx).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["h"].copy_(h)
    return {"out": y.to(s["x"].dtype), "h": s["h"]}


def _plain_ssm_bwd(s):
    x, raw, dt, a, Bx, Cx, M, D, N, G = _ssm_terms(s)
    h, prev, h0, t, q, start, end, first = _ssm_states(s, x, dt, a, Bx, M, D, N)
    dout = s["dy"].reshape(M, D).float()
    dz, dy = None, dout
    if s["z"] is not None:
        z = s["z"].reshape(M, D).float()
        sg = torch.sigmoid(z)
        y = (h * Cx).sum(-1) + s["D"] * x
        dz = (dout * y * sg * (1.0 + z * (1.0 - sg))).to(s["x"].dtype).reshape(s["x"].shape)
        dy = dout * z * sg
    dC = (dy[..., None] * h).reshape(M, G, D // G, N).sum(2)
    del h
    last = (t == end[q] - 1)
    v = dy[..., None] * Cx
    if s["dh"] is not None:
        v = v + s["dh"][q] * last[:, None, None]
    anext = torch.cat([a[1:], a[:1]])
    anext = torch.where(last[:, None, None], 0.0, anext)
    dh = _scan(anext.flip(0), v.flip(0)).flip(0)
    del anext, v, Cx
    w = dh * a * prev                                           # through the decay
    dA = (w * dt[..., None]).sum(0)
    ddt = (w * s["A"]).sum(-1)
    del w
    p = (dh * Bx).sum(-1)
    dB = (dh * (dt * x)[..., None]).reshape(M, G, D // G, N).sum(2)
    ddt = (ddt + p * x) * torch.sigmoid(raw)
    dx = p * dt + s["D"] * dy
    dh0 = None
    if s["h"] is not None:
        at = start.clamp(max=M - 1)
        dh0 = a[at] * dh[at]
        empty = s["dh"] if s["dh"] is not None else torch.zeros_like(dh0)
        dh0 = torch.where((end > start)[:, None, None], dh0, empty)
    like = lambda v, to: v.to(to.dtype).reshape(to.shape)  # noqa: E731
    return {"dx": like(dx, s["x"]), "ddt": like(ddt, s["dt"]), "dA": dA, "dB": like(dB, s["B"]), "dC": like(dC, s["C"]),
            "dD": (dy * x).sum(0), "dz": dz, "ddt_bias": ddt.sum(0), "dh0": dh0}


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = (d.square().mean(-1) + EPS).rsqrt()
    return {"out": (d * rstd[..., None] * s["w"] + s["b"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][..., None]) * s["rstd"][..., None]
    gy = dy * s["w"]
    dx = s["rstd"][..., None] * (gy - gy.mean(-1, keepdim=True) - xh * (gy * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


_OWN = {("conv", "step"): _own_conv_step, ("conv", "fwd"): _own_conv_fwd, ("conv", "bwd"): _own_conv_bwd,
        ("ssm", "step"): _own_ssm_step, ("ssm", "fwd"): _own_ssm_fwd, ("ssm", "bwd"): _own_ssm_bwd,
        ("norm", "fwd"): _own_norm_fwd, ("norm", "bwd"): _own_norm_bwd}
_PLAIN = {("conv", "step"): _plain_conv_step, ("conv", "fwd"): _plain_conv_fwd, ("conv", "bwd"): _plain_conv_bwd,
          ("ssm", "step"): _plain_ssm_step, ("ssm", "fwd"): _plain_ssm_fwd, ("ssm", "bwd"): _plain_ssm_bwd,
          ("norm", "fwd"): _plain_norm_fwd, ("norm", "bwd"): _plain_norm_bwd}


# ---------------------------------------------------------------- work


def work(case):
    c = case
    el = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        e = c["M"] * c["G"] * c["D"]
        par = 4 * c["G"] * c["D"]
        if c["do"] == "fwd":   # x, out; weight, bias; mean, rstd
            return {"bytes": 2 * el * e + 2 * par + 8 * c["M"] * c["G"], "flops": 8 * e}
        return {"bytes": 3 * el * e + 3 * par + 8 * c["M"] * c["G"], "flops": 14 * e}
    M, n = c["B"] * c["T"], c["seqs"] or c["B"]
    e = M * c["D"]
    if c["op"] == "conv":
        st = n * (c["W"] - 1) * c["D"] * el
        par = 4 * c["D"] * (c["W"] + bool(c["bias"]))
        had = 1 if c["state"] else 0
        if c["do"] == "bwd":   # x, dy in, dx out; the states and their gradients
            return {"bytes": 3 * el * e + 2 * par + 3 * had * st, "flops": (6 * c["W"] + 8) * e}
        return {"bytes": 2 * el * e + par + (1 + had) * st, "flops": (2 * c["W"] + 5) * e}
    N = c["N"]
    st = 4 * n * c["D"] * N
    bc = 2 * M * c["G"] * N * el
    par = 4 * c["D"] * (N + 2)
    z = 1 if c["gate"] else 0
    had = 1 if c["state"] else 0
    if c["do"] == "bwd":       # x, dt, z, dy in; dx, ddt, dz out; B, C and their gradients
        return {"bytes": (5 + 2 * z) * el * e + 2 * bc + 2 * par + 3 * had * st, "flops": 24 * e * N}
    return {"bytes": (3 + z) * el * e + bc + par + (1 + (had or c["do"] == "step")) * st, "flops": 7 * e * N}


# ---------------------------------------------------------------- 64 bits, from the definitions


def _seq_list(s):
    c = s["case"]
    if s["cu"] is not None:
        cu = s["cu"].tolist()
    else:
        cu = [i * c["T"] for i in range(c["B"] + 1)]
    return list(zip(cu[:-1], cu[1:]))


def _exact_conv(s):
    c, f = s["case"], torch.float64
    W, D = c["W"], c["D"]
    w = s["w"].to(f)
    bias = s["bias"].to(f) if s["bias"] is not None else torch.zeros(D, device=w.device, dtype=f)
    n = c["seqs"] or c["B"]
    st = s["state"].to(f) if s["state"] is not None else torch.zeros(n, W - 1, D, device=w.device, dtype=f)
    x = s["x"].reshape(-1, D)
    outs, fins = [], []
    dx, dst = [], []
    dw, db = torch.zeros(W, D, device=w.device, dtype=f), torch.zeros(D, device=w.device, dtype=f)
    for i, (b, e) in enumerate(_seq_list(s)):
        L = e - b
        line = torch.cat([st[i], x[b:e].to(f)])               # W-1 earlier inputs, then the tokens
        pre = bias.expand(L, D).clone()
        for j in range(W):
            pre += w[:, j] * line[j:j + L]
        sg = 1.0 / (1.0 + torch.exp(-pre))
        if c["do"] != "bwd":
            outs.append(pre * sg if c["silu"] else pre)
            fins.append(line[L:])
            continue
        dy = s["dy"].reshape(-1, D)[b:e].to(f)
        dp = dy * (sg + pre * sg * (1 - sg)) if c["silu"] else dy
        dl = torch.zeros_like(line)
        for j in range(W):
            dl[j:j + L] += w[:, j] * dp
            dw[j] += (dp * line[j:j + L]).sum(0)
        db += dp.sum(0)
        if s["dstate"] is not None:
            dl[L:] += s["dstate"][i].to(f)
        dx.append(dl[W - 1:])
        dst.append(dl[:W - 1])
    if c["do"] != "bwd":
        return {"out": torch.cat(outs).reshape(s["x"].shape), "state": torch.stack(fins)}
    return {"dx": torch.cat(dx).reshape(s["x"].shape), "dw": dw.t().contiguous(), "db": db if s["bias"] is not None else None,
            "dstate": torch.stack(dst) if s["state"] is not None else None}


def _exact_ssm(s):
    c, f = s["case"], torch.float64
    D, N, G = c["D"], c["N"], c["G"]
    A, Dk = s["A"].to(f), s["D"].to(f)
    dev = A.device
    flat = lambda v, *sh: v.reshape(-1, *sh)  # noqa: E731
    x, raw = flat(s["x"], D).to(f), flat(s["dt"], D).to(f) + s["dt_bias"].to(f)
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    Bm, Cm = flat(s["B"], G, N).to(f), flat(s["C"], G, N).to(f)
    z = flat(s["z"], D).to(f) if s["z"] is not None else None
    sg = torch.sigmoid(z) if z is not None else None
    M, n = x.shape[0], c["seqs"] or c["B"]
    bwd = c["do"] == "bwd"
    seqs = _seq_list(s)
    if c["seqs"]:
        runs = [([i], b, e) for i, (b, e) in enumerate(seqs)]
    else:   # sequences of one length walk together
        runs = [(list(range(n)), 0, c["T"])]
    grp = torch.arange(D, device=dev) // (D // G)
    y = torch.zeros(M, D, device=dev, dtype=f)
    hT = torch.zeros(n, D, N, device=dev, dtype=f)
    r = {k: torch.zeros_like(y) for k in ("dx", "ddt")} if bwd else {}
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dh0 = torch.zeros_like(hT)
    dout = flat(s["dy"], D).to(f) if bwd else None
    dy = None
    if bwd:
        dy = dout * z * sg if z is not None else dout
    for who, b, e in runs:
        base = torch.tensor([seqs[i][0] for i in who], device=dev)
        idx = torch.tensor(who, device=dev)
        h = s["h"][idx].to(f) if s["h"] is not None else torch.zeros(len(who), D, N, device=dev, dtype=f)
        kept = [h]
        for t in range(e - b):
            at = base + t
            h = torch.exp(dt[at][..., None] * A) * h + (dt[at] * x[at])[..., None] * Bm[at][:, grp]
            y[at] = (h * Cm[at][:, grp]).sum(-1)
            if bwd:
                kept.append(h)
        hT[idx] = h
        if not bwd:
            continue
        g = s["dh"][idx].to(f) if s["dh"] is not None else torch.zeros_like(h)
        for t in reversed(range(e - b)):
            at = base + t
            g = g + dy[at][..., None] * Cm[at][:, grp]
            dC.index_add_(0, at, (dy[at][..., None] * kept[t + 1]).reshape(len(who), G, D // G, N).sum(2))
            dB.index_add_(0, at, (g * (dt[at] * x[at])[..., None]).reshape(len(who), G, D // G, N).sum(2))
            gb = (g * Bm[at][:, grp]).sum(-1)
            g = g * torch.exp(dt[at][..., None] * A)
            gh = g * kept[t]
            dA += (gh * dt[at][..., None]).sum(0)
            r["dx"][at] = gb * dt[at]
            r["ddt"][at] = (gh * A).sum(-1) + gb * x[at]
        dh0[idx] = g
    y += Dk * x
    if not bwd:
        return {"out": (y * z * sg if z is not None else y).reshape(s["x"].shape), "h": hT}
    ddt = r["ddt"] * torch.sigmoid(raw)
    return {"dx": (r["dx"] + Dk * dy).reshape(s["x"].shape), "ddt": ddt.reshape(s["dt"].shape), "dA": dA,
            "dB": dB.reshape(s["B"].shape), "dC": dC.reshape(s["C"].shape), "dD": (dy * x).sum(0),
            "dz": (dout * y * (sg + z * sg * (1 - sg))).reshape(s["x"].shape) if z is not None else None,
            "ddt_bias": ddt.sum(0), "dh0": dh0 if s["h"] is not None else None}


def _exact_norm(s):
    f = torch.float64
    x, w = s["x"].to(f), s["w"].to(f)
    D = x.shape[-1]
    if s["case"]["do"] == "fwd":
        mean = x.sum(-1) / D
        var = ((x - mean[..., None]) ** 2).sum(-1) / D
        rstd = 1.0 / torch.sqrt(var + EPS)
        return {"out": (x - mean[..., None]) * rstd[..., None] * w + s["b"].to(f), "mean": mean, "rstd": rstd}
    r = s["rstd"].to(f)[..., None]
    xh, dy = (x - s["mean"].to(f)[..., None]) * r, s["dy"].to(f)
    gy = dy * w
    c1, c2 = gy.sum(-1, keepdim=True) / D, (gy * xh).sum(-1, keepdim=True) / D
    return {"dx": r * (gy - c1 - xh * c2), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    tokens = case["T"]
    # a token loop of small launches, twice for gradients, and every state kept: minutes past this
    if case["op"] == "ssm" and tokens * (3 if case["do"] == "bwd" else 1) > 60000:
        return None
    return _exact_conv(s) if case["op"] == "conv" else _exact_ssm(s)
