"""The selective state space scan: forward, one-row step and gradients against the float64
reference, over state counts, groups, types, alignments, packed and dense batches, sequences of
zero, one and a few rows, tiles and segments that sequences end inside of, rows behind the last
sequence; refusals; the reference's gradients against differences.

Steps (see block_cases).  Every row multiplies the state by a decay e^{dt A}: the hardware
exponential of dt A log2(e) is off by 2 units plus |dt A log2 e| <= 8 units of the argument's
rounding, a softplus by 8 units (times |dt A| in the exponent), and each row adds two roundings;
so T rows give 32 T + 64 steps on the states.  A gradient walks the rows once more in reverse
over such states, 64 T + 128, and a sum over R rows or channels adds R."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_22_b200 as kda
from block_cases import close, dev, lengths, rnd, strided_like
from kimi_delta_attention_22_b200 import build as kbuild
from oracle import block as ob
from test_block_conv import _differences

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def draw(B, T, D, N, G, dtype, cu=None, state=True, gate=True, skip=True, bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    return dict(x=rnd(g, B, T, D, dtype=dtype), dt=rnd(g, B, T, D, dtype=dtype) - 1,
                A=-torch.exp(rnd(g, D, N, scale=0.7)), B=rnd(g, B, T, G, N, dtype=dtype), C=rnd(g, B, T, G, N, dtype=dtype),
                D=rnd(g, D) if skip else None, z=rnd(g, B, T, D, dtype=dtype) if gate else None,
                dt_bias=rnd(g, D) if bias else None, h0=rnd(g, n, D, N) if state else None,
                dy=rnd(g, B, T, D, dtype=dtype), dh=rnd(g, n, D, N) if state else None,
                cu=None if cu is None else torch.tensor(cu, dtype=torch.int32))


def reference(d, softplus=True, bwd=False, mag=False):
    B, T, D = d["x"].shape
    G, N = d["B"].shape[2:]
    cu = None if d["cu"] is None else d["cu"].tolist()
    f = ob.f64
    r2 = lambda t: None if t is None else f(t).reshape(-1, D)  # noqa: E731
    r3 = lambda t: f(t).reshape(-1, G, N)  # noqa: E731
    return ob.ssm(r2(d["x"]), r2(d["dt"]), f(d["A"]), r3(d["B"]), r3(d["C"]), f(d["D"]), r2(d["z"]), f(d["dt_bias"]),
                  f(d["h0"]), ob.bounds(B, T, cu), softplus, r2(d["dy"]) if bwd else None,
                  f(d["dh"]) if bwd and d["dh"] is not None else None, mag)


def forward(o, **kw):
    return kda.kda_ssm_fwd(o["x"], o["dt"], o["A"], o["B"], o["C"], D=o["D"], z=o["z"], dt_bias=o["dt_bias"], h0=o["h0"],
                           cu_seqlens=o["cu"], **kw)


def backward(o, **kw):
    return kda.kda_ssm_bwd(o["x"], o["dt"], o["A"], o["B"], o["C"], o["dy"], D=o["D"], z=o["z"], dt_bias=o["dt_bias"],
                           h0=o["h0"], d_hT=o["dh"], cu_seqlens=o["cu"], **kw)


# B, T, D, N, G, dtype, sequence lengths (None: dense), options
CASES = [
    (2, 70, 64, 16, 1, BF, None, {}),
    (1, 1, 8, 16, 1, BF, None, {}),
    (1, 3, 1, 1, 1, F32, None, {}),
    (2, 64, 40, 16, 2, F32, None, {}),
    (1, 33, 37, 5, 1, BF, None, {}),                             # odd channels: element accesses
    (3, 45, 24, 3, 3, F32, None, dict(gate=False)),
    (1, 50, 136, 8, 1, BF, None, dict(state=False, skip=False)),
    (1, 40, 32, 24, 2, F32, None, dict(bias=False)),
    (1, 66, 16, 32, 1, BF, None, {}),
    (1, 65, 24, 64, 1, BF, None, {}),
    (2, 30, 12, 50, 1, F32, None, {}),
    (1, 35, 16, 128, 2, BF, None, {}),
    (1, 29, 9, 100, 1, F32, None, {}),
    (1, 0, 16, 16, 1, BF, [0, 0, 0], {}),
    (2, 0, 16, 16, 1, F32, None, {}),
    (1, 200, 48, 16, 1, BF, [0, 1, 63, 0, 64, 2, 65, 5, 0], {}),
    (1, 150, 40, 16, 1, F32, [31, 33, 1, 1, 70], {}),            # 14 rows behind the last sequence
    (1, 97, 21, 4, 1, F32, [40, 57], {}),
    (1, 130, 8, 7, 1, BF, [127, 3], dict(gate=False, skip=False, bias=False, state=False)),
    (1, 700, 24, 16, 1, BF, None, {}),                           # cut into segments
    (1, 900, 24, 16, 1, F32, [5, 300, 1, 594], {}),
    (2, 520, 16, 33, 1, F32, None, {}),
    (1, 1100, 72, 8, 3, BF, [512, 128, 0, 448], {}),             # boundaries on segments' and tiles' edges
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,N,G,dtype,lens,opt", CASES)
def test_forward(B, T, D, N, G, dtype, lens, opt):
    cu = None if lens is None else lengths(lens)
    d = draw(B, T, D, N, G, dtype, cu, seed=T + D, **opt)
    o = dev(d)
    out = torch.full((B, T, D), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, hT = forward(o, out=out, dev_status=st)
    assert st.item() == 0
    r, m = reference(d), reference(d, mag=True)
    n = B * T if cu is None else cu[-1]
    longest = T if cu is None else max(lens)
    flat = out.reshape(B * T, D)
    close(flat[:n], r["out"][:n], m["out"][:n], 32 * longest + 64 + N, "out")
    assert (flat[n:] == 7.0).all()
    close(hT, r["hT"], m["hT"], 32 * longest + 64, "hT")


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,N,G,dtype,lens,opt", CASES)
def test_backward(B, T, D, N, G, dtype, lens, opt):
    cu = None if lens is None else lengths(lens)
    d = draw(B, T, D, N, G, dtype, cu, seed=T + 2 * D, **opt)
    o = dev(d)
    keep = {k: torch.full(o["x"].shape if k != "dB" else o["B"].shape, 7.0, dtype=dtype, device="cuda")
            for k in ("dx", "ddt", "dB")}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = backward(o, grads=keep, want_dh0=d["h0"] is not None, dev_status=st)
    assert st.item() == 0
    r, m = reference(d, bwd=True), reference(d, bwd=True, mag=True)
    n = B * T if cu is None else cu[-1]
    longest = T if cu is None else max(lens)
    steps = 64 * longest + 128 + N
    for k, extra in (("dx", 0), ("ddt", 0), ("dz", 0), ("dB", D), ("dC", D)):
        if k == "dz" and d["z"] is None:
            assert g["dz"] is None
            continue
        flat = g[k].reshape(B * T, r[k][:1].size if r[k].size else 1)
        close(flat[:n], r[k][:n].reshape(flat[:n].shape), m[k][:n].reshape(flat[:n].shape), steps + extra, k)
        if k in keep:
            assert (flat[n:] == 7.0).all()
    close(g["dA"], r["dA"], m["dA"], steps + n, "dA")
    if d["D"] is not None:
        close(g["dD"], r["dD"], m["dD"], steps + n, "dD")
    if d["dt_bias"] is not None:
        close(g["ddt_bias"], r["ddt_bias"], m["ddt_bias"], steps + n, "ddt_bias")
    if d["h0"] is not None:
        close(g["dh0"], r["dh0"], m["dh0"], steps, "dh0")
    else:
        assert g["dh0"] is None


@pytest.mark.gpu
def test_without_softplus_growing_states():
    """dt as given: with negative steps the states grow, here past the range of fp32 in most
    channels (the reference reaches 10^48).  A state over 3.4e38 has no fp32 value and is infinite
    from then on, so the channels whose terms stay below 10^36 are compared."""
    d = draw(1, 20, 16, 16, 1, F32, seed=4)
    d["dt"] = d["dt"] * 0.1
    o = dev(d)
    out, hT = forward(o, softplus=False)
    r, m = reference(d, False), reference(d, False, mag=True)
    ok = (m["out"].max(0) < 1e36) & (m["hT"][0].max(-1) < 1e36)
    assert 4 <= ok.sum() < 16
    close(out.reshape(-1, 16)[:, torch.from_numpy(ok)], r["out"][:, ok], m["out"][:, ok], 32 * 20 + 80, "out")
    close(hT[:, torch.from_numpy(ok)], r["hT"][:, ok], m["hT"][:, ok], 32 * 20 + 64, "hT")


@pytest.mark.gpu
def test_without_softplus():
    """dt as given, a few negative steps among them: the decay is whatever dt A says."""
    d = draw(1, 20, 16, 16, 1, F32, bias=False, seed=4)
    d["dt"] = d["dt"] * 0.1 + 0.2
    assert (d["dt"] < 0).any()
    o = dev(d)
    out, hT = forward(o, softplus=False)
    r, m = reference(d, False), reference(d, False, mag=True)
    close(out.reshape(-1, 16), r["out"], m["out"], 32 * 20 + 80, "out")
    close(hT, r["hT"], m["hT"], 32 * 20 + 64, "hT")
    g = backward(o, softplus=False)
    r, m = reference(d, False, True), reference(d, False, True, True)
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
        close(g[k], r[k], m[k], 64 * 20 + 200, k)


@pytest.mark.gpu
def test_extreme_step_sizes():
    """Steps of e^-30 and of 60 (a decay of zero), infinite delta (dt = inf, x = 0 there): no NaN
    where the definition has none, and softplus keeps its relative accuracy at tiny steps."""
    d = draw(1, 40, 8, 16, 1, F32, state=True, bias=False, seed=6)
    d["dt"][0, :10] = -30.0
    d["dt"][0, 10:20] = 60.0
    d["dt"][0, 25] = -float("inf")
    o = dev(d)
    out, hT = forward(o)
    with np.errstate(over="ignore", invalid="ignore"):
        r, m = reference(d), reference(d, mag=True)
    close(out.reshape(-1, 8), r["out"], m["out"], 32 * 40 + 80 + 1000, "out")   # |dt A| reaches 10^3 where it decays to 0
    close(hT, r["hT"], m["hT"], 32 * 40 + 64, "hT")
    tiny = dict(d, x=d["x"][:, :1], dt=d["dt"][:, :1], B=d["B"][:, :1], C=d["C"][:, :1], z=d["z"][:, :1], h0=None)
    _, h = forward(dev(dict(tiny, A=d["A"])))
    want = np.logaddexp(ob.f64(tiny["dt"])[0, 0], 0) * ob.f64(tiny["x"])[0, 0]
    want = want[:, None] * ob.f64(tiny["B"])[0, 0, 0]
    close(h[0], want, np.abs(want), 16 + 64, "dt of e^-30")   # the argument 30 log2(e) rounds by 64 units


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,S,G,dtype,gate", [(1, 8, 16, 1, BF, True), (5, 40, 16, 2, F32, True), (3, 13, 5, 1, BF, False),
                                                (9, 24, 1, 1, F32, True), (2, 17, 64, 1, BF, True), (4, 8, 128, 1, F32, True),
                                                (2, 6, 20, 3, BF, True), (6, 33, 8, 1, BF, True)])
def test_steps_against_reference(N, D, S, G, dtype, gate):
    T = 6
    d = draw(N, T, D, S, G, dtype, gate=gate, seed=N + S)
    o = dev(d)
    h = o["h0"].clone()
    rows = [kda.kda_ssm_step(o["x"][:, t], o["dt"][:, t], o["A"], o["B"][:, t], o["C"][:, t], h, D=o["D"],
                             z=None if not gate else o["z"][:, t], dt_bias=o["dt_bias"]) for t in range(T)]
    r, m = reference(d), reference(d, mag=True)
    close(torch.stack(rows, 1).reshape(-1, D), r["out"], m["out"], 32 * T + 64 + S, "out")
    close(h, r["hT"], m["hT"], 32 * T + 64, "h")


@pytest.mark.gpu
def test_split_prompt_then_steps():
    """A packed prompt, then steps from its states, equal one longer prompt."""
    T, D, N = 90, 32, 16
    d = draw(1, T, D, N, 1, BF, [0, 50, 90], seed=12)
    o = dev(d)
    out, hT = forward(o)
    cu1 = torch.tensor([0, 45, 80], dtype=torch.int32, device="cuda")
    rows = torch.cat([torch.arange(0, 45), torch.arange(50, 85)]).cuda()
    pick = {k: o[k][:, rows].contiguous() for k in ("x", "dt", "B", "C", "z")}
    o1, h = kda.kda_ssm_fwd(pick["x"], pick["dt"], o["A"], pick["B"], pick["C"], D=o["D"], z=pick["z"], dt_bias=o["dt_bias"],
                            h0=o["h0"], cu_seqlens=cu1)
    last = []
    for k in range(5):
        at = torch.tensor([45 + k, 85 + k], device="cuda")
        last.append(kda.kda_ssm_step(o["x"][0, at], o["dt"][0, at], o["A"], o["B"][0, at], o["C"][0, at], h, D=o["D"],
                                     z=o["z"][0, at], dt_bias=o["dt_bias"]))
    r, m = reference(d), reference(d, mag=True)
    close(h, r["hT"], m["hT"], 32 * 50 + 64, "h after the steps")
    close(torch.stack(last)[:, 0], r["out"][45:50], m["out"][45:50], 32 * 50 + 80, "rows of the first")
    close(torch.stack(last)[:, 1], r["out"][85:90], m["out"][85:90], 32 * 50 + 80, "rows of the second")


@pytest.mark.gpu
@pytest.mark.parametrize("shift,pad", [(0, 8), (8, 24), (1, 3)])
def test_row_strided_inputs(shift, pad):
    """Slices of wider rows give the same values as contiguous inputs."""
    o = dev(draw(2, 75, 40, 16, 1, BF, seed=14))
    s = dict(o)
    for k in ("x", "dt", "z"):
        s[k] = strided_like(o[k], pad + shift, shift)
    wide = torch.zeros(2, 75, 4 + 32 + shift, dtype=BF, device="cuda")   # a projection's [dt, B, C] columns
    wide[..., 4 + shift:20 + shift] = o["B"][:, :, 0]
    wide[..., 20 + shift:] = o["C"][:, :, 0]
    s["B"], s["C"] = wide[..., 4 + shift:20 + shift], wide[..., 20 + shift:]
    a, b = forward(o), forward(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = backward(o), backward(s)
    for k in ga:
        assert torch.equal(ga[k].reshape(-1), gb[k].reshape(-1)), k


@pytest.mark.gpu
def test_inconsistent_cu_seqlens_is_flagged():
    o = dev(draw(1, 640, 16, 16, 1, BF, [0, 200, 400, 640], seed=8))
    for bad in ([0, 200, 700, 640], [0, 400, 200, 640], [0, 200, -5, 640], [5, 200, 400, 640]):
        o["cu"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (forward, backward):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(o, dev_status=st)
            assert st.item() == kda.KDA_DEV_BAD_SEQLENS, (bad, call)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[90, 70, 200, 33], [400, 300, 500, 70], [3, 2, 5, 4]])
def test_bad_values_stay_in_their_sequence(lens):
    """NaN and infinities in one sequence's rows, states and state gradients leave every other
    sequence's outputs and gradients as they were, bit for bit; the same in rows of no sequence."""
    cu = lengths(lens)
    T = cu[-1] + 9
    d = draw(1, T, 24, 16, 2, F32, cu, seed=21)
    o = dev(d)
    good, hT = forward(o)
    gg = backward(o)
    for bad in (1, 2):
        b, e = cu[bad], cu[bad + 1]
        for value in (float("nan"), float("inf")):
            p = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in o.items()}
            for k in ("x", "dt", "B", "C", "z", "dy"):
                p[k][:, b:e] = value
                p[k][:, cu[-1]:] = value
            p["h0"][bad] = value
            p["dh"][bad] = value
            out, h = forward(p)
            g = backward(p)
            keep = [n for n in range(len(lens)) if n != bad]
            rows = torch.cat([torch.arange(cu[n], cu[n + 1]) for n in keep]).cuda()
            assert torch.equal(out[:, rows], good[:, rows]) and torch.equal(h[keep], hT[keep])
            for k in ("dx", "ddt", "dz", "dB", "dC"):
                assert torch.equal(g[k][:, rows], gg[k][:, rows]), (bad, value, k)
            assert torch.equal(g["dh0"][keep], gg["dh0"][keep])
    p = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in o.items()}
    for k in ("x", "dt", "B", "C", "z", "dy"):
        p[k][:, cu[-1]:] = float("nan")
    g = backward(p)
    for k in ("dA", "dD", "ddt_bias", "dh0"):
        assert torch.equal(g[k], gg[k]), k


@pytest.mark.gpu
def test_binding_refusals():
    o = dev(draw(2, 8, 16, 16, 1, BF, seed=1))
    args = [o[k] for k in ("x", "dt", "A", "B", "C")]

    def call(**kw):
        a = [kw.pop(k, v) for k, v in zip(("x", "dt", "A", "B", "C"), args)]
        return kda.kda_ssm_fwd(*a, **kw)

    call()
    with pytest.raises(TypeError):
        call(dt=o["dt"].float())
    with pytest.raises(TypeError):
        call(A=o["A"].bfloat16())
    with pytest.raises(ValueError):
        call(B=o["B"].expand(2, 8, 3, 16), C=o["C"].expand(2, 8, 3, 16))   # 3 groups of 16 channels
    with pytest.raises(ValueError):
        call(C=o["C"][..., :8])
    with pytest.raises(ValueError):
        call(h0=o["h0"][:1])
    with pytest.raises(ValueError):
        call(z=o["z"].transpose(0, 1))
    with pytest.raises(ValueError):
        call(D=o["D"].cpu())
    with pytest.raises(kda.KDAError):
        call(h0=o["h0"], hT=o["h0"])
    with pytest.raises(kda.KDAError):
        call(out=o["x"])
    with pytest.raises(ValueError):
        kda.kda_ssm_bwd(*args, o["dy"], grads=dict(dX=o["dy"].clone()))
    with pytest.raises(kda.KDAError):
        kda.kda_ssm_bwd(*args, o["dy"], grads=dict(dx=o["dy"]))
    with pytest.raises(kda.KDAError):
        kda.kda_ssm_fwd(o["x"], o["dt"], torch.zeros(16, 129, device="cuda"), torch.zeros(2, 8, 129, dtype=BF, device="cuda"),
                        torch.zeros(2, 8, 129, dtype=BF, device="cuda"))


def test_validation(lib):
    P = ctypes.c_void_p
    A = P(0x10000)

    def sh(B=0, T=8, D=16, N=16, G=1, n=None, dt=kda.KDA_BF16, sp=1, st=(0, 0, 0, 0, 0)):
        return kda.SsmShape(B, T, D, N, G, B if n is None else n, dt, sp, *st, None)

    def fwd(s, x=A, Am=A, h0=None, cu=None, hT=None, ws=None, nb=0, out=A):
        return lib.kda_ssm_fwd(None if s is None else ctypes.byref(s), x, A, Am, A, A, None, None, None, h0, cu, out, hT,
                               ws, nb, None)

    assert fwd(None) == 1 and fwd(sh()) == 0
    assert fwd(sh(n=2)) == 1 and fwd(sh(B=2, n=0), cu=A) == 1
    assert fwd(sh(D=0)) == 1 and fwd(sh(N=0)) == 1 and fwd(sh(G=3)) == 1 and fwd(sh(G=0)) == 1 and fwd(sh(N=129)) == 2
    assert fwd(sh(dt=7)) == 1 and fwd(sh(sp=2)) == 1 and fwd(sh(T=-1)) == 1
    assert fwd(sh(st=(8, 0, 0, 0, 0))) == 1 and fwd(sh(st=(0, 0, 0, 15, 0))) == 1 and fwd(sh(st=(32, 16, 20, 16, 40))) == 0
    assert fwd(sh(), Am=None) == 1 and fwd(sh(B=1), x=None) == 1 and fwd(sh(), h0=A, hT=A) == 1
    assert fwd(sh(), x=P(0x10001)) == 3 and fwd(sh(), Am=P(0x10002)) == 3 and fwd(sh(dt=kda.KDA_F32), out=P(0x10002)) == 3
    # few channels and a long axis need scratch; many channels and sequences none
    long = sh(B=1, T=4096, n=1)
    need = lib.kda_ssm_fwd_workspace_size(ctypes.byref(long), 0)
    assert need > 0 and lib.kda_ssm_fwd_workspace_size(None, 0) == 0
    assert fwd(long, ws=A, nb=need - 1) == 1 and fwd(long, ws=P(0x10010), nb=need) == 3
    many = sh(B=64, T=256, D=4096)
    assert lib.kda_ssm_fwd_workspace_size(ctypes.byref(many), 0) == 0

    def step(s, h=A):
        return lib.kda_ssm_step(ctypes.byref(s), A, A, A, A, A, None, None, None, h, A, None)

    assert step(sh(T=1)) == 0 and step(sh(T=2)) == 1 and step(sh(B=3, T=1), h=None) == 1

    def bwd(s, z=None, dz=None, D=None, dD=None, b=None, db=None, ws=A, nb=0, dA=A):
        return lib.kda_ssm_bwd(ctypes.byref(s), A, A, A, A, A, D, z, b, None, None, A, None, A, A, dA, A, A, dD, dz, db,
                               None, ws, nb, None)

    s = sh(B=1, T=64)
    need = lib.kda_ssm_bwd_workspace_size(ctypes.byref(s), 0)
    assert need > 0
    assert bwd(s, nb=need - 1) == 1 and bwd(s, ws=P(0x10010), nb=need) == 3
    assert bwd(s, z=A, nb=need) == 1 and bwd(s, dz=A, nb=need) == 1
    assert bwd(s, D=A, nb=need) == 1 and bwd(s, db=A, nb=need) == 1 and bwd(s, dA=None, nb=need) == 1


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(1)
    M, D, N, G = 6, 4, 3, 2
    seqs = [(0, 2), (2, 2), (2, 6)]
    v = dict(x=rng.standard_normal((M, D)), dt=rng.standard_normal((M, D)), A=-np.exp(rng.standard_normal((D, N))),
             B=rng.standard_normal((M, G, N)), C=rng.standard_normal((M, G, N)), D=rng.standard_normal(D),
             z=rng.standard_normal((M, D)), b=rng.standard_normal(D), h0=rng.standard_normal((3, D, N)))
    dy, dh = rng.standard_normal((M, D)), rng.standard_normal((3, D, N))
    for sp in (True, False):
        def loss():
            r = ob.ssm(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["b"], v["h0"], seqs, sp)
            return (r["out"] * dy).sum() + (r["hT"] * dh).sum()

        r = ob.ssm(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["b"], v["h0"], seqs, sp, dy, dh)
        for name, grad in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                           ("b", "ddt_bias"), ("h0", "dh0")):
            _differences(loss, v[name], r[grad], name)
