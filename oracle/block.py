"""float64 references of the recurrent block's operators (test infrastructure): the short
causal convolution, the selective state space scan and layer norm, written row by row from
their definitions, with gradients by the chain rule.

Every function takes `mag`: False gives the values; True gives, in their place, the sums of
the absolute values of the terms that make them up, which is what rounding errors of a
computation in fewer bits are proportional to."""
from __future__ import annotations

import numpy as np


def f64(t):
    """A torch tensor (or None) as a float64 array."""
    return None if t is None else t.detach().cpu().double().numpy()


def _abs(mag):
    return np.abs if mag else (lambda v: v)


def silu(v):
    return v / (1.0 + np.exp(-v))


def silu_grad(v):
    s = 1.0 / (1.0 + np.exp(-v))
    return s * (1.0 + v * (1.0 - s))


def bounds(B, T, cu):
    return [(n * T, (n + 1) * T) for n in range(B)] if cu is None else list(zip(cu[:-1], cu[1:]))


# ---------------------------------------------------------------- convolution


def conv(x, w, bias, state, seqs, act, d_out=None, d_fin=None, mag=False):
    """x [M, D]; w [D, W]; state [n, W-1, D] or None; seqs: (first row, row past the last) of
    each sequence.  Returns out [M, D], final [n, W-1, D] and, with d_out, dx, dw, db, dstate.
    Rows in no sequence stay zero."""
    a = _abs(mag)
    M, D = x.shape
    W, n = w.shape[1], len(seqs)
    r = dict(out=np.zeros((M, D)), final=np.zeros((n, W - 1, D)))
    if d_out is not None:
        r.update(dx=np.zeros((M, D)), dw=np.zeros((D, W)), db=np.zeros(D), dstate=np.zeros((n, W - 1, D)))
    for q, (b, e) in enumerate(seqs):
        before = state[q] if state is not None else np.zeros((W - 1, D))
        line = np.concatenate([before, x[b:e]])
        dline = np.zeros_like(line)
        for t in range(e - b):
            pre = np.zeros(D) if bias is None else bias.copy()
            big = np.abs(pre)
            for j in range(W):
                pre += w[:, j] * line[t + j]
                big += np.abs(w[:, j] * line[t + j])
            if mag:   # |silu'| <= 1.1
                r["out"][b + t] = 1.1 * big if act else big
            else:
                r["out"][b + t] = silu(pre) if act else pre
            if d_out is None:
                continue
            g = a(d_out[b + t])
            if act:   # an error of pre moves silu' by at most half as much
                g = g * (np.abs(silu_grad(pre)) + 0.5 * big if mag else silu_grad(pre))
            for j in range(W):
                dline[t + j] += a(w[:, j]) * g
                r["dw"][:, j] += a(line[t + j]) * g
            r["db"] += g
        r["final"][q] = a(line[e - b:])
        if d_out is not None:
            if d_fin is not None:
                dline[e - b:] += a(d_fin[q])
            r["dx"][b:e] = dline[W - 1:]
            r["dstate"][q] = dline[:W - 1]
    return r


# ---------------------------------------------------------------- selective scan


def ssm(x, delta, A, Bm, Cm, D, z, bias, h0, seqs, softplus=True, d_out=None, d_hT=None, mag=False):
    """x, delta, z [M, D]; A [D, N]; Bm, Cm [M, G, N].  Returns out, hT and, with d_out, dx, ddt,
    dA, dB, dC, dD, dz, ddt_bias, dh0."""
    a = _abs(mag)
    M, Dc = x.shape
    G, N = Bm.shape[1:]
    n = len(seqs)
    grp = np.arange(Dc) // (Dc // G)
    raw = delta + (bias if bias is not None else 0.0)
    dt = np.logaddexp(raw, 0.0) if softplus else raw
    dD = D if D is not None else np.zeros(Dc)
    gate = a(silu(z)) if z is not None else np.ones_like(x)
    r = dict(out=np.zeros((M, Dc)), hT=np.zeros((n, Dc, N)))
    if d_out is not None:
        r.update(dx=np.zeros((M, Dc)), ddt=np.zeros((M, Dc)), dA=np.zeros((Dc, N)), dB=np.zeros((M, G, N)),
                 dC=np.zeros((M, G, N)), dD=np.zeros(Dc), dz=np.zeros((M, Dc)), ddt_bias=np.zeros(Dc),
                 dh0=np.zeros((n, Dc, N)))
    for q, (b, e) in enumerate(seqs):
        h = a(h0[q]).copy() if h0 is not None else np.zeros((Dc, N))
        hs = [h]
        for t in range(b, e):
            h = np.exp(dt[t][:, None] * A) * h + a(dt[t] * x[t])[:, None] * a(Bm[t][grp])
            hs.append(h)
            y = (h * a(Cm[t][grp])).sum(-1) + a(dD * x[t])
            r["out"][t] = y * gate[t]
            if d_out is not None and z is not None:
                r["dz"][t] = a(d_out[t]) * y * (1.1 if mag else silu_grad(z[t]))
        r["hT"][q] = h
        if d_out is None:
            continue
        g = a(d_hT[q]).copy() if d_hT is not None else np.zeros((Dc, N))
        for t in range(e - 1, b - 1, -1):
            dy = a(d_out[t]) * gate[t]
            B, C = a(Bm[t][grp]), a(Cm[t][grp])
            hp = hs[t - b]
            g = g + dy[:, None] * C
            cont = dy[:, None] * hs[t - b + 1]
            contB = g * a(dt[t] * x[t])[:, None]
            for k in range(G):
                r["dC"][t, k] = cont[grp == k].sum(0)
                r["dB"][t, k] = contB[grp == k].sum(0)
            p = (g * B).sum(-1)
            g = g * np.exp(dt[t][:, None] * A)
            w = g * hp
            r["dA"] += w * a(dt[t])[:, None]
            dd = (w * a(A)).sum(-1) + p * a(x[t])
            if softplus:
                dd = dd / (1.0 + np.exp(-raw[t]))
            r["ddt"][t] = dd
            r["ddt_bias"] += dd
            r["dx"][t] = p * a(dt[t]) + a(dD) * dy
            r["dD"] += dy * a(x[t])
        r["dh0"][q] = g
    return r


# ---------------------------------------------------------------- layer norm


def norm(x, w, b, eps, d_out=None, mag=False):
    """x [R, G, D]; w, b [G, D].  Returns out, mean, rstd and, with d_out, dx, dw, db."""
    a = _abs(mag)
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    xh = (a(x) + a(mean)) * rstd if mag else (x - mean) * rstd
    r = dict(out=xh * a(w) + a(b), mean=(a(x).mean(-1, keepdims=True))[..., 0], rstd=rstd[..., 0])
    if d_out is not None:
        g = a(d_out)
        gy = g * a(w)
        c1, c2 = gy.mean(-1, keepdims=True), (gy * xh).mean(-1, keepdims=True)
        r["dx"] = rstd * (gy + c1 + xh * c2) if mag else rstd * (gy - c1 - xh * c2)
        r["dw"], r["db"] = (g * xh).sum(0), g.sum(0)
    return r
