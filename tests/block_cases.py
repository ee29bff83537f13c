"""Inputs and comparisons that the recurrent block's tests share.

Tolerances.  A result computed in fp32 differs from the exact one by a number of roundings
(2^-24 each, relative) on terms whose absolute values sum to `mag` (the references' mag=True
result); a bf16 output adds half a step of its own, 2^-8 of the value.  So every comparison is
    |got - ref| <= half(dtype) * |ref| + steps * 2^-24 * mag * (1 + half(dtype)) + tiny
with `steps` the length of the longest chain of roundings, stated at each test."""
import numpy as np
import torch

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}   # an fp32 output's own rounding is one of the steps


def close(got, ref, mag, steps, what):
    if got is None:
        raise AssertionError(f"{what}: no result")
    h = HALF[got.dtype]
    g = got.detach().cpu().double().numpy().reshape(ref.shape)
    lim = h * np.abs(ref) + steps * 2.0 ** -24 * mag * (1.0 + h) + 1e-37
    bad = ~(np.abs(g - ref) <= lim)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / lim, 0)), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; worst at {at}: {g[at]!r} for {ref[at]!r}, "
                             f"allowed {lim[at]:.3e}")


def rnd(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * scale).to(dtype)


def lengths(spec):
    """cu_seqlens (list) of the sequence lengths."""
    cu = [0]
    for n in spec:
        cu.append(cu[-1] + n)
    return cu


def dev(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def strided_like(t, pad=3, shift=1):
    """The same values as a slice of a wider matrix whose rows start `shift` elements in."""
    D = t.shape[-1]
    wide = torch.zeros(*t.shape[:-1], D + pad, dtype=t.dtype, device=t.device)
    wide[..., shift:shift + D] = t
    return wide[..., shift:shift + D]
