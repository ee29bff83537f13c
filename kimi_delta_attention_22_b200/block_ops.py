"""Binding of the recurrent block's other operators (include/kda.h): the short causal
convolution, the selective state space scan and layer norm.

As in the package's other functions, every arithmetic step runs in the library's kernels,
on the current stream of the tensors' device, and nothing synchronises.  Activations are
bf16 or fp32; parameters and recurrent states are fp32.  Inputs marked "row-strided" may be
slices of a wider matrix (the last axis contiguous, rows at one common distance); all other
tensors are contiguous.  Rows that no sequence of `cu_seqlens` covers are not written.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

import kimi_delta_attention_22_b200 as _b

__all__ = ["kda_conv_fwd", "kda_conv_step", "kda_conv_bwd", "kda_ssm_fwd", "kda_ssm_step", "kda_ssm_bwd",
           "kda_layer_norm_fwd", "kda_layer_norm_bwd", "ConvShape", "SsmShape", "NormShape"]

_i32, _i64, _P, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class ConvShape(ctypes.Structure):
    """kda_conv_shape_t"""
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("num_seqs", _i32), ("width", _i32), ("dtype", _i32),
                ("grad_dtype", _i32), ("activation", _i32), ("x_stride", _i64), ("dev_status", _P)]


class SsmShape(ctypes.Structure):
    """kda_ssm_shape_t"""
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("N", _i32), ("G", _i32), ("num_seqs", _i32), ("dtype", _i32),
                ("softplus", _i32), ("x_stride", _i64), ("delta_stride", _i64), ("z_stride", _i64),
                ("b_stride", _i64), ("c_stride", _i64), ("dev_status", _P)]


class NormShape(ctypes.Structure):
    """kda_norm_shape_t"""
    _fields_ = [("rows", _i64), ("groups", _i32), ("D", _i32), ("dtype", _i32), ("eps", ctypes.c_float),
                ("x_stride", _i64)]


@functools.lru_cache(maxsize=1024)
def _sizes(cls, *fields):
    return ctypes.byref(cls(*fields))


def _shape(cls, *fields):
    """A shape structure by reference.  The library only reads it, so calls of the same sizes share
    one (building it takes a good part of the host's time of a small call); one with a status
    word's address in it is the call's own."""
    return _sizes(cls, *fields) if fields[-1] is None or cls is NormShape else ctypes.byref(cls(*fields))


def declare(lib) -> None:
    """Argument types of this file's entry points."""
    C, S, N = ctypes.POINTER(ConvShape), ctypes.POINTER(SsmShape), ctypes.POINTER(NormShape)
    sig = {
        "kda_conv_fwd": [C] + [_P] * 8, "kda_conv_step": [C] + [_P] * 6, "kda_conv_bwd": [C] + [_P] * 12 + [_SZ, _P],
        "kda_ssm_fwd": [S] + [_P] * 13 + [_SZ, _P], "kda_ssm_step": [S] + [_P] * 11,
        "kda_ssm_bwd": [S] + [_P] * 22 + [_SZ, _P],
        "kda_layer_norm_fwd": [N] + [_P] * 7, "kda_layer_norm_bwd": [N] + [_P] * 9 + [_SZ, _P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    for name, args in {"kda_conv_bwd_workspace_size": [C], "kda_ssm_fwd_workspace_size": [S, ctypes.c_int],
                       "kda_ssm_bwd_workspace_size": [S, ctypes.c_int], "kda_layer_norm_bwd_workspace_size": [N]}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, _SZ


# ------------------------------------------------------------------ argument checks

_DTYPE = {torch.bfloat16: _b.KDA_BF16, torch.float32: _b.KDA_F32}


def _code(t, what):
    c = _DTYPE.get(t.dtype)
    if c is None:
        raise TypeError(f"{what} must be bfloat16 or float32, got {t.dtype}")
    return c


def _want(t, what, shape, dtype, device):
    """A contiguous tensor of this shape, type and device; None passes."""
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, what, inner: int, width: int):
    """Distance in elements of consecutive rows of t, whose last `inner` axes (`width` elements)
    make up a row and are contiguous; 0 where the rows are contiguous."""
    if t.is_contiguous():
        return 0
    lead = t.dim() - inner
    step = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != step:
            raise ValueError(f"{what}: the last {inner} axes must be contiguous")
        step *= t.shape[i]
    stride, dist = 0, None
    for i in range(lead - 1, -1, -1):   # the leading axes, innermost first, walk one row at a time
        if t.shape[i] == 1:
            continue
        if dist is None:
            stride, dist = t.stride(i), t.stride(i)
        elif t.stride(i) != dist:
            raise ValueError(f"{what}: rows must lie at one common distance")
        dist *= t.shape[i]
    if dist is None:
        return 0
    if t.numel() and stride < width:
        raise ValueError(f"{what}: rows overlap (broadcast tensors are not taken)")
    return stride


def _strided(t, what, shape, dtype, device, inner, width):
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _rows(t, what, inner, width)


def _cuda(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: libkda takes device tensors (copy host data to the GPU first)")
    return t.device


def _batch(x, cu, device, step=False):
    """(B, T, num_seqs) of x [B, T, ..] (or [B, ..] for one row per sequence)."""
    B, T = (x.shape[0], 1) if step else (x.shape[0], x.shape[1])
    if cu is None:
        return B, T, B
    if cu.device != device or cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 1 or not cu.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 tensor [num_seqs + 1] on the inputs' device")
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) come as one batch row")
    return B, T, cu.numel() - 1


def _status_ptr(t, device):
    if t is None:
        return None
    if t.device != device or t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on the inputs' device")
    return t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(ws, nbytes, device):
    """(tensor kept alive, pointer, bytes): True allocates with torch, None / False leaves it to the library."""
    if ws is True:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    elif ws is False or ws is None:
        ws = None
    else:
        if ws.device != device or not ws.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return (None, None, 0) if ws is None else (ws, ws.data_ptr(), ws.numel() * ws.element_size())


_NULL = contextlib.nullcontext()
# The current stream's handle without building a torch.cuda.Stream object (a microsecond of the
# few that a small call takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device):
    """The device of the tensors as the current one, for the launch."""
    return _NULL if _current() == device.index else torch.cuda.device(device)


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _out(given, what, shape, dtype, device, like=None):
    """(tensor, pointer): the caller's buffer, checked, or a new one (`like`: a tensor of its type and device)."""
    if given is None:
        t = torch.empty(shape, dtype=dtype, device=device) if like is None else like.new_empty(shape)
        return t, t.data_ptr()
    return given, _want(given, what, shape, dtype, device)


def _grads(given, **computed):
    """The caller's gradient buffers by name; `computed` tells of every gradient whether the call writes it."""
    given = given or {}
    if unknown := set(given) - set(computed):
        raise ValueError(f"unknown gradients {sorted(unknown)}: expected some of {tuple(computed)}")
    if idle := sorted(k for k, v in given.items() if v is not None and not computed[k]):
        raise ValueError(f"buffers for gradients that this call does not compute: {idle} (their input is None, or they are not wanted)")
    return given


def _check(st, name):
    if st != 0:
        raise _b.KDAError(st, name)


# ------------------------------------------------------------------ short causal convolution


def _conv_common(x, weight, bias, device, step):
    lead = 2 if step else 3
    if x.dim() != lead:
        raise ValueError(f"x must have {lead} axes, got {x.dim()}")
    D = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be [{D}, width], got {tuple(weight.shape)}")
    W = weight.shape[1]
    w = _want(weight, "weight", weight.shape, torch.float32, device)
    b = _want(bias, "bias", (D,), torch.float32, device)
    xs = _strided(x, "x", x.shape, x.dtype, device, 1, D)
    return D, W, w, b, xs


def kda_conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, silu: bool = True, out=None, final_state=None,
                 want_state: bool = True, dev_status=None, lib=None):
    """Short causal depthwise convolution (kda_conv_fwd of include/kda.h).

    x [B,T,D] (bf16 or fp32, row-strided); weight [D,W] and bias [D] fp32, W from 2 to 8;
    state [N,W-1,D] of x's dtype or None (the inputs before each sequence, oldest first);
    cu_seqlens int32 [N+1] with B == 1 for packed sequences.  Returns (out [B,T,D],
    final_state [N,W-1,D]); final_state is None when want_state is False and no buffer is given.
    """
    dev = _cuda(x, "x")
    D, W, w, b, xs = _conv_common(x, weight, bias, dev, False)
    B, T, N = _batch(x, cu_seqlens, dev)
    st = (N, max(W - 1, 0), D)
    sp = _want(state, "state", st, x.dtype, dev)
    out, op = _out(out, "out", x.shape, x.dtype, dev, x)
    fp = None
    if final_state is not None or want_state:
        final_state, fp = _out(final_state, "final_state", st, x.dtype, dev, x)
    sh = _shape(ConvShape, B, T, D, N, W, _code(x, "x"), 0, int(bool(silu)), xs, _status_ptr(dev_status, dev))
    lib = lib or _b.load_library()
    with _on(dev):
        _check(lib.kda_conv_fwd(sh, x.data_ptr(), w, b, sp, _ptr(cu_seqlens), op, fp, _stream(dev)),
               "kda_conv_fwd")
    return out, final_state


def kda_conv_step(x, weight, state, bias=None, silu: bool = True, out=None, lib=None):
    """One row of the convolution per sequence (kda_conv_step of include/kda.h).

    x [N,D] (row-strided); state [N,W-1,D] of x's dtype, shifted by x in place.  Returns out [N,D].
    """
    dev = _cuda(x, "x")
    D, W, w, b, xs = _conv_common(x, weight, bias, dev, True)
    N = x.shape[0]
    if state is None:
        raise ValueError("state is required")
    sp = _want(state, "state", (N, max(W - 1, 0), D), x.dtype, dev)
    out, op = _out(out, "out", x.shape, x.dtype, dev, x)
    sh = _shape(ConvShape, N, 1, D, N, W, _code(x, "x"), 0, int(bool(silu)), xs, None)
    lib = lib or _b.load_library()
    with _on(dev):
        _check(lib.kda_conv_step(sh, x.data_ptr(), w, b, sp, op, _stream(dev)), "kda_conv_step")
    return out


def kda_conv_bwd(x, weight, d_out, bias=None, state=None, d_final_state=None, cu_seqlens=None, silu: bool = True,
                 want_dstate: bool = True, grads=None, dev_status=None, workspace=True, lib=None):
    """Gradients of kda_conv_fwd (kda_conv_bwd of include/kda.h).

    d_out [B,T,D] of x's dtype or fp32 (such as the dq, dk, dv of kda_chunk_bwd);
    d_final_state [N,W-1,D] of x's dtype or None.  Returns a dict of dx [B,T,D] (x's dtype),
    dweight [D,W], dbias [D] (fp32; None without a bias) and dstate [N,W-1,D] (x's dtype; None
    unless want_dstate) for the loss sum(out * d_out) + sum(final_state * d_final_state).
    grads: a dict of buffers to write instead of new ones, by the same names.
    workspace: as kda_chunk_fwd.
    """
    dev = _cuda(x, "x")
    D, W, w, b, xs = _conv_common(x, weight, bias, dev, False)
    B, T, N = _batch(x, cu_seqlens, dev)
    grads = _grads(grads, dx=True, dweight=True, dbias=bias is not None, dstate=want_dstate)
    st = (N, max(W - 1, 0), D)
    sp = _want(state, "state", st, x.dtype, dev)
    dsp = _want(d_final_state, "d_final_state", st, x.dtype, dev)
    if d_out.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"d_out must be {x.dtype} or float32, got {d_out.dtype}")
    dp = _want(d_out, "d_out", x.shape, d_out.dtype, dev)
    dx, dxp = _out(grads.get("dx"), "dx", x.shape, x.dtype, dev, x)
    dw, dwp = _out(grads.get("dweight"), "dweight", weight.shape, torch.float32, dev, weight)
    db = dbp = dst = dstp = None
    if bias is not None:
        db, dbp = _out(grads.get("dbias"), "dbias", (D,), torch.float32, dev, weight)
    if want_dstate:
        dst, dstp = _out(grads.get("dstate"), "dstate", st, x.dtype, dev, x)
    sh = _shape(ConvShape, B, T, D, N, W, _code(x, "x"), _code(d_out, "d_out"), int(bool(silu)), xs, _status_ptr(dev_status, dev))
    lib = lib or _b.load_library()
    with _on(dev):
        ws, wp, wn = _workspace(workspace, lib.kda_conv_bwd_workspace_size(sh) if workspace is True else 0, dev)
        _check(lib.kda_conv_bwd(sh, x.data_ptr(), w, b, sp, _ptr(cu_seqlens), dp, dsp, dxp, dwp, dbp, dstp,
                                wp, wn, _stream(dev)), "kda_conv_bwd")
    return dict(dx=dx, dweight=dw, dbias=db, dstate=dst)


# ------------------------------------------------------------------ selective state space scan


def _ssm_common(x, dt, A, Bm, Cm, D, z, dt_bias, device, step):
    lead = 2 if step else 3
    if x.dim() != lead:
        raise ValueError(f"x must have {lead} axes, got {x.dim()}")
    Dc = x.shape[-1]
    if A.dim() != 2 or A.shape[0] != Dc:
        raise ValueError(f"A must be [{Dc}, states], got {tuple(A.shape)}")
    N = A.shape[1]
    if Bm.dim() == lead:   # one group without its axis
        G, inner = 1, 1
        bshape = (*x.shape[:-1], N)
    else:
        if Bm.dim() != lead + 1:
            raise ValueError(f"B must be [.., groups, {N}] or [.., {N}]")
        G, inner = Bm.shape[-2], 2
        bshape = (*x.shape[:-1], G, N)
    if G <= 0 or Dc % G != 0:
        raise ValueError(f"the groups of B and C ({G}) must divide the channels ({Dc})")
    strides = [_strided(x, "x", x.shape, x.dtype, device, 1, Dc), _strided(dt, "dt", x.shape, x.dtype, device, 1, Dc),
               0 if z is None else _strided(z, "z", x.shape, x.dtype, device, 1, Dc),
               _strided(Bm, "B", bshape, x.dtype, device, inner, G * N),
               _strided(Cm, "C", bshape, x.dtype, device, inner, G * N)]
    ptrs = [x.data_ptr(), dt.data_ptr(), _want(A, "A", A.shape, torch.float32, device), Bm.data_ptr(), Cm.data_ptr(),
            _want(D, "D", (Dc,), torch.float32, device), _ptr(z), _want(dt_bias, "dt_bias", (Dc,), torch.float32, device)]
    return Dc, N, G, strides, ptrs


def kda_ssm_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, softplus: bool = True, out=None,
                hT=None, want_state: bool = True, dev_status=None, workspace=True, lib=None):
    """Selective state space scan (kda_ssm_fwd of include/kda.h).

    x, dt, z [b,T,D] and B, C [b,T,G,N] (or [b,T,N]) of one dtype (bf16 or fp32; all row-strided);
    A [D,N], the skip D [D] and dt_bias [D] fp32; h0 [n,D,N] fp32 or None; cu_seqlens int32 [n+1]
    with b == 1 for packed sequences.  N from 1 to 128.  Returns (out [b,T,D], hT [n,D,N]); hT is
    None when want_state is False and no buffer is given.  workspace: as kda_chunk_fwd.
    """
    dev = _cuda(x, "x")
    Dc, N, G, st, p = _ssm_common(x, dt, A, B, C, D, z, dt_bias, dev, False)
    b, T, n = _batch(x, cu_seqlens, dev)
    hp = _want(h0, "h0", (n, Dc, N), torch.float32, dev)
    out, op = _out(out, "out", x.shape, x.dtype, dev, x)
    tp = None
    if hT is not None or want_state:
        hT, tp = _out(hT, "hT", (n, Dc, N), torch.float32, dev, A)
    sh = _shape(SsmShape, b, T, Dc, N, G, n, _code(x, "x"), int(bool(softplus)), *st, _status_ptr(dev_status, dev))
    lib = lib or _b.load_library()
    with _on(dev):
        need = lib.kda_ssm_fwd_workspace_size(sh, int(cu_seqlens is not None)) if workspace is True else 0
        ws, wp, wn = _workspace(workspace, need, dev)
        _check(lib.kda_ssm_fwd(sh, *p, hp, _ptr(cu_seqlens), op, tp, wp, wn, _stream(dev)), "kda_ssm_fwd")
    return out, hT


def kda_ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, softplus: bool = True, out=None, lib=None):
    """One row of the scan per sequence (kda_ssm_step of include/kda.h).

    x, dt, z [n,D]; B, C [n,G,N] (or [n,N]); h [n,D,N] fp32, updated in place.  Returns out [n,D].
    """
    dev = _cuda(x, "x")
    Dc, N, G, st, p = _ssm_common(x, dt, A, B, C, D, z, dt_bias, dev, True)
    n = x.shape[0]
    if h is None:
        raise ValueError("h is required")
    hp = _want(h, "h", (n, Dc, N), torch.float32, dev)
    out, op = _out(out, "out", x.shape, x.dtype, dev, x)
    sh = _shape(SsmShape, n, 1, Dc, N, G, n, _code(x, "x"), int(bool(softplus)), *st, None)
    lib = lib or _b.load_library()
    with _on(dev):
        _check(lib.kda_ssm_step(sh, *p, hp, op, _stream(dev)), "kda_ssm_step")
    return out


def kda_ssm_bwd(x, dt, A, B, C, d_out, D=None, z=None, dt_bias=None, h0=None, d_hT=None, cu_seqlens=None,
                softplus: bool = True, want_dh0: bool = True, grads=None, dev_status=None, workspace=True, lib=None):
    """Gradients of kda_ssm_fwd (kda_ssm_bwd of include/kda.h).

    Inputs as kda_ssm_fwd, with d_out [b,T,D] of x's dtype and d_hT [n,D,N] fp32 or None.  Returns
    a dict of dx, ddt, dz [b,T,D], dB, dC (shape of B) of x's dtype, and fp32 dA [D,N], dD [D],
    ddt_bias [D], dh0 [n,D,N]; dz, dD and ddt_bias are None where their input is, dh0 unless
    want_dh0, for the loss sum(out * d_out) + sum(hT * d_hT).  grads: a dict of buffers to write
    instead of new ones, by the same names.  workspace: as kda_chunk_fwd.
    """
    dev = _cuda(x, "x")
    Dc, N, G, st, p = _ssm_common(x, dt, A, B, C, D, z, dt_bias, dev, False)
    b, T, n = _batch(x, cu_seqlens, dev)
    grads = _grads(grads, dx=True, ddt=True, dA=True, dB=True, dC=True, dD=D is not None, dz=z is not None,
                   ddt_bias=dt_bias is not None, dh0=want_dh0)
    hp = _want(h0, "h0", (n, Dc, N), torch.float32, dev)
    dtp = _want(d_hT, "d_hT", (n, Dc, N), torch.float32, dev)
    dop = _want(d_out, "d_out", x.shape, x.dtype, dev)
    f32, like = torch.float32, x.dtype
    r, q = {}, {}
    for name, shape, dtype, on in (("dx", x.shape, like, True), ("ddt", x.shape, like, True), ("dA", A.shape, f32, True),
                                   ("dB", B.shape, like, True), ("dC", B.shape, like, True), ("dD", (Dc,), f32, D is not None),
                                   ("dz", x.shape, like, z is not None), ("ddt_bias", (Dc,), f32, dt_bias is not None),
                                   ("dh0", (n, Dc, N), f32, want_dh0)):
        r[name], q[name] = _out(grads.get(name), name, shape, dtype, dev, A if dtype is f32 and like is not f32 else x) if on else (None, None)
    sh = _shape(SsmShape, b, T, Dc, N, G, n, _code(x, "x"), int(bool(softplus)), *st, _status_ptr(dev_status, dev))
    lib = lib or _b.load_library()
    with _on(dev):
        need = lib.kda_ssm_bwd_workspace_size(sh, int(cu_seqlens is not None)) if workspace is True else 0
        ws, wp, wn = _workspace(workspace, need, dev)
        _check(lib.kda_ssm_bwd(sh, *p, hp, _ptr(cu_seqlens), dop, dtp, q["dx"], q["ddt"], q["dA"], q["dB"],
                               q["dC"], q["dD"], q["dz"], q["ddt_bias"], q["dh0"], wp, wn, _stream(dev)), "kda_ssm_bwd")
    return r


# ------------------------------------------------------------------ layer norm


def _norm_common(x, weight, bias, device):
    """(rows, groups, D, row stride): weight [D] norms x [.., D], weight [G, D] norms x [.., G, D]."""
    if x.dim() < 1:
        raise ValueError("x needs at least one axis")
    D = x.shape[-1]
    par = weight if weight is not None else bias
    G, inner = 1, 1
    if par is not None and par.dim() == 2:
        G, inner = par.shape[0], 2
        if x.dim() < 2 or x.shape[-2] != G:
            raise ValueError(f"weights of {G} groups need x [.., {G}, {D}], got {tuple(x.shape)}")
    pshape = (D,) if inner == 1 else (G, D)
    w = _want(weight, "weight", pshape, torch.float32, device)
    b = _want(bias, "bias", pshape, torch.float32, device)
    rows = x.numel() // (G * D) if G * D else 0
    return rows, G, D, pshape, inner, w, b


def kda_layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, out=None, want_stats: bool = True, lib=None):
    """Layer norm over the last axis (kda_layer_norm_fwd of include/kda.h).

    x [.., D] (bf16 or fp32, row-strided) with weight, bias [D] fp32, or x [.., G, D] with weight,
    bias [G, D] (such as the out [B,T,H,d_v] of kda_chunk_fwd with weights per head); each may be
    None.  Returns (out, mean, rstd): out as x, contiguous; mean and rstd fp32 [..] (without the
    last axis), or None unless want_stats.
    """
    dev = _cuda(x, "x")
    rows, G, D, _, inner, w, b = _norm_common(x, weight, bias, dev)
    xs = _strided(x, "x", x.shape, x.dtype, dev, inner, G * D)
    out, op = _out(out, "out", x.shape, x.dtype, dev, x)
    mean = rstd = mp = rp = None
    if want_stats:
        shape = (2, *x.shape[:-1])
        f32 = x if x.dtype == torch.float32 else weight
        mean, rstd = (torch.empty(shape, dtype=torch.float32, device=dev) if f32 is None else f32.new_empty(shape)).unbind(0)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    sh = _shape(NormShape, rows, G, D, _code(x, "x"), float(eps), xs)
    lib = lib or _b.load_library()
    with _on(dev):
        _check(lib.kda_layer_norm_fwd(sh, x.data_ptr(), w, b, op, mp, rp, _stream(dev)), "kda_layer_norm_fwd")
    return out, mean, rstd


def kda_layer_norm_bwd(d_out, x, mean, rstd, weight=None, want_params: bool = True, groups: int | None = None, grads=None,
                       workspace=True, lib=None):
    """Gradients of kda_layer_norm_fwd (kda_layer_norm_bwd of include/kda.h).

    d_out as x (contiguous), mean and rstd from the forward.  Returns a dict of dx (as x,
    contiguous), dweight and dbias (fp32, shape of weight; None unless want_params) for the loss
    sum(out * d_out).  groups: without a weight, the number of groups (x [.., G, D]) whose
    parameter gradients are kept apart; the gradients are then [G, D].  grads: a dict of
    buffers to write instead of new ones, by the same names.  workspace: as kda_chunk_fwd.
    """
    dev = _cuda(x, "x")
    rows, G, D, pshape, inner, w, _ = _norm_common(x, weight, None, dev)
    if weight is None and groups is not None:
        if groups < 1 or x.dim() < 2 or x.shape[-2] != groups:
            raise ValueError(f"{groups} groups need x [.., {groups}, {D}], got {tuple(x.shape)}")
        G, inner, pshape = groups, 2, (groups, D)
        rows = x.numel() // (G * D) if G * D else 0
    xs = _strided(x, "x", x.shape, x.dtype, dev, inner, G * D)
    grads = _grads(grads, dx=True, dweight=want_params, dbias=want_params)
    dp = _want(d_out, "d_out", x.shape, x.dtype, dev)
    mp = _want(mean, "mean", x.shape[:-1], torch.float32, dev)
    rp = _want(rstd, "rstd", x.shape[:-1], torch.float32, dev)
    dx, dxp = _out(grads.get("dx"), "dx", x.shape, x.dtype, dev, x)
    dw = dwp = db = dbp = None
    if want_params:
        dw, dwp = _out(grads.get("dweight"), "dweight", pshape, torch.float32, dev)
        db, dbp = _out(grads.get("dbias"), "dbias", pshape, torch.float32, dev)
    sh = _shape(NormShape, rows, G, D, _code(x, "x"), 0.0, xs)
    lib = lib or _b.load_library()
    with _on(dev):
        need = lib.kda_layer_norm_bwd_workspace_size(sh) if workspace is True and want_params else 0
        ws, wp, wn = _workspace(workspace, need, dev)
        _check(lib.kda_layer_norm_bwd(sh, dp, x.data_ptr(), w, mp, rp, dxp, dwp, dbp, wp, wn, _stream(dev)),
               "kda_layer_norm_bwd")
    return dict(dx=dx, dweight=dw, dbias=db)
