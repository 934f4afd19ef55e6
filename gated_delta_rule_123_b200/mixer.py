"""The parts of a selective state-space mixer: layer norm, a projection with a bias, an activation and a
residual, the short causal convolution and the selective scan -- thin bindings like the rest of the package.

Every function checks shapes, types, strides and devices, allocates its outputs, and makes one call of
``include/kda.h`` on the tensors' device and its current stream."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _check, _lib, KDA_BF16, KDA_FP32

_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "softplus": 4}


class ScanParams(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("channels", ctypes.c_int), ("groups", ctypes.c_int), ("state", ctypes.c_int),
                ("dt_softplus", ctypes.c_int)]


def _declare():
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    sp = ctypes.POINTER(ScanParams)
    for name, args in {
        "kda_layer_norm_fwd": [vp, ll, vp, vp, vp, ll, vp, vp, i, i, i, f, vp],
        "kda_layer_norm_bwd": [vp, ll, vp, ll, vp, vp, vp, vp, ll, vp, vp, i, i, i, vp, sz, vp],
        "kda_linear_act_bf16": [vp, i, vp, i, vp, vp, i, vp, i, vp, i, i, i, i, i, vp],
        "kda_linear_act_bwd_bf16": [vp, i, vp, i, vp, i, vp, i, vp, i, vp, i, vp, i, i, i, i, vp, sz, vp],
        "kda_short_conv_fwd": [vp, ll, vp, vp, vp, ll, vp, vp, vp, i, i, i, i, i, i, i, vp],
        "kda_short_conv_bwd": [vp, ll, vp, ll, vp, vp, vp, vp, vp, ll, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp],
        "kda_short_conv_step": [vp, ll, vp, vp, vp, vp, ll, i, i, i, i, i, vp],
        "kda_selective_scan_fwd": [vp, ll, vp, ll, vp, ll, vp, ll, vp, ll, sp, vp, vp, vp, ll, vp, i, i, i, i, vp, sz, vp],
        "kda_selective_scan_bwd": [vp, ll, vp, ll, vp, ll, vp, ll, vp, ll, vp, ll, sp, vp, vp, vp, ll, vp, ll, vp, ll,
                                   vp, ll, vp, ll, vp, vp, vp, vp, vp, i, i, i, i, vp, sz, vp],
        "kda_selective_scan_step": [vp, ll, vp, ll, vp, ll, vp, ll, vp, ll, sp, vp, vp, ll, i, i, vp],
    }.items():
        getattr(_lib, name).argtypes = args
        getattr(_lib, name).restype = i
    for name, n in (("kda_layer_norm_bwd_workspace", 2), ("kda_linear_act_bwd_workspace", 2),
                    ("kda_short_conv_bwd_workspace", 3), ("kda_selective_scan_fwd_workspace", 6),
                    ("kda_selective_scan_bwd_workspace", 6)):
        getattr(_lib, name).argtypes = [i] * n
        getattr(_lib, name).restype = sz


_declare()


_device_now = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_stream_of = (torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream")
              else lambda index: torch.cuda.current_stream(index).cuda_stream)


def _p(t):
    return None if t is None else t.data_ptr()


def _run(device, name, *args):
    """One library call with the tensors' device current, on that device's current stream."""
    index = device.index
    if index == _device_now():
        rc = getattr(_lib, name)(*args, _stream_of(index))
    else:
        with torch.cuda.device(device):
            rc = getattr(_lib, name)(*args, _stream_of(index))
    if rc:
        _check(rc, name)


@functools.lru_cache(maxsize=4096)
def _query(device, name, *args):
    """A workspace size for that device (a function of the sizes alone)."""
    if device.index == _device_now():
        return getattr(_lib, name)(*args)
    with torch.cuda.device(device):
        return getattr(_lib, name)(*args)


def _first(t, what, dtypes=(torch.bfloat16, torch.float32)):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    return t.device


def _like(t, what, shape, dtype, device):
    """Check an operand against what the first one fixes; None passes."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    return t


def _whole(t, what, shape, dtype, device):
    """An operand without a stride of its own: contiguous."""
    if _like(t, what, shape, dtype, device) is not None and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _ld(t, what, inner=1):
    """Row stride of a tensor whose last ``inner`` axes are contiguous and whose leading axes form one axis of rows."""
    shape = t.shape
    want = shape[-1] if inner == 1 else shape[-1] * shape[-2]
    numel = t.numel()
    if numel <= want:  # no rows to step over: any stride does
        _ld_inner(t, what, inner)
        return (want + 7) // 8 * 8
    if t.is_contiguous():
        return want
    _ld_inner(t, what, inner)
    stride, ld, rows = t.stride(), None, 1
    for k in range(len(shape) - inner - 1, -1, -1):
        if shape[k] == 1:
            continue
        if ld is None:
            ld, rows = stride[k], shape[k]
        elif stride[k] != ld * rows:
            raise ValueError(f"{what}: rows of the leading axes must be evenly spaced")
        else:
            rows *= shape[k]
    if ld < want:
        raise ValueError(f"{what}: rows must not overlap")
    return ld


def _ld_inner(t, what, inner):
    shape, stride, step = t.shape, t.stride(), 1
    for k in range(1, inner + 1):
        if shape[-k] > 1 and stride[-k] != step:
            raise ValueError(f"{what}: the last {inner} axes must be contiguous")
        step *= shape[-k]


def _sizes(*values):
    """Refuse what the library's int arguments cannot hold (a conversion would cut it off)."""
    if max(values) > 0x7fffffff:
        raise ValueError("sizes and the projection's row strides must be below 2^31")


def _ld32(t, what):
    """Row stride for the projection, whose strides are ints; 0 without a tensor."""
    if t is None:
        return 0
    ld = _ld(t, what)
    if ld > 0x7fffffff:
        _sizes(ld)
    return ld


def _scratch(workspace, need, device):
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {device}")
        return workspace, workspace.numel() * workspace.element_size()
    return (None, 0) if need == 0 else (torch.empty(need, device=device, dtype=torch.uint8), need)


def _seqs(cu_seqlens, B, device):
    _sizes(B if cu_seqlens is None else cu_seqlens.numel())
    if cu_seqlens is None:
        return 0, B
    if B != 1:
        raise ValueError("packed input (cu_seqlens) must have a leading axis of 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    _whole(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, device)
    return cu_seqlens.numel() - 1, cu_seqlens.numel() - 1


def _new(like):
    """An output of that shape and type, contiguous."""
    return torch.empty_like(like, memory_format=torch.contiguous_format)


# ---------------------------------------------------------------- layer norm
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None):
    """Layer norm over the last axis (``kda_layer_norm_fwd``).  x [..., N] bf16 or fp32; weight, bias fp32 [N] or None.

    Returns (y, mean, rstd); mean and rstd fp32 of x's leading shape, as layer_norm_bwd takes them."""
    dev = _first(x, "x")
    N, lead = x.shape[-1], x.shape[:-1]
    _whole(weight, "weight", (N,), torch.float32, dev)
    _whole(bias, "bias", (N,), torch.float32, dev)
    y = _new(x) if out is None else _like(out, "out", x.shape, x.dtype, dev)
    mean = torch.empty(lead, device=dev, dtype=torch.float32)
    rstd = torch.empty_like(mean)
    M = mean.numel()
    _sizes(M, N)
    _run(dev, "kda_layer_norm_fwd", _p(x), _ld(x, "x"), _p(weight), _p(bias), _p(y), _ld(y, "out"), _p(mean), _p(rstd), M,
         N, _CODE[x.dtype], float(eps))
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, weight_grad=True, bias_grad=True, workspace=None):
    """Gradients of layer_norm_fwd (``kda_layer_norm_bwd``).  Returns (dx, dweight, dbias): dx of x's dtype, the others
    fp32 [N], or None where not asked for."""
    dev = _first(x, "x")
    N, lead = x.shape[-1], x.shape[:-1]
    _like(dy, "dy", x.shape, x.dtype, dev)
    _whole(weight, "weight", (N,), torch.float32, dev)
    _whole(mean, "mean", lead, torch.float32, dev)
    _whole(rstd, "rstd", lead, torch.float32, dev)
    M = mean.numel()
    _sizes(M, N)
    dx = _new(x)
    dw = torch.empty(N, device=dev, dtype=torch.float32) if weight_grad else None
    db = torch.empty(N, device=dev, dtype=torch.float32) if bias_grad else None
    ws, n = _scratch(workspace, _query(dev, "kda_layer_norm_bwd_workspace", M, N), dev)
    _run(dev, "kda_layer_norm_bwd", _p(dy), _ld(dy, "dy"), _p(x), _ld(x, "x"), _p(weight), _p(mean), _p(rstd), _p(dx), N,
         _p(dw), _p(db), M, N, _CODE[x.dtype], _p(ws), n)
    return dx, dw, db


# ---------------------------------------------------------------- projection
def _padded(M, N, dev):
    """[M, N] bf16 with a row stride of a multiple of 8 elements."""
    n8 = (N + 7) // 8 * 8
    t = torch.empty((M, n8), device=dev, dtype=torch.bfloat16)
    return t if n8 == N else t[:, :N]


def linear_act(x, W, bias=None, residual=None, act="none", output_pre=False, out=None):
    """act(x W^T + bias) + residual (``kda_linear_act_bf16``).  x [M, K], W [N, K], residual [M, N] bf16, bias fp32 [N];
    act one of "none", "relu", "gelu", "silu", "softplus".

    Returns y [M, N] bf16, or (y, pre) with output_pre: the value before the activation, for linear_act_bwd.  Both have
    a row stride padded to 8 elements when N is not a multiple of 8."""
    dev = _first(x, "x", (torch.bfloat16,))
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x [M, K] and W [N, K] must have two axes")
    (M, K), N = x.shape, W.shape[0]
    _sizes(M, N, K)
    _like(W, "W", (N, K), torch.bfloat16, dev)
    _whole(bias, "bias", (N,), torch.float32, dev)
    _like(residual, "residual", (M, N), torch.bfloat16, dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    y = _padded(M, N, dev) if out is None else _like(out, "out", (M, N), torch.bfloat16, dev)
    pre = _padded(M, N, dev) if output_pre else None
    _run(dev, "kda_linear_act_bf16", _p(x), _ld32(x, "x"), _p(W), _ld32(W, "W"), _p(bias), _p(residual),
         _ld32(residual, "residual"), _p(y), _ld32(y, "out"), _p(pre),
         0 if pre is None else pre.stride(0), M, N, K, ACTIVATIONS[act])
    return (y, pre) if output_pre else y


def linear_act_bwd(dy, x, W, pre=None, act="none", bias_grad=True, workspace=None):
    """Gradients of linear_act (``kda_linear_act_bwd_bf16``); the residual's is dy.  pre (needed unless act is "none") is
    what linear_act kept.  Returns (dx, dW, dbias): bf16 [M, K], bf16 [N, K], fp32 [N] or None."""
    dev = _first(x, "x", (torch.bfloat16,))
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x [M, K] and W [N, K] must have two axes")
    (M, K), N = x.shape, W.shape[0]
    _sizes(M, N, K)
    _like(W, "W", (N, K), torch.bfloat16, dev)
    _like(dy, "dy", (M, N), torch.bfloat16, dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    if act != "none" and pre is None:
        raise ValueError("pre is required with an activation")
    _like(pre, "pre", (M, N), torch.bfloat16, dev)
    lddy, ldx, ldw, ldp = _ld32(dy, "dy"), _ld32(x, "x"), _ld32(W, "W"), _ld32(pre, "pre")
    dx, dW = _padded(M, K, dev), _padded(N, K, dev)
    db = torch.empty(N, device=dev, dtype=torch.float32) if bias_grad else None
    ws, n = _scratch(workspace, _query(dev, "kda_linear_act_bwd_workspace", M, N), dev)
    _run(dev, "kda_linear_act_bwd_bf16", _p(dy), lddy, _p(x), ldx, _p(W), ldw, _p(pre), ldp, _p(dx), dx.stride(0) if M else K, _p(dW), dW.stride(0) if N else K, _p(db),
         M, N, K, ACTIVATIONS[act], _p(ws), n)
    return dx, dW, db


# ---------------------------------------------------------------- short convolution
def _conv_operands(x, weight, bias, cu_seqlens, conv_state):
    dev = _first(x, "x")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x [B, T, C] must have three axes and weight [C, width] two")
    B, T, C = x.shape
    W = weight.shape[1]
    _sizes(B * T, C, W)
    _whole(weight, "weight", (C, W), x.dtype, dev)
    _whole(bias, "bias", (C,), torch.float32, dev)
    nseq, n = _seqs(cu_seqlens, B, dev)
    _whole(conv_state, "conv_state", (n, W - 1, C), x.dtype, dev)
    return dev, B, T, C, W, nseq, n


def short_conv_fwd(x, weight, bias=None, cu_seqlens=None, conv_state=None, silu=True, output_conv_state=False, out=None,
                   conv_state_out=None):
    """Short causal depthwise convolution (``kda_short_conv_fwd``).  x [B, T, C] or packed [1, Ttot, C], weight [C, width]
    of the same dtype, bias fp32 [C]; conv_state [N, width-1, C]: the inputs before each sequence (None: zeros).

    Returns (y, conv_state after the call or None)."""
    dev, B, T, C, W, nseq, n = _conv_operands(x, weight, bias, cu_seqlens, conv_state)
    y = _new(x) if out is None else _like(out, "out", x.shape, x.dtype, dev)
    cs = _whole(conv_state_out, "conv_state_out", (n, W - 1, C), x.dtype, dev)
    if cs is None and output_conv_state:
        cs = torch.empty((n, W - 1, C), device=dev, dtype=x.dtype)
    _run(dev, "kda_short_conv_fwd", _p(x), _ld(x, "x"), _p(weight), _p(bias), _p(y), _ld(y, "out"), _p(conv_state), _p(cs),
         _p(cu_seqlens), nseq, B, T, C, W, _CODE[x.dtype], int(silu))
    return y, cs


def short_conv_bwd(dy, x, weight, bias=None, cu_seqlens=None, conv_state=None, d_conv_state_out=None, silu=True,
                   workspace=None):
    """Gradients of short_conv_fwd (``kda_short_conv_bwd``).  Returns (dx, dweight, dbias, d_conv_state): dbias fp32 [C],
    d_conv_state None when conv_state is None."""
    dev, B, T, C, W, nseq, n = _conv_operands(x, weight, bias, cu_seqlens, conv_state)
    _like(dy, "dy", x.shape, x.dtype, dev)
    _whole(d_conv_state_out, "d_conv_state_out", (n, W - 1, C), x.dtype, dev)
    dx = _new(x)
    dw = torch.empty((C, W), device=dev, dtype=x.dtype)
    db = torch.empty(C, device=dev, dtype=torch.float32)
    dc = torch.empty((n, W - 1, C), device=dev, dtype=x.dtype) if conv_state is not None else None
    ws, size = _scratch(workspace, _query(dev, "kda_short_conv_bwd_workspace", B * T, C, W), dev)
    _run(dev, "kda_short_conv_bwd", _p(dy), _ld(dy, "dy"), _p(x), _ld(x, "x"), _p(weight), _p(bias), _p(conv_state),
         _p(d_conv_state_out), _p(dx), C, _p(dw), _p(db), _p(dc), _p(cu_seqlens), nseq, B, T, C, W, _CODE[x.dtype],
         int(silu), _p(ws), size)
    return dx, dw, db, dc


def short_conv_step(x, weight, conv_state, bias=None, silu=True, out=None):
    """One token for each of B sequences (``kda_short_conv_step``).  x [B, C]; conv_state [B, width-1, C] is updated in
    place.  Returns y [B, C]."""
    dev = _first(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x [B, C] and weight [C, width] must have two axes")
    B, C = x.shape
    W = weight.shape[1]
    _sizes(B, C, W)
    _whole(weight, "weight", (C, W), x.dtype, dev)
    _whole(bias, "bias", (C,), torch.float32, dev)
    _whole(conv_state, "conv_state", (B, W - 1, C), x.dtype, dev)
    y = _new(x) if out is None else _like(out, "out", x.shape, x.dtype, dev)
    _run(dev, "kda_short_conv_step", _p(x), _ld(x, "x"), _p(weight), _p(bias), _p(conv_state), _p(y), _ld(y, "out"), B, C, W,
         _CODE[x.dtype], int(silu))
    return y


# ---------------------------------------------------------------- selective scan
def _scan_operands(u, dt, A, B, C, D, z, dt_bias, dt_softplus):
    dev = _first(u, "u")
    if A.dim() != 2 or B.dim() != u.dim() + 1:
        raise ValueError("A must be [channels, state] and B [..., groups, state]")
    lead, ch = u.shape[:-1], u.shape[-1]
    G, N = B.shape[-2:]
    _sizes(math.prod(lead), ch, G, N)
    if G < 1 or ch % G:
        raise ValueError("channels must be a multiple of groups")
    _like(dt, "dt", u.shape, u.dtype, dev)
    _like(z, "z", u.shape, u.dtype, dev)
    _like(B, "B", (*lead, G, N), u.dtype, dev)
    _like(C, "C", (*lead, G, N), u.dtype, dev)
    _whole(A, "A", (ch, N), torch.float32, dev)
    _whole(D, "D", (ch,), torch.float32, dev)
    _whole(dt_bias, "dt_bias", (ch,), torch.float32, dev)
    params = ScanParams(_p(A), _p(D), _p(dt_bias), ch, G, N, int(dt_softplus))
    args = (_p(u), _ld(u, "u"), _p(dt), _ld(dt, "dt"), _p(B), _ld(B, "B", 2), _p(C), _ld(C, "C", 2), _p(z),
            0 if z is None else _ld(z, "z"), ctypes.byref(params))
    return dev, ch, G, N, params, args


def selective_scan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                       cu_seqlens=None, output_final_state=True, out=None, final_state=None, workspace=None):
    """Selective scan over whole sequences (``kda_selective_scan_fwd``).

    u, dt, z [B, T, channels] (or [1, Ttot, channels] with cu_seqlens); A fp32 [channels, state]; B, C [B, T, groups,
    state]; D, dt_bias fp32 [channels].  Returns (y, final_state or None); states fp32 [N, channels, state]."""
    if u.dim() != 3:
        raise ValueError("u [B, T, channels] must have three axes")
    dev, ch, G, N, params, args = _scan_operands(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    nb, T = u.shape[:2]
    nseq, n = _seqs(cu_seqlens, nb, dev)
    _whole(initial_state, "initial_state", (n, ch, N), torch.float32, dev)
    fs = _whole(final_state, "final_state", (n, ch, N), torch.float32, dev)
    if fs is None and output_final_state:
        fs = torch.empty((n, ch, N), device=dev, dtype=torch.float32)
    y = _new(u) if out is None else _like(out, "out", u.shape, u.dtype, dev)
    ws, size = _scratch(workspace, _query(dev, "kda_selective_scan_fwd_workspace", nb, T, ch, G, N, nseq), dev)
    _run(dev, "kda_selective_scan_fwd", *args, _p(initial_state), _p(fs), _p(y), _ld(y, "out"), _p(cu_seqlens), nseq, nb, T,
         _CODE[u.dtype], _p(ws), size)
    return y, fs


def selective_scan_bwd(dy, u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                       cu_seqlens=None, d_final_state=None, workspace=None):
    """Gradients of selective_scan_fwd (``kda_selective_scan_bwd``).

    Returns (du, ddt, dA, dB, dC, dD, dz, ddt_bias, d_initial_state); du, ddt, dB, dC, dz of u's dtype, the others fp32;
    dD, dz, ddt_bias and d_initial_state are None where D, z, dt_bias or initial_state is."""
    if u.dim() != 3:
        raise ValueError("u [B, T, channels] must have three axes")
    dev, ch, G, N, params, args = _scan_operands(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    nb, T = u.shape[:2]
    nseq, n = _seqs(cu_seqlens, nb, dev)
    _like(dy, "dy", u.shape, u.dtype, dev)
    _whole(initial_state, "initial_state", (n, ch, N), torch.float32, dev)
    _whole(d_final_state, "d_final_state", (n, ch, N), torch.float32, dev)
    du, ddt = (_new(u) for _ in range(2))
    dz = _new(u) if z is not None else None
    dB, dC = (_new(B) for _ in range(2))
    dA = torch.empty((ch, N), device=dev, dtype=torch.float32)
    dD = torch.empty(ch, device=dev, dtype=torch.float32) if D is not None else None
    db = torch.empty(ch, device=dev, dtype=torch.float32) if dt_bias is not None else None
    dh = torch.empty((n, ch, N), device=dev, dtype=torch.float32) if initial_state is not None else None
    ws, size = _scratch(workspace, _query(dev, "kda_selective_scan_bwd_workspace", nb, T, ch, G, N, nseq), dev)
    _run(dev, "kda_selective_scan_bwd", _p(dy), _ld(dy, "dy"), *args, _p(initial_state), _p(d_final_state), _p(du), ch,
         _p(ddt), ch, _p(dB), G * N, _p(dC), G * N, _p(dz), ch, _p(dA), _p(dD), _p(db), _p(dh), _p(cu_seqlens), nseq, nb,
         T, _CODE[u.dtype], _p(ws), size)
    return du, ddt, dA, dB, dC, dD, dz, db, dh


def selective_scan_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, out=None):
    """One token for each of B sequences (``kda_selective_scan_step``).  u, dt, z [B, channels]; B, C [B, groups, state];
    state [B, channels, state] fp32 is updated in place.  Returns y [B, channels]."""
    if u.dim() != 2:
        raise ValueError("u [B, channels] must have two axes")
    dev, ch, G, N, params, args = _scan_operands(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    _whole(state, "state", (u.shape[0], ch, N), torch.float32, dev)
    y = _new(u) if out is None else _like(out, "out", u.shape, u.dtype, dev)
    _run(dev, "kda_selective_scan_step", *args, _p(state), _p(y), _ld(y, "out"), u.shape[0], _CODE[u.dtype])
    return y
