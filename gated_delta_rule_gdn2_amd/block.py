"""The state space block's calls: scan, short convolution and layer norm.

    y, S_T = ssm_fwd(x, dt, B, C, A, D=None, dt_bias=None, initial_state=None)
    y, S_T = ssm_fwd_varlen(x, dt, B, C, A, cu_seqlens, D, dt_bias, initial_state)  # packed sequences
    y      = ssm_step(x, dt, B, C, A, state, D, dt_bias)        # state updated in place
    y, kept = short_conv(x, taps, bias=None, initial_state=None)
    y, kept = short_conv_varlen(x, taps, cu_seqlens, bias, initial_state)
    y      = short_conv_step(x, taps, state, bias)              # state updated in place
    y, mean, rstd = layer_norm(x, gamma, beta=None, eps=1e-5)
    grads  = layer_norm_bwd(dy, x, gamma, mean, rstd)           # dx, dgamma, dbeta

Layouts: x, y [B,T,H,dv]; dt [B,T,H]; B, C [B,T,G,dk]; A, D, dt_bias [H] fp32; states
[B,H,dk,dv] fp32 (packed: [total_T,...] for [B,T,...] and [N,H,dk,dv]; step: [N,...]).
Convolution: x, y [B,T,C], taps [C,4] and bias [C] fp32, the inputs kept [B,3,C] in x's dtype.
Norm: x, y [...,width], gamma, beta [width] and mean, rstd [...] fp32.  Everything else is bf16
or fp32, one dtype in a call.  x, dt, B and C may be parts of one wider tensor (a token stride of
their own, a token's elements contiguous); all other tensors are contiguous.  Addresses are 16-byte aligned
(dt's and the convolution's x to their elements), token strides of x, B and C whole 16-byte units in
the scan and its step, below 2^22 elements for prompts and 2^31 for steps; C of the convolution is a
multiple of 8.  The library's refusals of other calls are Gdn2Error.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPES, Gdn2Error, _check, _load, _ptr

__all__ = ["ssm_fwd", "ssm_fwd_varlen", "ssm_fwd_workspace_bytes", "ssm_fwd_varlen_workspace_bytes",
           "ssm_step", "short_conv", "short_conv_varlen",
           "short_conv_step", "layer_norm", "layer_norm_bwd", "layer_norm_bwd_workspace_bytes"]

_F32 = torch.float32


def _declare(lib):
    P, I64, I32, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, args, res in (
            ("ssm_fwd", [P] * 10 + [I64] * 10 + [I32, I32, P, SZ, P], I32),
            ("ssm_fwd_workspace_bytes", [I64] * 5 + [I32], SZ),
            ("ssm_fwd_varlen", [P] * 11 + [I64] * 10 + [I32, I32, P, SZ, P], I32),
            ("ssm_fwd_varlen_workspace_bytes", [I64] * 5 + [I32], SZ),
            ("ssm_step", [P] * 9 + [I64] * 9 + [I32, I32, P], I32),
            ("short_conv", [P] * 6 + [I64] * 4 + [I32, P], I32),
            ("short_conv_varlen", [P] * 7 + [I64] * 4 + [I32, P], I32),
            ("short_conv_step", [P] * 5 + [I64] * 3 + [I32, P], I32),
            ("layer_norm", [P] * 6 + [I64] * 2 + [F, I32, P], I32),
            ("layer_norm_bwd_workspace_bytes", [I64] * 2, SZ),
            ("layer_norm_bwd", [P] * 9 + [SZ] + [I64] * 2 + [I32, P], I32)):
        f = getattr(lib, "gdn2_" + name)
        f.argtypes, f.restype = args, res


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without a Stream object around it: 2 us less of the 5 that a small call's checks take
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(name, dev, *args):
    """The library call on dev's current stream, with dev the current device."""
    lib = _load()
    f = getattr(lib, name)
    if dev.index == torch.cuda.current_device():
        st = f(*args, _raw_stream(dev.index) if _raw_stream else _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _stream(dev))
    if st != 0:
        raise Gdn2Error(name, st, lib.gdn2_status_string(st).decode())


def _bytes(name, dev, *args):
    """A workspace's size as the library states it for dev."""
    f = getattr(_load(), name)
    if dev.index == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _on_gpu(fn, t, ndim, layout):
    """The dtype code and device of a call's first tensor, after its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError("x must be %s" % layout)
    if not t.is_cuda:
        raise ValueError("%s runs on the GPU; got tensors on %s" % (fn, t.device))
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("x dtype must be float32 or bfloat16")
    return code, t.device


def _tokens(name, t, shape, inner, dtype, dev):
    """Checks a token tensor whose last `inner` (1 or 2) dimensions are a token's own elements; returns
    the elements between tokens."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev):
        _check(name, t, shape, dtype, dev)  # says which
    own = shape[-1] if inner == 1 else shape[-1] * shape[-2]
    if t.is_contiguous():
        return own
    strides = t.stride()
    if len(shape) == inner + 1 and strides[-1] == 1 and (inner == 1 or strides[1] == shape[2]) and strides[0] >= own:
        return strides[0]  # the usual part of a wider tensor, one axis of tokens
    want, ok = 1, True
    for i in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        ok = ok and (shape[i] == 1 or strides[i] == want)
        want *= shape[i]
    stride = None
    for i in range(len(shape) - 1 - inner, -1, -1):  # the axes of tokens, the innermost first
        if shape[i] == 1:
            continue
        if stride is None:
            stride, want = strides[i], strides[i]
        ok = ok and strides[i] == want
        want *= shape[i]
    if stride is None:  # a single token
        stride = own
    if not ok or stride < own:
        raise ValueError("%s must have a token's elements contiguous and one stride between all tokens" % name)
    return stride


def _in(name, t, shape, dtype, dev):
    """The address of a contiguous tensor, after its checks."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous()):
        _check(name, t, shape, dtype, dev)  # says which
    return t.data_ptr()


def _opt(name, t, shape, dtype, dev):
    return None if t is None else _in(name, t, shape, dtype, dev)


def _out(name, t, shape, dtype, dev, like=None):
    """The caller's output after its checks, or a new one; `like`: a tensor of its shape and dtype, if
    there is one (a quicker way to a new one)."""
    if t is None:
        if like is None:
            return torch.empty(shape, dtype=dtype, device=dev)
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _check(name, t, shape, dtype, dev)
    return t


def _workspace(ws, need, align, dev):
    """(address, bytes) of the caller's workspace or of one made here, and its tensor."""
    if ws is None:
        ws = torch.empty(need + align, dtype=torch.uint8, device=dev)
    elif ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    off = -ws.data_ptr() % align
    if ws.numel() - off < need:
        raise ValueError("workspace holds %d bytes, %d needed" % (max(ws.numel() - off, 0), need))
    return ws.data_ptr() + off, need, ws


def _offsets(cu, dev):
    if cu.dim() != 1 or cu.numel() < 2:
        raise ValueError("cu_seqlens must be [N+1] with N >= 1")
    _check("cu_seqlens", cu, cu.shape, torch.int64, dev)
    return cu.numel() - 1


def _ssm_args(lead, x, dt, B, C, A, D, dt_bias, dev):
    """Sizes, strides and the seven input pointers of a scan."""
    H, dv = x.shape[-2:]
    if not isinstance(B, torch.Tensor) or B.dim() != len(lead) + 2:
        raise ValueError("B must be %s" % ("[B,T,G,dk]" if len(lead) == 2 else "[tokens,G,dk]"))
    G, dk = B.shape[-2:]
    t = x.dtype
    group = lead + (G, dk)
    xs = _tokens("x", x, x.shape, 2, t, dev)
    ds = _tokens("dt", dt, lead + (H,), 1, t, dev)
    bs = _tokens("B", B, group, 2, t, dev)
    cs = _tokens("C", C, group, 2, t, dev)
    ptrs = (x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), _in("A", A, (H,), _F32, dev), _opt("D", D, (H,), _F32, dev),
            _opt("dt_bias", dt_bias, (H,), _F32, dev))
    return (H, G, dk, dv), (xs, ds, bs, cs), ptrs


def ssm_fwd(x, dt, B, C, A, D=None, dt_bias=None, initial_state=None, *, y=None, final_state=None,
            output_final_state=True, softplus=True, workspace=None):
    """Selective state space scan of whole sequences.  Returns (y, S_T); S_T is None when
    ``output_final_state`` is False and no ``final_state`` is given (which may be
    ``initial_state`` itself).  Head h reads group h // (H // G) of B and C.  ``workspace``
    (uint8, at least ssm_fwd_workspace_bytes + 256) is allocated here unless passed."""
    code, dev = _on_gpu("ssm_fwd", x, 4, "[B,T,H,dv]")
    lead = tuple(x.shape[:2])
    (H, G, dk, dv), strides, ptrs = _ssm_args(lead, x, dt, B, C, A, D, dt_bias, dev)
    n, T = lead
    sshape = (n, H, dk, dv)
    s0 = _opt("initial_state", initial_state, sshape, _F32, dev)
    y = _out("y", y, lead + (H, dv), x.dtype, dev, x)
    if final_state is not None or output_final_state:
        final_state = _out("final_state", final_state, sshape, _F32, dev, initial_state)
    need = _bytes("gdn2_ssm_fwd_workspace_bytes", dev, n, T, H, dk, dv, code)
    ws, ws_bytes, keep = _workspace(workspace, need, 256, dev) if need else (None, 0, None)
    _launch("gdn2_ssm_fwd", dev, *ptrs, s0, y.data_ptr(), _ptr(final_state), n, T, H, G, dk, dv, *strides, code,
            int(softplus), ws, ws_bytes)
    return y, final_state


def ssm_fwd_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) with which ssm_fwd is fastest for these sizes (0: it takes none)."""
    return int(_load().gdn2_ssm_fwd_workspace_bytes(B, T, H, dk, dv, _DTYPES[dtype]))


def ssm_fwd_varlen_workspace_bytes(N, total_T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) with which ssm_fwd_varlen is fastest for these sizes (0: it takes none)."""
    return int(_load().gdn2_ssm_fwd_varlen_workspace_bytes(N, total_T, H, dk, dv, _DTYPES[dtype]))


def ssm_fwd_varlen(x, dt, B, C, A, cu_seqlens, D=None, dt_bias=None, initial_state=None, *, y=None, final_state=None,
                   output_final_state=True, softplus=True, workspace=None):
    """ssm_fwd over N sequences packed along the token axis: x [total_T,H,dv], dt [total_T,H],
    B, C [total_T,G,dk], cu_seqlens int64 [N+1] on the device, states [N,H,dk,dv], which
    ssm_step continues from."""
    code, dev = _on_gpu("ssm_fwd_varlen", x, 3, "[total_T,H,dv]")
    lead = (x.shape[0],)
    (H, G, dk, dv), strides, ptrs = _ssm_args(lead, x, dt, B, C, A, D, dt_bias, dev)
    n = _offsets(cu_seqlens, dev)
    sshape = (n, H, dk, dv)
    s0 = _opt("initial_state", initial_state, sshape, _F32, dev)
    y = _out("y", y, lead + (H, dv), x.dtype, dev, x)
    if final_state is not None or output_final_state:
        final_state = _out("final_state", final_state, sshape, _F32, dev, initial_state)
    need = _bytes("gdn2_ssm_fwd_varlen_workspace_bytes", dev, n, lead[0], H, dk, dv, code)
    ws, ws_bytes, keep = _workspace(workspace, need, 256, dev) if need else (None, 0, None)
    _launch("gdn2_ssm_fwd_varlen", dev, *ptrs, s0, y.data_ptr(), _ptr(final_state), cu_seqlens.data_ptr(), n, lead[0],
            H, G, dk, dv, *strides, code, int(softplus), ws, ws_bytes)
    return y, final_state


def ssm_step(x, dt, B, C, A, state, D=None, dt_bias=None, *, y=None, softplus=True):
    """One token for each of N sequences: x [N,H,dv], dt [N,H], B, C [N,G,dk]; ``state``
    [N,H,dk,dv] fp32 is updated in place.  Returns y."""
    code, dev = _on_gpu("ssm_step", x, 3, "[N,H,dv]")
    lead = (x.shape[0],)
    (H, G, dk, dv), strides, ptrs = _ssm_args(lead, x, dt, B, C, A, D, dt_bias, dev)
    ps = _in("state", state, (lead[0], H, dk, dv), _F32, dev)
    y = _out("y", y, lead + (H, dv), x.dtype, dev, x)
    _launch("gdn2_ssm_step", dev, *ptrs, ps, y.data_ptr(), lead[0], H, G, dk, dv, *strides, code,
            int(softplus))
    return y


def short_conv(x, taps, bias=None, initial_state=None, *, y=None, final_state=None, output_final_state=True):
    """Causal depthwise convolution of four taps with bias and SiLU: x [B,T,C].  Returns
    (y, kept): kept [B,3,C] are the last three inputs, the next call's ``initial_state``
    (None when ``output_final_state`` is False and no ``final_state`` is given, which may be
    ``initial_state`` itself)."""
    code, dev = _on_gpu("short_conv", x, 3, "[B,T,C]")
    n, T, ch = x.shape
    xs = _tokens("x", x, x.shape, 1, x.dtype, dev)
    y, ptrs, final_state = _conv_args(x, taps, bias, initial_state, y, final_state, output_final_state, n, dev)
    _launch("gdn2_short_conv", dev, *ptrs, n, T, ch, xs, code)
    return y, final_state


def short_conv_varlen(x, taps, cu_seqlens, bias=None, initial_state=None, *, y=None, final_state=None,
                      output_final_state=True):
    """short_conv over N sequences packed along the token axis: x [total_T,C], cu_seqlens int64
    [N+1] on the device, the inputs kept [N,3,C]."""
    code, dev = _on_gpu("short_conv_varlen", x, 2, "[total_T,C]")
    total, ch = x.shape
    xs = _tokens("x", x, x.shape, 1, x.dtype, dev)
    n = _offsets(cu_seqlens, dev)
    y, ptrs, final_state = _conv_args(x, taps, bias, initial_state, y, final_state, output_final_state, n, dev)
    _launch("gdn2_short_conv_varlen", dev, *ptrs, cu_seqlens.data_ptr(), n, total, ch, xs, code)
    return y, final_state


def _conv_args(x, taps, bias, initial_state, y, final_state, output_final_state, n, dev):
    ch = x.shape[-1]
    pt = _in("taps", taps, (ch, 4), _F32, dev)
    b = _opt("bias", bias, (ch,), _F32, dev)
    s0 = _opt("initial_state", initial_state, (n, 3, ch), x.dtype, dev)
    y = _out("y", y, tuple(x.shape), x.dtype, dev, x)
    if final_state is not None or output_final_state:
        final_state = _out("final_state", final_state, (n, 3, ch), x.dtype, dev, initial_state)
    return y, (x.data_ptr(), pt, b, s0, y.data_ptr(), _ptr(final_state)), final_state


def short_conv_step(x, taps, state, bias=None, *, y=None):
    """One token for each of N sequences: x [N,C]; ``state`` [N,3,C], the inputs kept, is updated
    in place.  Returns y."""
    code, dev = _on_gpu("short_conv_step", x, 2, "[N,C]")
    n, ch = x.shape
    xs = _tokens("x", x, x.shape, 1, x.dtype, dev)
    pt = _in("taps", taps, (ch, 4), _F32, dev)
    ps = _in("state", state, (n, 3, ch), x.dtype, dev)
    b = _opt("bias", bias, (ch,), _F32, dev)
    y = _out("y", y, (n, ch), x.dtype, dev, x)
    _launch("gdn2_short_conv_step", dev, x.data_ptr(), pt, b, ps, y.data_ptr(), n, ch, xs,
            code)
    return y


def layer_norm(x, gamma, beta=None, eps=1e-5, *, y=None, stats=True):
    """Layer norm over the last axis.  Returns (y, mean, rstd); mean and rstd [...] fp32 are what
    layer_norm_bwd takes (None with ``stats=False``)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be [...,width]")
    code, dev = _on_gpu("layer_norm", x, x.dim(), "[...,width]")
    shape = x.shape
    width = shape[-1]
    px = _in("x", x, shape, x.dtype, dev)
    pg = _in("gamma", gamma, (width,), _F32, dev)
    b = _opt("beta", beta, (width,), _F32, dev)
    y = _out("y", y, shape, x.dtype, dev, x)
    mean = rstd = None
    if stats:
        mean = torch.empty(tuple(shape[:-1]), dtype=_F32, device=dev)
        rstd = torch.empty_like(mean)
    _launch("gdn2_layer_norm", dev, px, pg, b, y.data_ptr(), _ptr(mean), _ptr(rstd),
            x.numel() // max(width, 1), width, float(eps), code)
    return y, mean, rstd


def layer_norm_bwd_workspace_bytes(rows, width) -> int:
    """Device workspace (bytes) that layer_norm_bwd needs for these sizes."""
    return int(_load().gdn2_layer_norm_bwd_workspace_bytes(rows, width))


def layer_norm_bwd(dy, x, gamma, mean, rstd, *, grads=None, want_beta_grad=True, workspace=None):
    """Gradients of sum(dy * y) for layer_norm(x, gamma, beta), from the statistics it returned.
    Returns a dict dx (x's dtype), dgamma and dbeta (fp32; dbeta None when not requested).
    ``grads`` may hold preallocated outputs and ``workspace`` (uint8, at least
    layer_norm_bwd_workspace_bytes + 16) the scratch memory."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be [...,width]")
    code, dev = _on_gpu("layer_norm_bwd", x, x.dim(), "[...,width]")
    shape = x.shape
    width = shape[-1]
    rows = x.numel() // max(width, 1)
    lead = tuple(shape[:-1])
    ptrs = (_in("dy", dy, shape, x.dtype, dev), _in("x", x, shape, x.dtype, dev),
            _in("gamma", gamma, (width,), _F32, dev), _in("mean", mean, lead, _F32, dev),
            _in("rstd", rstd, lead, _F32, dev))
    out = {} if grads is None else dict(grads)
    out["dx"] = _out("dx", out.get("dx"), shape, x.dtype, dev, x)
    out["dgamma"] = _out("dgamma", out.get("dgamma"), (width,), _F32, dev, gamma)
    out["dbeta"] = _out("dbeta", out.get("dbeta"), (width,), _F32, dev, gamma) if want_beta_grad else None
    need = layer_norm_bwd_workspace_bytes(rows, width)
    ws, ws_bytes, keep = _workspace(workspace, need, 16, dev) if need else (None, 0, None)
    _launch("gdn2_layer_norm_bwd", dev, *ptrs, out["dx"].data_ptr(), out["dgamma"].data_ptr(), _ptr(out["dbeta"]), ws, ws_bytes, rows,
            width, code)
    return out
