"""The attention block's calls: attention, its gradients and its step, rotary positions and RMS norm.

    o, lse = attn_fwd(q, k, v, window=None, scale=None)
    o, lse = attn_fwd_varlen(q, k, v, cu_seqlens, cu_seqlens_k=None, window=None)   # packed sequences
    grads  = attn_bwd(d_o, q, k, v, o, lse, window=None)              # dq, dk, dv
    grads  = attn_bwd_varlen(d_o, q, k, v, o, lse, cu_seqlens)
    o      = attn_step(q, k, v, k_cache, v_cache, positions, window=None)   # caches updated in place
    q, k   = rotary(q, k, freq, positions=None, interleaved=False)
    freq   = rotary_frequencies(rot, base=10000.0)                    # the table, also for long contexts
    y, h, rstd = rms_norm(x, gamma, eps=1e-6, residual=None)          # h = x + residual
    y, scales, h, rstd = rms_norm_fp8(x, gamma, eps=1e-6, residual=None)
    grads  = rms_norm_bwd(dy, h, gamma, rstd, dh=None)                # dx, dgamma

Layouts: q, o, d_o [B,T,H,d]; k, v [B,S,G,d], head h reading key head h // (H // G); lse [B,T,H] fp32
(packed: [total,...] for [B,T,...]; step: [N,...], caches [N,C,G,d] and int64 positions [N]).  Queries are the
last T of the S tokens; a query sees the keys at and before its own position, with a ``window`` the last
``window`` of them.  Norm: x, y, h [...,width], gamma [width] and rstd [...] fp32; the residual, h, dh and dx
may be fp32 beside bf16 activations.  Everything else is bf16 or fp32, one dtype in a call; d is 64 or 128 for
attention, at most 512 for rotary.  q, k and v may be parts of one wider tensor (a token stride of their own, a
token's elements contiguous; in whole 16-byte units for attention); all other tensors are contiguous.
Addresses are 16-byte aligned (rotary's to their elements).  The library's refusals of other calls are
Gdn2Error.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _DTYPES, _load, _ptr
from .block import _bytes, _F32, _in, _launch, _offsets, _on_gpu, _opt, _out, _tokens, _workspace

__all__ = ["attn_fwd", "attn_fwd_varlen", "attn_fwd_workspace_bytes", "attn_fwd_varlen_workspace_bytes", "attn_bwd",
           "attn_bwd_varlen", "attn_bwd_workspace_bytes", "attn_bwd_varlen_workspace_bytes", "attn_step", "attn_step_workspace_bytes", "rotary",
           "rotary_frequencies", "rms_norm", "rms_norm_fp8", "rms_norm_bwd", "rms_norm_bwd_workspace_bytes"]


def _declare(lib):
    P, I64, I32, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, args, res in (
            ("attn_fwd", [P] * 5 + [I64] * 10 + [F, I32, P, SZ, P], I32),
            ("attn_fwd_workspace_bytes", [I64] * 7 + [I32], SZ),
            ("attn_fwd_varlen", [P] * 7 + [I64] * 10 + [F, I32, P, SZ, P], I32),
            ("attn_fwd_varlen_workspace_bytes", [I64] * 7 + [I32], SZ),
            ("attn_bwd", [P] * 9 + [I64] * 10 + [F, I32, P, SZ, P], I32),
            ("attn_bwd_varlen", [P] * 11 + [I64] * 10 + [F, I32, P, SZ, P], I32),
            ("attn_bwd_workspace_bytes", [I64] * 7 + [I32], SZ),
            ("attn_bwd_varlen_workspace_bytes", [I64] * 7 + [I32], SZ),
            ("attn_step", [P] * 7 + [I64] * 9 + [F, I32, P, SZ, P], I32),
            ("attn_step_workspace_bytes", [I64] * 6 + [I32], SZ),
            ("rotary", [P] * 6 + [I64] * 10 + [I32, I32, F, I32, P], I32),
            ("rms_norm", [P] * 6 + [I64] * 2 + [F, I32, I32, P], I32),
            ("rms_norm_fp8", [P] * 7 + [I64] * 2 + [F, I32, I32, P], I32),
            ("rms_norm_bwd_workspace_bytes", [I64] * 2, SZ),
            ("rms_norm_bwd", [P] * 8 + [SZ] + [I64] * 2 + [I32, I32, P], I32)):
        f = getattr(lib, "gdn2_" + name)
        f.argtypes, f.restype = args, res


def _window(window):
    if window is None:
        return 0
    window = int(window)
    if window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    return window


def _qkv(q, k, v, lead_q, lead_k, dev):
    """Sizes, strides and pointers of attention's inputs."""
    H, d = q.shape[-2:]
    G = k.shape[-2]
    kshape = lead_k + (G, d)
    t = q.dtype
    strides = (_tokens("q", q, q.shape, 2, t, dev), _tokens("k", k, kshape, 2, t, dev), _tokens("v", v, kshape, 2, t, dev))
    return (H, G, d), strides, (q.data_ptr(), k.data_ptr(), v.data_ptr())


def _keys(k, ndim, layout):
    if not isinstance(k, torch.Tensor) or k.dim() != ndim:
        raise ValueError("k must be %s" % layout)


def _scale(scale, d):
    return 1.0 / math.sqrt(max(d, 1)) if scale is None else float(scale)


def _parts(workspace, need, dev):
    return _workspace(workspace, need, 16, dev) if need else (None, 0, None)


def attn_fwd(q, k, v, *, window=None, scale=None, o=None, lse=None, stats=True, workspace=None):
    """Causal attention of whole sequences: q [B,T,H,d], k, v [B,S,G,d].  Returns (o, lse); lse
    [B,T,H] is what attn_bwd takes (None with ``stats=False`` and no ``lse``).  ``scale`` is
    1 / sqrt(d) unless given.  ``workspace`` (uint8, at least attn_fwd_workspace_bytes + 16) is
    allocated here unless passed."""
    code, dev = _on_gpu("attn_fwd", q, 4, "[B,T,H,d]")
    _keys(k, 4, "[B,S,G,d]")
    (B, T), S = q.shape[:2], k.shape[1]
    dims, strides, ptrs = _qkv(q, k, v, (B, T), (B, S), dev)
    w = _window(window)
    o, lse = _fwd_out(q, o, lse, stats, (B, T) + dims[:1], dev)
    need = _bytes("gdn2_attn_fwd_workspace_bytes", dev, B, T, S, *dims, w, code)
    ws, ws_bytes, keep = _parts(workspace, need, dev)
    _launch("gdn2_attn_fwd", dev, *ptrs, o.data_ptr(), _ptr(lse), B, T, S, *dims, *strides, w, _scale(scale, dims[2]), code,
            ws, ws_bytes)
    return o, lse


def _fwd_out(q, o, lse, stats, lse_shape, dev):
    o = _out("o", o, tuple(q.shape), q.dtype, dev, q)
    if lse is not None or stats:
        lse = _out("lse", lse, lse_shape, _F32, dev)
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens, *, cu_seqlens_k=None, window=None, scale=None, o=None, lse=None, stats=True,
                    workspace=None):
    """attn_fwd over N sequences packed along the token axis: q [total_T,H,d], k, v [total_S,G,d],
    cu_seqlens int64 [N+1] on the device, lse [total_T,H].  ``cu_seqlens_k`` are the keys' offsets where
    sequences go on from keys before their queries; without it they are the queries'.  Tokens of no
    sequence are left as they were in ``o`` and ``lse``."""
    code, dev = _on_gpu("attn_fwd_varlen", q, 3, "[total_T,H,d]")
    _keys(k, 3, "[total_S,G,d]")
    T, S = q.shape[0], k.shape[0]
    dims, strides, ptrs = _qkv(q, k, v, (T,), (S,), dev)
    n, cu, cu_k = _both_offsets(cu_seqlens, cu_seqlens_k, dev)
    w = _window(window)
    o, lse = _fwd_out(q, o, lse, stats, (T,) + dims[:1], dev)
    need = _bytes("gdn2_attn_fwd_varlen_workspace_bytes", dev, n, T, S, *dims, w, code)
    ws, ws_bytes, keep = _parts(workspace, need, dev)
    _launch("gdn2_attn_fwd_varlen", dev, *ptrs, o.data_ptr(), _ptr(lse), cu, cu_k, n, T, S, *dims, *strides, w,
            _scale(scale, dims[2]), code, ws, ws_bytes)
    return o, lse


def _both_offsets(cu, cu_k, dev):
    n = _offsets(cu, dev)
    if cu_k is None:
        return n, cu.data_ptr(), cu.data_ptr()
    if _offsets(cu_k, dev) != n:
        raise ValueError("cu_seqlens_k must have as many offsets as cu_seqlens")
    return n, cu.data_ptr(), cu_k.data_ptr()


def attn_fwd_workspace_bytes(B, T, S, H, G, d, window=None, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) with which attn_fwd is fastest for these sizes (0: it takes none)."""
    return int(_load().gdn2_attn_fwd_workspace_bytes(B, T, S, H, G, d, _window(window), _DTYPES[dtype]))


def attn_fwd_varlen_workspace_bytes(N, total_T, total_S, H, G, d, window=None, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) with which attn_fwd_varlen is fastest for these sizes (0: it takes none)."""
    return int(_load().gdn2_attn_fwd_varlen_workspace_bytes(N, total_T, total_S, H, G, d, _window(window), _DTYPES[dtype]))


def attn_bwd_workspace_bytes(B, T, S, H, G, d, window=None, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) that attn_bwd needs for these sizes (0: none)."""
    return int(_load().gdn2_attn_bwd_workspace_bytes(B, T, S, H, G, d, _window(window), _DTYPES[dtype]))


def attn_bwd_varlen_workspace_bytes(N, total_T, total_S, H, G, d, window=None, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) that attn_bwd_varlen needs for these sizes (0: none)."""
    return int(_load().gdn2_attn_bwd_varlen_workspace_bytes(N, total_T, total_S, H, G, d, _window(window), _DTYPES[dtype]))


def _bwd(name, d_o, q, k, v, o, lse, lead_q, lead_k, sizes, offsets, window, scale, grads, workspace, code, dev):
    dims, strides, ptrs = _qkv(q, k, v, lead_q, lead_k, dev)
    H, G, d = dims
    qs, ks = lead_q + (H, d), lead_k + (G, d)
    first = _in("d_o", d_o, qs, q.dtype, dev)
    kept = (_in("o", o, qs, q.dtype, dev), _in("lse", lse, lead_q + (H,), _F32, dev))
    out = {} if grads is None else dict(grads)
    out["dq"] = _out("dq", out.get("dq"), qs, q.dtype, dev, q)
    out["dk"] = _out("dk", out.get("dk"), ks, q.dtype, dev, k)
    out["dv"] = _out("dv", out.get("dv"), ks, q.dtype, dev, v)
    w = _window(window)
    need = _bytes(name + "_workspace_bytes", dev, *sizes, *dims, w, code)
    ws, ws_bytes, keep = _parts(workspace, need, dev)
    _launch(name, dev, first, *ptrs, *kept, out["dq"].data_ptr(), out["dk"].data_ptr(), out["dv"].data_ptr(), *offsets, *sizes,
            *dims, *strides, w, _scale(scale, d), code, ws, ws_bytes)
    return out


def attn_bwd(d_o, q, k, v, o, lse, *, window=None, scale=None, grads=None, workspace=None):
    """Gradients of sum(d_o * o) for attn_fwd(q, k, v), from the o and lse it returned.  Returns a dict dq,
    dk, dv (contiguous, in the inputs' dtype).  ``grads`` may hold preallocated outputs and ``workspace``
    (uint8, at least attn_bwd_workspace_bytes + 16) the scratch memory."""
    code, dev = _on_gpu("attn_bwd", q, 4, "[B,T,H,d]")
    _keys(k, 4, "[B,S,G,d]")
    (B, T), S = tuple(q.shape[:2]), k.shape[1]
    return _bwd("gdn2_attn_bwd", d_o, q, k, v, o, lse, (B, T), (B, S), (B, T, S), (), window, scale, grads, workspace, code, dev)


def attn_bwd_varlen(d_o, q, k, v, o, lse, cu_seqlens, *, cu_seqlens_k=None, window=None, scale=None, grads=None, workspace=None):
    """attn_bwd for attn_fwd_varlen.  Gradients of tokens of no sequence are left as they were.
    ``workspace``: at least attn_bwd_varlen_workspace_bytes + 16."""
    code, dev = _on_gpu("attn_bwd_varlen", q, 3, "[total_T,H,d]")
    _keys(k, 3, "[total_S,G,d]")
    T, S = q.shape[0], k.shape[0]
    n, cu, cu_k = _both_offsets(cu_seqlens, cu_seqlens_k, dev)
    return _bwd("gdn2_attn_bwd_varlen", d_o, q, k, v, o, lse, (T,), (S,), (n, T, S), (cu, cu_k), window, scale, grads, workspace,
                code, dev)


def attn_step_workspace_bytes(N, H, G, d, C, window=None, dtype=torch.bfloat16) -> int:
    """Device workspace (bytes) with which attn_step is fastest for these sizes (0: it takes none)."""
    return int(_load().gdn2_attn_step_workspace_bytes(N, H, G, d, C, _window(window), _DTYPES[dtype]))


def attn_step(q, k, v, k_cache, v_cache, positions, *, window=None, scale=None, o=None, workspace=None):
    """One token for each of N sequences: q [N,H,d], k, v [N,G,d] and its position (int64 [N], on the
    device).  The caches [N,C,G,d] keep the last C tokens, the token at position p in slot p mod C; the
    step writes its own there and sees the last min(p + 1, window, C) tokens.  A position below 0 is no
    token.  Returns o."""
    code, dev = _on_gpu("attn_step", q, 3, "[N,H,d]")
    _keys(k, 3, "[N,G,d]")
    N = q.shape[0]
    dims, strides, ptrs = _qkv(q, k, v, (N,), (N,), dev)
    H, G, d = dims
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [N,C,G,d]")
    C = k_cache.shape[1]
    caches = (_in("k_cache", k_cache, (N, C, G, d), q.dtype, dev), _in("v_cache", v_cache, (N, C, G, d), q.dtype, dev))
    places = _in("positions", positions, (N,), torch.int64, dev)
    w = _window(window)
    o = _out("o", o, (N, H, d), q.dtype, dev, q)
    need = _bytes("gdn2_attn_step_workspace_bytes", dev, N, H, G, d, C, w, code)
    ws, ws_bytes, keep = _parts(workspace, need, dev)
    _launch("gdn2_attn_step", dev, *ptrs, *caches, places, o.data_ptr(), N, H, G, d, C, *strides, w, _scale(scale, d), code, ws,
            ws_bytes)
    return o


def rotary_frequencies(rot, base=10000.0, *, factor=1.0, length=None, low=1.0, high=32.0, device=None):
    """The table that rotary takes: fp32 [rot / 2], base^(-2 i / rot) radians a position, formed in 64
    bits.  For contexts ``factor`` times as long as those a model has learned: without ``length`` every
    frequency is divided by ``factor`` (position interpolation); with ``length``, the context learned, only
    those that make fewer than ``low`` turns in it, those of more than ``high`` turns stay, and between them
    the share that is divided falls linearly with the turns: interpolation by parts as in Peng et al., "YaRN:
    Efficient Context Window Extension of Large Language Models" (arXiv:2309.00071, section 3.2), whose alpha
    and beta are the defaults of ``low`` and ``high``."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not factor > 0 or (length is not None and not (length > 0 and high > low)):
        raise ValueError("factor and length must be positive, and high above low")
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if length is None:
        freq = freq / factor
    else:
        kept = ((length * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        freq = freq * (kept + (1 - kept) / factor)
    return freq.to(torch.float32).to(device)


def rotary(q, k, freq, positions=None, *, interleaved=False, inverse=False, scale=1.0, q_out=None, k_out=None):
    """Rotary positions on the first 2 len(freq) channels of the heads of q [B,T,H,d] and k [B,T,G,d] (or
    [tokens,H,d] and [tokens,G,d]; ``k`` may be None): channels i and i + len(freq) of a head, or 2 i and
    2 i + 1 when ``interleaved``, turn by position * freq[i].  ``positions`` are int64, one a token; without
    them a token's is its place on the last token axis.  ``inverse`` turns back, which is also the gradient.
    Outputs are new tensors unless given; ``q_out`` may be ``q`` itself, and ``k_out`` ``k``, also as parts
    of one wider tensor.  Returns (q, k)."""
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be [B,T,H,d] or [tokens,H,d]")
    code, dev = _on_gpu("rotary", q, q.dim(), "[...,H,d]")
    lead = tuple(q.shape[:-2])
    H, d = q.shape[-2:]
    qs = _tokens("q", q, q.shape, 2, q.dtype, dev)
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise ValueError("freq must be [rot / 2]")
    pf = _in("freq", freq, freq.shape, _F32, dev)
    pp = _opt("positions", positions, lead, torch.int64, dev)
    q_out, qos = _rotary_out("q_out", q, q_out, dev)
    G, ks, kos = 0, 0, 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
            raise ValueError("k must be [...,G,d] with as many axes as q")
        G = k.shape[-2]
        if G == 0:
            raise ValueError("k must have at least one head (None: q alone)")
        ks = _tokens("k", k, lead + (G, d), 2, q.dtype, dev)
        k_out, kos = _rotary_out("k_out", k, k_out, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _launch("gdn2_rotary", dev, q.data_ptr(), _ptr(k), pf, pp, q_out.data_ptr(), _ptr(k_out), math.prod(lead), max(lead[-1], 1),
            H, G, d, 2 * freq.shape[0], qs, ks, qos, kos, int(bool(interleaved)), int(bool(inverse)), float(scale), code)
    return q_out, k_out


def _rotary_out(name, t, out, dev):
    """The output beside t, and the elements between its tokens."""
    if out is None:
        out = torch.empty_like(t, memory_format=torch.contiguous_format)
        return out, t.shape[-1] * t.shape[-2]
    return out, _tokens(name, out, t.shape, 2, t.dtype, dev)


def _norm_in(fn, x, gamma):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be [...,width]")
    code, dev = _on_gpu(fn, x, x.dim(), "[...,width]")
    width = x.shape[-1]
    px = _in("x", x, x.shape, x.dtype, dev)
    pg = _in("gamma", gamma, (width,), _F32, dev)
    return code, dev, width, px, pg


def _residual(x, residual, h, dev):
    """The residual's address and dtype code, and the sum's tensor."""
    if residual is None:
        if h is not None:
            raise ValueError("h without a residual")
        return None, _DTYPES[x.dtype], None
    if not isinstance(residual, torch.Tensor):
        raise TypeError("residual must be a torch.Tensor")
    if residual.dtype not in (x.dtype, _F32):
        raise TypeError("residual dtype must be x's or float32")
    p = _in("residual", residual, x.shape, residual.dtype, dev)
    return p, _DTYPES[residual.dtype], _out("h", h, x.shape, residual.dtype, dev, residual)


def rms_norm(x, gamma, eps=1e-6, *, residual=None, y=None, h=None, stats=True):
    """Root-mean-square norm of x + residual over the last axis.  Returns (y, h, rstd): h is the sum, in the
    residual's dtype (x's or fp32; None without a residual; ``h`` may be ``residual`` itself), rstd [...] fp32
    what rms_norm_bwd takes (None with ``stats=False``)."""
    code, dev, width, px, pg = _norm_in("rms_norm", x, gamma)
    pr, rcode, h = _residual(x, residual, h, dev)
    y = _out("y", y, x.shape, x.dtype, dev, x)
    rstd = torch.empty(tuple(x.shape[:-1]), dtype=_F32, device=dev) if stats else None
    _launch("gdn2_rms_norm", dev, px, pr, pg, y.data_ptr(), _ptr(h), _ptr(rstd), x.numel() // max(width, 1), width, float(eps),
            code, rcode)
    return y, h, rstd


def rms_norm_fp8(x, gamma, eps=1e-6, *, residual=None, y=None, scales=None, h=None, stats=True):
    """rms_norm with its output in 8 bits (float8_e4m3fn) and a scale for each row: y * scales[..., None]
    stands for the norm's output, scales being the row's largest size / 448.  Returns (y, scales, h, rstd)."""
    code, dev, width, px, pg = _norm_in("rms_norm_fp8", x, gamma)
    pr, rcode, h = _residual(x, residual, h, dev)
    y = _out("y", y, x.shape, torch.float8_e4m3fn, dev)
    lead = tuple(x.shape[:-1])
    scales = _out("scales", scales, lead, _F32, dev)
    rstd = torch.empty(lead, dtype=_F32, device=dev) if stats else None
    _launch("gdn2_rms_norm_fp8", dev, px, pr, pg, y.data_ptr(), scales.data_ptr(), _ptr(h), _ptr(rstd),
            x.numel() // max(width, 1), width, float(eps), code, rcode)
    return y, scales, h, rstd


def rms_norm_bwd_workspace_bytes(rows, width) -> int:
    """Device workspace (bytes) that rms_norm_bwd needs for these sizes."""
    return int(_load().gdn2_rms_norm_bwd_workspace_bytes(rows, width))


def rms_norm_bwd(dy, h, gamma, rstd, *, dh=None, grads=None, workspace=None):
    """Gradients of sum(dy * y) + sum(dh * h) for rms_norm, from the sum h (x where there was no residual) and
    the rstd it returned.  Returns a dict dx (h's dtype; the gradient of x and of the residual) and dgamma
    (fp32).  ``grads`` may hold preallocated outputs (``dx`` may be ``dh`` itself) and ``workspace`` (uint8, at
    least rms_norm_bwd_workspace_bytes + 16) the scratch memory."""
    if not isinstance(dy, torch.Tensor) or dy.dim() < 1:
        raise ValueError("dy must be [...,width]")
    code, dev = _on_gpu("rms_norm_bwd", dy, dy.dim(), "[...,width]")
    if not isinstance(h, torch.Tensor) or h.dtype not in (dy.dtype, _F32):
        raise TypeError("h must be a torch.Tensor of dy's dtype or float32")
    shape = dy.shape
    width = shape[-1]
    rows = dy.numel() // max(width, 1)
    lead = tuple(shape[:-1])
    ptrs = (_in("dy", dy, shape, dy.dtype, dev), _in("h", h, shape, h.dtype, dev), _in("gamma", gamma, (width,), _F32, dev),
            _in("rstd", rstd, lead, _F32, dev), _opt("dh", dh, shape, h.dtype, dev))
    out = {} if grads is None else dict(grads)
    out["dx"] = _out("dx", out.get("dx"), shape, h.dtype, dev, h)
    out["dgamma"] = _out("dgamma", out.get("dgamma"), (width,), _F32, dev, gamma)
    need = rms_norm_bwd_workspace_bytes(rows, width)
    ws, ws_bytes, keep = _parts(workspace, need, dev)
    _launch("gdn2_rms_norm_bwd", dev, *ptrs, out["dx"].data_ptr(), out["dgamma"].data_ptr(), ws, ws_bytes, rows, width, code,
            _DTYPES[h.dtype])
    return out
