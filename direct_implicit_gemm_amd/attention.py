"""Tensor-level helpers of the attention-layer operators of ``include/libconv.h``.

    lora_linear        a projection with each request's low-rank adapter beside it
    qk_norm_rope       norms of queries and keys, position rotation, cache write
    prefix_attention   attention over keys a batch shares and each entry's own

They allocate outputs (and workspaces, through torch), enqueue on the current
stream or ``stream``, and raise ``LibconvError`` on a status other than OK.
Tensors may be strided (slices of a fused projection, caches in any order of
axes) as long as their last axis is dense and their rows lie on 16-byte
boundaries.  There is no backward pass: libconv runs networks forward.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

_STRIDES12 = ctypes.c_longlong * 12
_STRIDES16 = ctypes.c_longlong * 16


def _base():
    import direct_implicit_gemm_amd as L
    return L


def _check(what, tensors, like, dims=None):
    """Device, dtype and dense last axis of the operands that are given."""
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda or t.device != like.device:
            raise ValueError(f"{what}: operands must be device tensors of one device")
        if t.dtype != like.dtype:
            raise ValueError(f"{what}: operands must have one dtype")
        if t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"{what}: expected {dims} axes with the last one dense")


def _ints(what, t, shape, device):
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() or \
            t.device != device:
        raise ValueError(f"{what} must be a contiguous int32 device tensor of shape {shape}")
    return t.data_ptr()


def _call(device, stream, what, call, need=0, workspace=True):
    """Runs call(workspace pointer, bytes, stream) with `device` current."""
    import torch
    L = _base()
    with torch.cuda.device(device):
        foreign = stream is not None
        if not foreign:
            stream = torch.cuda.current_stream(device).cuda_stream
        ptr, size, buf = None, 0, None
        if workspace is not None and workspace is not False:
            if workspace is True:
                if need > 0:
                    buf = torch.empty(need, dtype=torch.uint8, device=device)
                    ptr, size = buf.data_ptr(), need
            else:
                ptr, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        st = call(ptr, size, stream)
        if buf is not None and foreign:  # its memory is used on that stream until then
            buf.record_stream(torch.cuda.ExternalStream(stream, device=device))
    if st != 0:
        raise L.LibconvError(st, what)


def rotary_frequencies(rot_dim: int, theta: float = 10000.0,
                       sections: Optional[Sequence[int]] = None, device="cuda"):
    """Radians a position of each of the rot_dim / 2 pairs, in 64 bits: theta^(-i / n)
    for pair i of a section of n pairs (one section by default)."""
    import torch
    sections = [rot_dim // 2] if sections is None else list(sections)
    if sum(sections) != rot_dim // 2:
        raise ValueError("the sections must add up to rot_dim / 2 pairs")
    f = [theta ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections if n > 0]
    return (torch.cat(f) if f else torch.empty(0, dtype=torch.float64)).to(device)


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps: float = 1e-6,
                 sections: Optional[Sequence[int]] = None, interleaved: bool = False, v=None,
                 slots=None, q_out=None, k_out=None, v_out=None, stream=None):
    """Per-head RMS norm of q [T, Hq, D] and k [T, Hk, D], and their rotation by
    positions (int32 [axes, T] or [T]) times freqs (float64 [pairs]); sections:
    pairs that turn with each axis.  With v, values are copied to v_out; with
    slots (int32 [T]), keys and values go to rows slots[t] of k_out / v_out.
    Returns (q_out, k_out) or (q_out, k_out, v_out)."""
    import torch
    L = _base()
    _check("qk_norm_rope", (q, k, v), q, 3)
    T, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape != (T, Hk, D) or (v is not None and v.shape != k.shape):
        raise ValueError("qk_norm_rope: q [T, Hq, D], k and v [T, Hk, D]")
    if slots is not None and (k_out is None or (v is not None and v_out is None)):
        raise ValueError("qk_norm_rope: slots need k_out (and v_out)")
    if v is None and v_out is not None:
        raise ValueError("qk_norm_rope: v_out without v")
    pos = positions if positions.dim() == 2 else positions.unsqueeze(0)
    pairs = freqs.numel()
    sections = [pairs] if sections is None else [int(n) for n in sections]
    if len(sections) > 3 or sum(sections) != pairs or min(sections, default=0) < 0 or \
            2 * pairs > D or pos.shape[0] < len(sections):
        raise ValueError("qk_norm_rope: up to 3 sections that add up to the pairs of freqs, "
                         "with a row of positions each")
    pos_ptr = _ints("positions", pos, (pos.shape[0], T), q.device)
    if freqs.dtype != torch.float64 or not freqs.is_contiguous() or freqs.device != q.device:
        raise ValueError("freqs must be a contiguous float64 device tensor")
    for w in (q_weight, k_weight):
        if w is not None:
            _check("qk_norm_rope", (w,), q, 1)
            if w.shape[0] != D:
                raise ValueError("qk_norm_rope: weights [D]")
    q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device) if q_out is None else q_out
    k_out = torch.empty((T, Hk, D), dtype=q.dtype, device=q.device) if k_out is None else k_out
    if v is not None and v_out is None:
        v_out = torch.empty((T, Hk, D), dtype=q.dtype, device=q.device)
    _check("qk_norm_rope", (q_out, k_out, v_out), q, 3)
    rows = T if slots is None else k_out.shape[0]
    if q_out.shape != q.shape or k_out.shape != (rows, Hk, D) or \
            (v is not None and v_out.shape != (rows, Hk, D)):
        raise ValueError("qk_norm_rope: bad output tensor")
    slot_ptr = None if slots is None else _ints("slots", slots, (T,), q.device)
    result = (q_out, k_out) if v is None else (q_out, k_out, v_out)
    if T == 0:
        return result
    st = []
    for t in (q, k, v, q_out, k_out, v_out):
        st += [0, 0] if t is None else [t.stride(0), t.stride(1)]
    n = sections + [0] * (3 - len(sections))
    _call(q.device, stream, "libconv_qk_norm_rope", lambda _p, _n, s: L.libconv_qk_norm_rope(
        L._ptr(q), L._ptr(k), L._ptr(v), L._ptr(q_out), L._ptr(k_out), L._ptr(v_out),
        L._ptr(q_weight), L._ptr(k_weight), freqs.data_ptr(), pos_ptr, slot_ptr,
        _STRIDES12(*st), T, Hq, Hk, D, 2 * pairs, n[0], n[1], n[2], int(bool(interleaved)), rows,
        float(eps), L._dtype_code(q), s))
    return result


def prefix_attention(q, k_prefix, v_prefix, k, v, lengths, scale: Optional[float] = None,
                     causal: bool = True, out=None, return_lse: bool = False, stream=None,
                     workspace=True):
    """Attention of q [B, Sq, Hq, D] over the shared k_prefix, v_prefix [P, Hk, D]
    and each entry's first lengths[b] (int32 [B]) rows of k, v [B, S, Hk, D].
    causal: query i sees the own keys up to lengths[b] - Sq + i.  k_prefix and
    v_prefix, or k and v, may be None (no such keys).  Returns out, or (out, lse
    [B, Hq, Sq] float32).  workspace: True (allocate what the best plan takes),
    False (none), or a uint8 device tensor."""
    import torch
    L = _base()
    _check("prefix_attention", (q, k, v, out), q, 4)
    _check("prefix_attention", (k_prefix, v_prefix), q, 3)
    B, Sq, Hq, D = q.shape
    if (k is None) != (v is None) or (k_prefix is None) != (v_prefix is None):
        raise ValueError("prefix_attention: keys and values come together")
    if k is None and k_prefix is None:
        raise ValueError("prefix_attention: neither a prefix nor own keys")
    Hk = (k if k is not None else k_prefix).shape[-2]
    P = 0 if k_prefix is None else k_prefix.shape[0]
    S = 0 if k is None else k.shape[1]
    if (k is not None and (k.shape != (B, S, Hk, D) or v.shape != k.shape)) or \
            (P and (k_prefix.shape != (P, Hk, D) or v_prefix.shape != k_prefix.shape)):
        raise ValueError("prefix_attention: k, v [B, S, Hk, D], k_prefix, v_prefix [P, Hk, D]")
    len_ptr = _ints("lengths", lengths, (B,), q.device)
    out = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device) if out is None else out
    if out.shape != q.shape:
        raise ValueError("prefix_attention: bad output tensor")
    lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device) if return_lse else None
    if B == 0 or Sq == 0:
        return (out, lse) if return_lse else out
    scale = D ** -0.5 if scale is None else float(scale)
    dt = L._dtype_code(q)
    need = L.load().libconv_prefix_attention_workspace(B, Sq, P, S, Hq, Hk, D, dt) \
        if workspace is True else 0
    st = []
    for t, n in ((q, 3), (k_prefix, 2), (v_prefix, 2), (k, 3), (v, 3), (out, 3)):
        st += [0] * n if t is None else t.stride()[:n]
    _call(q.device, stream, "libconv_prefix_attention",
          lambda p, n, s: L.libconv_prefix_attention(
              L._ptr(q), L._ptr(k_prefix), L._ptr(v_prefix), L._ptr(k), L._ptr(v), len_ptr,
              L._ptr(out), L._ptr(lse), _STRIDES16(*st), B, Sq, P, S, Hq, Hk, D, scale,
              int(bool(causal)), dt, p, n, s), need, workspace)
    return (out, lse) if return_lse else out


def lora_linear(x, w, bias, a, b, scales, row_starts, adapters, out=None, stream=None,
                workspace=True):
    """y = x w^T + bias + scales[i] (x a[i]^T) b[i]^T for the rows row_starts[r] ..
    row_starts[r + 1] - 1 of request r, whose adapter is i = adapters[r].
    x [T, K], w [N, K], a [n, rank, K], b [n, N, rank], scales float32 [n],
    row_starts int32 [R + 1], adapters int32 [R] (outside [0, n): none).
    a .. adapters may all be None: the projection alone."""
    import torch
    L = _base()
    _check("lora_linear", (x, w, out), x, 2)
    T, K = x.shape
    N = w.shape[0]
    if w.shape != (N, K) or not w.is_contiguous():
        raise ValueError("lora_linear: w must be a contiguous [N, K]")
    if bias is not None:
        _check("lora_linear", (bias,), x, 1)
        if bias.shape != (N,):
            raise ValueError("lora_linear: bias must be [N]")
    low = (a, b, scales, row_starts, adapters)
    n = rank = R = 0
    starts_ptr = adapters_ptr = None
    if any(t is not None for t in low):
        if any(t is None for t in low):
            raise ValueError("lora_linear: a, b, scales, row_starts and adapters come together")
        _check("lora_linear", (a, b), x, 3)
        n, rank = a.shape[0], a.shape[1]
        if a.shape != (n, rank, K) or b.shape != (n, N, rank) or not a.is_contiguous() or \
                not b.is_contiguous():
            raise ValueError("lora_linear: contiguous a [n, rank, K] and b [n, N, rank]")
        if scales.dtype != torch.float32 or scales.shape != (n,) or \
                not scales.is_contiguous() or scales.device != x.device:
            raise ValueError("lora_linear: scales must be a contiguous float32 device tensor [n]")
        R = adapters.shape[0]
        adapters_ptr = _ints("adapters", adapters, (R,), x.device)
        starts_ptr = _ints("row_starts", row_starts, (R + 1,), x.device)
    out = torch.empty((T, N), dtype=x.dtype, device=x.device) if out is None else out
    if out.shape != (T, N):
        raise ValueError("lora_linear: bad output tensor")
    if T == 0:
        return out
    dt = L._dtype_code(x)
    need = L.load().libconv_lora_workspace(T, K, N, rank, n, R, dt)
    _call(x.device, stream, "libconv_lora_linear", lambda p, m, s: L.libconv_lora_linear(
        L._ptr(x), L._ptr(w), L._ptr(bias), L._ptr(a), L._ptr(b), L._ptr(scales), starts_ptr,
        adapters_ptr, L._ptr(out), T, K, N, rank, n, R, x.stride(0), out.stride(0), dt, p, m, s),
        need, workspace)
    return out
