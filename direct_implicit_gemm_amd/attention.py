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
import functools
from typing import Optional, Sequence

_STRIDES12 = ctypes.c_longlong * 12
_STRIDES16 = ctypes.c_longlong * 16

# The calls below take as long on the host as small ones take on the GPU, so
# what does not change from call to call is looked up once, by _load().
_lib = _codes = _int32 = _float32 = _raw_stream = _current_device = None


def _load():
    import torch
    import direct_implicit_gemm_amd as L
    global _lib, _codes, _int32, _float32, _raw_stream, _current_device
    _int32, _float32 = torch.int32, torch.float32
    _codes = {torch.float32: L.F32, torch.float16: L.F16, torch.bfloat16: L.BF16}
    # as torch.cuda.current_stream() and current_device() have them, without
    # the objects (a call that gets this far has a device tensor)
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    _lib = L.load()
    return _lib


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, *sizes):
    return getattr(_lib, name)(*sizes)


def _refuse(what, why):
    raise ValueError(f"{what}: {why}")


_OPERANDS = "operands must be device tensors of one device and dtype, their last axis dense"


def _bad(t, device, dtype, strides, shape):
    """Whether an operand (its strides given) is not as _OPERANDS says or not of `shape`."""
    return (t.get_device() != device or t.dtype is not dtype or t.shape != shape or
            (strides[-1] != 1 and shape[-1] > 1))


def _bad_ints(t, device, shape):
    return (t.get_device() != device or t.dtype is not _int32 or t.shape != shape or
            not t.is_contiguous())


def _run(what, function, args, device, stream, buffer=None):
    """Enqueue on `stream` (a handle; None: the current stream), raise what it reports;
    buffer: a workspace that torch allocated for this call."""
    handle = _raw_stream(device) if stream is None else stream
    if _current_device() == device:
        status = function(*args, handle)
    else:
        import torch
        with torch.cuda.device(device):
            status = function(*args, handle)
    if buffer is not None and stream is not None:
        import torch
        # its memory is that stream's until then
        buffer.record_stream(torch.cuda.ExternalStream(stream, device=device))
    if status != 0:
        import direct_implicit_gemm_amd as L
        raise L.LibconvError(status, what)


def _given_workspace(workspace):
    """(address, bytes) of the caller's workspace, or of none."""
    if workspace is None or workspace is False:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


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
    what = "qk_norm_rope"
    lib, dev, dtype = _lib or _load(), q.get_device(), q.dtype
    qs, ks, qt, kt = q.shape, k.shape, q.stride(), k.stride()
    if dev < 0 or len(qs) != 3 or len(ks) != 3 or dtype not in _codes:
        _refuse(what, _OPERANDS)
    T, Hq, D = qs
    Hk = ks[1]
    if _bad(q, dev, dtype, qt, qs) or _bad(k, dev, dtype, kt, (T, Hk, D)):
        _refuse(what, "q [T, Hq, D], k and v [T, Hk, D]; " + _OPERANDS)
    if slots is not None and (k_out is None or (v is not None and v_out is None)):
        _refuse(what, "slots need k_out (and v_out)")
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    pairs = freqs.numel()
    n0, n1, n2 = pairs, 0, 0
    if sections is not None:
        n0, n1, n2, *more = (*sections, 0, 0, 0)
        if any(more) or n0 + n1 + n2 != pairs or min(n0, n1, n2) < 0:
            _refuse(what, "up to 3 sections that add up to the pairs of freqs")
    rows = positions.shape[0]
    if 2 * pairs > D or rows < (3 if n2 else 2 if n1 else 1):
        _refuse(what, "a row of positions for each section, and at most D / 2 pairs")
    if _bad_ints(positions, dev, (rows, T)):
        _refuse(what, "positions must be a contiguous int32 device tensor [axes, T]")
    if freqs.itemsize != 8 or not freqs.is_floating_point() or not freqs.is_contiguous() or \
            freqs.get_device() != dev:
        _refuse(what, "freqs must be a contiguous float64 device tensor")
    qw = kw = slot_ptr = v_ptr = vo_ptr = None
    if q_weight is not None:
        if _bad(q_weight, dev, dtype, q_weight.stride(), (D,)):
            _refuse(what, "weights [D]; " + _OPERANDS)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if _bad(k_weight, dev, dtype, k_weight.stride(), (D,)):
            _refuse(what, "weights [D]; " + _OPERANDS)
        kw = k_weight.data_ptr()
    rows = T
    if slots is not None:
        rows = k_out.shape[0]
        if _bad_ints(slots, dev, (T,)):
            _refuse(what, "slots must be a contiguous int32 device tensor [T]")
        slot_ptr = slots.data_ptr()
    qo, ko, vt, vo = (Hq * D, D), (Hk * D, D), (0, 0), (0, 0)
    if q_out is None:
        q_out = q.new_empty((T, Hq, D))
    else:
        qo = q_out.stride()
        if _bad(q_out, dev, dtype, qo, (T, Hq, D)):
            _refuse(what, "bad output tensor; " + _OPERANDS)
    if k_out is None:
        k_out = q.new_empty((T, Hk, D))
    else:
        ko = k_out.stride()
        if _bad(k_out, dev, dtype, ko, (rows, Hk, D)):
            _refuse(what, "bad output tensor; " + _OPERANDS)
    if v is not None:
        vt, vo = v.stride(), (Hk * D, D)
        if _bad(v, dev, dtype, vt, (T, Hk, D)):
            _refuse(what, "v [T, Hk, D]; " + _OPERANDS)
        if v_out is None:
            v_out = q.new_empty((T, Hk, D))
        else:
            vo = v_out.stride()
            if _bad(v_out, dev, dtype, vo, (rows, Hk, D)):
                _refuse(what, "v_out as k_out; " + _OPERANDS)
        v_ptr, vo_ptr = v.data_ptr(), v_out.data_ptr()
    elif v_out is not None:
        _refuse(what, "v_out without v")
    if T > 0:
        strides = _STRIDES12(qt[0], qt[1], kt[0], kt[1], vt[0], vt[1], qo[0], qo[1], ko[0], ko[1],
                             vo[0], vo[1])
        _run("libconv_qk_norm_rope", lib.libconv_qk_norm_rope,
             (q.data_ptr(), k.data_ptr(), v_ptr, q_out.data_ptr(), k_out.data_ptr(), vo_ptr, qw, kw,
              freqs.data_ptr(), positions.data_ptr(), slot_ptr, strides, T, Hq, Hk, D, 2 * pairs,
              n0, n1, n2, 1 if interleaved else 0, rows, eps, _codes[dtype]), dev, stream)
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def prefix_attention(q, k_prefix, v_prefix, k, v, lengths, scale: Optional[float] = None,
                     causal: bool = True, out=None, return_lse: bool = False, stream=None,
                     workspace=True):
    """Attention of q [B, Sq, Hq, D] over the shared k_prefix, v_prefix [P, Hk, D]
    and each entry's first lengths[b] (int32 [B]) rows of k, v [B, S, Hk, D].
    causal: query i sees the own keys up to lengths[b] - Sq + i.  k_prefix and
    v_prefix, or k and v, may be None (no such keys).  Returns out, or (out, lse
    [B, Hq, Sq] float32).  workspace: True (allocate what the best plan takes),
    False (none), or a uint8 device tensor."""
    what = "prefix_attention"
    lib, dev, dtype = _lib or _load(), q.get_device(), q.dtype
    qs, qt = q.shape, q.stride()
    if dev < 0 or len(qs) != 4 or dtype not in _codes or (qt[3] != 1 and qs[3] > 1):
        _refuse(what, "q [B, Sq, Hq, D]; " + _OPERANDS)
    B, Sq, Hq, D = qs
    if (k is None) != (v is None) or (k_prefix is None) != (v_prefix is None):
        _refuse(what, "keys and values come together")
    if k is None and k_prefix is None:
        _refuse(what, "neither a prefix nor own keys")
    P = S = Hk = 0
    kp_ptr = vp_ptr = k_ptr = v_ptr = None
    kp_st = vp_st = k_st = v_st = (0, 0, 0)
    if k is not None:
        ks, k_st, v_st = k.shape, k.stride(), v.stride()
        if len(ks) != 4:
            _refuse(what, "k, v [B, S, Hk, D]")
        S, Hk = ks[1], ks[2]
        shape = (B, S, Hk, D)
        if _bad(k, dev, dtype, k_st, shape) or _bad(v, dev, dtype, v_st, shape):
            _refuse(what, "k, v [B, S, Hk, D]; " + _OPERANDS)
        k_ptr, v_ptr = k.data_ptr(), v.data_ptr()
    if k_prefix is not None:
        ps, kp_st, vp_st = k_prefix.shape, k_prefix.stride(), v_prefix.stride()
        if len(ps) != 3:
            _refuse(what, "k_prefix, v_prefix [P, Hk, D]")
        P, Hk = ps[0], Hk if k is not None else ps[1]
        shape = (P, Hk, D)
        if _bad(k_prefix, dev, dtype, kp_st, shape) or _bad(v_prefix, dev, dtype, vp_st, shape):
            _refuse(what, "k_prefix, v_prefix [P, Hk, D]; " + _OPERANDS)
        kp_ptr, vp_ptr = k_prefix.data_ptr(), v_prefix.data_ptr()
    if _bad_ints(lengths, dev, (B,)):
        _refuse(what, "lengths must be a contiguous int32 device tensor [B]")
    if out is None:
        out, ot = q.new_empty(qs), (Sq * Hq * D, Hq * D, D)
    else:
        ot = out.stride()
        if _bad(out, dev, dtype, ot, qs):
            _refuse(what, "bad output tensor; " + _OPERANDS)
    lse = lse_ptr = buffer = None
    if return_lse:
        lse = q.new_empty((B, Hq, Sq), dtype=_float32)
        lse_ptr = lse.data_ptr()
    if B > 0 and Sq > 0:
        dt = _codes[dtype]
        if workspace is True:
            ws, size = None, _workspace_bytes("libconv_prefix_attention_workspace", B, Sq, P, S,
                                              Hq, Hk, D, dt)
            if size > 0:
                buffer = q.new_empty((size + 1) // 2 if dt else (size + 3) // 4)
                ws = buffer.data_ptr()
            else:   # none, or invalid sizes: the call says which
                size = 0
        else:
            ws, size = _given_workspace(workspace)
        strides = _STRIDES16(qt[0], qt[1], qt[2], kp_st[0], kp_st[1], vp_st[0], vp_st[1], k_st[0],
                             k_st[1], k_st[2], v_st[0], v_st[1], v_st[2], ot[0], ot[1], ot[2])
        _run("libconv_prefix_attention", lib.libconv_prefix_attention,
             (q.data_ptr(), kp_ptr, vp_ptr, k_ptr, v_ptr, lengths.data_ptr(), out.data_ptr(),
              lse_ptr, strides, B, Sq, P, S, Hq, Hk, D, D ** -0.5 if scale is None else scale,
              1 if causal else 0, dt, ws, size), dev, stream, buffer)
    return (out, lse) if return_lse else out


def lora_linear(x, w, bias, a, b, scales, row_starts, adapters, out=None, stream=None,
                workspace=True):
    """y = x w^T + bias + scales[i] (x a[i]^T) b[i]^T for the rows row_starts[r] ..
    row_starts[r + 1] - 1 of request r, whose adapter is i = adapters[r].
    x [T, K], w [N, K], a [n, rank, K], b [n, N, rank], scales float32 [n],
    row_starts int32 [R + 1], adapters int32 [R] (outside [0, n): none).
    a .. adapters may all be None: the projection alone."""
    what = "lora_linear"
    lib, dev, dtype = _lib or _load(), x.get_device(), x.dtype
    xs, xt = x.shape, x.stride()
    if dev < 0 or len(xs) != 2 or dtype not in _codes or (xt[1] != 1 and xs[1] > 1):
        _refuse(what, "x [T, K]; " + _OPERANDS)
    T, K = xs
    N = w.shape[0]
    if _bad(w, dev, dtype, w.stride(), (N, K)) or not w.is_contiguous():
        _refuse(what, "w must be a contiguous [N, K]; " + _OPERANDS)
    bias_ptr = a_ptr = b_ptr = scales_ptr = starts_ptr = adapters_ptr = None
    if bias is not None:
        if _bad(bias, dev, dtype, bias.stride(), (N,)):
            _refuse(what, "bias must be [N]; " + _OPERANDS)
        bias_ptr = bias.data_ptr()
    n = rank = R = 0
    if a is not None and b is not None and scales is not None and row_starts is not None and \
            adapters is not None:
        n, rank, _ = a.shape if a.dim() == 3 else (0, 0, 0)
        R = adapters.shape[0]
        if _bad(a, dev, dtype, a.stride(), (n, rank, K)) or not a.is_contiguous() or \
                _bad(b, dev, dtype, b.stride(), (n, N, rank)) or not b.is_contiguous():
            _refuse(what, "contiguous a [n, rank, K] and b [n, N, rank]; " + _OPERANDS)
        if scales.get_device() != dev or scales.shape != (n,) or \
                scales.dtype is not _float32 or not scales.is_contiguous():
            _refuse(what, "scales must be a contiguous float32 device tensor [n]")
        if _bad_ints(adapters, dev, (R,)) or _bad_ints(row_starts, dev, (R + 1,)):
            _refuse(what, "row_starts [R + 1] and adapters [R] must be contiguous int32 device "
                          "tensors")
        a_ptr, b_ptr, scales_ptr = a.data_ptr(), b.data_ptr(), scales.data_ptr()
        starts_ptr, adapters_ptr = row_starts.data_ptr(), adapters.data_ptr()
    elif not (a is None and b is None and scales is None and row_starts is None and
              adapters is None):
        _refuse(what, "a, b, scales, row_starts and adapters come together")
    y_stride = N
    if out is None:
        out = x.new_empty((T, N))
    else:
        ot = out.stride()
        if _bad(out, dev, dtype, ot, (T, N)):
            _refuse(what, "bad output tensor; " + _OPERANDS)
        y_stride = ot[0]
    if T > 0:
        dt, buffer = _codes[dtype], None
        if workspace is True:
            ws, size = None, _workspace_bytes("libconv_lora_workspace", T, K, N, rank, n, R, dt)
            if size > 0:
                buffer = x.new_empty((size + 1) // 2 if dt else (size + 3) // 4)
                ws = buffer.data_ptr()
            else:   # none, or invalid sizes: the call says which
                size = 0
        else:
            ws, size = _given_workspace(workspace)
        _run("libconv_lora_linear", lib.libconv_lora_linear,
             (x.data_ptr(), w.data_ptr(), bias_ptr, a_ptr, b_ptr, scales_ptr, starts_ptr,
              adapters_ptr, out.data_ptr(), T, K, N, rank, n, R, xt[0], y_stride, dt, ws, size), dev,
             stream, buffer)
    return out
