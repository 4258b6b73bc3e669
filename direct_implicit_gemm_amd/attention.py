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


def _check(what, t, device, dtype, dims):
    """Device (its index), dtype and dense last axis of an operand."""
    if t.get_device() != device or device < 0:
        raise ValueError(f"{what}: operands must be device tensors of one device")
    if t.dtype != dtype:
        raise ValueError(f"{what}: operands must have one dtype")
    if t.dim() != dims or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{what}: expected {dims} axes with the last one dense")


def _ints(what, t, shape, device):
    import torch
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous() or \
            t.get_device() != device:
        raise ValueError(f"{what} must be a contiguous int32 device tensor of shape {shape}")
    return t.data_ptr()


class _Launch:
    """The stream and workspace of one call: ``stream`` is a handle (default: the
    current stream of the device), ``workspace`` True (allocate ``need`` bytes
    through torch), False / None (none) or a device tensor.  The calls are
    short: nothing here is done twice or for later."""

    __slots__ = ("stream", "ptr", "size", "_buffer", "_foreign", "_device")

    def __init__(self, device, stream, need, workspace):
        import torch
        self._device, self._foreign, self._buffer = device, stream is not None, None
        # the current stream's handle, as torch.cuda.current_stream() has it,
        # without the stream object
        self.stream = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream
        self.ptr, self.size = None, 0
        if workspace is True:
            if need > 0:
                self._buffer = torch.empty(need, dtype=torch.uint8, device=device)
                self.ptr, self.size = self._buffer.data_ptr(), need
        elif workspace is not None and workspace is not False:
            self.ptr = workspace.data_ptr()
            self.size = workspace.numel() * workspace.element_size()

    def run(self, what, function, *args):
        import torch
        if torch.cuda.current_device() == self._device:
            status = function(*args, self.stream)
        else:
            with torch.cuda.device(self._device):
                status = function(*args, self.stream)
        if self._foreign and self._buffer is not None:
            # its memory is that stream's until then
            self._buffer.record_stream(
                torch.cuda.ExternalStream(self.stream, device=self._device))
        if status != 0:
            raise _base().LibconvError(status, what)


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
    what = "qk_norm_rope"
    lib, dev, dtype = _base().load(), q.get_device(), q.dtype
    _check(what, q, dev, dtype, 3)
    _check(what, k, dev, dtype, 3)
    T, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape != (T, Hk, D):
        raise ValueError("qk_norm_rope: q [T, Hq, D], k and v [T, Hk, D]")
    if slots is not None and (k_out is None or (v is not None and v_out is None)):
        raise ValueError("qk_norm_rope: slots need k_out (and v_out)")
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    pairs = freqs.numel()
    n0, n1, n2, *more = list(sections) + [0, 0, 0] if sections is not None else (pairs, 0, 0)
    axes = 3 if n2 else 2 if n1 else 1
    if any(more) or n0 + n1 + n2 != pairs or min(n0, n1, n2) < 0 or 2 * pairs > D or \
            positions.shape[0] < axes:
        raise ValueError("qk_norm_rope: up to 3 sections that add up to the pairs of freqs, "
                         "with a row of positions each")
    pos_ptr = _ints("positions", positions, (positions.shape[0], T), dev)
    if freqs.dtype != torch.float64 or not freqs.is_contiguous() or freqs.get_device() != dev:
        raise ValueError("freqs must be a contiguous float64 device tensor")
    w_ptr = [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is not None:
            _check(what, w, dev, dtype, 1)
            if w.shape[0] != D:
                raise ValueError("qk_norm_rope: weights [D]")
            w_ptr[i] = w.data_ptr()
    rows, slot_ptr = T, None
    if slots is not None:
        rows, slot_ptr = k_out.shape[0], _ints("slots", slots, (T,), dev)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dtype, device=dev)
    else:
        _check(what, q_out, dev, dtype, 3)
    if k_out is None:
        k_out = torch.empty((T, Hk, D), dtype=dtype, device=dev)
    else:
        _check(what, k_out, dev, dtype, 3)
    if q_out.shape != q.shape or k_out.shape != (rows, Hk, D):
        raise ValueError("qk_norm_rope: bad output tensor")
    v_ptr = vo_ptr = None
    v_st = vo_st = (0, 0, 0)
    if v is not None:
        _check(what, v, dev, dtype, 3)
        v_out = torch.empty((T, Hk, D), dtype=dtype, device=dev) if v_out is None else v_out
        _check(what, v_out, dev, dtype, 3)
        if v.shape != k.shape or v_out.shape != (rows, Hk, D):
            raise ValueError("qk_norm_rope: v [T, Hk, D] and v_out as k_out")
        v_ptr, vo_ptr, v_st, vo_st = v.data_ptr(), v_out.data_ptr(), v.stride(), v_out.stride()
    elif v_out is not None:
        raise ValueError("qk_norm_rope: v_out without v")
    result = (q_out, k_out) if v is None else (q_out, k_out, v_out)
    if T == 0:
        return result
    a, b, c, d = q.stride(), k.stride(), q_out.stride(), k_out.stride()
    strides = _STRIDES12(a[0], a[1], b[0], b[1], v_st[0], v_st[1], c[0], c[1], d[0], d[1],
                         vo_st[0], vo_st[1])
    _Launch(dev, stream, 0, False).run(
        "libconv_qk_norm_rope", lib.libconv_qk_norm_rope, q.data_ptr(), k.data_ptr(), v_ptr,
        q_out.data_ptr(), k_out.data_ptr(), vo_ptr, w_ptr[0], w_ptr[1], freqs.data_ptr(), pos_ptr,
        slot_ptr, strides, T, Hq, Hk, D, 2 * pairs, n0, n1, n2, 1 if interleaved else 0, rows,
        eps, _base()._dtype_code(q))
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
    what = "prefix_attention"
    L = _base()
    lib, dev, dtype = L.load(), q.get_device(), q.dtype
    _check(what, q, dev, dtype, 4)
    B, Sq, Hq, D = q.shape
    if (k is None) != (v is None) or (k_prefix is None) != (v_prefix is None):
        raise ValueError("prefix_attention: keys and values come together")
    if k is None and k_prefix is None:
        raise ValueError("prefix_attention: neither a prefix nor own keys")
    Hk = (k if k is not None else k_prefix).shape[-2]
    P = S = 0
    kp_ptr = vp_ptr = k_ptr = v_ptr = None
    kp_st = vp_st = k_st = v_st = (0, 0, 0)
    if k_prefix is not None:
        _check(what, k_prefix, dev, dtype, 3)
        _check(what, v_prefix, dev, dtype, 3)
        P = k_prefix.shape[0]
        if k_prefix.shape != (P, Hk, D) or v_prefix.shape != (P, Hk, D):
            raise ValueError("prefix_attention: k_prefix, v_prefix [P, Hk, D]")
        kp_ptr, vp_ptr = k_prefix.data_ptr(), v_prefix.data_ptr()
        kp_st, vp_st = k_prefix.stride(), v_prefix.stride()
    if k is not None:
        _check(what, k, dev, dtype, 4)
        _check(what, v, dev, dtype, 4)
        S = k.shape[1]
        if k.shape != (B, S, Hk, D) or v.shape != (B, S, Hk, D):
            raise ValueError("prefix_attention: k, v [B, S, Hk, D]")
        k_ptr, v_ptr, k_st, v_st = k.data_ptr(), v.data_ptr(), k.stride(), v.stride()
    len_ptr = _ints("lengths", lengths, (B,), dev)
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=dtype, device=dev)
    else:
        _check(what, out, dev, dtype, 4)
        if out.shape != q.shape:
            raise ValueError("prefix_attention: bad output tensor")
    lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=dev) if return_lse else None
    if B == 0 or Sq == 0:
        return (out, lse) if return_lse else out
    dt = L._dtype_code(q)
    need = lib.libconv_prefix_attention_workspace(B, Sq, P, S, Hq, Hk, D, dt) \
        if workspace is True else 0
    a, o = q.stride(), out.stride()
    strides = _STRIDES16(a[0], a[1], a[2], kp_st[0], kp_st[1], vp_st[0], vp_st[1], k_st[0],
                         k_st[1], k_st[2], v_st[0], v_st[1], v_st[2], o[0], o[1], o[2])
    call = _Launch(dev, stream, need, workspace)
    call.run("libconv_prefix_attention", lib.libconv_prefix_attention, q.data_ptr(), kp_ptr,
             vp_ptr, k_ptr, v_ptr, len_ptr, out.data_ptr(), L._ptr(lse), strides, B, Sq, P, S, Hq,
             Hk, D, D ** -0.5 if scale is None else scale, 1 if causal else 0, dt, call.ptr,
             call.size)
    return (out, lse) if return_lse else out


def lora_linear(x, w, bias, a, b, scales, row_starts, adapters, out=None, stream=None,
                workspace=True):
    """y = x w^T + bias + scales[i] (x a[i]^T) b[i]^T for the rows row_starts[r] ..
    row_starts[r + 1] - 1 of request r, whose adapter is i = adapters[r].
    x [T, K], w [N, K], a [n, rank, K], b [n, N, rank], scales float32 [n],
    row_starts int32 [R + 1], adapters int32 [R] (outside [0, n): none).
    a .. adapters may all be None: the projection alone."""
    import torch
    what = "lora_linear"
    L = _base()
    lib, dev, dtype = L.load(), x.get_device(), x.dtype
    _check(what, x, dev, dtype, 2)
    _check(what, w, dev, dtype, 2)
    T, K = x.shape
    N = w.shape[0]
    if w.shape != (N, K) or not w.is_contiguous():
        raise ValueError("lora_linear: w must be a contiguous [N, K]")
    if bias is not None:
        _check(what, bias, dev, dtype, 1)
        if bias.shape[0] != N:
            raise ValueError("lora_linear: bias must be [N]")
    n = rank = R = 0
    a_ptr = b_ptr = scales_ptr = starts_ptr = adapters_ptr = None
    given = [t is not None for t in (a, b, scales, row_starts, adapters)]
    if all(given):
        _check(what, a, dev, dtype, 3)
        _check(what, b, dev, dtype, 3)
        n, rank = a.shape[0], a.shape[1]
        if a.shape != (n, rank, K) or b.shape != (n, N, rank) or not a.is_contiguous() or \
                not b.is_contiguous():
            raise ValueError("lora_linear: contiguous a [n, rank, K] and b [n, N, rank]")
        if scales.dtype != torch.float32 or scales.shape != (n,) or \
                not scales.is_contiguous() or scales.get_device() != dev:
            raise ValueError("lora_linear: scales must be a contiguous float32 device tensor [n]")
        R = adapters.shape[0]
        adapters_ptr = _ints("adapters", adapters, (R,), dev)
        starts_ptr = _ints("row_starts", row_starts, (R + 1,), dev)
        a_ptr, b_ptr, scales_ptr = a.data_ptr(), b.data_ptr(), scales.data_ptr()
    elif any(given):
        raise ValueError("lora_linear: a, b, scales, row_starts and adapters come together")
    if out is None:
        out = torch.empty((T, N), dtype=dtype, device=dev)
    else:
        _check(what, out, dev, dtype, 2)
        if out.shape != (T, N):
            raise ValueError("lora_linear: bad output tensor")
    if T == 0:
        return out
    dt = L._dtype_code(x)
    need = lib.libconv_lora_workspace(T, K, N, rank, n, R, dt) if workspace is True else 0
    call = _Launch(dev, stream, need, workspace)
    call.run("libconv_lora_linear", lib.libconv_lora_linear, x.data_ptr(), w.data_ptr(),
             L._ptr(bias), a_ptr, b_ptr, scales_ptr, starts_ptr, adapters_ptr, out.data_ptr(), T,
             K, N, rank, n, R, x.stride(0), out.stride(0), dt, call.ptr, call.size)
    return out
