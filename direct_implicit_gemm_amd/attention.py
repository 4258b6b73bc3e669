"""Tensor-level helpers of the attention-layer operators of ``include/libconv.h``.

    lora_linear        a projection with each request's low-rank adapter beside it
    qk_norm_rope       norms of queries and keys, position rotation, cache write
    prefix_attention   attention over keys a batch shares and each entry's own

They allocate outputs (and workspaces, through torch), enqueue on the current
stream or ``stream`` (a handle), and raise ``LibconvError`` on a status other than
OK.  What they allocate for another ``stream`` than the current one is allocated
there, as under ``torch.cuda.stream``; an output may be dropped at any time.  That
the stream waits for the operands, and the reader for the stream, and that operands
live until the stream is done with them, is the caller's affair.
Tensors may be strided (slices of a fused projection, caches in any order of
axes) as long as their last axis is dense and their rows lie on 16-byte
boundaries.  There is no backward pass: libconv runs networks forward, and an
operand that requires gradients outside ``torch.no_grad()`` gets a warning.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

CALLS_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_torch_calls.so")
_calls = None


def _load():
    """The module that checks the tensors and calls libconv, bound to the loaded library."""
    import importlib.util

    import torch
    import direct_implicit_gemm_amd as L
    global _calls

    def stream_id(handle, device):
        return torch.cuda.ExternalStream(handle, device=device).stream_id

    def fail(status, what):
        raise L.LibconvError(status, what)

    lib = L.load()
    if not os.path.exists(CALLS_PATH):
        raise ImportError(f"{CALLS_PATH} is missing: build it with "
                          "`python -m direct_implicit_gemm_amd.build`")
    spec = importlib.util.spec_from_file_location("_torch_calls", CALLS_PATH)
    calls = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    functions = (lib.libconv_qk_norm_rope, lib.libconv_prefix_attention,
                 lib.libconv_prefix_attention_workspace, lib.libconv_lora_linear,
                 lib.libconv_lora_workspace)
    calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in functions),
               # as torch.cuda.current_stream() has it, without the object
               getattr(torch._C, "_cuda_getCurrentRawStream", None), stream_id, fail)
    _calls = calls
    return calls


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
    return (_calls or _load()).qk_norm_rope(
        q, k, positions, freqs, q_weight, k_weight, eps, sections, interleaved, v, slots, q_out,
        k_out, v_out, stream)


def prefix_attention(q, k_prefix, v_prefix, k, v, lengths, scale: Optional[float] = None,
                     causal: bool = True, out=None, return_lse: bool = False, stream=None,
                     workspace=True):
    """Attention of q [B, Sq, Hq, D] over the shared k_prefix, v_prefix [P, Hk, D]
    and each entry's first lengths[b] (int32 [B]) rows of k, v [B, S, Hk, D].
    causal: query i sees the own keys up to lengths[b] - Sq + i.  k_prefix and
    v_prefix, or k and v, may be None (no such keys).  Returns out, or (out, lse
    [B, Hq, Sq] float32).  workspace: True (allocate what the best plan takes),
    False (none), or a uint8 device tensor."""
    return (_calls or _load()).prefix_attention(
        q, k_prefix, v_prefix, k, v, lengths, scale, causal, out, return_lse, stream, workspace)


def lora_linear(x, w, bias, a, b, scales, row_starts, adapters, out=None, stream=None,
                workspace=True):
    """y = x w^T + bias + scales[i] (x a[i]^T) b[i]^T for the rows row_starts[r] ..
    row_starts[r + 1] - 1 of request r, whose adapter is i = adapters[r].
    x [T, K], w [N, K], a [n, rank, K], b [n, N, rank], scales float32 [n],
    row_starts int32 [R + 1], adapters int32 [R] (outside [0, n): none).
    a .. adapters may all be None: the projection alone."""
    return (_calls or _load()).lora_linear(
        x, w, bias, a, b, scales, row_starts, adapters, out, stream, workspace)
