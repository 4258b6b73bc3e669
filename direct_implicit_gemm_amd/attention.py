"""Tensor-level helpers of the attention-layer operators of ``include/libconv.h``.

    lora_linear        a projection with each request's low-rank adapter beside it
    qk_norm_rope       norms of queries and keys, position rotation, cache write
    prefix_attention   attention over keys a batch shares and each entry's own
    kv_cache_write     keys and values of new tokens into a cache of 8-bit blocks
    kv_cache_read      ... and back, in the activations' type
    cache_attention    attention of a ragged batch over such a cache
    linear             a projection with bias, activation and residual

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
                 lib.libconv_lora_workspace, lib.libconv_kv_cache_write, lib.libconv_kv_cache_read,
                 lib.libconv_cache_attention, lib.libconv_cache_attention_workspace,
                 lib.libconv_linear, lib.libconv_linear_workspace)
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


def kv_cache_write(k, v, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table,
                   stream=None):
    """Appends rows k, v [T, Hk, D] to a cache of codes (int8 or float8_e4m3fn)
    k_cache, v_cache [blocks, block, Hk, D] with scales k_scale, v_scale (float32
    [blocks, Hk]).  Entry b has rows row_starts[b] .. row_starts[b + 1] - 1 (int32
    [B + 1]), which become the last of its lengths[b] (int32 [B]) tokens; position p
    lies in block block_table[b, p // block] (int32 [B, any]).  A block's scale is the
    least power of two that holds its largest value, and grows with new tokens.

        shape = (blocks, heads, block, head_dim)     # each head's tokens side by side
        k_cache = torch.zeros(shape, dtype=torch.int8, device="cuda").transpose(1, 2)
        k_scale = torch.zeros(blocks, heads, device="cuda")"""
    return (_calls or _load()).kv_cache_write(
        k, v, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table, stream)


def kv_cache_read(k_cache, v_cache, k_scale, v_scale, lengths, block_table, k_out=None, v_out=None,
                  dtype=None, rows: Optional[int] = None, stream=None):
    """The first lengths[b] tokens of every entry, as prefix_attention takes them:
    (k_out, v_out) [B, S, Hk, D].  Rows from lengths[b] on are left as they were.
    Outputs not given are made, zero where nothing is written, of `dtype` (bfloat16)
    with S = rows (all positions of the table)."""
    like = None
    if k_out is None or v_out is None:
        import torch
        like = torch.empty(0, dtype=torch.bfloat16 if dtype is None else dtype)
    return (_calls or _load()).kv_cache_read(
        k_cache, v_cache, k_scale, v_scale, lengths, block_table, k_out, v_out, like, rows, stream)


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table,
                    max_rows: Optional[int] = None, scale: Optional[float] = None,
                    causal: bool = True, out=None, return_lse: bool = False, stream=None,
                    workspace=True):
    """Attention of q [T, Hq, D] over a cache (see kv_cache_write): row t of entry b
    over the entry's lengths[b] tokens, causal: up to its own position.  max_rows: the
    rows of the entry with the most (T will do; 1 for single tokens plans best).
    Returns out, or (out, lse [T, Hq] float32); rows of no entry are not written.
    workspace: True (allocate what the best plan takes), False (none), or a uint8
    device tensor."""
    return (_calls or _load()).cache_attention(
        q, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table, max_rows, scale,
        causal, out, return_lse, stream, workspace)


_LINEAR_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def linear(x, w, bias=None, act: str = "none", residual=None, out=None, stream=None,
           workspace=True):
    """y = act(x w^T + bias) + residual for x [T, K], w [N, K], bias [N], residual
    [T, N] (out may be the residual).  act: none, relu, gelu, gelu_tanh or silu."""
    number = _LINEAR_ACTS.get(act)
    if number is None:
        raise ValueError(f"linear: act must be one of {', '.join(_LINEAR_ACTS)}")
    return (_calls or _load()).linear(x, w, bias, number, residual, out, stream, workspace)
