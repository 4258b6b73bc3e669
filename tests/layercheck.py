"""Plain 64-bit forms of the attention-layer operators and the error each result may have.

The bounds count roundings: half a step of a type relative to the value (U),
and for a sum of n products in fp32 at most n half steps of 2^-24 of the sum
of their magnitudes."""
import math

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {t: torch.finfo(t).eps / 2 for t in TYPES.values()}
U32 = 2.0 ** -24


def tiny(t):
    """Half a step of the smallest numbers of a type (results near 0)."""
    return torch.finfo(t).tiny * U[t] * 2


def attention(q, kp, vp, k, v, lengths, scale, causal):
    """(out, its bound, lse, its bound) in 64 bits, on the CPU."""
    t = q.dtype
    q = q.double().cpu()
    B, Sq, Hq, D = q.shape
    Hk = (k if k is not None else kp).shape[-2]
    P = 0 if kp is None else kp.shape[0]
    out, bound = torch.zeros(B, Sq, Hq, D).double(), torch.zeros(B, Sq, Hq, D).double()
    lse, lse_bound = torch.full((B, Hq, Sq), -math.inf).double(), torch.zeros(B, Hq, Sq).double()
    dense = lambda x: None if x is None else x.double().cpu()
    kp, vp, k, v = dense(kp), dense(vp), dense(k), dense(v)
    for b, n in enumerate(lengths.tolist()):
        n = max(0, min(n, 0 if k is None else k.shape[1]))
        for h in range(Hq):
            g = h // (Hq // Hk)
            keys = torch.cat(([kp[:, g]] if P else []) + ([k[b, :n, g]] if n else [])) \
                if P or n else torch.zeros(0, D).double()
            vals = torch.cat(([vp[:, g]] if P else []) + ([v[b, :n, g]] if n else [])) \
                if P or n else torch.zeros(0, D).double()
            if not len(keys):
                continue
            s = scale * q[b, :, h] @ keys.t()
            size = abs(scale) * q[b, :, h].abs() @ keys.abs().t()
            seen = torch.ones(Sq, P + n, dtype=torch.bool)
            if causal:
                i, j = torch.arange(Sq)[:, None], torch.arange(n)[None, :]
                seen[:, P:] = j <= n - Sq + i
            some = seen.any(-1)
            if not some.any():
                continue
            s = s.masked_fill(~seen, -math.inf)
            p = torch.where(some[:, None], torch.softmax(s, -1), torch.zeros(()).double())
            mag = p @ vals.abs()
            # a score is off by D + 4 half steps of the size of its products, which every
            # probability and their sum take over; the probabilities are rounded to the type
            # once, sums of P + n terms and the joins to fp32, the output to the type
            a = torch.where(seen, size, torch.zeros(()).double()).amax(-1)
            off = U32 * (2 * (D + 4) * a + 2 * (P + n) + 64)
            out[b, :, h] = p @ vals
            bound[b, :, h] = (2 * U[t] + off)[:, None] * mag + tiny(t)
            lse[b, h] = torch.where(some, torch.logsumexp(s, -1), torch.full((), -math.inf).double())
            lse_bound[b, h] = off + U32 * 8 * (1 + a)
    return out, bound, lse, lse_bound


def rope(x, weight, positions, freqs, sections, eps, interleaved):
    """(out, bound) of one operand [T, H, D], in 64 bits on the CPU."""
    t = x.dtype
    x, D, half = x.double().cpu(), x.shape[-1], freqs.numel()
    w = torch.ones(D).double() if weight is None else weight.double().cpu()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    pos = positions.double().cpu()
    pos = pos if pos.dim() == 2 else pos[None]
    axis = torch.tensor([a for a, m in enumerate(sections) for _ in range(m)], dtype=torch.long)
    angle = pos[axis].t() * freqs.cpu() if half else torch.zeros(x.shape[0], 0).double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    first = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
    second = first + 1 if interleaved else first + half
    out, mag = n.clone(), n.abs()
    out[..., first] = n[..., first] * c - n[..., second] * s
    out[..., second] = n[..., second] * c + n[..., first] * s
    pair = n[..., first].abs() + n[..., second].abs()
    mag[..., first] = pair
    mag[..., second] = pair
    # the sum of D squares, root, division, two products; cos and sin are off by at most
    # 8 half steps of 1 (the reduced angle's rounding, up to pi, and the functions' own)
    return out, U[t] * out.abs() + U32 * (D / 2 + 24) * mag + tiny(t)


def lora(x, w, bias, a, b, scales, starts, ids):
    """(y, bound), in 64 bits on the CPU."""
    t = x.dtype
    x, w = x.double().cpu(), w.double().cpu()
    K = x.shape[1]
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    off = U32 * (K + 8) * mag
    if bias is not None:
        y = y + bias.double().cpu()
        off = off + U32 * 4 * bias.double().cpu().abs()
    if a is not None:
        n, r = a.shape[0], a.shape[1]
        st = starts.tolist()
        for i, lo, hi in zip(ids.tolist(), st, st[1:]):
            if not 0 <= i < n or hi <= lo:
                continue
            A, Bm, s = a[i].double().cpu(), b[i].double().cpu(), scales[i].double().cpu()
            low = x[lo:hi] @ A.t()
            size = s.abs() * (x[lo:hi].abs() @ A.abs().t())
            y[lo:hi] += s * low @ Bm.t()
            # low-rank values: K half steps of fp32, then two bfloat16 terms (16 bits) on
            # either side for the 16-bit types
            parts = 0.0 if t == torch.float32 else 3 * 2.0 ** -16
            off[lo:hi] += U32 * (K + 3 * r + 16) * (size @ Bm.abs().t()) + \
                parts * (s * low).abs() @ Bm.abs().t()
    return y, U[t] * y.abs() + (1 + U[t]) * off + tiny(t)


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    same = (got == want)   # infinities
    bad &= ~same
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        worst = float(((got - want).abs() / bound)[bad].max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: "
                             f"{float(got[at])} for {float(want[at])}, worst {worst:.3g} bounds")
