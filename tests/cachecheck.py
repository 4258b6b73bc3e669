"""Plain 64-bit forms of the operators around the 8-bit cache of keys and values, and of the
projection with activation and residual, with the error each result may have.

The bounds count roundings, as in layercheck: half a step of a type relative to the value (U), and
for a sum of n products in fp32 at most n half steps of 2^-24 of the sum of their magnitudes."""
import math

import torch

from layercheck import TYPES, U, U32, assert_within, tiny  # noqa: F401  (the tests' names)

CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
MOST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
# roundings of a probability for the second product: one bfloat16 term, one fp16 number (of a few
# rows: two bfloat16 terms, 2^-16, which is less), three bfloat16 terms
P_ROUNDING = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


class Cache:
    """A cache on the GPU: codes [blocks, block, Hk, D] (each head's tokens of a block side by
    side, or, tokens_first, each token's heads), scales, the entries' table."""

    def __init__(self, B, lengths, block, hk, d, codes, seed=0, tokens_first=False, spare=3,
                 width=None, empty=False):
        g = torch.Generator().manual_seed(seed)
        longest = max([1] + [n for n in lengths])
        self.width = -(-longest // block) if width is None else width
        blocks = B * self.width + spare
        self.block = block
        for name in ("k", "v"):
            x = torch.randint(-127, 128, (blocks, hk, block, d), generator=g)
            if codes == "e4m3":
                x = (x / 16.0).exp2() * torch.randint(0, 2, x.shape, generator=g).mul(2).sub(1)
                x = x.clamp(-448, 448)
            x = x.float().to(CODES[codes])
            if empty:
                x = torch.zeros_like(x)
            x = x.transpose(1, 2).contiguous() if tokens_first else x
            x = x.cuda()
            setattr(self, name, x if tokens_first else x.transpose(1, 2))
            scale = torch.randint(-9, -5, (blocks, hk), generator=g).float().exp2()
            setattr(self, name + "s", scale.cuda())
        self.table = torch.randperm(blocks, generator=g)[:B * self.width].view(B, -1).int().cuda()
        self.lengths = torch.tensor(lengths).int().cuda()

    def operands(self):
        return self.k, self.v, self.ks, self.vs

    def host(self, name):
        """(codes as 64-bit values, scales) on the CPU."""
        return getattr(self, name).cpu().float().double(), getattr(self, name + "s").cpu().double()


def starts(rows):
    return torch.tensor([0] + rows).cumsum(0).int().cuda()


def of_entry(cache, b, name):
    """(values [n, Hk, D] in 64 bits, which positions lie in a block)."""
    codes, scale = getattr(cache, name), getattr(cache, name + "s").cpu().double()
    table = cache.table[b].cpu().long()
    n = max(0, min(int(cache.lengths[b]), table.numel() * cache.block))
    p = torch.arange(n)
    at = table[p // cache.block]
    there = (at >= 0) & (at < len(codes))
    at = torch.where(there, at, torch.zeros_like(at))
    used, of = at.unique(return_inverse=True)   # (the entry's blocks only: caches are large)
    part = codes.view(torch.uint8)[used.to(codes.device)].view(codes.dtype).cpu().float().double()
    value = part[of, p % cache.block] * scale[at][..., None]
    return torch.where(there[:, None, None], value, torch.zeros(()).double()), there


def round_codes(x, codes):
    """To the nearest code, ties to even; infinities the largest, NaN 0 or NaN."""
    most = MOST[codes]
    if codes == torch.int8:
        return torch.nan_to_num(x, nan=0.0, posinf=most, neginf=-most).round().clamp(-most, most)
    y = x.clamp(-most, most)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = (e - 3).exp2()
    y = (y / step).round() * step   # (a sum that reaches the next power of two is one of its codes)
    return torch.where(torch.isnan(x), x, y)


def scale_of(top, codes):
    """The least power of two >= 2^-126 with top / 2^e <= the largest code."""
    e = -126
    while top > MOST[codes] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def write(cache, k, v, row_starts):
    """(codes as values, scales) of keys and of values after the call, in 64 bits."""
    out = []
    st = row_starts.tolist()
    for name, x in (("k", k), ("v", v)):
        codes, scale = cache.host(name)
        t = getattr(cache, name).dtype
        x = x.double().cpu()
        for b, n in enumerate(cache.lengths.tolist()):
            width = cache.table.shape[1]
            n = max(0, min(n, width * cache.block))
            lo, hi = max(0, st[b]), min(len(x), st[b + 1])
            for i in range(width):
                p0, p1 = i * cache.block, (i + 1) * cache.block
                at = int(cache.table[b, i])
                rows = [r for r in range(lo, hi) if p0 <= n - hi + r < p1]
                if not rows or not 0 <= at < len(codes):
                    continue
                first = n - hi + rows[0] - p0
                for h in range(x.shape[1]):
                    new = x[rows, h]
                    fine = new[torch.isfinite(new)].abs()
                    s = scale_of(float(fine.max()) if fine.numel() else 0.0, t)
                    if first > 0:
                        old = float(scale[at, h])
                        old = old if math.isfinite(old) and old > 0 else 0.0
                        s = max(s, old)
                        if s != old:
                            codes[at, :first, h] = round_codes(codes[at, :first, h] * (old / s), t)
                    codes[at, first:first + len(rows), h] = round_codes(new / s, t)
                    scale[at, h] = s
        out.append((codes, scale))
    return out


def attention(q, cache, row_starts, scale, causal):
    """(out, its bound, lse, its bound) in 64 bits; rows of no entry are NaN."""
    t = q.dtype
    q = q.double().cpu()
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), math.nan).double()
    lse = torch.full((T, Hq), math.nan).double()
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    terms = 3 if t == torch.float32 else 1
    st = row_starts.tolist()
    for b in range(len(st) - 1):
        lo, hi = max(0, st[b]), min(T, st[b + 1])
        if hi <= lo:
            continue
        k, there = of_entry(cache, b, "k")
        v, _ = of_entry(cache, b, "v")
        n, Hk = k.shape[0], cache.k.shape[2]
        seen = there[None].expand(hi - lo, -1)
        if causal:
            i = torch.arange(hi - lo)[:, None]
            seen = seen & (torch.arange(n)[None] <= n - (hi - lo) + i)
        some = seen.any(-1) if n else torch.zeros(hi - lo, dtype=torch.bool)
        zero = torch.zeros(()).double()
        for h in range(Hq):
            g = h // (Hq // Hk)
            x = q[lo:hi, h]
            if not n:
                out[lo:hi, h], lse[lo:hi, h] = 0.0, -math.inf
                continue
            s = (scale * x @ k[:, g].t()).masked_fill(~seen, -math.inf)
            size = abs(scale) * x.abs() @ k[:, g].abs().t()
            p = torch.where(some[:, None], torch.softmax(s, -1), zero)
            a = torch.where(seen, size, zero).amax(-1)
            # a score is off by a half step of its products for each sum of D * terms products
            # and a few more for its scales, which every probability and their sum take over;
            # sums of n terms and the joins in fp32
            off = U32 * (2 * (terms * D + 8) * a + 2 * n + 64)
            mag = p @ v[:, g].abs()
            out[lo:hi, h] = p @ v[:, g]
            # a probability (or it times its scale) below 2^-126 is 0 in the matrix
            # instructions, which take numbers that small for 0: n terms of less than 2^-126
            # times a code (or a value) are missing then
            gone = n * 2.0 ** -126 * (448 + v[:, g].abs().amax())
            if t == torch.float16:
                # as fp16 numbers, probabilities are multiplied by 2^11 relative to a maximum that
                # theirs is not below: below 2^-14 each is off by half of fp16's last step, 2^-25,
                # so 2^-36 of a sum that is 1 at least
                gone = gone + n * 2.0 ** -36 * v[:, g].abs().amax()
            bound[lo:hi, h] = (U[t] + P_ROUNDING[t] + off)[:, None] * mag + tiny(t) + gone
            lse[lo:hi, h] = torch.where(some, torch.logsumexp(s, -1), torch.full((), -math.inf).double())
            lse_bound[lo:hi, h] = off + U32 * 8 * (1 + a)
    return out, bound, lse, lse_bound


def activation(v, act):
    """(act(v), how much an error of v counts, the error of act itself) in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v), torch.zeros_like(v)
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), torch.ones_like(v), torch.zeros_like(v)
    if act == "gelu":
        # 1 + erf: erf is off by 4 half steps of 1 at most, and so is the sum
        return v * torch.special.ndtr(v), 1.13 * torch.ones_like(v), U32 * 6 * v.abs()
    # v / (1 + exp(-u)): the exponent is off by half steps of |u| log2 e (3 of them, and one of the
    # function's own), the sum and the quotient by one or two
    u = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    s = torch.sigmoid(u)
    own = U32 * (6 + 6 * u.abs()) * (v * s).abs()
    # below 2^-126 the reciprocal is 0
    return v * s, 1.13 * torch.ones_like(v), own + v.abs() * 2.0 ** -125


def linear(x, w, bias, act, residual):
    """(y, bound) in 64 bits on the CPU."""
    t = x.dtype
    x, w = x.double().cpu(), w.double().cpu()
    v, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        v, mag = v + bias.double().cpu(), mag + bias.double().cpu().abs()
    y, slope, own = activation(v, act)
    off = slope * U32 * (x.shape[1] + 8) * mag + own
    if residual is not None:
        r = residual.double().cpu()
        y, off = y + r, off + U32 * (y.abs() + (y + r).abs())
    return y, U[t] * y.abs() + (1 + U[t]) * off + tiny(t)
