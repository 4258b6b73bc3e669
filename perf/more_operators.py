"""Measured cases of the operators around an 8-bit cache of keys and values: what a caller has in
hand, one pass through each operator, and its plain form in elementary torch operations.

Three operators of a decoder layer that answers many prompts:
  cache      keys and values of new tokens appended to a cache of 8-bit blocks, each with a power
             of two as its scale for every head, and all entries read back for dense attention
  attention  attention of a ragged batch (prompts and single tokens) over such a cache
  linear     a projection with bias, activation and residual: the output projection and the MLP

`own` selects between the plain form (False) and the calls of the package (True).
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
_MOST = {"i8": 127.0, "e4m3": 448.0}  # the largest code


# ------------------------------------------------------------------------------------- the cases
def _cache(B, n, rows, lo, hi, hk, d, block, codes, dtype):
    return {"op": "cache", "B": B, "n": n, "rows": rows, "lo": lo, "hi": hi, "hk": hk, "d": d,
            "block": block, "codes": codes, "dtype": dtype}


def _attention(B, n, rows, lo, hi, hq, hk, d, block, causal, codes, dtype):
    return {"op": "attention", "B": B, "n": n, "rows": rows, "lo": lo, "hi": hi, "hq": hq,
            "hk": hk, "d": d, "block": block, "causal": causal, "codes": codes, "dtype": dtype}


def _linear(T, K, N, act, bias, residual, dtype):
    return {"op": "linear", "T": T, "K": K, "N": N, "act": act, "bias": bias,
            "residual": residual, "dtype": dtype}


def listed():
    return [
        # one decoding step of 64 requests, ragged lengths, and a snapshot of all of them
        {"name": "cache decode 64", **_cache(64, 1, "all", 1, 2048, 8, 128, 16, "e4m3", "bf16")},
        # chunks of 9 prompts behind what they have, heads of 80, read back for dense attention
        {"name": "cache chunks i8", **_cache(9, 517, "ragged", 300, 1400, 4, 80, 32, "i8", "f16")},
        # 12 windows of a video's tokens written at once and read back
        {"name": "cache windows", **_cache(12, 3200, "all", 3200, 3200, 20, 128, 64, "e4m3",
                                           "bf16")},
        # one decoding step of 4 prompts about one page's features: latency
        {"name": "attention decode 4", **_attention(4, 1, "all", 961, 1000, 20, 20, 64, 32, True,
                                                    "i8", "bf16")},
        # one decoding step of 64 requests of very different lengths, shared heads of keys
        {"name": "attention decode 64", **_attention(64, 1, "all", 1, 8192, 32, 8, 128, 16, True,
                                                     "e4m3", "bf16")},
        # two long documents, one token each: the keys have to be split
        {"name": "attention long i8", **_attention(2, 1, "all", 65537, 131072, 16, 4, 128, 64,
                                                   True, "i8", "bf16")},
        # a batch in service: half of it decodes, the others read chunks of their prompts
        {"name": "attention mixed f16", **_attention(9, 517, "mixed", 300, 4096, 16, 4, 80, 32,
                                                     True, "e4m3", "f16")},
        # short texts in single precision
        {"name": "attention f32", **_attention(2, 130, "all", 463, 523, 8, 8, 64, 16, True, "i8",
                                               "f32")},
        # prompts read in at once behind what they have in the cache
        {"name": "attention prompts", **_attention(8, 2048, "all", 2048, 6144, 32, 8, 128, 64,
                                                   True, "e4m3", "bf16")},
        # one decoding step of 64 requests: the output projection added to the residual stream
        {"name": "linear decode 64", **_linear(64, 4096, 4096, "none", False, True, "bf16")},
        # two 32x32 maps of 1280 channels and a ragged tail of text rows, into an MLP, in half
        {"name": "linear ragged f16", **_linear(2167, 1280, 3840, "gelu", True, False, "f16")},
        # prompts read in at once, through an MLP's first product
        {"name": "linear prefill", **_linear(8192, 4096, 8192, "gelu_tanh", True, True, "bf16")},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache", "attention", "attention", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    codes, block = rng.choice(["i8", "e4m3"]), rng.choice([16, 32, 64, 128])
    most = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        hk, d = _log(rng, 1, 20), rng.choice([64, 80, 128])
        rows = rng.choice(["all", "ragged", "mixed"])
        if op == "linear":
            c = _linear(_log(rng, 1, 8192), 8 * _log(rng, 16, 512), _log(rng, 64, 8192),
                        rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                        rng.random() < 0.5, rng.random() < 0.5, dtype)
        elif op == "cache":
            hi = _log(rng, 1, 8192)
            c = _cache(_log(rng, 1, 64), rng.choice([1, _log(rng, 1, 3200)]), rows,
                       _log(rng, 1, hi), hi, hk, d, block, codes, dtype)
        else:
            hi = _log(rng, 1, 131072)
            c = _attention(_log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 2048)]), rows,
                           _log(rng, 1, hi), hi, hk * rng.choice([1, 2, 4, 8]), hk, d, block,
                           rng.random() < 0.7, codes, dtype)
        w = work(c)
        slow = 8 if dtype == "f32" and op == "linear" else 4 if dtype == "f32" else 1
        if op != "linear" and _room(c) > 1 << 29:  # the plain form holds all of it in 32 bits
            continue
        if op == "attention" and c["B"] * c["n"] * c["hq"] * _longest(c) > 3 << 30:
            continue                               # and every score
        if slow * w["flops"] <= most["flops"] and (op == "linear" or w["bytes"] <= most["bytes"]):
            return c


def _spread(case):
    """(new tokens, tokens in all) of each entry: new ones 1 to n, lengths from lo to hi."""
    B, n, lo, hi = (case[k] for k in ("B", "n", "lo", "hi"))
    got = []
    for b in range(B):
        length = hi if B == 1 else lo + (hi - lo) * b // (B - 1)
        new = n
        if case["rows"] == "ragged":
            new = 1 + (n - 1) * ((5 * b + 3) % B) // max(1, B - 1)
        elif case["rows"] == "mixed" and b % 2 == 0:
            new = 1
        got.append((new, max(new, length)))
    return got


def _longest(case):
    return max(length for _, length in _spread(case))


def _room(case):
    """Elements of keys in a table of blocks for every entry."""
    return case["B"] * (_longest(case) + case["block"]) * case["hk"] * case["d"]


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": e * (T * K + N * K + T * N * (2 if case["residual"] else 1) +
                              (N if case["bias"] else 0)),
                "flops": 2 * T * K * N}
    hk, d, block = case["hk"], case["d"], case["block"]
    new, keys = (sum(x) for x in zip(*_spread(case)))
    scales = 8 * hk * sum(-(-length // block) for _, length in _spread(case))
    if case["op"] == "cache":
        # the new rows read and their codes written; all codes read and their values written
        return {"bytes": 2 * hk * d * (new * (e + 1) + keys * (1 + e)) + scales,
                "flops": 4 * hk * d * (new + keys)}
    hq = case["hq"]
    pairs = sum(n * length - (n * (n - 1) // 2 if case["causal"] else 0)
                for n, length in _spread(case))
    return {"bytes": 2 * e * d * hq * new + 2 * d * hk * keys + scales, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------------- their inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(t)

    s = {"case": dict(case)}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        s.update(x=normal(T, K), w=normal(N, K, by=K ** -0.5),
                 bias=normal(N, by=0.05) if case["bias"] else None,
                 residual=normal(T, N) if case["residual"] else None)
        return s
    B, hk, d, block = (case[k] for k in ("B", "hk", "d", "block"))
    pairs = _spread(case)
    pairs = [pairs[i] for i in torch.randperm(B, generator=h).tolist()]
    new, lengths = torch.tensor([p[0] for p in pairs]), torch.tensor([p[1] for p in pairs])
    width = -(-int(lengths.max()) // block)
    blocks = B * width + 3
    starts = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
    # blocks of an entry lie anywhere in the cache, a head's tokens of a block one after another
    table = torch.randperm(blocks, generator=h)[:B * width].view(B, width)
    s.update(starts=starts.int().cuda(), lengths=lengths.int().cuda(), table=table.int().cuda(),
             max_rows=int(new.max()))
    for name in ("k", "v"):
        # what the tokens so far left: normed keys and values, about unit size
        codes = torch.empty(blocks, hk, block, d, dtype=_CODES[case["codes"]], device="cuda")
        scale = torch.empty(blocks, hk, device="cuda")
        step = max(1, (1 << 26) // (hk * block * d))
        for at in range(0, blocks, step):
            x = torch.randn(min(step, blocks - at), hk, block, d, device="cuda", generator=g)
            by = _needed(x.abs().amax((2, 3)), case["codes"])
            codes[at:at + step] = _rounded(x / by[..., None, None], case["codes"])
            scale[at:at + step] = by
        s.update({name + "_cache": codes.transpose(1, 2), name + "_scale": scale})
    T = int(starts[-1])
    if case["op"] == "cache":
        s.update(k=normal(T, hk, d), v=normal(T, hk, d),
                 k_out=torch.zeros(B, int(lengths.max()), hk, d, dtype=t, device="cuda"),
                 v_out=torch.zeros(B, int(lengths.max()), hk, d, dtype=t, device="cuda"))
    else:
        s.update(q=normal(T, case["hq"], d))
    return s


# ----------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import direct_implicit_gemm_amd as L
        if c["op"] == "linear":
            return L.linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"])
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "cache":
            L.kv_cache_write(s["k"], s["v"], *cache, s["starts"], s["lengths"], s["table"])
            L.kv_cache_read(*cache, s["lengths"], s["table"], k_out=s["k_out"], v_out=s["v_out"])
            return [s["k_out"], s["v_out"], s["k_scale"], s["v_scale"]]
        return list(L.cache_attention(s["q"], *cache, s["starts"], s["lengths"], s["table"],
                                      max_rows=s["max_rows"], causal=c["causal"],
                                      return_lse=True))
    return {"cache": _plain_cache, "attention": _plain_attention, "linear": _plain_linear}[
        c["op"]](s, c)


def _needed(top, codes):
    """The least power of two (from 2^-126 on) that brings `top` down to the largest code."""
    m, e = torch.frexp(top)
    most_m, most_e = math.frexp(_MOST[codes])
    e = torch.where(m <= most_m, e - most_e, e - most_e + 1).clamp(min=-126)
    e = torch.where(top > 0, e, torch.full_like(e, -126))
    return ((e + 127) << 23).view(torch.float32)  # 2^e


def _rounded(x, codes):
    return (x.round() if codes == "i8" else x).clamp(-_MOST[codes], _MOST[codes]).to(_CODES[codes])


def _entry_and_position(s, T):
    """Of every new row: its entry and its position among the entry's tokens."""
    row = torch.arange(T, device="cuda")
    entry = torch.searchsorted(s["starts"], row.int(), right=True) - 1
    return entry, s["lengths"].long()[entry] - (s["starts"].long()[entry + 1] - row)


def _plain_cache(s, c):
    block, table, lengths = c["block"], s["table"].long(), s["lengths"].long()
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    entry, at = _entry_and_position(s, len(s["k"]))
    to, row = table[entry, at // block], at % block
    # blocks that the new tokens share with earlier ones, and how many of those they hold
    first = (lengths - new) // block
    held = torch.where(new > 0, (lengths - new) % block, torch.zeros_like(new))
    shared = table.gather(1, first.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    old = torch.arange(block, device="cuda")[None] < held[:, None]
    for name, x in (("k", s["k"].float()), ("v", s["v"].float())):
        codes, scale = s[name + "_cache"], s[name + "_scale"]
        top = torch.zeros_like(scale).index_reduce_(0, to, x.abs().amax(-1), "amax")
        before = torch.zeros_like(scale)
        before[shared] = torch.where(held[:, None] > 0, scale[shared], before[shared])
        after = torch.maximum(before, _needed(top, c["codes"]))
        was = codes[shared].float() * (before / after)[shared][:, None, :, None]
        codes[shared] = torch.where(old[:, :, None, None], _rounded(was, c["codes"]).float(),
                                    codes[shared].float()).to(codes.dtype)
        codes[to, row] = _rounded(x / after[to][..., None], c["codes"])
        written = torch.zeros(len(scale), dtype=torch.bool, device="cuda").index_fill_(0, to, True)
        scale.copy_(torch.where(written[:, None], after, scale))
        out = s[name + "_out"]
        p = torch.arange(out.shape[1], device="cuda")
        here = table[:, p // block]
        value = codes[here, p % block].float() * scale[here][..., None]
        out.copy_(torch.where((p < lengths[:, None])[..., None, None], value.to(out.dtype), out))
    return [s["k_out"], s["v_out"], s["k_scale"], s["v_scale"]]


def _plain_attention(s, c):
    B, hq, hk, d, block, n = c["B"], c["hq"], c["hk"], c["d"], c["block"], s["max_rows"]
    T, lengths = len(s["q"]), s["lengths"].long()
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(n, device="cuda")
    row = (s["starts"][:-1].long()[:, None] + i).clamp(max=T - 1)  # [B, n]: each entry's rows
    # queries of one key head together: [B, hk, n * group, d]
    q = s["q"][row].float().view(B, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, d)
    j = torch.arange(int(s["table"].shape[1]) * block, device="cuda")
    here = s["table"].long()[:, j // block]
    inside = (j < lengths[:, None])[..., None, None]

    def dense(name):  # [B, hk, keys, d]
        x = s[name + "_cache"][here, j % block].float() * s[name + "_scale"][here][..., None]
        return x.masked_fill_(~inside, 0.0).transpose(1, 2).contiguous()

    score = torch.matmul(q * d ** -0.5, dense("k").transpose(2, 3).contiguous())
    seen = (j < lengths[:, None])[:, None].expand(B, n, -1)
    if c["causal"]:  # query i of an entry stands at position length - new + i
        seen = seen & (j <= ((lengths - new)[:, None] + i)[..., None])
    score.masked_fill_(~seen.repeat_interleave(hq // hk, 1)[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, dense("v")) / total).view(B, hk, n, hq // hk, d)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d)
    lse = (top + total.log()).view(B, hk, n, hq // hk).permute(0, 2, 1, 3).reshape(B, n, hq)
    entry = torch.searchsorted(s["starts"], torch.arange(T, device="cuda").int(), right=True) - 1
    at = torch.arange(T, device="cuda") - s["starts"].long()[entry]
    return [out[entry, at].to(s["q"].dtype), lse[entry, at]]


def _plain_linear(s, c):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y += s["bias"].float()
    if c["act"] == "relu":
        y = y.clamp_(min=0.0)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


# ------------------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"cache": _exact_cache, "attention": _exact_attention, "linear": _exact_linear}[
        case["op"]](s, case)


def _exact_cache(s, c):
    block, most, t = c["block"], _MOST[c["codes"]], _CODES[c["codes"]]
    starts, table = s["starts"].tolist(), s["table"].tolist()
    if sum(-(-length // block) for length in s["lengths"].tolist()) > 20000:
        return None

    def code(x):  # in units of the scale
        return (x.round() if t == torch.int8 else x).clamp(-most, most).to(t)

    for name in ("k", "v"):
        codes, scale, out = s[name + "_cache"], s[name + "_scale"].double(), s[name + "_out"].double()
        for b, length in enumerate(s["lengths"].tolist()):
            x = s[name][starts[b]:starts[b + 1]].double()
            begin = length - len(x)
            for i in range(begin // block, -(-length // block) if len(x) else 0):
                lo, hi = max(begin, i * block), min(length, (i + 1) * block)
                mine, at = x[lo - begin:hi - begin], table[b][i]
                # least power of two with largest / 2^e <= most
                ratio = (mine.abs().amax((0, 2)) / most).clamp(min=2.0 ** -126)
                need = torch.exp2(torch.ceil(torch.log2(ratio)))
                need = torch.where(need / 2 >= ratio, need / 2, torch.where(need < ratio, 2 * need,
                                                                           need))
                held = lo - i * block
                by = torch.maximum(need, scale[at]) if held else need
                if held:
                    codes[at, :held] = code(codes[at, :held].double() * (scale[at] / by)[:, None])
                codes[at, held:hi - i * block] = code(mine / by[:, None])
                scale[at] = by
            here = s["table"][b].long()
            dense = codes[here].double() * scale[here][:, None, :, None]
            out[b, :length] = dense.flatten(0, 1)[:length]
        s[name + "_scale"], s[name + "_out"] = scale, out
    return [s["k_out"], s["v_out"], s["k_scale"], s["v_scale"]]


def _exact_attention(s, c):
    hq, hk, block = c["hq"], c["hk"], c["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for b, length in enumerate(s["lengths"].tolist()):
        rows, here = slice(starts[b], starts[b + 1]), s["table"][b, :-(-length // block)].long()
        n = starts[b + 1] - starts[b]
        for h in range(hk):
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            k, v = ((s[x + "_cache"][here, :, h].double() *
                     s[x + "_scale"][here, h].double()[:, None, None]).flatten(0, 1)[:length]
                    for x in ("k", "v"))
            score = torch.einsum("ngd,jd->ngj", s["q"][rows, heads].double(), k) / math.sqrt(c["d"])
            if c["causal"]:
                i = torch.arange(n, device="cuda")[:, None, None]
                score.masked_fill_(torch.arange(length, device="cuda") > length - n + i, -math.inf)
            lse[rows, heads] = torch.logsumexp(score, -1)
            out[rows, heads] = torch.softmax(score, -1) @ v
    return [out, lse]


def _exact_linear(s, c):
    y = s["x"].double() @ s["w"].double().t()
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["act"] == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    elif c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif c["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
    elif c["act"] == "silu":
        y = y * torch.sigmoid(y)
    return y if s["residual"] is None else y + s["residual"].double()
