"""Measured cases of the attention-layer operators: what a caller has in hand, one pass through
each operator, and its plain form in elementary torch operations.

Three operators that run one after another in an attention layer:
  lora       a projection shared by all requests with each request's low-rank adapter beside it
  rope       norms of queries and keys for each head and the position rotation, keys and values
             written into a cache
  attention  attention of a batch over a prefix all its entries share and each entry's own keys

`own` selects between the plain form (False) and the calls of the package (True).
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-6


# ------------------------------------------------------------------------------------- the cases
def _lora(T, K, N, rank, adapters, requests, dtype, bias):
    return {"op": "lora", "T": T, "K": K, "N": N, "rank": rank, "adapters": adapters,
            "requests": requests, "dtype": dtype, "bias": bias}


def _rope(T, hq, hk, d, rot, axes, far, interleaved, cache, dtype):
    return {"op": "rope", "T": T, "hq": hq, "hk": hk, "d": d, "rot": rot, "axes": axes, "far": far,
            "interleaved": interleaved, "cache": cache, "dtype": dtype}


def _attention(B, Sq, P, lo, hi, hq, hk, d, causal, dtype):
    return {"op": "attention", "B": B, "Sq": Sq, "P": P, "lo": lo, "hi": hi, "hq": hq, "hk": hk,
            "d": d, "causal": causal, "dtype": dtype}


def listed():
    return [
        # one decoding step of 8 prompts about one image, q/k/v projection of 640 channels
        {"name": "lora decode 8", **_lora(8, 640, 1920, 8, 4, 8, "bf16", True)},
        # one decoding step of 64 requests over 24 adapters in a wide decoder
        {"name": "lora decode 64", **_lora(64, 4096, 4096, 16, 24, 64, "bf16", False)},
        # two 32x32 maps of 1280 channels and a ragged tail of text rows, 7 requests, in half
        {"name": "lora ragged f16", **_lora(2167, 1280, 3840, 64, 5, 7, "f16", True)},
        # prompts read in at once, 9 requests: a large product
        {"name": "lora prefill", **_lora(8192, 4096, 8192, 32, 6, 9, "bf16", False)},
        # one decoding step: queries, keys and values of 8 rows, keys and values into the cache
        {"name": "rope decode 8", **_rope(8, 20, 20, 64, 64, 1, 40000, False, True, "bf16")},
        # a long text far into its positions, pairs side by side, part of each head rotated, fp32
        {"name": "rope text f32", **_rope(2053, 16, 4, 128, 96, 1, 1 << 20, True, False, "f32")},
        # the tokens of a video of 5 frames of 64x120, rotated by frame, row and column
        {"name": "rope video", **_rope(38400, 20, 20, 128, 128, 3, 128, False, False, "bf16")},
        # the first steps of 4 prompts about one page's 960 features, few own keys
        {"name": "attention decode 4", **_attention(4, 1, 960, 1, 40, 20, 20, 64, True, "bf16")},
        # decoding with 64 requests behind one long prompt, shared heads of keys
        {"name": "attention decode 64", **_attention(64, 1, 8192, 1, 2048, 32, 8, 128, True,
                                                     "bf16")},
        # prompts of ragged length read in behind a shared one; heads of 80, half
        {"name": "attention prefill f16", **_attention(3, 517, 1023, 300, 1400, 16, 4, 80, True,
                                                       "f16")},
        # short texts in single precision behind a shared one
        {"name": "attention f32", **_attention(2, 130, 333, 130, 190, 8, 8, 64, True, "f32")},
        # 12 windows of a video of 38400 tokens, all with the same 77 text tokens
        {"name": "attention windows", **_attention(12, 3200, 77, 3200, 3200, 20, 20, 128, False,
                                                   "bf16")},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "rope", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = {c["op"]: work(c) for c in listed()}  # the last listed case of each is its largest
    while True:
        if op == "lora":
            T = _log(rng, 1, 8192)
            c = _lora(T, 8 * _log(rng, 16, 512), _log(rng, 64, 8192), rng.choice([4, 8, 16, 32, 64]),
                      _log(rng, 1, 24), min(T, _log(rng, 1, 64)), dtype, rng.random() < 0.5)
        elif op == "rope":
            d = rng.choice([64, 80, 128])
            hk = _log(rng, 1, 20)
            c = _rope(_log(rng, 1, 38400), hk * rng.choice([1, 2, 4]), hk, d,
                      rng.choice([d, d // 2 // 16 * 16]), rng.choice([1, 3]),
                      _log(rng, 128, 1 << 20), rng.random() < 0.5, rng.random() < 0.5, dtype)
        else:
            hk, hi, Sq = _log(rng, 1, 20), _log(rng, 1, 4096), rng.choice([1, 1, _log(rng, 2, 3200)])
            c = _attention(_log(rng, 1, 64), Sq, _log(rng, 1, 8192), _log(rng, 1, hi), hi,
                           hk * rng.choice([1, 2, 4]), hk, rng.choice([64, 80, 128]),
                           rng.random() < 0.6, dtype)
        w, cap = work(c), most[op]
        # the plain form of attention holds every score: keep it within the largest listed case's
        scores = 0 if op != "attention" else c["B"] * c["Sq"] * c["hq"] * (c["P"] + c["hi"])
        slow = 8 if dtype == "f32" else 1
        if (w["bytes"] <= cap["bytes"] or op != "rope") and slow * w["flops"] <= cap["flops"] \
                and scores <= 12 * 3200 * 20 * 3277:
            return c


def _lengths(case):
    """Own keys of each entry: spread evenly from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "lora":
        T, K, N, r = case["T"], case["K"], case["N"], case["rank"]
        used = min(case["adapters"], case["requests"])
        return {"bytes": e * (T * K + N * K + T * N + used * r * (K + N)),
                "flops": 2 * T * (K * N + r * (K + N))}
    if case["op"] == "rope":
        heads = case["hq"] + case["hk"] * (2 if case["cache"] else 1)
        return {"bytes": 2 * e * case["T"] * heads * case["d"] + 4 * case["T"] * case["axes"],
                "flops": 8 * case["T"] * (case["hq"] + case["hk"]) * case["d"]}
    B, Sq, P, d = case["B"], case["Sq"], case["P"], case["d"]
    keys = sum(_lengths(case))
    pairs = B * Sq * P + sum(
        sum(max(0, n - Sq + i + 1) for i in range(Sq)) if case["causal"] else Sq * n
        for n in _lengths(case))
    return {"bytes": e * d * (2 * B * Sq * case["hq"] + 2 * (P + keys) * case["hk"]),
            "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------------------------- their inputs
def _starts(case, g):
    """Where each request's rows begin, and the end: cut at random places, every request a row."""
    T, R = case["T"], case["requests"]
    cuts = torch.randperm(T - 1, generator=g)[:R - 1].sort().values + 1
    return torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(t)

    s = {"case": dict(case)}
    if case["op"] == "lora":
        T, K, N, r, n = (case[k] for k in ("T", "K", "N", "rank", "adapters"))
        ids = torch.randint(0, n, (case["requests"],), generator=h).int()
        ids[torch.rand(case["requests"], generator=h) < 0.1] = -1  # some requests have none
        s.update(x=normal(T, K), w=normal(N, K, by=K ** -0.5),
                 bias=normal(N, by=0.05) if case["bias"] else None,
                 a=normal(n, r, K, by=K ** -0.5), b=normal(n, N, r, by=0.3 * r ** -0.5),
                 scales=(0.5 + torch.rand(n, device="cuda", generator=g)),
                 starts=_starts(case, h).cuda(), ids=ids.cuda())
    elif case["op"] == "rope":
        T, hq, hk, d, rot, axes = (case[k] for k in ("T", "hq", "hk", "d", "rot", "axes"))
        qkv = normal(T, (hq + 2 * hk) * d, by=2.0)  # one projection's output
        q, k, v = (x.view(T, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], 1))
        half = rot // 2
        # pairs of each axis: the first axis takes what is left over
        sections = [half - (axes - 1) * (half // axes)] + (axes - 1) * [half // axes]
        freqs = torch.cat([10000.0 ** (-torch.arange(m, dtype=torch.float64) / m)
                           for m in sections])
        rows = 2 * T + 3
        s.update(q=q, k=k, v=v, q_weight=(1 + 0.2 * normal(d).float()).to(t),
                 k_weight=(1 + 0.2 * normal(d).float()).to(t), sections=sections,
                 freqs=freqs.cuda(),
                 positions=torch.randint(0, case["far"], (axes, T), generator=h).int().cuda(),
                 slots=torch.randperm(rows, generator=h)[:T].int().cuda() if case["cache"] else None,
                 cache_k=normal(rows, hk, d) if case["cache"] else None,
                 cache_v=normal(rows, hk, d) if case["cache"] else None)
    else:
        B, Sq, P, hq, hk, d = (case[k] for k in ("B", "Sq", "P", "hq", "hk", "d"))
        lengths = torch.tensor(_lengths(case))[torch.randperm(B, generator=h)]
        # normed and rotated queries and keys: about unit size in every component
        s.update(q=normal(B, Sq, hq, d), kp=normal(P, hk, d), vp=normal(P, hk, d),
                 k=normal(B, case["hi"], hk, d), v=normal(B, case["hi"], hk, d),
                 lengths=lengths.int().cuda())
    return s


# ----------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import direct_implicit_gemm_amd as L
        if c["op"] == "lora":
            return L.lora_linear(s["x"], s["w"], s["bias"], s["a"], s["b"], s["scales"],
                                 s["starts"], s["ids"])
        if c["op"] == "rope":
            out = L.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], s["q_weight"],
                                 s["k_weight"], eps=_EPS, sections=s["sections"],
                                 interleaved=c["interleaved"], v=s["v"] if c["cache"] else None,
                                 slots=s["slots"], k_out=s["cache_k"], v_out=s["cache_v"])
            return list(out)
        out, lse = L.prefix_attention(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lengths"],
                                      causal=c["causal"], return_lse=True)
        return [out, lse]
    return {"lora": _plain_lora, "rope": _plain_rope, "attention": _plain_attention}[c["op"]](s, c)


def _plain_lora(s, c):
    x, n, r = s["x"].float(), c["adapters"], c["rank"]
    rows = torch.arange(c["T"], device="cuda", dtype=torch.int32)
    ids = s["ids"][torch.searchsorted(s["starts"], rows, right=True) - 1]  # each row's adapter
    # every adapter's low-rank values, those of other adapters than the row's own set to 0
    mine = (ids[:, None] == torch.arange(n, device="cuda")) * s["scales"]
    low = (x @ s["a"].float().view(n * r, -1).t()).view(-1, n, r) * mine[:, :, None]
    y = x @ s["w"].float().t()
    y += low.view(-1, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    if s["bias"] is not None:
        y += s["bias"].float()
    return y.to(s["x"].dtype)


def _plain_rope(s, c):
    half, t = c["rot"] // 2, s["q"].dtype
    axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=half)
    angle = s["positions"].double()[axis].t() * s["freqs"]  # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight.float()
        if c["interleaved"]:
            a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:c["rot"]]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., c["rot"]:]], -1).to(t)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not c["cache"]:
        return [q, k]
    s["cache_k"][s["slots"].long()] = k
    s["cache_v"][s["slots"].long()] = s["v"]
    return [q, s["cache_k"], s["cache_v"]]


def _plain_attention(s, c):
    B, Sq, P, hq, hk, d = (c[k] for k in ("B", "Sq", "P", "hq", "hk", "d"))
    # queries of one key head together: [B, hk, Sq * group, d]
    q = s["q"].float().view(B, Sq, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, d)
    q = q * d ** -0.5
    prefix = torch.matmul(q, s["kp"].float().permute(1, 2, 0).contiguous())
    mine = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1).contiguous())
    n = s["lengths"][:, None, None]
    j = torch.arange(c["hi"], device="cuda")
    seen = (j < n).expand(B, Sq, -1)
    if c["causal"]:
        seen = seen & (j <= n - Sq + torch.arange(Sq, device="cuda")[:, None])
    seen = seen.repeat_interleave(hq // hk, 1)[:, None]
    score = torch.cat([prefix, mine.masked_fill_(~seen, -math.inf)], -1)
    del prefix, mine
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p[..., :P], s["vp"].float().transpose(0, 1).contiguous())
    out += torch.matmul(p[..., P:], s["v"].float().transpose(1, 2).contiguous())
    out = (out / total).view(B, hk, Sq, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, Sq, hq, d)
    lse = (top + total.log()).view(B, hk, Sq, hq // hk).transpose(2, 3).reshape(B, hq, Sq)
    return [out.to(s["q"].dtype), lse]


# ------------------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "rope": _exact_rope, "attention": _exact_attention}[case["op"]](
        s, case)


def _exact_lora(s, c):
    y = s["x"].double() @ s["w"].double().t()
    if s["bias"] is not None:
        y += s["bias"].double()
    starts, ids = s["starts"].tolist(), s["ids"].tolist()
    for lo, hi, i in zip(starts, starts[1:], ids):
        if i >= 0:
            low = s["x"][lo:hi].double() @ s["a"][i].double().t()
            y[lo:hi] += s["scales"][i].double() * (low @ s["b"][i].double().t())
    return y


def _exact_rope(s, c):
    d, rot = c["d"], c["rot"]
    first, second, turn, at = [], [], [], 0
    for axis, m in enumerate(s["sections"]):  # pair by pair: where its two halves lie, its angle
        for i in range(at, at + m):
            first.append(2 * i if c["interleaved"] else i)
            second.append(2 * i + 1 if c["interleaved"] else i + rot // 2)
            turn.append(s["positions"][axis].double() * s["freqs"][i])
        at += m
    turn = torch.polar(torch.ones_like(turn[0]).expand(len(turn), -1), torch.stack(turn)).t()

    def one(x, weight):
        x = x.double()
        x = weight.double() * x / (x.square().sum(-1, keepdim=True) / d + _EPS).sqrt()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not c["cache"]:
        return [q, k]
    keys, values = s["cache_k"].double(), s["cache_v"].double()
    keys[s["slots"].long()] = k
    values[s["slots"].long()] = s["v"].double()
    return [q, keys, values]


def _exact_attention(s, c):
    Sq, hq, hk = c["Sq"], c["hq"], c["hk"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["B"], hq, Sq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        for h in range(hk):
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            q = s["q"][b, :, heads].double().transpose(0, 1)
            k = torch.cat([s["kp"][:, h], s["k"][b, :n, h]]).double()
            v = torch.cat([s["vp"][:, h], s["v"][b, :n, h]]).double()
            score = (q.reshape(-1, c["d"]) @ k.t()).view(-1, Sq, c["P"] + n) / math.sqrt(c["d"])
            if c["causal"]:  # query i stands at own key n - Sq + i
                i = torch.arange(Sq, device="cuda")[:, None]
                j = torch.arange(-c["P"], n, device="cuda")
                score.masked_fill_((j >= 0) & (j > n - Sq + i), -math.inf)
            lse[b, heads] = torch.logsumexp(score, -1)
            p = torch.softmax(score, -1).view(-1, c["P"] + n)
            out[b, :, heads] = (p @ v).view(-1, Sq, c["d"]).transpose(0, 1)
    return [out, lse]
