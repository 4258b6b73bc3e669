"""examples/decoder_layer.py in fp32 against 64 bits, step by step: the codes and scales that a step
writes, number for number, and its outputs from the keys and values that the cache holds, each within
what the roundings of fp32 add up to."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
import cachecheck as C  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu
U32 = C.U32


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def host(t):
    return t.double().cpu()


def product(x, w, b=None, off=0.0):
    """(x w^T + b, its error) for x that is off by `off`: half a step of 2^-24 of every product and
    sum, and what an error of x moves it by."""
    v, mag = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        v, mag = v + b, mag + b.abs()
    moved = off @ w.abs().t() if torch.is_tensor(off) else 0.0
    return v, U32 * (x.shape[-1] + 9) * mag + moved


def normed_and_turned(t, off, w, freqs, positions):
    """(t, its error) after the norm over a head and the rotation."""
    d = t.shape[-1]
    rms = torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
    # the norm moves by no more than the error's own norm
    moved = off / rms + t.abs() / rms * (off.norm(dim=-1, keepdim=True) / (rms * d ** 0.5))
    t = t / rms * w
    off = moved * w.abs() + U32 * (d + 16) * t.abs()
    angle = positions[:, None] * freqs
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b, ea, eb = t[..., :d // 2], t[..., d // 2:], off[..., :d // 2], off[..., d // 2:]
    size = a.abs() + b.abs()   # sines and cosines, products and a sum: 8 half steps
    return (torch.cat([a * cos - b * sin, b * cos + a * sin], -1),
            torch.cat([ea * cos.abs() + eb * sin.abs() + 8 * U32 * size,
                       eb * cos.abs() + ea * sin.abs() + 8 * U32 * size], -1))


def cache_of(m, lengths):
    c = C.Cache.__new__(C.Cache)
    c.k, c.v, c.ks, c.vs = (t.clone() for t in (m.k_cache, m.v_cache, m.k_scale, m.v_scale))
    c.table, c.block, c.lengths = m.table, m.k_cache.shape[1], lengths
    return c


def check_codes(before, after, k, v, starts, turn):
    """The cache after the step is what the definition makes of k and v (pairs of values and their
    errors): each code is that of a number within the error.  Returns how many of them that leaves
    a choice, and how many there are."""
    low = C.write(before, k[0] - k[1], v[0] - v[1], starts)
    high = C.write(before, k[0] + k[1], v[0] + v[1], starts)
    other = 0
    for name, (c0, s0), (c1, s1) in zip("kv", low, high):
        got, scale = after.host(name)
        assert torch.equal(s0, s1) and torch.equal(scale, s0), (turn, name)
        assert bool((c0 <= got).all()) and bool((got <= c1).all()), (turn, name)
        other += int((c0 != c1).sum())
    return other, 2 * k[0].numel()


def check_outputs(m, x, cache, q, starts, got, turn):
    d, hq = m.head_dim, m.q_heads
    out, bound, _, _ = C.attention(q[0], cache, starts, d ** -0.5, True)
    # an error of q moves each score, and each probability relative to their sum by twice the most
    # that one moves by; (64-bit queries: the bound's own roundings are those of fp32)
    T = len(x)
    moved = torch.zeros(T, hq, dtype=torch.float64)
    mag = torch.zeros_like(out)
    st = starts.tolist()
    for b in range(len(st) - 1):
        k, v = (C.of_entry(cache, b, n)[0] for n in "kv")
        for h in range(hq):
            g = h // (hq // m.k_heads)
            rows = slice(st[b], st[b + 1])
            if rows.start == rows.stop:
                continue
            moved[rows, h] = d ** -0.5 * (q[1][rows, h] @ k[:, g].abs().t()).amax(-1)
            mag[rows, h] = v[:, g].abs().amax(0)      # no less than the weighted mean of |v|
    bound = bound + 2 * moved[..., None] * mag
    out, bound = out.view(T, -1), bound.view(T, -1)
    y, off = product(out, host(m.w_out), off=bound)
    x, off = x + y, off + U32 * (x.abs() + y.abs())
    up, off_up = product(x, host(m.w_up), host(m.b_up), off)
    act, slope, own = C.activation(up, "gelu_tanh")
    down, off_down = product(act, host(m.w_down), off=slope * off_up + own)
    want = x + down
    C.assert_within(got, want, off + off_down + 2 * U32 * (x.abs() + down.abs()), f"turn {turn}")


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn], ids=["i8", "e4m3"])
def test_prompts_chunks_and_steps(codes, monkeypatch):
    import decoder_layer
    # queries in 64 bits, kernels in fp32: its roundings, and nothing for the output's own
    monkeypatch.setitem(C.P_ROUNDING, torch.float64, C.P_ROUNDING[torch.float32])
    monkeypatch.setitem(C.U, torch.float64, U32)
    B, channels = 3, 128
    m = decoder_layer.DecoderLayer(channels, 4, 2, 32, 256, B, 90, block=16, codes=codes,
                                   dtype=torch.float32)
    g = torch.Generator().manual_seed(7)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    # prompts; a chunk of one while the others decode; none of one; single tokens, then captured
    turns = [[40, 7, 33], [1, 30, 1], [2, 0, 1]] + [[1, 1, 1]] * 4
    graph = y = None
    choices = numbers = 0
    for turn, rows in enumerate(turns):
        starts, T = C.starts(rows), sum(rows)
        lengths += torch.tensor(rows, device="cuda").int()
        x = torch.randn(T, channels, generator=g).cuda()
        at = decoder_layer.positions_of(starts, lengths, T)
        before = cache_of(m, lengths)
        if turn < 4:
            got = m(x, starts, lengths, at, max(rows))
        else:
            if graph is None:
                x_in, at_in, starts_in = x.clone(), at.clone(), starts
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    y = m(x_in, starts_in, lengths, at_in, 1)
            x_in.copy_(x)
            at_in.copy_(at)
            graph.replay()
            got = y
        torch.cuda.synchronize()
        after = cache_of(m, lengths)
        d, hq, hk = m.head_dim, m.q_heads, m.k_heads
        qkv, off = product(host(x), host(m.w_qkv), host(m.b_qkv))
        parts, offs = ([p.view(T, -1, d) for p in t.split([hq * d, hk * d, hk * d], 1)]
                       for t in (qkv, off))
        q = normed_and_turned(parts[0], offs[0], host(m.q_norm), host(m.freqs), host(at))
        k = normed_and_turned(parts[1], offs[1], host(m.k_norm), host(m.freqs), host(at))
        n = check_codes(before, after, k, (parts[2], offs[2]), starts, turn)
        choices, numbers = choices + n[0], numbers + n[1]
        check_outputs(m, host(x), after, q, starts, got, turn)
    # Few codes may be either of two: numbers of about 1 are off by 1.2e-4 here (140 half steps of
    # sums of 128 products of about 12 in all, and the norm's), so 2 * 1.2e-4 of them lie that near to a
    # border for each border in 1: 2^5 of int8's (s = 2^-5), 0.8 %; E4M3's lie 1/8 to 1/16 of the
    # number apart, half as many above 1/2 and more below: no more than 2 %.
    assert choices < 0.02 * numbers, (choices, numbers)
