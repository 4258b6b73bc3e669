"""The operators around the 8-bit cache together: examples/decoder_layer.py against one plain pass
over every request's tokens in 64 bits, with the keys and values that the cache holds."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
import cachecheck as C  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Plain:
    """The layer in 64 bits on the CPU, its cache written by the definition."""

    def __init__(self, m):
        self.m = m
        self.cache = C.Cache.__new__(C.Cache)
        self.cache.k, self.cache.v = m.k_cache.clone(), m.v_cache.clone()
        self.cache.ks, self.cache.vs = m.k_scale.clone(), m.v_scale.clone()
        self.cache.table, self.cache.block = m.table, m.k_cache.shape[1]

    def __call__(self, x, starts, lengths, positions):
        m, c = self.m, lambda t: t.double().cpu()
        d, hq, hk = m.head_dim, m.q_heads, m.k_heads
        x, T = c(x), len(x)
        qkv = x @ c(m.w_qkv).t() + c(m.b_qkv)
        q, k, v = (p.view(T, -1, d) for p in qkv.split([hq * d, hk * d, hk * d], 1))
        angle = c(positions)[:, None] * c(m.freqs)
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]

        def turned(t, w):
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * c(w)
            a, b = t[..., :d // 2], t[..., d // 2:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

        q, k = turned(q, m.q_norm), turned(k, m.k_norm)
        self.cache.lengths = lengths
        for name, (codes, scale) in zip("kv", C.write(self.cache, k, v, starts)):
            setattr(self.cache, name, codes.float().to(getattr(m, name + "_cache").dtype))
            setattr(self.cache, name + "s", scale.float())
        out = C.attention(q, self.cache, starts, d ** -0.5, True)[0]
        x = x + out.view(T, hq * d) @ c(m.w_out).t()
        up = C.activation(x @ c(m.w_up).t() + c(m.b_up), "gelu_tanh")[0]
        return x + up @ c(m.w_down).t()


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn], ids=["i8", "e4m3"])
def test_prompts_chunks_and_steps(codes):
    import decoder_layer
    C.P_ROUNDING.setdefault(torch.float64, 0.0)
    C.U.setdefault(torch.float64, 2.0 ** -53)
    B, channels = 3, 128
    m = decoder_layer.DecoderLayer(channels, 4, 2, 32, 256, B, 90, block=16, codes=codes,
                                   dtype=torch.float32)
    plain = Plain(m)
    g = torch.Generator().manual_seed(5)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    # prompts; a chunk of one while the others decode; none of one; single tokens
    turns = [[40, 7, 33], [1, 30, 1], [2, 0, 1], [1, 1, 1]]
    graph = y = None
    for turn, rows in enumerate(turns + [[1, 1, 1]] * 3):
        starts, T = C.starts(rows), sum(rows)
        lengths += torch.tensor(rows, device="cuda").int()
        x = torch.randn(T, channels, generator=g).cuda()
        at = decoder_layer.positions_of(starts, lengths, T)
        want = plain(x, starts, lengths, at)
        if turn < len(turns):
            got = m(x, starts, lengths, at, max(rows))
        else:   # captured; every replay is another step
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
        # Codes differ by a step where fp32 keys and 64-bit keys round to either side: a step is
        # at most 1/64 (i8) or 1/8 (e4m3: 2^-3 of the value) of a block's largest, on 1 value in
        # 1000 at most (an fp32 key is off by 200 half steps of 2^-24 of it, 2^-16, against a step
        # of 2^-6); so a score of 32 products moves by less than a step of one of them.  The rest
        # is six fp32 passes of up to 256 sums.
        step = 1 / 64 if codes == torch.int8 else 1 / 8
        off = (got.double().cpu() - want).abs()
        scale = want.abs().max()
        assert float((off > 6 * 256 * 40 * 2.0 ** -24 * scale).float().mean()) < 0.2, turn
        assert float(off.max()) <= step * float(scale), turn


def test_the_command_runs(capsys, monkeypatch):
    import decoder_layer
    for codes in ("e4m3", "i8"):
        monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--steps", "3", "--prompt", "80",
                                          "--codes", codes])
        decoder_layer.main()
    assert capsys.readouterr().out.count("us a step") == 2
