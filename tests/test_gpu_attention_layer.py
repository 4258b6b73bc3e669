"""The attention-layer operators together: examples/attention_layer.py against one plain pass
over every request's whole sequence in 64 bits."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plain(m, x, adapter, n_prefix):
    """x [T, channels]: the prefix and one request's tokens, in 64 bits on the CPU."""
    def c(t):
        return t.double().cpu()

    def project(x, w, bias, a, up):
        y = x @ c(w).t() + (0 if bias is None else c(bias))
        if adapter >= 0:
            low = c(m.scales)[adapter] * (x[n_prefix:] @ c(a)[adapter].t()) @ c(up)[adapter].t()
            y[n_prefix:] += low
        return y

    T, d, hq, hk = len(x), m.head_dim, m.q_heads, m.k_heads
    x = c(x)
    q, k, v = (p.view(T, -1, d) for p in project(x, m.w_qkv, m.b_qkv, m.a_qkv, m.up_qkv).split(
        [hq * d, hk * d, hk * d], 1))
    angle = torch.arange(T).double()[:, None] * c(m.freqs)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turned(t, w):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * c(w)
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = turned(q, m.q_norm), turned(k, m.k_norm)
    out = torch.empty(T, hq, d).double()
    for h in range(hq):
        s = (q[:, h] @ k[:, h // (hq // hk)].t() * d ** -0.5).masked_fill(
            torch.ones(T, T, dtype=torch.bool).triu(1), float("-inf"))
        out[:, h] = torch.softmax(s, -1) @ v[:, h // (hq // hk)]
    return project(out.reshape(T, hq * d), m.w_out, None, m.a_out, m.up_out)


@pytest.mark.parametrize("k_heads", [1, 4])
def test_prefix_prompts_and_steps(k_heads):
    import attention_layer
    B, P, n, steps, channels = 3, 150, 7, 4, 192
    m = attention_layer.AttentionLayer(channels, 4, k_heads, 48, 2, 8, B, P, n + steps,
                                       torch.float32)
    g = torch.Generator().manual_seed(5)
    shared = torch.randn(P, channels, generator=g).cuda()
    own = torch.randn(B, n + steps, channels, generator=g).cuda()
    ids = [1, -1, 0]
    adapters = torch.tensor(ids).int().cuda()
    first = torch.zeros(B, dtype=torch.int32, device="cuda")
    y_prefix = m.read_prefix(shared)
    ys = [m.read(own[:, :n].contiguous(), first, adapters)]
    first += n
    x = own[:, n:n + 1].contiguous()
    ys.append(m.read(x, first, adapters))
    first += 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.read(x, first, adapters)
        first += 1
    for i in range(1, steps):
        x.copy_(own[:, n + i:n + i + 1])
        graph.replay()
        torch.cuda.synchronize()
        ys.append(y.clone())
    got = torch.cat(ys, 1).double().cpu()
    # four fp32 passes of up to 200 sums each, scores of up to 20 whose error the exponential
    # takes over: 4 * 200 * 20 half steps of the largest output
    for b in range(B):
        want = plain(m, torch.cat([shared, own[b]]), ids[b], P)
        bound = 4 * 200 * 20 * 2.0 ** -24 * float(want.abs().max())
        assert float((got[b] - want[P:]).abs().max()) <= bound, b
        assert float((y_prefix.double().cpu() - want[:P]).abs().max()) <= bound


def test_the_command_runs(capsys, monkeypatch):
    import attention_layer
    monkeypatch.setattr(sys, "argv", ["attention_layer.py", "--steps", "3", "--prefix", "100"])
    attention_layer.main()
    assert "us a step" in capsys.readouterr().out
