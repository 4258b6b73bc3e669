"""prefix_attention on the GPU against its plain form in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, Sq, P, S, hq, hk, d, dtype, lengths, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = C.TYPES[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t).cuda()
    n = torch.tensor(lengths).int().cuda()
    return r(B, Sq, hq, d), r(P, hk, d), r(P, hk, d), r(B, S, hk, d), r(B, S, hk, d), n


def check(q, kp, vp, k, v, n, causal, scale=None, what="", **kw):
    print(f"[gpu] attention {what} q{tuple(q.shape)} causal={causal}", flush=True)
    out, lse = L.prefix_attention(q, kp, vp, k, v, n, scale=scale, causal=causal, return_lse=True,
                                  **kw)
    torch.cuda.synchronize()
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want, bound, wl, bl = C.attention(q, kp, vp, k, v, n, s, causal)
    C.assert_within(out, want, bound, f"out {what}")
    C.assert_within(lse, wl, bl, f"lse {what}")
    return out


CASES = [  # B, Sq, P, S, query heads, key heads, head_dim, causal, dtype, lengths
    (1, 1, 1, 1, 1, 1, 64, True, "bf16", [1]),
    (1, 1, 0, 5, 2, 1, 128, True, "bf16", [3]),
    (2, 1, 300, 40, 4, 4, 64, True, "bf16", [0, 40]),
    (3, 1, 129, 700, 8, 2, 128, True, "f16", [1, 513, 700]),
    (5, 2, 2000, 33, 8, 1, 80, True, "bf16", [0, 1, 2, 17, 33]),
    (2, 7, 65, 65, 6, 3, 72, True, "f16", [3, 65]),
    (1, 130, 0, 130, 2, 2, 64, True, "bf16", [130]),
    (2, 65, 77, 200, 4, 2, 128, True, "bf16", [64, 200]),
    (2, 100, 31, 96, 2, 2, 128, False, "f16", [95, 0]),
    (1, 257, 77, 257, 2, 1, 128, False, "bf16", [257]),
    (1, 33, 200, 0, 2, 1, 40, False, "bf16", [0]),
    (2, 40, 0, 64, 2, 2, 64, True, "f16", [0, 20]),
    (2, 1, 500, 300, 4, 1, 64, True, "f32", [7, 300]),
    (2, 70, 40, 90, 2, 1, 128, True, "f32", [90, 30]),
    (1, 129, 5, 130, 1, 1, 80, False, "f32", [130]),
    (9, 3, 4100, 64, 16, 2, 128, True, "bf16", [0, 1, 2, 3, 4, 30, 31, 63, 64]),
    (3, 16, 600, 50, 4, 1, 64, True, "bf16", [16, 3, 50]),
    (1, 1, 0, 9000, 1, 1, 128, True, "bf16", [8999]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("workspace", [True, False])
def test_against_64_bits(case, workspace):
    B, Sq, P, S, hq, hk, d, causal, dtype, lengths = case
    check(*make(B, Sq, P, S, hq, hk, d, dtype, lengths), causal, what=str(case),
          workspace=workspace)


def test_stale_rows_past_the_length_are_not_read():
    """NaN and infinity in cache rows past the length, and in rows between sequences."""
    for Sq, P in ((1, 200), (40, 0), (1, 0)):
        q, kp, vp, k, v, n = make(3, Sq, P, 300, 4, 2, 64, "bf16", [0, 70, 129])
        want = check(q, kp, vp, k, v, n, True, what="clean")
        for b, m in enumerate(n.tolist()):
            k[b, m:], v[b, m:] = math.nan, math.inf
        got = L.prefix_attention(q, kp, vp, k, v, n, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(got, want), (Sq, P)


def test_rows_without_a_key_are_zero():
    q, _, _, k, v, n = make(3, 5, 1, 20, 4, 2, 64, "f16", [0, 2, 20])
    out, lse = L.prefix_attention(q, None, None, k, v, n, return_lse=True)
    torch.cuda.synchronize()
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    # two own keys, five queries: the first three see none
    assert bool((out[1, :3] == 0).all()) and bool((lse[1, :, :3] == -math.inf).all())
    assert bool(torch.isfinite(lse[1, :, 3:]).all())


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.7])
def test_scales(scale):
    check(*make(2, 9, 90, 50, 4, 2, 64, "bf16", [50, 20]), True, scale=scale, what=f"scale {scale}")


def test_lengths_out_of_range_are_clamped():
    q, kp, vp, k, v, n = make(2, 1, 30, 40, 2, 2, 64, "bf16", [-5, 4000])
    check(q, kp, vp, k, v, n, True, what="clamped")


def test_strides():
    """Head-major caches, queries from a fused projection, a strided output."""
    B, Sq, hq, hk, d, P, S = 2, 33, 4, 2, 64, 70, 90
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    fused = r(B, Sq, hq + 2 * hk, d)
    kc, vc = r(B, hk, S, d).transpose(1, 2), r(B, hk, S, d).transpose(1, 2)
    kp, vp = r(hk, P, d).transpose(0, 1), r(P, 2, hk, d)[:, 1]
    out = torch.full((B, Sq, hq, 2 * d), 5.0, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([90, 41]).int().cuda()
    q = fused[:, :, :hq]
    check(q, kp, vp, kc, vc, n, True, what="strided", out=out[..., :d])
    assert bool((out[..., d:] == 5.0).all())


def test_expanded_keys():
    """One head of keys given to all through a stride of 0."""
    q, kp, vp, k, v, n = make(2, 4, 70, 60, 4, 1, 64, "bf16", [60, 9])
    kp, vp = kp.expand(70, 4, 64), vp.expand(70, 4, 64)
    check(q, kp, vp, k.expand(2, 60, 4, 64), v.expand(2, 60, 4, 64), n, True, what="expanded")


def test_large_scores():
    """Scores of hundreds: the maximum moves from tile to tile."""
    q, kp, vp, k, v, n = make(2, 3, 500, 90, 2, 1, 128, "f32", [90, 50])
    ramp = torch.linspace(0.1, 8.0, 500, device="cuda")[:, None, None]
    check(q * 4, kp * ramp, vp, k, v, n, True, what="large")


def test_another_stream_and_repeats():
    q, kp, vp, k, v, n = make(6, 1, 1500, 200, 8, 2, 128, "bf16", [1, 20, 60, 100, 150, 200])
    first = check(q, kp, vp, k, v, n, True, what="first")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        out = L.prefix_attention(q, kp, vp, k, v, n, stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(out, first)   # fixed order of sums


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements, the entry's rows far apart."""
    hk, d, S = 1, 64, 40
    q, kp, vp, _, _, n = make(2, 1, 40, S, 2, 1, d, "bf16", [40, 33])
    stride = (1 << 31) + 64
    big = torch.zeros(stride + S * d, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((2, S, hk, d), (stride, d, d, 1))
    k.copy_(torch.randn(2, S, hk, d, generator=torch.Generator().manual_seed(2)).bfloat16())
    check(q, kp, vp, k, k, n, True, what="far")


def test_graph_replays():
    q, kp, vp, k, v, n = make(4, 1, 900, 128, 8, 2, 64, "bf16", [1, 50, 99, 128])
    L.prefix_attention(q, kp, vp, k, v, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.prefix_attention(q, kp, vp, k, v, n)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(20 + i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.prefix_attention(q, kp, vp, k, v, n)), i
        torch.cuda.synchronize()


MORE = [  # B, Sq, P, S, query heads, key heads, head_dim, causal, dtype, lengths
    # more workgroups of 128 rows than half the compute units: tiles shared by their waves
    (2, 300, 77, 310, 33, 33, 64, True, "bf16", [310, 171]),
    (2, 290, 150, 200, 50, 25, 80, True, "f16", [200, 1]),
    (3, 260, 65, 128, 22, 22, 128, False, "bf16", [128, 0, 65]),
    (1, 700, 0, 700, 25, 25, 96, True, "f16", [640]),
    (2, 200, 191, 64, 35, 35, 128, True, "bf16", [64, 40]),
    (2, 280, 33, 130, 30, 30, 72, True, "f32", [130, 20]),
    # the prefix once, own keys in several runs, one ending at a run's end
    (4, 1, 700, 3000, 4, 1, 64, True, "bf16", [0, 256, 257, 3000]),
    (6, 2, 2500, 1200, 16, 2, 128, True, "f16", [1200, 1, 128, 129, 384, 700]),
    (40, 1, 1100, 300, 8, 2, 80, True, "bf16", [7 * i for i in range(40)]),
    (3, 9, 300, 500, 4, 1, 128, True, "f32", [500, 5, 131]),
    # many keys for few rows: more than 8 partial results to join
    (1, 1, 5000, 6000, 2, 1, 64, True, "bf16", [5555]),
    (2, 17, 130, 0, 4, 2, 8, False, "f16", [0, 0]),
]


@pytest.mark.parametrize("case", MORE, ids=str)
@pytest.mark.parametrize("workspace", [True, False])
def test_more_shapes_against_64_bits(case, workspace):
    B, Sq, P, S, hq, hk, d, causal, dtype, lengths = case
    check(*make(B, Sq, P, S, hq, hk, d, dtype, lengths, seed=6), causal, what=str(case),
          workspace=workspace)


def test_stale_rows_with_shared_tiles():
    """As above, for rows enough that the waves of a workgroup share their tiles."""
    q, kp, vp, k, v, n = make(3, 270, 70, 300, 24, 24, 64, "bf16", [0, 70, 129])
    want = check(q, kp, vp, k, v, n, True, what="clean")
    for b, m in enumerate(n.tolist()):
        k[b, m:], v[b, m:] = math.nan, math.inf
    got = L.prefix_attention(q, kp, vp, k, v, n, causal=True)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("Sq,hk", [(1, 2), (300, 33)])
def test_scores_that_climb_and_fall(Sq, hk):
    """Keys in order of growing and of falling scores, far beyond what the exponential holds."""
    q, kp, vp, k, v, n = make(2, Sq, 400, 90, hk, hk, 64, "f16", [90, 50])
    q = q.abs()
    for ramp in (torch.linspace(-3.0, 3.0, 400), torch.linspace(3.0, -3.0, 400)):
        keys = kp.abs() * ramp.half().cuda()[:, None, None]
        check(q * 3, keys, vp, k, v, n, True, what=f"ramp from {float(ramp[0])}")


def test_not_finite_values_stay_with_their_entry():
    q, kp, vp, k, v, n = make(5, 1, 300, 200, 4, 2, 64, "bf16", [200, 150, 1, 0, 64])
    want = check(q, kp, vp, k, v, n, True, what="finite")
    k[1, 7], v[1, 7], q[4] = math.nan, math.inf, math.nan
    got = L.prefix_attention(q, kp, vp, k, v, n)
    torch.cuda.synchronize()
    for b in (0, 2, 3):
        assert torch.equal(got[b], want[b]), b
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[4]).all())
