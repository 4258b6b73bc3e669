"""linear on the GPU against its plain form in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(T, K, N, dtype, bias=True, residual=True, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = C.TYPES[dtype]
    r = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).to(t).cuda()
    return r(T, K), r(N, K, by=2 * K ** -0.5), r(N) if bias else None, r(T, N) if residual else None


def check(x, w, b, act, r, what="", **kw):
    print(f"[gpu] linear {what} {tuple(x.shape)} x {w.shape[0]} {act}", flush=True)
    y = L.linear(x, w, b, act=act, residual=r, **kw)
    torch.cuda.synchronize()
    want, bound = C.linear(x, w, b, act, r)
    C.assert_within(y, want, bound, f"y {what}")
    return y


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("T,K,N", [(1, 8, 1), (1, 1280, 3840), (3, 72, 130), (8, 640, 1920),
                                   (16, 4096, 256), (17, 520, 999), (33, 1000, 64), (64, 2048, 515),
                                   (65, 264, 260), (100, 640, 640), (130, 4096, 384),
                                   (257, 392, 1031), (700, 1280, 1280)])
def test_against_64_bits(T, K, N, dtype, workspace):
    x, w, b, r = make(T, K, N, dtype)
    act = ACTS[(T + K + N) % 5]
    check(x, w, b, act, r, workspace=workspace)
    check(x, w, None, ACTS[(T + K + N + 2) % 5], None, workspace=workspace)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", C.TYPES)
def test_activations(act, dtype):
    """Every activation over small and large sums, in tiles of each size and in runs."""
    for T, K, N in ((3, 520, 700), (300, 136, 530), (2500, 64, 3900)):
        x, w, b, r = make(T, K, N, dtype, seed=2)
        w = w * 4
        check(x, w, b, act, r, what=f"{act} {T}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_tiles(dtype):
    check(*(lambda x, w, b, r: (x, w, b, "gelu", r))(*make(4200, 200, 4300, dtype)), what="256 x 256")
    check(*(lambda x, w, b, r: (x, w, b, "silu", r))(*make(4097, 1032, 4101, dtype)), what="odd")


@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("T,K,N", [(1000, 72, 2500), (1030, 640, 3700), (513, 1032, 5000)])
def test_tiles_of_128_with_a_compute_unit_each(T, K, N, dtype):
    """Stages that lie further ahead, fewer of them than places too."""
    x, w, b, r = make(T, K, N, dtype, seed=3)
    check(x, w, b, "silu", r, what="4 stages")


def test_strides_and_in_place():
    x, w, b, r = make(70, 264, 130, "bf16")
    wide = torch.zeros(70, 700, dtype=torch.bfloat16, device="cuda")   # rows of 1400 bytes
    with pytest.raises(L.LibconvError, match="MISALIGNED"):
        L.linear(wide[:, 8:272], w, b)
    wide = torch.zeros(70, 704, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:272] = x
    wide[:, 400:530] = r
    want = check(x, w, b, "gelu", r)
    # rows of one buffer: inputs, residual and outputs (one byte off 16-byte boundaries)
    check(wide[:, 8:272], w, b, "gelu", wide[:, 400:530], out=wide[:, 531:661])
    assert torch.equal(wide[:, 531:661], want)
    before = wide.clone()
    y = wide[:, 400:530]
    L.linear(wide[:, 8:272], w, b, act="gelu", residual=y, out=y)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(wide[:, 530:], before[:, 530:])
    assert torch.equal(wide[:, :400], before[:, :400])
    one = r[:1].expand(70, 130)     # one residual for all
    assert torch.equal(check(x, w, b, "none", one), L.linear(x, w, b, residual=one.contiguous()))
    # a single row twice over
    same = x[:1].expand(70, 264)
    assert torch.equal(check(same, w, b, "none", r)[3:4],
                       L.linear(same, w, b, residual=r)[3:4])


@pytest.mark.parametrize("T", [5, 400])
@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_nan_stay_in_their_rows(T, act):
    x, w, b, r = make(T, 128, 300, "bf16")
    want = check(x, w, b, act, r)
    x[1], x[3, 5], r[4, 7] = float("inf"), float("nan"), float("-inf")
    got = L.linear(x, w, b, act=act, residual=r)
    torch.cuda.synchronize()
    keep = torch.ones(T, dtype=torch.bool)
    keep[[1, 3]] = False
    keep = keep.cuda()
    got[4, 7], want[4, 7] = 0, 0
    assert torch.equal(got[keep], want[keep])
    if act != "relu":   # which gives 0 for NaN
        assert bool(torch.isnan(got[3]).all())


def test_graph_replays():
    for T in (8, 300):
        x, w, b, r = make(T, 1024, 640, "bf16")
        L.linear(x, w, b, act="silu", residual=r)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = L.linear(x, w, b, act="silu", residual=r)
        for i in range(4):
            x.copy_(make(T, 1024, 640, "bf16", seed=40 + i)[0])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, L.linear(x, w, b, act="silu", residual=r)), i
            torch.cuda.synchronize()


def test_no_rows():
    x, w, b, _ = make(1, 64, 32, "f32")
    assert L.linear(x[:0], w, b).shape == (0, 32)


def test_linear_of_many_outputs():
    g = torch.Generator().manual_seed(2)
    N, K = (1 << 27) + 20, 8
    print(f"[gpu] linear 1 row of {N} outputs", flush=True)
    x, w = torch.randn(1, K, generator=g).bfloat16().cuda(), torch.randn(N, K, dtype=torch.bfloat16,
                                                                         device="cuda")
    r = torch.randn(1, N, dtype=torch.bfloat16, device="cuda")
    y = L.linear(x, w, act="silu", residual=r)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(300), torch.randint(300, N - 300, (3000,), generator=g),
                    torch.arange(N - 300, N)]).cuda()
    want, bound = C.linear(x, w[at], None, "silu", r[:, at])
    C.assert_within(y[:, at], want, bound, "outputs")
    assert bool(torch.isfinite(y[:, ::97]).all())
    del x, w, y, r
    torch.cuda.empty_cache()
