"""lora_linear on the GPU against its plain form in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(T, K, N, rank, n, starts, ids, dtype, bias=True, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = C.TYPES[dtype]
    r = lambda *s, by=1.0: (by * torch.randn(*s, generator=g)).to(t).cuda()
    return dict(x=r(T, K), w=r(N, K, by=K ** -0.5), bias=r(N) if bias else None,
                a=r(n, rank, K, by=K ** -0.5), b=r(n, N, rank), scales=torch.rand(n).cuda() + 0.5,
                row_starts=torch.tensor(starts).int().cuda(), adapters=torch.tensor(ids).int().cuda())


def check(s, what, **kw):
    print(f"[gpu] lora {what}", flush=True)
    y = L.lora_linear(*s.values(), **kw)
    torch.cuda.synchronize()
    want, bound = C.lora(*s.values())
    C.assert_within(y, want, bound, what)
    return y


CASES = [  # T, K, N, rank, adapters, row_starts, ids, dtype, bias
    (1, 8, 1, 1, 1, [0, 1], [0], "bf16", True),
    (1, 640, 1920, 8, 2, [0, 1], [1], "bf16", False),
    (8, 648, 130, 4, 3, [0, 1, 2, 5, 8], [2, -1, 0, 1], "bf16", True),
    (16, 136, 64, 3, 2, [0, 16], [1], "f16", True),
    (17, 256, 72, 64, 2, [0, 5, 17], [0, 1], "f16", False),
    (33, 320, 77, 128, 2, [0, 3, 20, 33], [1, 0, 1], "bf16", True),
    (64, 1024, 200, 16, 64, list(range(65)), list(range(63, -1, -1)), "bf16", True),
    (65, 104, 65, 16, 2, [0, 1, 64, 65], [1, 0, 5], "bf16", True),
    (130, 512, 384, 40, 3, [0, 100, 100, 130], [2, 1, 0], "f16", True),
    (300, 1000, 513, 32, 40, list(range(0, 301, 6)) + [300], [i % 40 for i in range(51)], "bf16",
     True),
    (2100, 648, 1283, 12, 5, [0, 7, 600, 1999, 2100], [4, 3, -1, 0], "bf16", True),
    (1100, 264, 2052, 5, 2, [0, 550, 1100], [0, 1], "f16", False),
    (4, 72, 33, 8, 2, [0, 2, 4], [0, 1], "f32", True),
    (50, 520, 96, 17, 3, [0, 20, 50], [2, 0], "f32", True),
    (500, 264, 300, 100, 2, [0, 13, 500], [1, 0], "f32", True),
    (1500, 136, 1100, 32, 2, [0, 700, 1500], [1, 0], "f32", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + "-" + c[7])
def test_against_64_bits(case):
    T, K, N, rank, n, starts, ids, dtype, bias = case
    check(make(T, K, N, rank, n, starts, ids, dtype, bias), str(case[:5]))


@pytest.mark.parametrize("T", [5, 40, 200])
def test_without_adapters(T):
    s = make(T, 128, 96, 8, 1, [0, T], [0], "bf16")
    for k in ("a", "b", "scales", "row_starts", "adapters"):
        s[k] = None
    check(s, f"plain {T}")


@pytest.mark.parametrize("T", [12, 300])
def test_rows_of_no_request(T):
    """Rows before the first and after the last request, adapters out of range."""
    s = make(T, 64, 64, 8, 2, [3, 5, 9, T - 2], [1, 2, 0], "bf16")
    check(s, "uncovered rows")


@pytest.mark.parametrize("T", [6, 150])
def test_strided_rows(T):
    s = make(T, 128, 70, 16, 2, [0, 3, T], [1, 0], "f16")
    wide = torch.full((T, 200), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 8:136] = s["x"]
    s["x"] = wide[:, 8:136]
    out = torch.full((T, 75), 9.0, dtype=torch.float16, device="cuda")
    check(s, "strided", out=out[:, 3:73])
    assert bool((out[:, :3] == 9.0).all()) and bool((out[:, 73:] == 9.0).all())


@pytest.mark.parametrize("T", [9, 100])
def test_half_precision_low_rank_values_past_its_range(T):
    """a x reaches 10^6 in fp16 types, where y does not."""
    s = make(T, 512, 64, 8, 1, [0, T], [0], "f16")
    s["a"].mul_(2e4)
    s["b"].mul_(1e-3)
    s["scales"].fill_(0.01)
    check(s, "past fp16's range")


def test_repeats_and_another_stream():
    s = make(64, 2048, 256, 16, 8, list(range(0, 65, 8)), [7, 6, 5, 4, 3, 2, 1, 0], "bf16")
    first = check(s, "first")
    st = torch.cuda.Stream()
    for _ in range(3):
        y = L.lora_linear(*s.values(), stream=st.cuda_stream)
        st.synchronize()
        assert torch.equal(y, first)   # fixed order of sums


def test_graph_replays():
    s = make(20, 512, 256, 16, 3, [0, 9, 20], [2, 0], "bf16")
    L.lora_linear(*s.values())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = L.lora_linear(*s.values())
    for i in range(4):
        s["x"].copy_(torch.randn(20, 512, generator=torch.Generator().manual_seed(i)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, L.lora_linear(*s.values())), i
        torch.cuda.synchronize()


MORE = [  # T, K, N, rank, adapters, row_starts, ids, dtype, bias
    # runs of the sums' axis beside the low-rank values; groups of 4 rows with up to 4 adapters
    (66, 2056, 200, 8, 4, [0, 1, 2, 3, 64, 66], [3, -1, 1, 0, 2], "bf16", True),
    (128, 4096, 320, 33, 2, [0, 63, 128], [1, 0], "f16", True),
    (257, 1544, 129, 64, 3, [0, 2, 129, 130, 257], [0, 1, 2, 0], "bf16", False),
    (1000, 1032, 4104, 16, 9, list(range(0, 1000, 125)) + [1000], list(range(8)), "bf16", True),
    (1024, 72, 65, 128, 2, [0, 1022, 1024], [0, 1], "f16", True),
    (130, 2064, 70, 9, 3, [0, 65, 130], [2, 0], "f32", True),
    (700, 520, 1100, 32, 3, [0, 300, 301, 700], [1, 0, 2], "f32", True),
    # low-rank values first, then the product
    (1025, 136, 192, 128, 3, [0, 500, 501, 1025], [2, 0, 1], "f16", True),
    (3000, 264, 2500, 64, 6, [0, 1, 40, 700, 701, 2999, 3000], [5, 4, -1, 2, 1, 0], "bf16", True),
    (1500, 520, 2052, 24, 2, [0, 1499, 1500], [0, 1], "f32", True),
    (1100, 2048, 70, 128, 2, [0, 40, 1100], [0, 1], "f32", False),
]


@pytest.mark.parametrize("case", MORE, ids=lambda c: "-".join(map(str, c[:5])) + "-" + c[7])
def test_more_rows_against_64_bits(case):
    T, K, N, rank, n, starts, ids, dtype, bias = case
    check(make(T, K, N, rank, n, starts, ids, dtype, bias, seed=4), str(case[:5]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [7, 200, 1400])
def test_an_adapter_that_is_not_finite_stays_with_its_rows(T, dtype):
    """Infinities and NaN in one request's adapter do not reach the others' rows."""
    cut = [0, 3, T // 2, T - 2, T]
    s = make(T, 128, 96, 16, 4, cut, [0, 1, 2, -1], dtype)
    want, bound = C.lora(*s.values())
    s["a"][1].fill_(float("inf"))
    s["b"][1].fill_(float("nan"))
    s["b"][3].fill_(float("nan"))   # nobody's
    y = L.lora_linear(*s.values())
    torch.cuda.synchronize()
    rows = torch.tensor([t for t in range(T) if not 3 <= t < T // 2])
    C.assert_within(y.cpu()[rows], want[rows], bound[rows], f"rows of other adapters, {T}")
    assert bool(torch.isnan(y[3:T // 2]).all())
