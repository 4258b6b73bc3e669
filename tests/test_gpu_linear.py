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
