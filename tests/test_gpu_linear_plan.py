"""linear on the GPU at sizes where its tiles leave compute units idle, in runs and without."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402
from test_gpu_linear import _needs_gpu, check, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,dtype", [
    (136, 3624, 3934, "f32"), (367, 3848, 2691, "f32"), (223, 2360, 469, "f32"), (5, 3992, 6718, "f32"),
    (79, 648, 82, "f32"), (2000, 4096, 330, "f32"), (98, 3864, 6037, "bf16"), (300, 4104, 2700, "f16"),
    (1462, 688, 188, "bf16")], ids=str)
def test_runs_beside_more_tiles(T, K, N, dtype):
    x, w, b, r = make(T, K, N, dtype, seed=5)
    first = check(x, w, b, "silu", r)
    assert torch.equal(first, L.linear(x, w, b, act="silu", residual=r))
    check(x, w, None, "none", None, workspace=False)


def test_more_rows_than_a_launch_has():
    """Rows past 65535, which are not in runs."""
    x, w, b, r = make(65600, 2056, 70, "bf16", seed=6)
    y = L.linear(x, w, b, act="relu", residual=r)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(100), torch.arange(65500, 65600)])
    want, bound = C.linear(x[at], w, b, "relu", r[at])
    C.assert_within(y[at.cuda()], want, bound, "ends")
