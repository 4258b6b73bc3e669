"""linear's GELU over its whole range, relative to its values: also where they are small, in its negative
tail."""
import math

import pytest

torch = pytest.importorskip("torch")
scipy_special = pytest.importorskip("scipy.special")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gelu(v):
    """v Phi(v) in 64 bits, right in both tails."""
    a = v.abs().numpy() / math.sqrt(2.0)
    c = torch.from_numpy(0.5 * scipy_special.erfcx(a)) * torch.exp(-0.5 * v * v)
    return v * torch.where(v > 0, 1 - c, c)


@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("T,N", [(8, 1400), (600, 700)])   # in runs or small tiles; in large ones
def test_gelu_relative_to_its_values(T, N, dtype):
    t = C.TYPES[dtype]
    x = torch.zeros(T, 8, dtype=t)
    x[:, 0] = 1
    w = torch.zeros(N, 8, dtype=t)
    w[:, 0] = torch.linspace(-14, 14, N).to(t)       # sums of one product, which is exact
    print(f"[gpu] gelu {dtype} {T} x {N}", flush=True)
    y = L.linear(x.cuda(), w.cuda(), act="gelu").double().cpu()
    torch.cuda.synchronize()
    v = w[:, 0].double().expand(T, N)
    want = gelu(v)
    if dtype == "f32":
        # half steps of 2^-24: erfcx 16 (8 last places), its argument 3 (a relative error of the
        # argument counts once at most), exp 4, the square's correction 2, products 4, v Phi 1
        rel = 30 * C.U32 * torch.ones_like(v)
    else:
        # the polynomial 2^-17.4 (its fit and its coefficients' rounding), its steps, the reciprocal
        # and the products 20 half steps, the exponent v^2 / 2 off by 3 of its own
        rel = C.U[t] + (1 + C.U[t]) * (2.0 ** -17.4 + C.U32 * (20 + 3 * v * v / 2))
    # exponentials below 2^-126 may be 0 or have fewer bits
    C.assert_within(y, want, rel * want.abs() + C.tiny(t) + 16 * 2.0 ** -126, dtype)


@pytest.mark.parametrize("dtype", C.TYPES)
def test_gelu_at_the_ends(dtype):
    t = C.TYPES[dtype]
    most = torch.finfo(t).max
    x = torch.tensor([0.0, -0.0, 100.0, -100.0, most, -most, math.inf, math.nan]).to(t)
    rows = torch.zeros(len(x), 8, dtype=t)
    rows[:, 0] = x
    w = torch.zeros(3, 8, dtype=t)
    w[:, 0] = 1
    y = L.linear(rows.cuda(), w.cuda(), act="gelu")[:, 0].cpu()
    torch.cuda.synchronize()
    assert y[:2].tolist() == [0, 0] and y[2] == 100 and y[3] == 0 and y[4] == most and y[5] == 0
    assert math.isinf(y[6]) and y[6] > 0 and math.isnan(y[7])
