"""lora_linear with infinities and NaN: what the formula gives, whatever the number of rows."""
import math

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(T, K, N, rank, starts, ids, dtype, seed=5):
    g = torch.Generator().manual_seed(seed)
    t = C.TYPES[dtype]
    r = lambda *s, by=1.0: (by * torch.randn(*s, generator=g)).to(t)
    n = 3
    return dict(x=r(T, K), w=r(N, K, by=K ** -0.5), bias=r(N), a=r(n, rank, K, by=K ** -0.5),
                b=r(n, N, rank), scales=torch.rand(n, generator=g) + 0.5,
                row_starts=torch.tensor(starts).int(), adapters=torch.tensor(ids).int())


# what is planted; even outputs have rows of b of one sign, so that infinities of one sign there
# do not meet
def x_infinite(s):
    s["a"][:, :, 3] = s["a"][:, :, 3].abs()
    s["x"][5, 3], s["x"][-2, 3] = INF, -INF


def x_nan(s):
    s["x"][7, 0] = NAN


def a_infinite(s):
    s["a"][1, :, 2] = INF


def a_one_rank(s):
    s["a"][1, 1, 2], s["a"][2, 0, 4] = -INF, INF


def b_infinite(s):
    s["b"][1, 4, 0], s["b"][1, 6, 1], s["b"][2, 7, 0] = INF, -INF, INF


def b_two(s):
    s["b"][1, 4, 0], s["b"][1, 4, 2], s["b"][0, 10, 1] = INF, -INF, NAN


def a_and_b(s):
    s["a"][1, 0, 2], s["b"][1, 4, 0], s["b"][1, 6, 1], s["b"][1, 7, 0] = INF, INF, -INF, NAN


def a_infinite_b_zero(s):
    s["a"][1, 0, 2] = INF
    s["b"][1, 4, 0] = 0.0


PLANT = [x_infinite, x_nan, a_infinite, a_one_rank, b_infinite, b_two, a_and_b, a_infinite_b_zero]
SIZES = [  # T, K, N, rank, row_starts, ids
    (9, 64, 40, 4, [0, 4, 9], [1, 2]),
    (200, 64, 70, 8, [0, 90, 150, 200], [0, 1, 2]),
    (1000, 72, 70, 4, [0, 3, 500, 1000], [1, 2, 1]),
    (1100, 72, 70, 4, [0, 3, 500, 1100], [1, 2, 1]),        # tiles of several adapters
    (1100, 72, 70, 8, [0, 1100], [1]),                       # of one
    (1300, 136, 1100, 33, [0, 3, 512, 1300], [2, 1, -1]),
    (2200, 72, 2052, 16, [0, 1024, 1030, 2200], [1, 2, 0]),
]


@pytest.mark.parametrize("plant", PLANT, ids=lambda f: f.__name__)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_as_the_formula_has_it(size, dtype, plant):
    print(f"[gpu] lora {size} {dtype} {plant.__name__}", flush=True)
    s = make(*size, dtype)
    s["b"][:, ::2] = s["b"][:, ::2].abs()
    plant(s)
    y = L.lora_linear(*[v.cuda() for v in s.values()]).cpu().double()
    want, bound = C.lora(*s.values())
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    infinite = torch.isinf(want)
    assert torch.equal(torch.isinf(y), infinite)
    assert torch.equal(y[infinite], want[infinite])
    finite = torch.isfinite(want)
    assert bool((~finite).any())
    C.assert_within(y[finite], want[finite], bound[finite], str(size))


@pytest.mark.parametrize("T", [40, 1100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_low_rank_value_at_the_end_of_the_range(T, dtype):
    """A finite value that bfloat16 would round to an infinity."""
    s = make(T, 64, 48, 2, [0, T], [1], dtype)
    s["x"].zero_()
    s["a"].zero_()
    s["x"][:, 0], s["a"][1, 0, 0] = 1.0, 1.0
    s["b"].mul_(1e-30)
    s["scales"].fill_(3.4e38)   # past 2^128 (1 - 2^-9)
    y = L.lora_linear(*[v.cuda() for v in s.values()])
    want, bound = C.lora(*s.values())
    C.assert_within(y, want, bound, "large")
