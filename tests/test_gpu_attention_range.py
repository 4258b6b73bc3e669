"""prefix_attention with probabilities far apart: one key far above tens of thousands of others."""
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


# Sq, heads, keys, log2 of how far the others lie below: few rows, whose waves take a quarter of
# the keys each, and many, whose waves share their keys
CASES = [(1, 1, 65536, 25.0), (1, 2, 65536, 14.5), (3, 1, 65536, 30.25), (130, 70, 32768, 25.0),
         (130, 70, 32768, 14.5), (130, 70, 65536, 30.25)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_probabilities_count(case, workspace, dtype):
    """Each of the others is less than the type's smallest number beside the one key, together
    they are not; the one key's values are 0, so that they alone make up the output."""
    Sq, H, N, below = case
    t, D, scale = C.TYPES[dtype], 8, math.log(2.0)
    print(f"[gpu] attention {case} {dtype}", flush=True)
    g = torch.Generator().manual_seed(3)
    q = torch.zeros(1, Sq, H, D, dtype=t)
    q[..., 0] = 1.0
    k = torch.zeros(1, N + 1, H, D, dtype=t)
    k[..., 0] = 32.0 - below
    k[:, 0, :, 0] = 32.0
    v = torch.rand(1, N + 1, H, D, generator=g).to(t)
    v[:, 0] = 0.0
    n = torch.tensor([N + 1]).int().cuda()
    out, lse = L.prefix_attention(q.cuda(), None, None, k.cuda(), v.cuda(), n, scale=scale,
                                  causal=False, return_lse=True, workspace=workspace)
    torch.cuda.synchronize()
    r = 2.0 ** (float(k[0, 1, 0, 0]) - 32.0)
    total = 1.0 + N * r
    want = (r / total * v.double().sum(1))[:, None].expand(1, Sq, H, D)
    # as in layercheck: scores off by D + 4 half steps of their size, sums of N + 1 terms, the
    # probabilities and the output rounded to the type.  Half a step of fp16's smallest numbers
    # (2^-25) for each probability beside a largest one of 2^11 or more.
    off = C.U32 * (2 * (D + 4) * 32 * scale + 2 * (N + 1) + 64)
    smallest = 2.0 ** -36 / total * v.double().sum(1) if dtype == "f16" else torch.zeros(1)
    bound = (2 * C.U[t] + off) * want + smallest.reshape(1, 1, -1, D if dtype == "f16" else 1) + \
        C.tiny(t)
    C.assert_within(out, want, bound, f"out {case}")
    want = torch.full((1, H, Sq), 32.0 * scale + math.log(total)).double()
    C.assert_within(lse, want, torch.full_like(want, off + C.U32 * 8 * (1 + 32 * scale)), "lse")
