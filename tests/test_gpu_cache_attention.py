"""cache_attention on the GPU against its plain form in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def queries(T, hq, d, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, hq, d, generator=g).to(C.TYPES[dtype]).cuda()


def check(q, cache, starts, causal, scale=None, what="", **kw):
    print(f"[gpu] cache attention {what} q{tuple(q.shape)} causal={causal}", flush=True)
    out, lse = L.cache_attention(q, *cache.operands(), starts, cache.lengths, cache.table,
                                 scale=scale, causal=causal, return_lse=True, **kw)
    torch.cuda.synchronize()
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want, bound, wl, bl = C.attention(q, cache, starts, s, causal)
    mine = ~torch.isnan(wl[:, 0])
    C.assert_within(out[mine.cuda()], want[mine], bound[mine], f"out {what}")
    C.assert_within(lse[mine.cuda()], wl[mine], bl[mine], f"lse {what}")
    return out


CASES = [  # rows, lengths, query heads, key heads, head_dim, block, codes, causal, dtype
    ([1], [1], 1, 1, 64, 16, "i8", True, "bf16"),
    ([1, 1], [0, 17], 4, 2, 128, 16, "e4m3", True, "bf16"),
    ([1] * 5, [31, 32, 33, 127, 129], 8, 2, 128, 32, "i8", True, "f16"),
    ([1] * 3, [1000, 3, 700], 6, 3, 80, 64, "e4m3", True, "f32"),
    ([1, 1], [4097, 260], 16, 1, 64, 128, "i8", True, "bf16"),
    ([1] * 9, [1, 2, 15, 16, 17, 300, 511, 512, 513], 8, 8, 48, 16, "e4m3", True, "f16"),
    ([2, 0, 3, 1], [40, 10, 3, 900], 4, 1, 96, 32, "i8", True, "bf16"),
    ([7, 1, 33], [7, 300, 50], 4, 4, 64, 16, "e4m3", True, "f32"),
    ([40, 1, 1, 65], [140, 600, 1, 65], 8, 2, 128, 64, "e4m3", True, "bf16"),
    ([130, 130], [463, 131], 4, 2, 64, 16, "i8", True, "f32"),
    ([100, 5], [100, 77], 6, 2, 80, 256, "i8", False, "f16"),
    ([257], [300], 2, 1, 128, 32, "e4m3", False, "bf16"),
    ([9], [4], 2, 1, 16, 16, "i8", True, "bf16"),          # more rows than tokens
    ([70, 3], [20, 0], 4, 2, 64, 16, "e4m3", True, "f16"),
    ([1] * 70, [5 * i for i in range(70)], 4, 2, 64, 16, "i8", True, "bf16"),
    ([3] * 3, [2000, 1, 900], 40, 2, 112, 128, "e4m3", True, "bf16"),   # 60 rows a key head
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:4]}-{c[1][:4]}-{c[2:]}")
@pytest.mark.parametrize("workspace", [True, False])
def test_against_64_bits(case, workspace):
    rows, lengths, hq, hk, d, block, codes, causal, dtype = case
    cache = C.Cache(len(rows), lengths, block, hk, d, codes)
    q = queries(sum(rows), hq, d, dtype)
    first = check(q, cache, C.starts(rows), causal, what=str(case), workspace=workspace)
    again = L.cache_attention(q, *cache.operands(), C.starts(rows), cache.lengths, cache.table,
                              causal=causal, workspace=workspace)
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    most = check(q, cache, C.starts(rows), causal, what="max_rows", workspace=workspace,
                 max_rows=max(rows))
    assert bool(torch.isfinite(most).all())
