"""kv_cache_write and kv_cache_read on the GPU against their definitions, code for code."""
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


def rows_of(T, hk, d, dtype, seed=1, by=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda: (torch.randn(T, hk, d, generator=g) * by).to(C.TYPES[dtype]).cuda()
    return r(), r()


def write_and_check(cache, k, v, starts, what=""):
    print(f"[gpu] cache write {what} {tuple(k.shape)}", flush=True)
    want = C.write(cache, k, v, starts)
    L.kv_cache_write(k, v, *cache.operands(), starts, cache.lengths, cache.table)
    torch.cuda.synchronize()
    for name, (codes, scale) in zip(("k", "v"), want):
        got, got_scale = cache.host(name)
        assert torch.equal(got_scale, scale), (what, name)
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(codes, nan=1e9)), \
            (what, name, torch.nonzero(got != codes)[:5].tolist())


CASES = [  # rows, lengths, heads, head_dim, block, codes, dtype
    ([1], [1], 1, 16, 16, "i8", "bf16"),
    ([1, 1, 1], [16, 17, 40], 4, 128, 16, "e4m3", "bf16"),
    ([1, 5, 0, 33], [1000, 5, 20, 64], 3, 80, 32, "i8", "f16"),
    ([100, 17], [130, 17], 2, 64, 64, "e4m3", "f32"),
    ([300, 1, 90], [300, 256, 257], 2, 128, 128, "i8", "f32"),
    ([517, 2], [600, 300], 5, 48, 256, "e4m3", "f16"),
    ([9], [4], 2, 32, 16, "i8", "bf16"),                   # the first 5 rows have no position
    ([1] * 40, [3 * i + 1 for i in range(40)], 2, 64, 32, "e4m3", "bf16"),
]


@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:4]}-{c[1][:4]}-{c[2:]}")
def test_write(case, tokens_first):
    rows, lengths, hk, d, block, codes, dtype = case
    cache = C.Cache(len(rows), lengths, block, hk, d, codes, tokens_first=tokens_first)
    k, v = rows_of(sum(rows), hk, d, dtype)
    write_and_check(cache, k, v, C.starts(rows), str(case))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("hk,d,block", [(1, 16, 16), (5, 80, 32), (8, 128, 64), (2, 112, 256)])
def test_read(hk, d, block, codes, out):
    lengths = [0, 1, block, 3 * block + 7, 41]
    cache = C.Cache(5, lengths, block, hk, d, codes)
    print(f"[gpu] cache read {hk} heads of {d}, blocks of {block}, {codes}, {out}", flush=True)
    S = max(lengths) - 3
    k_out, v_out = (torch.full((5, S, hk, d), 7.0, dtype=C.TYPES[out], device="cuda") for _ in "kv")
    L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, k_out=k_out, v_out=v_out)
    torch.cuda.synchronize()
    for name, got in (("k", k_out), ("v", v_out)):
        for b, n in enumerate(lengths):
            want, _ = C.of_entry(cache, b, name)
            n = min(n, S)
            assert torch.equal(got[b, :n].cpu(), want[:n].to(C.TYPES[out])), (name, b)
            assert bool((got[b, n:] == 7.0).all()), (name, b)
