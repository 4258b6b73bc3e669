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


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_appending_token_by_token(codes):
    """A block's scale grows with its largest value, earlier codes with it, and never falls."""
    cache = C.Cache(2, [80, 80], 16, 3, 64, codes)
    cache.lengths.zero_()
    g = torch.Generator().manual_seed(3)
    for step in range(40):
        k, v = (torch.randn(2, 3, 64, generator=g).mul(2.0 ** (step % 7 - 3)).bfloat16().cuda()
                for _ in "kv")
        cache.lengths += 1
        write_and_check(cache, k, v, C.starts([1, 1]), f"step {step}")


@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_extreme_values(codes, dtype):
    """Zeros, the smallest and largest numbers, infinities, NaN, numbers on a code's border."""
    t = C.TYPES[dtype]
    cache = C.Cache(6, [20] * 6, 16, 2, 64, codes, seed=2)
    k, v = rows_of(6 * 20, 2, 64, dtype)
    k[:20] = 0
    v[:20] = torch.finfo(t).tiny * 2.0 ** -3
    k[20:40] = torch.finfo(t).max
    k[40, 0, 3], k[41, 1, 5], v[45, 0, 0] = math.inf, -math.inf, math.nan
    k[60:80, :, ::2] = math.nan
    v[60:80] = math.inf
    steps = torch.arange(64, device="cuda") - 31.5
    k[80:100], v[80:100] = steps.to(t), (steps * 3).to(t)
    k[100:120, :, 0] = 127.0
    write_and_check(cache, k, v, C.starts([20] * 6), "extreme")


def test_old_scales_that_are_no_numbers():
    """What a block's earlier tokens are worth then: nothing."""
    cache = C.Cache(5, [9] * 5, 16, 1, 32, "i8", seed=4)
    for b, s in enumerate([math.nan, math.inf, -1.0, 0.0, 0.3]):
        cache.ks[cache.table[b, 0].long()] = s
    k, v = rows_of(5, 1, 32, "bf16")
    write_and_check(cache, k, v, C.starts([1] * 5), "old scales")


def test_blocks_that_are_not_there_and_clamps():
    cache = C.Cache(4, [70, 70, 70, 70], 16, 2, 64, "e4m3", seed=5)
    cache.table[0, 2] = -1
    cache.table[1] = 1 << 29
    cache.lengths = torch.tensor([70, 70, 1 << 30, -3]).int().cuda()
    k, v = rows_of(200, 2, 64, "bf16")
    write_and_check(cache, k, v, torch.tensor([-4, 60, 90, 140, 999]).int().cuda(), "missing")
    out = torch.full((4, 80, 2, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, k_out=out, v_out=out.clone())
    torch.cuda.synchronize()
    assert bool((out[1] == 4.0).all()) and bool((out[3] == 4.0).all())
    assert bool((out[0, 32:48] == 4.0).all()) and not bool((out[0, :32] == 4.0).all(-1).any())


def test_round_trip_into_dense_attention():
    """Written, read back and attended to by prefix_attention: as cache_attention does."""
    rows, lengths = [33, 1, 60], [33, 200, 180]
    cache = C.Cache(3, lengths, 32, 2, 64, "i8", empty=True)
    for s in (cache.ks, cache.vs):
        s.zero_()
    k, v = rows_of(sum(lengths), 2, 64, "f32")
    everything = C.starts(lengths)
    L.kv_cache_write(k, v, *cache.operands(), everything, cache.lengths, cache.table)
    kd, vd = L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, dtype=torch.float32,
                             rows=max(lengths))
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(lengths):
        # half a step of the scale at most: 1/2 of the 64th part of the largest in a block
        for got, x in ((kd, k), (vd, v)):
            assert float((got[b, :n] - x[at:at + n]).abs().max()) <= float(x[at:at + n].abs().max()) / 127
            assert bool((got[b, n:] == 0).all())
        at += n
    q = torch.randn(3, 60, 4, 64, generator=torch.Generator().manual_seed(2)).cuda()
    dense = L.prefix_attention(q, None, None, kd, vd, cache.lengths)
    ragged = L.cache_attention(torch.cat([q[b, 60 - n:] for b, n in enumerate(rows)]),
                               *cache.operands(), C.starts(rows), cache.lengths, cache.table)
    torch.cuda.synchronize()
    want = torch.cat([dense[b, 60 - n:] for b, n in enumerate(rows)])
    # either is off by about 200 half steps of fp32 of the values' magnitude
    assert float((ragged - want).abs().max()) <= 400 * 2.0 ** -24 * float(vd.abs().max())


def test_strides_and_offsets_past_32_bits():
    far = (1 << 32) + 4096
    room = torch.zeros(2 * far + 65536, dtype=torch.int8, device="cuda")
    cache = C.Cache(1, [40], 16, 2, 64, "i8", spare=0)
    k = room.as_strided((3, 16, 2, 64), (far, 64, 1024, 1))
    k.copy_(cache.k)
    cache.k = k
    fused = torch.randn(24, 8, 64, generator=torch.Generator().manual_seed(6)).half().cuda()
    write_and_check(cache, fused[:, 2:4], fused[:, 6:], C.starts([24]), "far")
    out = torch.zeros(1, 40, 2, 2, 64, dtype=torch.float16, device="cuda")
    L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, k_out=out[:, :, 0],
                    v_out=out[:, :, 1])
    torch.cuda.synchronize()
    for i, name in enumerate("kv"):
        assert torch.equal(out[0, :, i].cpu(), C.of_entry(cache, 0, name)[0].half())


def test_graph_replays():
    cache = C.Cache(3, [200] * 3, 16, 2, 64, "e4m3", seed=7)
    cache.lengths.copy_(torch.tensor([3, 50, 100]))
    k, v = rows_of(3, 2, 64, "bf16")
    out = torch.zeros(3, 208, 2, 64, dtype=torch.bfloat16, device="cuda")
    v_out = torch.zeros_like(out)

    def step():
        L.kv_cache_write(k, v, *cache.operands(), starts, cache.lengths, cache.table)
        L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, k_out=out, v_out=v_out)

    starts = C.starts([1, 1, 1])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        cache.lengths += 1
        k.copy_(rows_of(3, 2, 64, "bf16", seed=30 + i, by=1.0 + i)[0])
        want = C.write(cache, k, v, starts)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, dense, (codes, scale) in zip("kv", (out, v_out), want):
            assert torch.equal(cache.host(name)[0], codes) and torch.equal(cache.host(name)[1], scale)
            for b, n in enumerate(cache.lengths.tolist()):
                assert torch.equal(dense[b, :n].cpu(), C.of_entry(cache, b, name)[0].bfloat16())
