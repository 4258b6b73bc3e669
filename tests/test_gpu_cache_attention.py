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


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("case", [
    # enough rows that they share their tiles, in one share of the keys and in several
    ([300, 270], [700, 271], 64, 8, 64, 16, True, "bf16"),
    ([260, 1, 200], [300, 900, 1300], 32, 8, 128, 64, True, "bf16"),
    ([129, 400], [2000, 400], 16, 4, 80, 32, True, "f16"),
    ([513], [4200], 8, 4, 128, 128, True, "f16"),
    ([200, 333], [1500, 40], 16, 8, 64, 16, True, "f32"),
    ([300, 300], [290, 0], 32, 16, 96, 16, False, "bf16"),
    ([140] * 3, [1100, 640, 576], 24, 3, 112, 256, True, "f32"),
    ([40] * 9, [1000 + 31 * i for i in range(9)], 40, 10, 48, 32, True, "bf16"),
], ids=str)
def test_many_rows_against_64_bits(case, codes):
    rows, lengths, hq, hk, d, block, causal, dtype = case
    cache = C.Cache(len(rows), lengths, block, hk, d, codes, seed=3)
    q = queries(sum(rows), hq, d, dtype, seed=4)
    first = check(q, cache, C.starts(rows), causal, what=str(case), max_rows=max(rows))
    again = check(q, cache, C.starts(rows), causal, what="alone", max_rows=max(rows),
                  workspace=False)
    third = L.cache_attention(q, *cache.operands(), C.starts(rows), cache.lengths, cache.table,
                              causal=causal, max_rows=max(rows))
    torch.cuda.synchronize()
    assert torch.equal(first, third)
    assert bool(torch.isfinite(again).all())


SHAPES = [([1, 1, 1], [70, 1500, 2300], "bf16"), ([200, 300, 1], [700, 900, 2300], "bf16"),
          ([200, 300, 1], [700, 900, 2300], "f16"), ([3, 150, 2], [70, 600, 1100], "f32")]


@pytest.mark.parametrize("rows,lengths,dtype", SHAPES, ids=str)
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_scales_that_are_no_powers_of_two(rows, lengths, dtype, codes):
    cache = C.Cache(len(rows), lengths, 16, 8, 64, codes, seed=5)
    g = torch.Generator().manual_seed(6)
    for s in (cache.ks, cache.vs):
        s.mul_((0.5 + torch.rand(s.shape, generator=g)).cuda())
    check(queries(sum(rows), 32, 64, dtype), cache, C.starts(rows), True, what="scales")


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype,least,most", [("f16", -15, 7), ("bf16", -117, 100)])
def test_scales_at_the_ends_of_the_16_bit_types(codes, dtype, least, most):
    """Powers of two whose products with codes just fit the type, and the next ones.  (bfloat16's
    last ones, from 2^119 on, are past what the operator allows: sums of 1300 values of 2^126 pass
    fp32's range before they are divided.)"""
    rows, lengths = [300, 1], [900, 1300]
    q = queries(sum(rows), 16, 64, dtype)
    for e in (least - 1, least, most, most + 1):
        if dtype == "f16":   # (sums of products with bfloat16's would pass fp32's range)
            cache = C.Cache(2, lengths, 32, 4, 64, codes, seed=15)
            cache.ks.fill_(2.0 ** e)
            check(q, cache, C.starts(rows), True, scale=2.0 ** (-e - 9), what=f"keys 2^{e}")
        cache = C.Cache(2, lengths, 32, 4, 64, codes, seed=16)
        cache.vs.fill_(2.0 ** e)
        check(q, cache, C.starts(rows), True, what=f"values 2^{e}")


@pytest.mark.parametrize("rows,lengths,dtype", SHAPES, ids=str)
def test_blocks_that_are_not_there(rows, lengths, dtype):
    """A window that has moved on, and holes; an entry without any block."""
    cache = C.Cache(len(rows), lengths, 32, 8, 128, "e4m3", seed=7)
    cache.table[1, :9] = -1
    cache.table[2, 3::2] = 1 << 30
    cache.table[0] = -7
    out = check(queries(sum(rows), 16, 128, dtype), cache, C.starts(rows), True, what="holes")
    assert bool((out[:rows[0]] == 0).all())


@pytest.mark.parametrize("rows,lengths,dtype", SHAPES, ids=str)
@pytest.mark.parametrize("block", [16, 128])
def test_what_lies_past_the_length_is_not_read(rows, lengths, dtype, block):
    """NaN codes and scales in blocks of nobody, and NaN codes behind the last token."""
    cache = C.Cache(len(rows), lengths, block, 8, 64, "e4m3", seed=8, width=200)
    q = queries(sum(rows), 8, 64, dtype)
    want = check(q, cache, C.starts(rows), True, what="clean")
    used = torch.zeros(len(cache.k), dtype=torch.bool)
    for b, n in enumerate(lengths):
        at = cache.table[b].cpu().long()
        used[at[:-(-n // block)]] = True
        for x in (cache.k, cache.v):
            x.view(torch.uint8)[int(at[n // block]), n % block:] = 0x7f
    for x, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        x.view(torch.uint8)[~used.cuda()] = 0x7f
        s[~used.cuda()] = math.nan
    got = L.cache_attention(q, *cache.operands(), C.starts(rows), cache.lengths, cache.table)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.1])
@pytest.mark.parametrize("rows", [[1, 2], [250, 200]], ids=str)
def test_scales(scale, rows):
    cache = C.Cache(2, [300, 777], 16, 8, 64, "i8", seed=9)
    check(queries(sum(rows), 16, 64, "bf16"), cache, C.starts(rows), True, scale=scale,
          what=f"scale {scale}")


def test_lengths_and_starts_out_of_range_are_clamped():
    cache = C.Cache(3, [40, 40, 40], 16, 2, 64, "i8")
    cache.lengths = torch.tensor([-5, 1 << 30, 30]).int().cuda()
    starts = torch.tensor([-3, 2, 4, 900]).int().cuda()
    check(queries(7, 4, 64, "bf16"), cache, starts, True, what="clamped")


def test_rows_of_no_entry_and_past_max_rows_are_left():
    cache = C.Cache(2, [40, 700], 16, 2, 64, "e4m3")
    q = queries(60, 4, 64, "bf16")
    out = torch.full_like(q, 3.0)
    starts = torch.tensor([2, 4, 50]).int().cuda()
    check(q, cache, starts, True, what="gaps", out=out)
    assert bool((out[:2] == 3.0).all()) and bool((out[50:] == 3.0).all())
    want, out = out.clone(), torch.full_like(q, 3.0)
    L.cache_attention(q, *cache.operands(), starts, cache.lengths, cache.table, max_rows=10, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[2:14], want[2:14]) and bool((out[14:] == 3.0).all())


@pytest.mark.parametrize("rows", [[1, 1], [1, 300]], ids=str)
def test_strides(rows):
    """Queries from a fused projection, a strided output, keys and values of a block side by side."""
    cache = C.Cache(2, [333, 900], 32, 4, 64, "i8", seed=11)
    both = torch.empty(len(cache.k), 2, 32, 4, 64, dtype=torch.int8, device="cuda")
    both[:, 0], both[:, 1] = cache.k, cache.v
    cache.k, cache.v = both[:, 0], both[:, 1]
    T = sum(rows)
    fused = queries(T, 16, 64, "bf16")
    out = torch.full((T, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    check(fused[:, 3:11], cache, C.starts(rows), True, what="strided", out=out[..., :64])
    assert bool((out[..., 64:] == 5.0).all())


def test_offsets_past_32_bits():
    """Blocks more than 2^32 bytes apart."""
    far = (1 << 32) + 4096
    room = torch.zeros(2 * far + 65536, dtype=torch.int8, device="cuda")
    cache = C.Cache(1, [40], 16, 2, 64, "i8", spare=0)
    for rows in ([1], [70]):
        k = room.as_strided((3, 16, 2, 64), (far, 64, 1024, 1))
        k.copy_(cache.k)
        cache.k, v = k, cache.v
        check(queries(rows[0], 4, 64, "bf16"), cache, C.starts(rows), True, what="far")
        cache.v = k
        check(queries(rows[0], 4, 64, "bf16"), cache, C.starts(rows), True, what="far values")
        cache.v = v


@pytest.mark.parametrize("lengths", [[900, 1500, 2000], [100, 400, 5]], ids=str)
def test_graph_replays(lengths):
    """Lengths, tables and starts change between replays; a plan with partial results and one
    without."""
    cache = C.Cache(3, [2048] * 3, 16, 4, 128, "e4m3", seed=12)
    q, starts = queries(300, 16, 128, "bf16"), C.starts([1, 298, 1])
    cache.lengths = torch.tensor(lengths).int().cuda()
    call = lambda: L.cache_attention(q, *cache.operands(), starts, cache.lengths, cache.table)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        q.copy_(queries(300, 16, 128, "bf16", seed=20 + i))
        starts.copy_(C.starts([[1, 298, 1], [298, 1, 1], [100, 100, 100], [0, 290, 10]][i]))
        cache.lengths.copy_((cache.lengths + 7 * i) % 2048)
        cache.table.copy_(cache.table[:, torch.randperm(cache.width)])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()), i
        torch.cuda.synchronize()


def test_scores_that_climb_and_fall():
    """Scales of keys from 2^-20 to 2^6 from block to block: the maximum moves far."""
    for rows in ([1, 1], [260, 200]):
        for ramp in (range(-20, 7), range(6, -21, -1)):
            cache = C.Cache(2, [27 * 16, 300], 16, 8, 64, "i8", seed=13)
            for b in range(2):
                n = min(27, cache.width)
                cache.ks[cache.table[b, :n].long()] = torch.tensor(
                    [2.0 ** (e - 4) for e in ramp][:n], device="cuda")[:, None]
            check(queries(sum(rows), 8, 64, "bf16"), cache, C.starts(rows), True, what=str(ramp))


def test_more_entries_than_a_wave_has_lanes():
    n = 150
    cache = C.Cache(n, [(37 * i) % 1300 for i in range(n)], 16, 2, 64, "i8", seed=14)
    rows = [[1, 0, 2, 1, 40][i % 5] for i in range(n)]
    check(queries(sum(rows), 4, 64, "bf16"), cache, C.starts(rows), True, what="entries")
    one = C.starts([1] * n)
    check(queries(n, 4, 64, "bf16"), cache, one, True, what="single tokens", max_rows=1)


@pytest.mark.parametrize("B", [5, 64, 130])
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_keys_shared_by_workgroups(B, codes):
    """Entries of very different lengths, some empty, whose keys workgroups share."""
    g = torch.Generator().manual_seed(B)
    lengths = torch.randint(0, 200, (B,), generator=g).tolist()
    lengths[1], lengths[3], lengths[-1] = 4096, 0, 3001
    cache = C.Cache(B, lengths, 64, 2, 64, codes, seed=17, width=80)
    check(queries(B, 8, 64, "bf16"), cache, C.starts([1] * B), True, what=f"{B} entries")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_keys_are_shared(dtype, d):
    """Up to 32 rows of a key head, in parts of several workgroups."""
    cache = C.Cache(4, [5000, 33, 2500, 129], 32, 2, d, "e4m3", seed=18)
    check(queries(10, 16, d, dtype), cache, C.starts([3, 1, 4, 2]), True, max_rows=4, what="32 rows")


def test_nothing_to_do():
    cache = C.Cache(2, [5, 5], 16, 2, 64, "i8")
    q = queries(0, 4, 64, "bf16")
    assert L.cache_attention(q, *cache.operands(), C.starts([0, 0]), cache.lengths,
                             cache.table).shape == (0, 4, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    L.cache_attention(queries(3, 4, 64, "bf16"), *cache.operands(), C.starts([]), none,
                      torch.zeros(0, 4, dtype=torch.int32, device="cuda"), out=out)
    # a table of no blocks: entries without tokens
    L.cache_attention(queries(3, 4, 64, "bf16"), *cache.operands(), C.starts([1, 1]), cache.lengths,
                      cache.table[:, :0].contiguous(), out=out)
    torch.cuda.synchronize()
    assert bool((out[:2] == 0).all()) and bool((out[2] == 2.0).all())


@pytest.mark.parametrize("B", [3, 70, 600])
def test_many_entries_of_many_rows(B):
    """Sets of rows side by side and entry by entry, one with most of the rows among them."""
    rows = [[40, 0, 33, 1][i % 4] for i in range(B)]
    rows[B // 2] = 900
    cache = C.Cache(B, [n + 11 * (i % 20) for i, n in enumerate(rows)], 16, 2, 16, "i8", seed=15)
    q = queries(sum(rows), 4, 16, "bf16")
    first = check(q, cache, C.starts(rows), True, what=str(B))
    again = check(q, cache, C.starts(rows), True, what="max_rows", max_rows=900)
    assert torch.equal(first, again)


def test_the_most_entries():
    """65536 entries, few of them with rows; one with many."""
    n = 65536
    cache = C.Cache(n, [1 + i % 16 for i in range(n)], 16, 1, 16, "i8", seed=19)
    rows = [1 if i % 97 == 0 else 0 for i in range(n)]
    check(queries(sum(rows), 2, 16, "bf16"), cache, C.starts(rows), True, what="single", max_rows=1)
    rows[40000] = 50
    check(queries(sum(rows), 2, 16, "bf16"), cache, C.starts(rows), True, what="and one of 50")
    check(queries(sum(rows), 2, 16, "bf16"), cache, C.starts(rows), True, what="max_rows",
          max_rows=50)
