"""cache_attention's sets of 128 rows of a key head on the GPU against 64 bits.  Every call here says
which sets the plan takes for it, so that no change of the plan's rule takes a test to another kernel
unseen."""
import math

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402
from test_gpu_cache_attention import _needs_gpu, check, queries  # noqa: E402,F401

pytestmark = pytest.mark.gpu

CUS = 256   # that plans are made for


def plan(B, T, most, hq, hk, positions, workspace=True):
    """(rows of a set, shares of its keys) of a batch with an entry of more than 32 rows a key head,
    in a table of that many positions."""
    G = hq // hk
    sets = min(-(-most * G // 128) * B, T * G // 128 + B) * hk
    most = max(min(positions // 512, 32), positions // 2048)
    shares = max(1, min(4 * CUS // sets, most)) if workspace else 1
    return (128, shares) if sets * shares >= CUS // 2 or shares >= 4 else (32, 1)


def of_sets(q, cache, rows, causal=True, workspace=True, **kw):
    """check() of a call whose rows go in sets of 128; (output, tiles of 64 keys of the longest
    share)."""
    B, T, most = len(rows), sum(rows), max(rows)
    (_, hq, d), hk, positions = q.shape, cache.k.shape[2], cache.width * cache.block
    size, shares = plan(B, T, most, hq, hk, positions, workspace)
    assert size == 128
    # the same rule in the library, as far as its workspace tells: rows' partial results of each
    # share, and 64 for each of 512 workgroups that share the keys of few rows
    few = 512 if hq // hk <= 32 and positions >= max(1024, 16 * B * hk) else 0
    each = -(-most * (hq // hk) // 128) * B
    side = min(each, T * (hq // hk) // 128 + B)
    units = (each if each <= 2 * side else side) * hk
    want = (64 * few + (units * 128 * shares if shares > 1 else 0)) * (d + 1) * 4
    if workspace:
        assert L.libconv_cache_attention_workspace(
            B, T, most, cache.block, cache.width, hq, hk, d,
            {torch.float32: L.F32, torch.float16: L.F16, torch.bfloat16: L.BF16}[q.dtype]) == want
    tiles = -(-int(cache.lengths.max()) // 64)
    out = check(q, cache, C.starts(rows), causal, max_rows=most, workspace=workspace, **kw)
    return out, -(-tiles // max(1, min(shares, tiles // 6)))


def test_the_rule():
    assert plan(8, 8 * 2048, 2048, 32, 8, 6144) == (128, 1)
    assert plan(2, 301, 300, 16, 4, 1312) == (32, 1)      # too few sets
    assert plan(1, 513, 513, 8, 4, 4224) == (128, 8)
    assert plan(1, 513, 513, 8, 4, 4224, False) == (32, 1)
    assert plan(1, 16, 16, 16, 4, 131072) == (128, 64)    # few sets, many keys
    assert plan(1, 1, 1, 64, 1, 16384) == (128, 32)
    assert plan(1, 16, 16, 16, 4, 2032) == (32, 1)


ROWS, LENGTHS, HEADS = [400, 300], [520, 333], 20   # 140 sets


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype,least,most", [("f16", -15, 7), ("bf16", -117, 100)])
def test_scales_at_the_ends_of_the_16_bit_types(codes, dtype, least, most):
    """Powers of two whose products with codes just fit the type, and are taken into the widened
    numbers, and the next ones, which are not."""
    q = queries(sum(ROWS), HEADS, 64, dtype)
    for e in (least - 1, least, most, most + 1):
        cache = C.Cache(2, LENGTHS, 32, HEADS, 64, codes, seed=15)
        cache.ks.fill_(2.0 ** e)
        of_sets(q, cache, ROWS, scale=2.0 ** (-e - 9), what=f"keys 2^{e}")
        cache = C.Cache(2, LENGTHS, 32, HEADS, 64, codes, seed=16)
        cache.vs.fill_(2.0 ** e)
        of_sets(q, cache, ROWS, what=f"values 2^{e}")


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.1])
@pytest.mark.parametrize("dtype", C.TYPES)
def test_scales(scale, dtype):
    cache = C.Cache(2, LENGTHS, 16, HEADS, 64, "i8", seed=9)
    of_sets(queries(sum(ROWS), HEADS, 64, dtype), cache, ROWS, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("dtype", C.TYPES)
def test_scores_that_climb_and_fall(dtype):
    """Scales of keys from 2^-20 to 2^6 from block to block: the maximum moves far."""
    for ramp in (range(-20, 7), range(6, -21, -1)):
        cache = C.Cache(2, [27 * 16, 300], 16, HEADS, 64, "i8", seed=13)
        for b in range(2):
            n = min(27, cache.width)
            cache.ks[cache.table[b, :n].long()] = torch.tensor(
                [2.0 ** (e - 4) for e in ramp][:n], device="cuda")[:, None]
        of_sets(queries(sum(ROWS), HEADS, 64, dtype), cache, ROWS, what=str(ramp))


@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_scales_that_are_no_powers_of_two(dtype, codes):
    cache = C.Cache(2, LENGTHS, 16, HEADS, 80, codes, seed=5)
    g = torch.Generator().manual_seed(6)
    for s in (cache.ks, cache.vs):
        s.mul_((0.5 + torch.rand(s.shape, generator=g)).cuda())
    of_sets(queries(sum(ROWS), HEADS, 80, dtype), cache, ROWS, what="scales")


@pytest.mark.parametrize("dtype", C.TYPES)
def test_blocks_that_are_not_there(dtype):
    cache = C.Cache(3, [500, 520, 333], 32, HEADS, 128, "e4m3", seed=7)
    cache.table[1, :9] = -1
    cache.table[2, 3::2] = 1 << 30
    cache.table[0] = -7
    out, _ = of_sets(queries(840, HEADS, 128, dtype), cache, [140, 400, 300], what="holes")
    assert bool((out[:140] == 0).all())


@pytest.mark.parametrize("dtype", C.TYPES)
def test_what_lies_past_the_length_is_not_read(dtype):
    """NaN codes and scales in blocks of nobody, and NaN codes behind the last token."""
    cache = C.Cache(2, LENGTHS, 128, HEADS, 64, "e4m3", seed=8, width=9)
    q = queries(sum(ROWS), HEADS, 64, dtype)
    want, _ = of_sets(q, cache, ROWS, what="clean")
    used = torch.zeros(len(cache.k), dtype=torch.bool)
    for b, n in enumerate(LENGTHS):
        at = cache.table[b].cpu().long()
        used[at[:-(-n // 128)]] = True
        for x in (cache.k, cache.v):
            x.view(torch.uint8)[int(at[n // 128]), n % 128:] = 0x7f
    for x, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        x.view(torch.uint8)[~used.cuda()] = 0x7f
        s[~used.cuda()] = math.nan
    got = L.cache_attention(q, *cache.operands(), C.starts(ROWS), cache.lengths, cache.table,
                            max_rows=max(ROWS))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", C.TYPES)
def test_strides(dtype):
    """Queries from a fused projection, a strided output, keys and values of a block side by side."""
    cache = C.Cache(2, LENGTHS, 32, HEADS, 64, "i8", seed=11)
    both = torch.empty(len(cache.k), 2, 32, HEADS, 64, dtype=torch.int8, device="cuda")
    both[:, 0], both[:, 1] = cache.k, cache.v
    cache.k, cache.v = both[:, 0], both[:, 1]
    T = sum(ROWS)
    fused = queries(T, 2 * HEADS + 3, 64, dtype)
    out = torch.full((T, HEADS, 128), 5.0, dtype=C.TYPES[dtype], device="cuda")
    of_sets(fused[:, 3:3 + HEADS], cache, ROWS, what="strided", out=out[..., :64])
    assert bool((out[..., 64:] == 5.0).all())


def test_offsets_past_32_bits():
    """Blocks more than 2^32 bytes apart."""
    far, hk = (1 << 32) + 4096, 24
    room = torch.zeros(2 * far + 65536, dtype=torch.int8, device="cuda")
    cache = C.Cache(1, [40], 16, hk, 64, "i8", spare=0)
    k = room.as_strided((3, 16, hk, 64), (far, 64, 1024, 1))
    k.copy_(cache.k)
    q = queries(700, hk, 64, "bf16")
    v = cache.v
    cache.k = k
    of_sets(q, cache, [700], causal=False, what="far")
    cache.k, cache.v = v, k
    of_sets(q, cache, [700], causal=False, what="far values")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scales", ["powers of two", "others", "holes"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "f16"), (64, "f32"), (128, "bf16")])
def test_long_keys_in_one_share(d, dtype, scales, causal):
    """More tiles than a wave holds blocks and scales of: 132, filled in again by halves (and, of
    scales that are multiplied with, every 16 tiles)."""
    rows, lengths, hk = [129], [8403], 64
    cache = C.Cache(1, lengths, 32, hk, d, "e4m3" if causal else "i8", seed=20)
    g = torch.Generator().manual_seed(21)
    if scales == "others":
        for s in (cache.ks, cache.vs):
            s.mul_((0.5 + torch.rand(s.shape, generator=g)).cuda())
    if scales == "holes":
        cache.table[0, torch.randperm(cache.width, generator=g)[:20].cuda()] = -1
    _, tiles = of_sets(queries(129, hk, d, dtype), cache, rows, causal=causal, workspace=False,
                       what=scales)
    assert tiles > 128


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_keys_in_shares(dtype):
    """Shares that begin past a wave's first tiles, each with more than one fill."""
    for rows, hk, least in (([300, 1], 16, 16), ([129, 1], 80, 64)):
        cache = C.Cache(2, [20011, 6000], 64, hk, 64, "i8", seed=22)
        _, tiles = of_sets(queries(sum(rows), hk, 64, dtype), cache, rows, what="shares")
        assert tiles > least


@pytest.mark.parametrize("codes,dtype", [("i8", "bf16"), ("e4m3", "f16"), ("i8", "f32")])
@pytest.mark.parametrize("rows,lengths,hq,hk,d", [
    ([16], [20011], 16, 4, 128),            # a chunk of one long request
    ([1], [20011], 64, 1, 64),              # a token of heads that all share one
    ([1] * 4, [9001, 3, 8192, 5000], 64, 1, 128),
    ([100], [16400], 2, 2, 64),
    ([3, 40, 0, 1], [700, 12345, 9000, 2049], 4, 1, 80),
    ([40], [70001], 1, 1, 64),              # shares of more than 512 keys
], ids=str)
def test_few_sets_of_long_keys(rows, lengths, hq, hk, d, codes, dtype):
    cache = C.Cache(len(rows), lengths, 16, hk, d, codes, seed=23)
    q = queries(sum(rows), hq, d, dtype)
    first, tiles = of_sets(q, cache, rows, what="few sets")
    assert tiles <= max(32, -(-max(lengths) // 64) // 4)
    alone = check(q, cache, C.starts(rows), True, max_rows=max(rows), workspace=False, what="alone")
    assert bool(torch.isfinite(alone).all()) and bool(torch.isfinite(first).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_padded_batch_in_shares(dtype):
    """Rows of no entry before, between and behind, in a buffer of far more rows than sets."""
    cache = C.Cache(3, [5000, 300, 9000], 16, 2, 64, "i8", seed=24)
    q = queries(3000, 8, 64, dtype)
    starts = torch.tensor([7, 47, 48, 178]).int().cuda()
    out = torch.full_like(q, 3.0)
    check(q, cache, starts, True, what="padded", max_rows=130, out=out)
    assert bool((out[:7] == 3.0).all()) and bool((out[178:] == 3.0).all())
