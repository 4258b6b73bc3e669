"""kv_cache_write behind scales that are no powers of two (a cache that others wrote): codes on and
next to the borders between two codes, as the definition has them in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import cachecheck as C  # noqa: E402
from test_gpu_kv_cache import _needs_gpu, write_and_check  # noqa: E402,F401

pytestmark = pytest.mark.gpu

SCALES = [0.3, 0.1, 7.0, 1 / 3, 2.5 / 127, 0.7 * 2.0 ** -80, 1.1 * 2.0 ** 100]


def borders(codes):
    """The numbers half-way between two codes, and the codes."""
    if codes == "i8":
        c = torch.arange(-127, 128).double()
    else:
        c = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
        c = c.float().double()
        c = c[torch.isfinite(c)].unique()
    return torch.cat([(c[1:] + c[:-1]) / 2, c])


def on_borders(codes, scale, dtype, n, most=1e9):
    """[n] numbers of the type, on the borders times the scale or one or two of the type's last
    places beside them."""
    b = borders(codes)
    b = b[b.abs() <= most]
    x = (b[torch.arange(n) % len(b)] * scale).to(C.TYPES[dtype])
    ints = torch.int32 if dtype == "f32" else torch.int16
    x = (x.view(ints) + (torch.arange(n) // len(b) % 5 - 2).to(ints)).view(x.dtype)
    return torch.where(torch.isfinite(x), x, torch.zeros_like(x))


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("scale,dtype", [(s, t) for s in SCALES for t in C.TYPES
                                         if t != "f16" or 2.0 ** -14 < s < 2.0 ** 8])
def test_new_tokens_under_an_older_scale(scale, dtype, codes):
    """The block's scale is larger than the new values need, and stays."""
    scale = float(torch.tensor(scale))
    cache = C.Cache(2, [16, 14], 16, 2, 64, codes, seed=3)
    cache.ks.fill_(scale)
    cache.vs.fill_(scale)
    # (values that need no larger scale: below the last code's half)
    most = 60 if codes == "i8" else 200
    x = on_borders(codes, scale, dtype, 25 * 2 * 64, most).view(25, 2, 64).cuda()
    before = cache.ks.clone()
    write_and_check(cache, x, x.flip(0).contiguous(), C.starts([13, 12]), f"{codes} under {scale}")
    assert torch.equal(cache.ks, before)


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("scale", SCALES + [3e-39])
def test_earlier_codes_when_such_a_scale_grows(scale, codes):
    cache = C.Cache(12, [15] * 12, 16, 2, 64, codes, seed=4)
    # every code, times scales from all over a power of two and more
    for s in (cache.ks, cache.vs):
        s.copy_(scale * (1 + torch.arange(s.numel()).view(s.shape) / 7).float())
    x = (cache.ks.max() * 448 * torch.linspace(0.5, 3, 12, device="cuda")).view(12, 1, 1)
    x = x.expand(12, 2, 64).contiguous()
    write_and_check(cache, x, -x, C.starts([1] * 12), f"{codes} from {scale}")


@pytest.mark.parametrize("codes", ["i8", "e4m3"])
def test_more_heads_than_a_launch_has_rows_of_workgroups(codes):
    """Tokens of 150000 key heads, written and read back."""
    hk = 150000
    cache = C.Cache(1, [3], 16, hk, 16, codes, seed=9, spare=0, empty=True)
    cache.ks.zero_()
    cache.vs.zero_()
    k = torch.randn(3, hk, 16, generator=torch.Generator().manual_seed(3)).cuda()
    print(f"[gpu] cache write {hk} heads {codes}", flush=True)
    L.kv_cache_write(k, -k, *cache.operands(), C.starts([3]), cache.lengths, cache.table)
    got, minus = L.kv_cache_read(*cache.operands(), cache.lengths, cache.table, dtype=torch.float32,
                                 rows=3)
    torch.cuda.synchronize()
    # half a step of a code: of a power of two up to 1/64 of a head's largest value (i8), or of the
    # value's own 4 bits, and of the smallest 2^-9 scales (E4M3)
    top = k.abs().amax((0, 2), keepdim=True)
    bound = top / 127 if codes == "i8" else k.abs() / 16 + top / 448 * 2.0 ** -9
    assert bool(((got[0] - k).abs() <= bound).all())
    assert torch.equal(got, -minus)


def test_outputs_made_in_a_graph():
    """kv_cache_read makes its outputs, zero behind the tokens, again at every replay."""
    cache = C.Cache(3, [200, 40, 64], 16, 2, 64, "e4m3", seed=10)
    call = lambda: L.kv_cache_read(*cache.operands(), cache.lengths, cache.table)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for lengths in ([200, 40, 64], [3, 0, 208], [100, 41, 1], [200, 200, 200]):
        cache.lengths.copy_(torch.tensor(lengths))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), lengths
            for e, n in enumerate(lengths):
                assert bool((a[e, n:] == 0).all())
