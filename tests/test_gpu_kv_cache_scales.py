"""kv_cache_write behind scales that are no powers of two (a cache that others wrote): codes on and
next to the borders between two codes, as the definition has them in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
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


@pytest.mark.parametrize("dtype", C.TYPES)
@pytest.mark.parametrize("codes", ["i8", "e4m3"])
@pytest.mark.parametrize("scale", SCALES)
def test_new_tokens_under_an_older_scale(scale, codes, dtype):
    """The block's scale is larger than the new values need, and stays."""
    scale = float(torch.tensor(scale))
    if dtype == "f16" and not 2.0 ** -14 < scale < 2.0 ** 8:
        pytest.skip("past the type's range")
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
