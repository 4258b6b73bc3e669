"""Operands of prefix_attention beside one another in the rows of one buffer."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

ALIAS, DEVICE = 5, 7
BUF, KEYS, N = 0x10000000, 0x20000000, 0x30000000   # fake addresses: never read


def status(B, Sq, at_out, q=(0, 0), out=(0, 0), key_at=None, keys=(0, 0)):
    """4 heads of 64, bf16, one key head: queries at the buffer's start, `out` from byte at_out on;
    (entry, row) strides in elements."""
    k = KEYS if key_at is None else BUF + key_at
    s = (ctypes.c_longlong * 16)(*q, 64, 0, 0, 0, 0, *keys, 64, *keys, 64, *out, 64)
    return L.libconv_prefix_attention(BUF, None, None, k, k, N, BUF + at_out, None, s, B, Sq, 0, 8,
                                      4, 1, 64, 0.125, 1, L.BF16, None, 0, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")
@pytest.mark.parametrize("kw,want", [
    # a row of 512: the queries' 256, then the output's
    (dict(B=5, Sq=3, at_out=512, q=(1536, 512), out=(1536, 512)), DEVICE),
    (dict(B=5, Sq=1, at_out=512, q=(512, 0), out=(512, 0)), DEVICE),          # single tokens
    (dict(B=1, Sq=7, at_out=512, q=(0, 512), out=(0, 512)), DEVICE),
    (dict(B=3, Sq=5, at_out=512, q=(512, 1536), out=(512, 1536)), DEVICE),    # entries inside rows
    (dict(B=5, Sq=1, at_out=512, q=(512, 0), out=(1024, 0)), DEVICE),         # every second row
    (dict(B=5, Sq=3, at_out=512, q=(0, 512), out=(1536, 512)), DEVICE),       # shared queries
    (dict(B=1, Sq=1, at_out=512), DEVICE),
    # one entry's only query before the output's rows, and in their middle
    (dict(B=2, Sq=1, at_out=512, q=(0, 0), out=(512, 0)), DEVICE),
    (dict(B=5, Sq=1, at_out=496, q=(512, 0), out=(512, 0)), ALIAS),           # its last 8 elements
    (dict(B=5, Sq=1, at_out=528, q=(512, 0), out=(512, 0)), ALIAS),           # the next query
    (dict(B=5, Sq=1, at_out=512, q=(512, 0), out=(768, 0)), ALIAS),
    (dict(B=5, Sq=1, at_out=512, q=(520, 0), out=(512, 0)), ALIAS),
    (dict(B=5, Sq=3, at_out=512, q=(1544, 512), out=(1536, 512)), ALIAS),
    (dict(B=1, Sq=1, at_out=496), ALIAS),
    # keys of 64 behind both, in rows of 576 each; then with the output over them
    (dict(B=5, Sq=1, at_out=512, q=(576, 0), out=(576, 0), key_at=1024, keys=(576, 576)), DEVICE),
    (dict(B=5, Sq=1, at_out=512, q=(576, 0), out=(576, 0), key_at=1008, keys=(576, 576)), ALIAS),
])
def test_which_operands_meet(kw, want):
    assert status(**kw) == want


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 3])
def test_output_beside_the_queries(Sq):
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    rows, kp, vp, k, v = r(5, Sq, 8, 64), r(40, 1, 64), r(40, 1, 64), r(5, 9, 1, 64), r(5, 9, 1, 64)
    n = torch.tensor([0, 9, 3, 1, 5]).int().cuda()
    q, out = rows[:, :, :4], rows[:, :, 4:]
    before = q.clone()
    L.prefix_attention(q, kp, vp, k, v, n, out=out)
    torch.cuda.synchronize()
    want, bound, _, _ = C.attention(before, kp, vp, k, v, n, 64 ** -0.5, True)
    C.assert_within(out, want, bound, "beside")
    assert torch.equal(q, before)
