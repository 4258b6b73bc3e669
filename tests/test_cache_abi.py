"""Argument checks of the operators around the 8-bit cache and of the projection with activation
and residual, which return before anything is enqueued (no GPU), and their workspace sizes."""
import ctypes

import pytest
import torch

import direct_implicit_gemm_amd as L

NULL, SHAPE, DTYPE, ACT, ALIAS, UNSUPPORTED, DEVICE, LARGE, ALIGN = 1, 2, 3, 4, 5, 6, 7, 10, 12
# fake addresses: never read
Q, K, V, KC, VC, KS, VS, ST, LN, TB, OUT, LSE, WS = (0x10000000 * i for i in range(1, 14))

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")


def with_strides(a, s):
    if a["strides"] is not None:
        v = list(a["strides"])
        for i, x in (s or {}).items():
            v[i] = x
        a["strides"] = (ctypes.c_longlong * len(v))(*v)
    return a.values()


# a block of 16 tokens of 2 heads of 64, each head's tokens side by side: 2048 bytes
CODES = (2048, 64, 1024)
CACHE = dict(B=3, T=5, blocks=9, block_size=16, table_width=4, k_heads=2, head_dim=64,
             format=L.CACHE_I8, dtype=L.BF16)
WRITE = dict(k=K, v=V, k_cache=KC, v_cache=VC, k_scale=KS, v_scale=VS, row_starts=ST, lengths=LN,
             block_table=TB, strides=(128, 64, 128, 64) + CODES + CODES, **CACHE)


def write(s=None, **kw):
    return L.libconv_kv_cache_write(*with_strides({**WRITE, **kw}, s), None)


COMMON = [
    (dict(k_cache=None), NULL), (dict(v_cache=None), NULL), (dict(k_scale=None), NULL),
    (dict(v_scale=None), NULL), (dict(lengths=None), NULL), (dict(block_table=None), NULL),
    (dict(strides=None), NULL),
    (dict(B=-1), SHAPE), (dict(blocks=-1), SHAPE), (dict(table_width=-1), SHAPE),
    (dict(k_heads=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(block_size=0), SHAPE),
    (dict(dtype=3), DTYPE), (dict(format=2), DTYPE), (dict(format=-1), DTYPE),
    (dict(head_dim=72), UNSUPPORTED), (dict(head_dim=144), UNSUPPORTED),
    (dict(block_size=8), UNSUPPORTED), (dict(block_size=48), UNSUPPORTED),
    (dict(block_size=512), UNSUPPORTED),
    (dict(table_width=1 << 28), LARGE), (dict(blocks=1 << 30), LARGE), (dict(k_heads=1 << 21), LARGE),
    (dict(B=1 << 24), LARGE), (dict(B=65537), LARGE),
    (dict(k_cache=KC + 8), ALIGN), (dict(v_scale=VS + 2), ALIGN), (dict(lengths=LN + 1), ALIGN),
    (dict(block_table=TB + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(row_starts=None), NULL),
    (dict(T=-1), SHAPE), (dict(T=1 << 26), LARGE), (dict(s={0: -128}), SHAPE),
    (dict(s={4: 1 << 40}), SHAPE), (dict(s={5: 1 << 23}), LARGE),
    (dict(k=K + 8), ALIGN), (dict(s={1: 60}), ALIGN), (dict(s={8: 65}), ALIGN),
    (dict(row_starts=ST + 2), ALIGN),
    (dict(v_cache=KC), ALIAS), (dict(v_cache=KC + 1024), ALIAS), (dict(k=KC), ALIAS),
    (dict(k_scale=KC), ALIAS), (dict(v_scale=KS), ALIAS), (dict(lengths=VC + 64), ALIAS),
    (dict(block_table=KS), ALIAS), (dict(row_starts=VS), ALIAS), (dict(v_scale=V), ALIAS),
    (dict(s={4: 1024}), ALIAS), (dict(s={5: 0}), SHAPE), (dict(s={5: 48}), SHAPE),
    (dict(s={0: 1 << 39, 2: 1 << 39}, T=1 << 25), LARGE), (dict(s={4: 1 << 39}, blocks=1 << 25), LARGE),
])
def test_write_refusals(kw, code):
    assert write(**kw) == code


def test_write_accepts():
    assert write(T=0) == 0 and write(B=0) == 0 and write(T=0, k=None, v=None) == 0
    assert write() == DEVICE
    assert write(s={4: 2048, 5: 128, 6: 64}) == DEVICE              # each token's heads
    # keys and values of a block side by side
    assert write(v_cache=KC + 2048, s={4: 4096, 7: 4096}) == DEVICE
    assert write(v_cache=KC + 2032, s={4: 4096, 7: 4096}) == ALIAS
    assert write(k=K, v=K + 256, s={0: 256, 2: 256}) == DEVICE       # rows of one projection
    assert write(blocks=0, k_cache=None, v_cache=None, k_scale=None, v_scale=None) == 0


READ = dict(k_cache=KC, v_cache=VC, k_scale=KS, v_scale=VS, lengths=LN, block_table=TB, k=K, v=V,
            strides=CODES + CODES + (8192, 128, 64) * 2, B=3, S=64, blocks=9, block_size=16,
            table_width=4, k_heads=2, head_dim=64, format=L.CACHE_E4M3, dtype=L.F16)


def read(s=None, **kw):
    return L.libconv_kv_cache_read(*with_strides({**READ, **kw}, s), None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(S=-1), SHAPE), (dict(s={6: -8}), SHAPE),
    (dict(B=1 << 20, S=1 << 20, table_width=1 << 20, s={6: 1 << 30, 9: 1 << 30}), LARGE),
    (dict(v=V + 2), ALIGN), (dict(s={8: 36}), ALIGN),
    (dict(k=V), ALIAS), (dict(k=KC), ALIAS), (dict(v=TB), ALIAS), (dict(k=KS), ALIAS),
    (dict(s={6: 128}), ALIAS), (dict(s={11: 0}), ALIAS),
])
def test_read_refusals(kw, code):
    assert read(**kw) == code


def test_read_accepts():
    assert read(B=0) == 0 and read(S=0) == 0 and read(table_width=0, block_table=None) == 0
    assert read() == DEVICE
    assert read(S=100000, s={6: 100000 * 128, 9: 100000 * 128}, v=V << 4) == DEVICE
    assert read(k=K, v=K + 256, s={6: 16384, 7: 256, 9: 16384, 10: 256}) == DEVICE


ATTN = dict(q=Q, k_cache=KC, v_cache=VC, k_scale=KS, v_scale=VS, row_starts=ST, lengths=LN,
            block_table=TB, out=OUT, lse=LSE, strides=(256, 64, 256, 64) + CODES + CODES, B=3, T=5,
            max_rows=5, blocks=9, block_size=16, table_width=4, q_heads=4, k_heads=2, head_dim=64,
            scale=0.125, causal=1, format=L.CACHE_I8, dtype=L.BF16, workspace=None,
            workspace_bytes=0)


def attention(s=None, **kw):
    return L.libconv_cache_attention(*with_strides({**ATTN, **kw}, s), None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(row_starts=None), NULL),
    (dict(T=-1), SHAPE), (dict(max_rows=-1), SHAPE), (dict(q_heads=3), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(workspace_bytes=-1), SHAPE), (dict(s={0: -1}), SHAPE), (dict(s={2: 1 << 40}), SHAPE),
    (dict(T=1 << 26), LARGE), (dict(T=1 << 25, q_heads=64), LARGE), (dict(B=1 << 23), LARGE),
    (dict(B=65537), LARGE),
    (dict(q=Q + 8), ALIGN), (dict(s={3: 60}), ALIGN), (dict(lse=LSE + 2), ALIGN),
    (dict(workspace=WS + 16, workspace_bytes=64), ALIGN),
    (dict(out=Q), ALIAS), (dict(out=KC), ALIAS), (dict(lse=OUT), ALIAS), (dict(lse=VC), ALIAS),
    (dict(out=KS), ALIAS), (dict(lse=TB), ALIAS), (dict(s={2: 0}), ALIAS),
    (dict(workspace=OUT, workspace_bytes=1 << 20), ALIAS),
    (dict(workspace=KC, workspace_bytes=1 << 20), ALIAS),
    (dict(workspace=LN, workspace_bytes=1 << 20), ALIAS),
])
def test_attention_refusals(kw, code):
    assert attention(**kw) == code


def test_attention_accepts():
    assert attention(B=0) == 0 and attention(T=0) == 0 and attention(max_rows=0) == 0
    assert attention() == DEVICE
    assert attention(lse=None) == DEVICE
    assert attention(out=Q + 512, s={0: 512, 2: 512}) == DEVICE       # beside the queries
    assert attention(workspace=WS, workspace_bytes=1) == DEVICE       # too small: a plan without
    assert attention(q_heads=128, k_heads=2, s={0: 8192, 2: 8192}) == DEVICE
    assert attention(v_cache=KC + 2048, s={4: 4096, 7: 4096}) == DEVICE


def test_attention_workspace():
    size = L.libconv_cache_attention_workspace
    assert size(3, 5, 5, 16, 4, 4, 2, 60, L.BF16) == -1
    assert size(3, 5, 5, 16, 4, 4, 3, 64, L.BF16) == -1
    assert size(3, 5, 5, 24, 4, 4, 2, 64, L.BF16) == -1
    assert size(3, 5, 5, 16, 4, 4, 2, 64, 9) == -1
    assert size(3, 0, 5, 16, 4, 4, 2, 64, L.BF16) == 0
    assert size(4, 4, 1, 32, 32, 20, 20, 64, L.BF16) == 0             # few keys: one launch
    few = size(64, 64, 1, 16, 512, 32, 8, 128, L.BF16)
    assert few > 0
    # as much for any length of the table, and for long rows no more than their shares
    assert size(64, 64, 1, 16, 8192, 32, 8, 128, L.BF16) == few
    assert size(8, 8 * 2048, 2048, 64, 96, 32, 8, 128, L.BF16) <= few
    assert size(9, 2594, 517, 32, 128, 16, 4, 80, L.F16) <= few + 16 * 2594 * 16 * 81 * 4


LINEAR = dict(x=Q, w=K, bias=V, residual=KC, y=OUT, T=5, K=64, N=48, x_stride=64,
              residual_stride=48, y_stride=48, act=2, dtype=L.F16, workspace=None,
              workspace_bytes=0)


def linear(**kw):
    return L.libconv_linear(*{**LINEAR, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(y_stride=47), SHAPE),
    (dict(x_stride=-64), SHAPE), (dict(residual_stride=-1), SHAPE), (dict(workspace_bytes=-1), SHAPE),
    (dict(dtype=3), DTYPE), (dict(act=5), ACT), (dict(act=-1), ACT), (dict(K=60), UNSUPPORTED),
    (dict(K=1 << 23), LARGE), (dict(x_stride=1 << 23), LARGE), (dict(T=1 << 26), LARGE),
    (dict(T=1 << 22, N=1 << 20), LARGE),
    (dict(x=Q + 8), ALIGN), (dict(x_stride=68), ALIGN), (dict(w=K + 2), ALIGN),
    (dict(y=OUT + 1), ALIGN), (dict(residual=KC + 1), ALIGN), (dict(bias=V + 1), ALIGN),
    (dict(workspace=WS + 128, workspace_bytes=9), ALIGN),
    (dict(y=Q), ALIAS), (dict(y=K + 16), ALIAS), (dict(y=V), ALIAS), (dict(y=KC + 2), ALIAS),
    (dict(y=KC, residual_stride=96), ALIAS), (dict(workspace=OUT, workspace_bytes=64), ALIAS),
    (dict(workspace=Q, workspace_bytes=64), ALIAS), (dict(workspace=KC, workspace_bytes=64), ALIAS),
])
def test_linear_refusals(kw, code):
    assert linear(**kw) == code


def test_linear_accepts():
    assert linear(T=0) == 0 and linear(T=0, x=None, y=None) == 0
    assert linear() == DEVICE
    assert linear(bias=None, residual=None, residual_stride=0) == DEVICE
    assert linear(y=KC) == DEVICE                                     # in place
    assert linear(residual_stride=0, x_stride=0) == DEVICE            # one row for all
    assert linear(y=Q + 128, x_stride=128, y_stride=128) == DEVICE    # beside the inputs
    assert linear(workspace=WS, workspace_bytes=1) == DEVICE


def test_linear_workspace():
    size = L.libconv_linear_workspace
    assert size(5, 60, 48, L.F16) == -1 and size(5, 64, 48, 7) == -1
    assert size(0, 64, 48, L.F16) == 0 and size(8192, 4096, 8192, L.BF16) == 0
    assert size(3, 64, 4096, L.BF16) == 0                             # a short sum
    n = size(64, 4096, 4096, L.BF16)
    assert n > 0 and n % (64 * 4096 * 4) == 0                         # whole runs
    assert size(1, 4096, 100, L.F32) % (128 * 4) == 0


def test_convolutions_take_no_other_activation():
    st = L.conv2d_forward(Q, K, V, OUT, 1, 4, 8, 8, 8, 3, 3, 1, 1, 1, 1, L.F32, L.ACT_SILU, None)
    assert st == ACT


def test_helpers_refuse_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        L.linear(x, x)
    with pytest.raises(ValueError):
        L.linear(x, x, act="swish")
    q, codes, s = torch.zeros(2, 1, 16), torch.zeros(3, 16, 1, 16, dtype=torch.int8), torch.zeros(3, 1)
    starts, n, table = (torch.zeros(*shape).int() for shape in ((3,), (2,), (2, 1)))
    with pytest.raises(ValueError):
        L.kv_cache_write(q, q, codes, codes, s, s, starts, n, table)
    with pytest.raises(ValueError):
        L.kv_cache_read(codes, codes, s, s, n, table)
    with pytest.raises(ValueError):
        L.cache_attention(q, codes, codes, s, s, starts, n, table)
