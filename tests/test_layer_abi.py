"""Argument checks of the attention-layer operators, which return before
anything is enqueued (no GPU), and their workspace sizes."""
import ctypes

import pytest

import direct_implicit_gemm_amd as L

NULL, SHAPE, DTYPE, ALIAS, UNSUPPORTED, DEVICE, LARGE, ALIGN, SCRATCH = 1, 2, 3, 5, 6, 7, 10, 12, 13
# fake addresses: never read
Q, K, V, QO, KO, VO, W1, W2, FR, POS, SL = (0x10000000 * i for i in range(1, 12))


def no_gpu():
    import torch
    return not torch.cuda.is_available()


# ------------------------------------------------------------------------- norms and rotation
ROPE = dict(q=Q, k=K, v=V, q_out=QO, k_out=KO, v_out=VO, q_weight=W1, k_weight=W2, freqs=FR,
            positions=POS, slots=None, strides=(256, 64, 128, 64, 128, 64) * 2, T=4, q_heads=4,
            k_heads=2, head_dim=64, rot_dim=64, pairs0=32, pairs1=0, pairs2=0, interleaved=0,
            out_rows=4, eps=1e-6, dtype=L.BF16)


def rope(**kw):
    a = {**ROPE, **kw}
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_longlong * 12)(*a["strides"])
    return L.libconv_qk_norm_rope(*a.values(), None)


def strides(**kw):
    s = list(ROPE["strides"])
    for i, v in kw.items():
        s[int(i[1:])] = v
    return tuple(s)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(v=None), NULL), (dict(v_out=None), NULL), (dict(freqs=None), NULL),
    (dict(positions=None), NULL), (dict(strides=None), NULL),
    (dict(T=-1), SHAPE), (dict(q_heads=0), SHAPE), (dict(k_heads=0), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(pairs0=31), SHAPE), (dict(pairs1=-1, pairs0=33), SHAPE),
    (dict(rot_dim=128, pairs0=64), SHAPE), (dict(rot_dim=33), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(out_rows=-1), SHAPE),
    (dict(strides=strides(_0=-256)), SHAPE), (dict(strides=strides(_6=1 << 41)), SHAPE),
    (dict(dtype=3), DTYPE),
    (dict(head_dim=264), UNSUPPORTED), (dict(head_dim=68), UNSUPPORTED),
    (dict(rot_dim=40, pairs0=20), UNSUPPORTED),
    (dict(q=Q + 8), ALIGN), (dict(v_out=VO + 2), ALIGN), (dict(strides=strides(_1=65)), ALIGN),
    (dict(q_weight=W1 + 4), ALIGN), (dict(positions=POS + 2), ALIGN), (dict(freqs=FR + 4), ALIGN),
    (dict(q_out=K), ALIAS), (dict(k_out=QO + 64), ALIAS), (dict(q_out=Q + 128), ALIAS),
    (dict(k_out=K, slots=SL), ALIAS), (dict(q_out=W1), ALIAS), (dict(k_out=POS), ALIAS),
    (dict(strides=strides(_6=0)), ALIAS), (dict(strides=strides(_7=0)), ALIAS),
    (dict(q_out=Q, strides=strides(_6=512)), ALIAS),
])
def test_rope_refusals(kw, code):
    assert rope(**kw) == code


def test_rope_accepts():
    assert rope(T=0) == 0
    if no_gpu():
        assert rope() == DEVICE
        assert rope(q_out=Q, k_out=K) == DEVICE                       # in place
        # slices of one buffer's rows: queries, keys and values of 512 elements
        row = dict(q=Q, k=Q + 512, v=Q + 768, q_out=Q, k_out=Q + 512,
                   strides=(512, 64) * 5 + (128, 64))
        assert rope(**row) == DEVICE
        assert rope(**{**row, "k_out": Q + 256}) == ALIAS             # the last queries' place
        assert rope(v=None, v_out=None, q_weight=None, k_weight=None) == DEVICE
        assert rope(rot_dim=0, pairs0=0, freqs=None, positions=None) == DEVICE
        assert rope(rot_dim=40, pairs0=20, interleaved=1) == DEVICE


# ---------------------------------------------------------------------------------- attention
WS = 0xc0000000
ATTN = dict(q=Q, kp=K, vp=V, k=W1, v=W2, lengths=POS, out=QO, lse=KO,
            strides=(512, 256, 64, 128, 64, 128, 64, 1280, 128, 64, 1280, 128, 64, 512, 256, 64),
            B=2, Sq=2, P=300, S=10, q_heads=4, k_heads=2, head_dim=64, scale=0.125, causal=1,
            dtype=L.BF16, workspace=None, workspace_bytes=0)


def attention(s=None, **kw):
    a = {**ATTN, **kw}
    if s:
        a["strides"] = tuple(s.get(i, v) for i, v in enumerate(a["strides"]))
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_longlong * 16)(*a["strides"])
    return L.libconv_prefix_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(kp=None), NULL), (dict(vp=None), NULL), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(lengths=None), NULL), (dict(out=None), NULL),
    (dict(strides=None), NULL),
    (dict(B=-1), SHAPE), (dict(Sq=-1), SHAPE), (dict(P=-1), SHAPE), (dict(S=-1), SHAPE),
    (dict(q_heads=3), SHAPE), (dict(k_heads=0), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(workspace_bytes=-1), SHAPE), (dict(s={3: -128}), SHAPE), (dict(s={15: 1 << 40}), SHAPE),
    (dict(dtype=-1), DTYPE), (dict(head_dim=136), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED),
    (dict(q=Q + 8), ALIGN), (dict(s={8: 132}), ALIGN), (dict(lengths=POS + 1), ALIGN),
    (dict(workspace=WS + 16, workspace_bytes=64), ALIGN),
    (dict(out=Q), ALIAS), (dict(out=W2 + 64), ALIAS), (dict(lse=QO), ALIAS), (dict(lse=V), ALIAS),
    (dict(s={14: 0}), ALIAS), (dict(workspace=QO, workspace_bytes=1 << 20), ALIAS),
    (dict(workspace=W1, workspace_bytes=1 << 20), ALIAS), (dict(lse=POS), ALIAS),
    (dict(B=1 << 20, Sq=1 << 10), LARGE), (dict(s={8: 1 << 23}), LARGE),
])
def test_attention_refusals(kw, code):
    assert attention(**kw) == code


def test_attention_accepts():
    assert attention(B=0) == 0 and attention(Sq=0) == 0
    if no_gpu():
        assert attention() == DEVICE
        assert attention(P=0, kp=None, vp=None) == DEVICE
        assert attention(S=0, k=None, v=None, lse=None) == DEVICE
        # keys and values beside the queries in a fused projection, the output over none of it
        assert attention(kp=Q + 512, s={0: 1024, 1: 512, 3: 512}) == DEVICE


def test_attention_workspace():
    size = L.libconv_prefix_attention_workspace
    assert size(2, 1, 300, 10, 4, 2, 60, L.BF16) == -1
    assert size(2, 1, 300, 10, 4, 3, 64, L.BF16) == -1
    assert size(2, 1, 300, 10, 4, 2, 64, 7) == -1
    assert size(0, 1, 300, 10, 4, 2, 64, L.BF16) == 0
    assert size(64, 4096, 77, 4096, 16, 16, 128, L.BF16) == 0       # many rows: nothing to join
    n = size(64, 1, 8192, 2048, 32, 8, 128, L.BF16)
    assert n > 0 and n % (64 * 32 * 129 * 4) == 0                   # whole slots


# ------------------------------------------------------------------------------------ adapters
LORA = dict(x=Q, w=K, bias=V, a=W1, b=W2, scales=FR, row_starts=POS, adapters=SL, y=QO, T=5, K=64,
            N=48, rank=8, n_adapters=2, n_requests=3, x_stride=64, y_stride=48, dtype=L.F16,
            workspace=WS, workspace_bytes=1 << 20)


def lora(**kw):
    return L.libconv_lora_linear(*{**LORA, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(a=None), NULL),
    (dict(b=None), NULL), (dict(scales=None), NULL), (dict(row_starts=None), NULL),
    (dict(adapters=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(rank=0), SHAPE),
    (dict(n_adapters=-1), SHAPE), (dict(n_requests=-1), SHAPE), (dict(y_stride=47), SHAPE),
    (dict(x_stride=-64), SHAPE), (dict(workspace_bytes=-1), SHAPE), (dict(dtype=9), DTYPE),
    (dict(K=60), UNSUPPORTED), (dict(rank=129), UNSUPPORTED),
    (dict(K=1 << 23), LARGE), (dict(N=1 << 30), LARGE), (dict(x_stride=1 << 23), LARGE),
    (dict(x=Q + 8), ALIGN), (dict(x_stride=68), ALIGN), (dict(w=K + 2), ALIGN),
    (dict(a=W1 + 8), ALIGN), (dict(y=QO + 1), ALIGN), (dict(workspace=WS + 128), ALIGN),
    (dict(scales=FR + 2), ALIGN),
    (dict(y=Q), ALIAS), (dict(y=K + 16), ALIAS), (dict(y=WS), ALIAS), (dict(y=W2), ALIAS),
    (dict(workspace=Q), ALIAS), (dict(workspace=W1), ALIAS), (dict(bias=QO + 2), ALIAS),
    (dict(workspace=None), SCRATCH), (dict(workspace_bytes=64), SCRATCH),
])
def test_lora_refusals(kw, code):
    assert lora(**kw) == code


def test_lora_accepts():
    assert lora(T=0) == 0
    if no_gpu():
        assert lora() == DEVICE
        none = dict(a=None, b=None, scales=None, row_starts=None, adapters=None, workspace=None,
                    workspace_bytes=0)
        assert lora(n_adapters=0, **none) == DEVICE and lora(n_requests=0, **none) == DEVICE
        assert lora(x_stride=0) == DEVICE                       # one row for all tokens
        # outputs beside the inputs in one buffer's rows
        assert lora(y=Q + 128, x_stride=128, y_stride=128) == DEVICE


def test_lora_workspace():
    assert L.libconv_lora_workspace(5, 64, 48, 8, 0, 3, L.F16) == 0
    assert L.libconv_lora_workspace(5, 64, 48, 8, 2, 0, L.F16) == 0
    assert L.libconv_lora_workspace(5, 60, 48, 8, 2, 3, L.F16) == -1
    n = L.libconv_lora_workspace(64, 4096, 4096, 16, 24, 64, L.BF16)
    assert n > 0 and n >= 64 * 16 * 4


def test_helpers_refuse_host_tensors():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        L.lora_linear(x, x, None, None, None, None, None, None)
    q = torch.zeros(2, 1, 8)
    with pytest.raises(ValueError):
        L.qk_norm_rope(q, q, torch.zeros(1, 2).int(), torch.zeros(4).double())
    with pytest.raises(ValueError):
        L.prefix_attention(q[None], q, q, None, None, torch.zeros(1).int())


def test_rotary_frequencies():
    f = L.rotary_frequencies(8, 10000.0, device="cpu")
    assert f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    f = L.rotary_frequencies(12, 100.0, [2, 2, 2], device="cpu")
    assert f.tolist() == pytest.approx([1.0, 0.1] * 3, rel=1e-15)
    with pytest.raises(ValueError):
        L.rotary_frequencies(8, 10000.0, [3], device="cpu")


# ------------------------------------------------------------------- sizes a launch cannot have
@pytest.mark.parametrize("kw", [dict(T=1 << 26), dict(T=(1 << 31) - 1), dict(q_heads=1 << 24)])
def test_rope_too_large(kw):
    assert rope(**{**kw, "strides": (1 << 31, 64) * 6}) == LARGE


@pytest.mark.parametrize("kw", [dict(B=1 << 24, Sq=1), dict(B=1 << 20, Sq=1024), dict(P=1 << 30, S=1 << 30)])
def test_attention_too_large(kw):
    assert attention(**kw) == LARGE
    a = {**ATTN, **kw}
    assert L.libconv_prefix_attention_workspace(a["B"], a["Sq"], a["P"], a["S"], a["q_heads"],
                                                a["k_heads"], a["head_dim"], a["dtype"]) == -1


@pytest.mark.parametrize("kw", [dict(T=1 << 26), dict(T=1 << 22, N=1 << 20)])
def test_lora_too_large(kw):
    assert lora(**kw) == LARGE


@pytest.mark.parametrize("T", [1, 16, 17, 64, 65, 700, 1024, 1025, 9000])
@pytest.mark.parametrize("dtype", [L.F32, L.F16, L.BF16])
def test_lora_workspace_holds_the_low_rank_values(T, dtype):
    """At least a row's low-rank values and its adapter; never more than the split product."""
    for K, N, rank in ((8, 1, 1), (640, 1920, 8), (4096, 4096, 128), (1000, 8192, 33)):
        n = L.libconv_lora_workspace(T, K, N, rank, 3, 2, dtype)
        low = T * (rank + 1) * 4
        assert low <= n <= T * (128 + 32 + 1) * 4 + 256 + 64 * T * (N + 63) * 4, (T, K, N, rank)


def test_attention_workspace_of_few_keys_is_none():
    assert L.libconv_prefix_attention_workspace(4, 1, 960, 40, 20, 20, 64, L.BF16) == 0
    assert L.libconv_prefix_attention_workspace(4, 1, 9600, 40, 20, 20, 64, L.BF16) > 0
