"""qk_norm_rope on the GPU against its plain form in 64 bits."""
import sys

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(T, hq, hk, d, rot, axes, far, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    t = C.TYPES[dtype]
    qkv = (2 * torch.randn(T, (hq + 2 * hk) * d, generator=g)).to(t).cuda()
    q, k, v = (x.view(T, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], 1))
    half = rot // 2
    sections = [half - (axes - 1) * (half // axes)] + (axes - 1) * [half // axes]
    freqs = L.rotary_frequencies(rot, 10000.0, sections)
    pos = torch.randint(-3, far, (axes, T), generator=g).int().cuda()
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(t).cuda() for _ in range(2)]
    return qkv, q, k, v, sections, freqs, pos, w


CASES = [  # T, query heads, key heads, head_dim, rot_dim, axes, positions to, interleaved, dtype
    (1, 1, 1, 64, 64, 1, 10, False, "bf16"),
    (1, 20, 5, 128, 128, 1, 1 << 30, False, "bf16"),
    (7, 3, 1, 80, 80, 3, 500, False, "f16"),
    (33, 5, 5, 96, 64, 2, 1 << 20, False, "bf16"),
    (5, 8, 2, 256, 256, 1, 1 << 20, False, "bf16"),
    (3, 2, 2, 8, 0, 1, 10, False, "f16"),
    (1031, 7, 7, 64, 64, 3, 64, False, "bf16"),
    (4099, 3, 1, 128, 96, 1, 1 << 20, True, "f32"),
    (9, 2, 1, 72, 36, 1, 1 << 20, True, "bf16"),
    (13, 4, 4, 256, 254, 2, 1000, True, "f32"),
    (17, 6, 3, 40, 32, 1, 1000, False, "f32"),
    (2, 1, 1, 16, 2, 1, 1000, True, "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_64_bits(case):
    T, hq, hk, d, rot, axes, far, inter, dtype = case
    print(f"[gpu] rope {case}", flush=True)
    _, q, k, v, sec, freqs, pos, w = make(T, hq, hk, d, rot, axes, far, dtype, 1)
    qo, ko = L.qk_norm_rope(q, k, pos, freqs, w[0], w[1], eps=1e-6, sections=sec, interleaved=inter)
    torch.cuda.synchronize()
    for got, x, wt, name in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want, bound = C.rope(x, wt, pos, freqs, sec, 1e-6, inter)
        C.assert_within(got, want, bound, f"{name} {case}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_write_and_skipped_slots(dtype):
    """Keys and values land in their slots, other rows stay, bad slots write nothing."""
    T, hq, hk, d = 19, 4, 2, 64
    _, q, k, v, sec, freqs, pos, w = make(T, hq, hk, d, d, 1, 4000, dtype, 2)
    rows = 50
    # a cache with a longer row (its values beside its keys)
    cache = torch.full((rows, 2, hk, d), 7.0, dtype=q.dtype, device="cuda")
    slots = torch.randperm(rows, generator=torch.Generator().manual_seed(3))[:T].int()
    slots[4], slots[9], slots[11] = -1, rows, 2 ** 31 - 1
    qo, ko, vo = L.qk_norm_rope(q, k, pos, freqs, w[0], None, sections=sec, v=v, slots=slots.cuda(),
                                k_out=cache[:, 0], v_out=cache[:, 1])
    torch.cuda.synchronize()
    want_k, bound = C.rope(k, None, pos, freqs, sec, 1e-6, False)
    written = torch.zeros(rows, dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < rows:
            written[s] = True
            C.assert_within(ko[s], want_k[t], bound[t], f"slot {s}")
            assert torch.equal(vo[s], v[t])
    assert bool((cache[~written.cuda()] == 7.0).all())
    want, bound = C.rope(q, w[0], pos, freqs, sec, 1e-6, False)
    C.assert_within(qo, want, bound, "q")


def test_in_place_in_a_fused_projection():
    qkv, q, k, v, sec, freqs, pos, w = make(77, 6, 3, 128, 128, 3, 900, "bf16", 4)
    want_q, bq = C.rope(q, w[0], pos, freqs, sec, 1e-6, False)
    want_k, bk = C.rope(k, w[1], pos, freqs, sec, 1e-6, False)
    values = v.clone()
    qo, ko = L.qk_norm_rope(q, k, pos, freqs, w[0], w[1], sections=sec, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert qo.data_ptr() == q.data_ptr()
    C.assert_within(q, want_q, bq, "q in place")
    C.assert_within(k, want_k, bk, "k in place")
    assert torch.equal(v, values)


def test_zero_rows_and_no_tokens():
    _, q, k, v, sec, freqs, pos, w = make(3, 2, 1, 64, 64, 1, 10, "f16", 5)
    q = torch.zeros_like(q.contiguous())
    qo, _ = L.qk_norm_rope(q, k, pos, freqs, w[0], w[1])
    torch.cuda.synchronize()
    assert bool((qo == 0).all())
    qo, ko = L.qk_norm_rope(q[:0], k[:0], pos[:, :0].contiguous(), freqs)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)


def test_head_major_outputs_and_another_stream():
    """Outputs laid out [head][token]; inputs made on the stream that is used."""
    _, q, k, v, sec, freqs, pos, w = make(129, 4, 2, 64, 64, 1, 3000, "bf16", 6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qo = torch.empty(4, 129, 64, dtype=q.dtype, device="cuda").transpose(0, 1)
    ko = torch.empty(2, 129, 64, dtype=q.dtype, device="cuda").transpose(0, 1)
    L.qk_norm_rope(q, k, pos, freqs, w[0], w[1], q_out=qo, k_out=ko, stream=s.cuda_stream)
    s.synchronize()
    for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
        want, bound = C.rope(x, wt, pos, freqs, sec, 1e-6, False)
        C.assert_within(got, want, bound, "head-major")


MORE = [  # T, query heads, key heads, head_dim, rot_dim, axes, positions to, interleaved, dtype
    (11, 9, 2, 24, 16, 1, 100, False, "bf16"),
    (5, 3, 3, 40, 16, 1, 100, False, "f16"),
    (6, 2, 1, 104, 48, 3, 5000, False, "bf16"),
    (9, 5, 1, 200, 176, 2, 5000, False, "bf16"),
    (21, 4, 2, 256, 16, 1, 5000, False, "f32"),
    (8, 3, 1, 8, 6, 1, 5000, True, "bf16"),
    (10, 2, 2, 136, 130, 3, 5000, True, "f16"),
    (2500, 1, 1, 128, 128, 1, 2500, False, "bf16"),
]


@pytest.mark.parametrize("case", MORE, ids=str)
def test_more_shapes_against_64_bits(case):
    test_against_64_bits(case)


@pytest.mark.parametrize("interleaved", [False, True])
def test_an_infinity_beside_what_does_not_turn(interleaved):
    """Of a head with an infinity only the infinity's own pair is lost; other heads are not."""
    _, q, k, v, sec, freqs, pos, w = make(4, 3, 1, 64, 32, 1, 100, "bf16", 8)
    want, bound = C.rope(q, w[0], pos, freqs, sec, 1e-6, interleaved)
    q = q.clone()
    q[2, 1, 50] = float("inf")    # past what turns
    got, _ = L.qk_norm_rope(q, k, pos, freqs, w[0], w[1], sections=sec, interleaved=interleaved)
    torch.cuda.synchronize()
    hit = torch.zeros(q.shape, dtype=torch.bool)
    hit[2, 1] = True
    C.assert_within(got.cpu()[~hit], want[~hit], bound[~hit], "other heads")
    rest = got.cpu()[2, 1].float()
    assert bool(torch.isnan(rest[50]))
    assert bool((torch.cat([rest[:50], rest[51:]]) == 0).all())   # divided by an infinite norm


def test_tiny_values_without_eps():
    """The root of a mean square below what its fast form takes."""
    _, q, k, v, sec, freqs, pos, w = make(3, 2, 1, 64, 64, 1, 100, "f32", 9)
    q = q * 1e-20
    got, _ = L.qk_norm_rope(q, k, pos, freqs, w[0], w[1], eps=0.0)
    torch.cuda.synchronize()
    want, bound = C.rope(q, w[0], pos, freqs, sec, 0.0, False)
    # squares of 1e-20 keep 10 to 20 bits of theirs: the norm of 64 of them is off by 2^-10
    C.assert_within(got, want, bound + 2.0 ** -10 * want.abs().amax(-1, keepdim=True), "tiny")
