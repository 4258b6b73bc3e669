"""Sizes of the attention-layer operators near what a launch holds (2^32 lanes an axis)."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402
import layercheck as C  # noqa: E402

MOST = (1 << 24) - 4096   # groups of rows that prefix_attention accepts


def test_attention_plans_fit_a_launch():
    """With the most entries that are accepted, sharing the prefix would add its workgroups to
    theirs, past what a launch holds: each entry reads it then, and nothing is joined."""
    size = L.libconv_prefix_attention_workspace
    assert size(16600000, 1, 1000, 1, 1, 1, 8, L.BF16) > 0
    assert size(MOST, 1, 1000, 1, 1, 1, 8, L.BF16) == 0
    assert size(MOST // 8, 1, 1000, 1, 8, 8, 8, L.F16) == 0
    assert size(MOST + 1, 1, 1000, 1, 1, 1, 8, L.BF16) == -1


@pytest.mark.gpu
def test_attention_of_the_most_entries():
    g = torch.Generator().manual_seed(1)
    print("[gpu] attention of 2^24 - 4096 entries", flush=True)
    h = dict(dtype=torch.bfloat16, device="cuda")
    some = torch.cat([torch.arange(8), torch.randint(8, MOST - 8, (16,), generator=g),
                      torch.arange(MOST - 8, MOST)])
    q, k = torch.randn(MOST, 1, 1, 8, **h), torch.randn(MOST, 1, 1, 8, **h)
    kp, vp = torch.randn(1000, 1, 8, **h), torch.randn(1000, 1, 8, **h)
    n = (torch.arange(MOST, device="cuda") % 2).int()
    out = L.prefix_attention(q, kp, vp, k, k, n)
    torch.cuda.synchronize()
    at = some.cuda()
    want, bound, _, _ = C.attention(q[at], kp, vp, k[at], k[at], n[at], 8 ** -0.5, True)
    C.assert_within(out[at], want, bound, "entries")
    assert bool(torch.isfinite(out).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,dtype", [(1, (1 << 27) + 20, "bf16"), (65, 180000000, "f32")])
def test_projections_of_many_outputs(T, N, dtype):
    """16 outputs a workgroup of 512 lanes, and tiles of 32 x 32, would be more than a launch
    holds."""
    g = torch.Generator().manual_seed(2)
    t, K = C.TYPES[dtype], 8
    print(f"[gpu] lora {T} rows of {N} outputs", flush=True)
    x, w = torch.randn(T, K, generator=g).to(t).cuda(), torch.randn(N, K, dtype=t, device="cuda")
    y = L.lora_linear(x, w, None, None, None, None, None, None)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(300), torch.randint(300, N - 300, (3000,), generator=g),
                    torch.arange(N - 300, N)]).cuda()
    want, bound = C.lora(x, w[at], None, None, None, None, None, None)
    C.assert_within(y[:, at], want, bound, "outputs")
    assert bool(torch.isfinite(y[:, ::97]).all())
    del x, w, y
    torch.cuda.empty_cache()
