"""Where the attention-layer helpers' outputs and workspaces live when a stream is given."""
import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rope():
    q, k = torch.ones(1200, 8, 128, device="cuda"), torch.ones(1200, 2, 128, device="cuda")
    at = torch.arange(1200, dtype=torch.int32, device="cuda")
    f = L.rotary_frequencies(128)
    return lambda **kw: L.qk_norm_rope(q, k, at, f, v=k, **kw)


def attention():
    """A plan with partial results."""
    h = dict(dtype=torch.bfloat16, device="cuda")
    q, kp, k = torch.ones(96, 16, 8, 128, **h), torch.ones(900, 2, 128, **h), \
        torch.ones(96, 40, 2, 128, **h)
    n = torch.full((96,), 40, dtype=torch.int32, device="cuda")
    return lambda **kw: L.prefix_attention(q, kp, kp, k, k, n, return_lse=True, **kw)


def lora():
    h = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.ones(1100, 512, **h), torch.ones(1536, 512, **h)
    a, b = torch.ones(2, 16, 512, **h), torch.ones(2, 1536, 16, **h)
    s, starts = torch.ones(2, device="cuda"), torch.tensor([0, 500, 1100]).int().cuda()
    ids = torch.tensor([1, 0]).int().cuda()
    return lambda **kw: (L.lora_linear(x, w, None, a, b, s, starts, ids, **kw),)


OPS = {"rope": rope, "attention": attention, "lora": lora}


def bytes_of(stream):
    """What torch's allocator holds for a stream."""
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream)


@pytest.mark.parametrize("op", OPS)
def test_outputs_on_a_given_stream(op):
    call = OPS[op]()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for turn in range(3):
        # blocks that the current stream may still use are not the call's outputs
        freed = [torch.empty_like(t) for t in want]
        places = {t.data_ptr() for t in freed}
        del freed
        out = call(stream=side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
        assert not places & {t.data_ptr() for t in out}
        # nor are the outputs, once dropped, the current stream's to write
        places = {t.data_ptr() for t in out}
        torch.cuda.synchronize()
        del out
        again = [torch.empty_like(t) for t in want]
        assert not places & {t.data_ptr() for t in again}
        del again


@pytest.mark.parametrize("op", ["attention", "lora"])
def test_workspace_on_a_given_stream(op):
    call = OPS[op]()
    out = torch.empty_like(call()[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    before = bytes_of(side.cuda_stream)
    call(stream=side.cuda_stream, out=out, workspace=False) if op == "attention" else None
    lse = bytes_of(side.cuda_stream) - before if op == "attention" else 0
    call(stream=side.cuda_stream, out=out)
    side.synchronize()
    assert bytes_of(side.cuda_stream) - before > lse


@pytest.mark.parametrize("op", OPS)
def test_the_current_stream_given(op):
    """By its handle, and the default stream by 0: outputs as without."""
    call = OPS[op]()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in
               zip(call(stream=torch.cuda.current_stream().cuda_stream), want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = call(stream=0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.cuda.current_stream() == side   # the caller's stream again
    with pytest.raises(TypeError):
        call(stream="0")
