"""What the tensor helpers of the attention-layer operators refuse before anything is launched."""
import pytest
import torch

import direct_implicit_gemm_amd as L

pytestmark = pytest.mark.gpu


def rope_args():
    h = dict(dtype=torch.float16, device="cuda")
    return dict(q=torch.randn(5, 4, 16, **h), k=torch.randn(5, 2, 16, **h),
                positions=torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5),
                freqs=L.rotary_frequencies(16, 100.0, [5, 3]), q_weight=torch.ones(16, **h),
                k_weight=torch.ones(16, **h), sections=(5, 3), v=torch.randn(5, 2, 16, **h),
                slots=torch.arange(5, dtype=torch.int32, device="cuda"),
                q_out=torch.empty(5, 4, 16, **h), k_out=torch.empty(9, 2, 16, **h),
                v_out=torch.empty(9, 2, 16, **h))


def attention_args():
    h = dict(dtype=torch.bfloat16, device="cuda")
    return dict(q=torch.randn(2, 3, 4, 16, **h), k_prefix=torch.randn(7, 2, 16, **h),
                v_prefix=torch.randn(7, 2, 16, **h), k=torch.randn(2, 6, 2, 16, **h),
                v=torch.randn(2, 6, 2, 16, **h),
                lengths=torch.tensor([3, 6], dtype=torch.int32, device="cuda"),
                out=torch.empty(2, 3, 4, 16, **h))


def lora_args():
    h = dict(dtype=torch.float32, device="cuda")
    return dict(x=torch.randn(5, 16, **h), w=torch.randn(8, 16, **h), bias=torch.randn(8, **h),
                a=torch.randn(3, 4, 16, **h), b=torch.randn(3, 8, 4, **h),
                scales=torch.ones(3, **h),
                row_starts=torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda"),
                adapters=torch.tensor([1, 0], dtype=torch.int32, device="cuda"),
                out=torch.empty(5, 8, **h))


def every_second(t):
    """The same shape and values, the last axis at twice the stride."""
    return torch.stack([t, t], -1)[..., 0]


OPS = {"rope": (L.qk_norm_rope, rope_args), "attention": (L.prefix_attention, attention_args),
       "lora": (L.lora_linear, lora_args)}


def names():
    return [("rope", n) for n in ("q", "k", "positions", "freqs", "q_weight", "k_weight", "v", "slots",
                                  "q_out", "k_out", "v_out")] + \
           [("attention", n) for n in ("q", "k_prefix", "v_prefix", "k", "v", "lengths", "out")] + \
           [("lora", n) for n in ("x", "w", "bias", "a", "b", "scales", "row_starts", "adapters",
                                  "out")]


CHANGES = {
    "host": lambda t: t.cpu(),
    "type": lambda t: t.to(torch.int64 if t.dtype == torch.int32 else
                           torch.float32 if t.dtype != torch.float32 else torch.float16),
    "stride": every_second,
    "an axis more": lambda t: t[None, None],
    "size": lambda t: torch.cat([t, t], -1),
}


@pytest.mark.parametrize("op", OPS)
def test_accepts(op):
    f, make = OPS[op]
    f(**make())
    torch.cuda.synchronize()


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("op,name", names())
def test_refuses(op, name, change):
    f, make = OPS[op]
    args = make()
    if (name, change) == ("freqs", "an axis more"):
        args["freqs"], change = args["freqs"][:-1], "size"   # a number of values is all it is
    args[name] = CHANGES[change](args[name])
    with pytest.raises(ValueError):
        f(**args)


@pytest.mark.parametrize("op,kw", [
    ("rope", dict(q=None)), ("rope", dict(positions=None)), ("rope", dict(v=3)),
    ("attention", dict(lengths=None)), ("attention", dict(q=[1.0])), ("attention", dict(scale="1")),
    ("lora", dict(w=None)), ("lora", dict(out=1)), ("lora", dict(stream="s")),
    ("lora", dict(workspace=7)),
])
def test_refuses_types(op, kw):
    f, make = OPS[op]
    with pytest.raises(TypeError):
        f(**{**make(), **kw})


@pytest.mark.parametrize("op,kw", [
    ("rope", dict(k_out=None)), ("rope", dict(v_out=None)), ("rope", dict(v=None)),
    ("rope", dict(sections=(5, 4))), ("rope", dict(sections=(9, -1))),
    ("rope", dict(sections=(2, 2, 2, 2))), ("rope", dict(sections=(2, 3, 3))),
    ("attention", dict(k=None)), ("attention", dict(v_prefix=None)),
    ("attention", dict(k=None, v=None, k_prefix=None, v_prefix=None)),
    ("attention", dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))),
    ("lora", dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))),
    ("lora", dict(a=None)), ("lora", dict(scales=None)), ("lora", dict(adapters=None)),
])
def test_refuses_missing(op, kw):
    f, make = OPS[op]
    with pytest.raises(ValueError):
        f(**{**make(), **kw})


def test_status_is_raised():
    args = lora_args()
    args["workspace"] = torch.empty(0, dtype=torch.uint8, device="cuda")
    args["x"] = args["x"].repeat(40, 1)
    args["out"] = torch.empty(200, 8, device="cuda")
    args["row_starts"] = torch.tensor([0, 2, 200], dtype=torch.int32, device="cuda")
    with pytest.raises(L.LibconvError) as e:
        L.lora_linear(**args)
    assert e.value.status == 13 and "libconv_lora_linear" in str(e.value)
    q = torch.randn(2, 1, 4, 16, dtype=torch.float16, device="cuda")
    with pytest.raises(L.LibconvError) as e:   # 4 query heads over 3
        L.prefix_attention(q, q.new_empty(5, 3, 16), q.new_empty(5, 3, 16), None, None,
                           torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert e.value.status == 2
