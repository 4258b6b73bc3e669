"""What the tensor helpers of the 8-bit cache's operators and of linear refuse before anything is
launched, what they say of gradients, and where their outputs and workspaces live."""
import warnings

import pytest
import torch

import direct_implicit_gemm_amd as L

pytestmark = pytest.mark.gpu


def cache_args():
    codes = lambda: torch.zeros(9, 2, 16, 32, dtype=torch.int8, device="cuda").transpose(1, 2)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return dict(k_cache=codes(), v_cache=codes(), k_scale=torch.ones(9, 2, device="cuda"),
                v_scale=torch.ones(9, 2, device="cuda"), lengths=ints(4, 17),
                block_table=ints(3, 1, 0, 2).view(2, 2)), ints(0, 2, 5)


def write_args():
    c, starts = cache_args()
    h = dict(dtype=torch.float16, device="cuda")
    return dict(k=torch.randn(5, 2, 32, **h), v=torch.randn(5, 2, 32, **h), row_starts=starts, **c)


def read_args():
    h = dict(dtype=torch.bfloat16, device="cuda")
    return dict(k_out=torch.zeros(2, 20, 2, 32, **h), v_out=torch.zeros(2, 20, 2, 32, **h),
                **cache_args()[0])


def attention_args():
    c, starts = cache_args()
    h = dict(dtype=torch.bfloat16, device="cuda")
    return dict(q=torch.randn(5, 4, 32, **h), row_starts=starts, out=torch.empty(5, 4, 32, **h), **c)


def linear_args():
    h = dict(device="cuda")
    return dict(x=torch.randn(5, 16, **h), w=torch.randn(8, 16, **h), bias=torch.randn(8, **h),
                residual=torch.randn(5, 8, **h), out=torch.empty(5, 8, **h), act="gelu")


def every_second(t):
    """The same shape and values, the last axis at twice the stride."""
    return torch.stack([t, t], -1)[..., 0]


OPS = {"write": (L.kv_cache_write, write_args), "read": (L.kv_cache_read, read_args),
       "attention": (L.cache_attention, attention_args), "linear": (L.linear, linear_args)}
CHANGES = {
    "host": lambda t: t.cpu(),
    "type": lambda t: t.to(torch.int64 if t.dtype == torch.int32 else torch.uint8
                           if t.dtype == torch.int8 else torch.float64),
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
@pytest.mark.parametrize("op", OPS)
def test_refuses(op, change):
    f, make = OPS[op]
    for name, t in make().items():
        if not torch.is_tensor(t) or (name, change) == ("block_table", "size"):
            continue   # (a wider table is a table)
        args = make()
        args[name] = CHANGES[change](args[name])
        with pytest.raises(ValueError):
            f(**args)
            print(op, name, change)


@pytest.mark.parametrize("op,kw", [
    ("write", dict(k=None)), ("write", dict(k_scale=2.0)), ("write", dict(row_starts=None)),
    ("read", dict(k_cache=None)), ("read", dict(k_out=3)), ("read", dict(lengths=[4, 17])),
    ("attention", dict(q=None)), ("attention", dict(block_table=None)),
    ("attention", dict(scale="1")), ("attention", dict(max_rows="a")), ("attention", dict(stream="s")),
    ("linear", dict(w=None)), ("linear", dict(out=1)), ("linear", dict(workspace=7)),
    ("linear", dict(stream="s")),
])
def test_refuses_types(op, kw):
    f, make = OPS[op]
    with pytest.raises(TypeError):
        f(**{**make(), **kw})


@pytest.mark.parametrize("op,kw", [
    ("attention", dict(max_rows=-1)), ("linear", dict(act="swish")), ("linear", dict(act=None)),
    ("read", dict(k_out=None, v_out=None, dtype=torch.float64)),
    ("read", dict(k_out=None, v_out=None, rows=-1)),
    ("attention", dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))),
    ("linear", dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))),
])
def test_refuses_values(op, kw):
    f, make = OPS[op]
    with pytest.raises(ValueError):
        f(**{**make(), **kw})


def test_status_is_raised():
    args = attention_args()
    args["q"], args["out"] = torch.cat([args["q"]] * 2, 1)[:, :5], None
    with pytest.raises(L.LibconvError) as e:     # 5 query heads over 2
        L.cache_attention(**args)
    assert e.value.status == 2 and "libconv_cache_attention" in str(e.value)
    args = write_args()
    args["v_cache"] = args["k_cache"]
    with pytest.raises(L.LibconvError) as e:
        L.kv_cache_write(**args)
    assert e.value.status == 5


@pytest.fixture
def every_time():
    torch.set_warn_always(True)
    yield
    torch.set_warn_always(False)


@pytest.mark.parametrize("op,name", [("write", "v"), ("attention", "q"), ("linear", "w"),
                                     ("linear", "residual")])
def test_a_leaf_that_requires_gradients_is_warned_of(op, name, every_time):
    f, make = OPS[op]
    args = make()
    args[name].requires_grad_()
    with pytest.warns(UserWarning, match="no backward pass"):
        y = f(**args)
    assert y is None or not y.requires_grad
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            f(**args)
    torch.cuda.synchronize()


def test_outputs_and_workspaces_on_a_given_stream():
    h = dict(dtype=torch.bfloat16, device="cuda")
    codes = torch.ones(300, 4, 16, 128, dtype=torch.int8, device="cuda").transpose(1, 2)
    scale = torch.full((300, 4), 0.125, device="cuda")
    table = torch.arange(288, dtype=torch.int32, device="cuda").view(3, 96)
    n = torch.tensor([1500, 30, 800], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2, 400], dtype=torch.int32, device="cuda")
    q, x, w = torch.ones(400, 16, 128, **h), torch.ones(64, 4096, **h), torch.ones(1024, 4096, **h)
    calls = {
        "read": lambda **kw: L.kv_cache_read(codes, codes, scale, scale, n, table, **kw),
        "attention": lambda **kw: L.cache_attention(q, codes, codes, scale, scale, starts, n, table,
                                                    return_lse=True, **kw),
        "linear": lambda **kw: (L.linear(x, w, **kw),),
    }
    held = lambda s: sum(m["total_size"] for m in torch.cuda.memory_snapshot() if m["stream"] == s)
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        before = held(side.cuda_stream)
        for turn in range(3):
            freed = [torch.empty_like(t) for t in want]
            places = {t.data_ptr() for t in freed}
            del freed
            out = call(stream=side.cuda_stream)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (name, turn)
            assert not places & {t.data_ptr() for t in out}, name
            del out
        assert held(side.cuda_stream) >= before
        # the default stream by its handle, from another current stream
        with torch.cuda.stream(side):
            out = call(stream=0)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            assert torch.cuda.current_stream() == side


def test_two_streams_at_once():
    """Each call has a workspace of its own."""
    h = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-127, 128, (600, 4, 16, 128), generator=g, device="cuda",
                          dtype=torch.int8).transpose(1, 2)
    scale = torch.full((600, 4), 2.0 ** -6, device="cuda")
    table = torch.randperm(600, device="cuda")[:576].int().view(3, 192)
    n = torch.tensor([3000, 2900, 1800], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2, 300], dtype=torch.int32, device="cuda")
    qs = [torch.randn(300, 16, 128, generator=g, **h) for _ in range(4)]
    xs = [torch.randn(64, 4096, generator=g, **h) for _ in range(4)]
    w = torch.randn(1024, 4096, generator=g, **h)
    run = lambda q, x: (L.cache_attention(q, codes, codes, scale, scale, starts, n, table),
                        L.linear(x, w, act="silu"))
    want = [run(q, x) for q, x in zip(qs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        got = []
        for s, q, x in zip(streams, qs, xs):
            with torch.cuda.stream(s):
                got.append(run(q, x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
