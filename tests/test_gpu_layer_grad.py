"""The attention-layer operators have no backward pass, and say so to who may expect one."""
import warnings

import pytest

torch = pytest.importorskip("torch")
import direct_implicit_gemm_amd as L  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture
def every_time():
    torch.set_warn_always(True)
    yield
    torch.set_warn_always(False)


def rope(leaf):
    q, k = torch.ones(4, 2, 16, device="cuda"), torch.ones(4, 1, 16, device="cuda")
    w = torch.ones(16, device="cuda", requires_grad=leaf)
    at = torch.arange(4, dtype=torch.int32, device="cuda")
    return L.qk_norm_rope(q, k, at, L.rotary_frequencies(16), w, w)[0]


def attention(leaf):
    q, k = torch.ones(2, 1, 2, 16, device="cuda"), torch.ones(2, 3, 1, 16, device="cuda")
    v = torch.ones(2, 3, 1, 16, device="cuda", requires_grad=leaf)
    return L.prefix_attention(q, None, None, k, v, torch.ones(2, dtype=torch.int32, device="cuda"))


def lora(leaf):
    w = torch.nn.Parameter(torch.ones(8, 16, device="cuda"), requires_grad=leaf)
    return L.lora_linear(torch.ones(3, 16, device="cuda"), w, None, None, None, None, None, None)


@pytest.mark.parametrize("op", [rope, attention, lora], ids=lambda f: f.__name__)
def test_a_leaf_that_requires_gradients_is_warned_of(op, every_time):
    with pytest.warns(UserWarning, match="no backward pass"):
        y = op(True)
    assert not y.requires_grad
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert torch.equal(op(False), y)
        with torch.no_grad():
            assert torch.equal(op(True), y)
        with torch.inference_mode():
            assert torch.equal(op(True), y)


@pytest.mark.parametrize("op", [rope, attention, lora], ids=lambda f: f.__name__)
def test_a_warning_that_is_an_error_is_raised(op, every_time):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):
            op(True)
    assert bool(torch.isfinite(op(False)).all())
