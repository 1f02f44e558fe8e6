"""Refusals of the layer operators' torch interface that need no GPU."""
import pytest

torch = pytest.importorskip("torch")

from language_fp32_gemm_gb300 import build as lib_build  # noqa: E402
from language_fp32_gemm_gb300 import layers  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    lib_build.build()


def test_what_requires_grad_is_refused():
    x, w = torch.zeros(4, 8), torch.zeros(8, 8)
    p, b = torch.zeros(8, 8, requires_grad=True), torch.zeros(8, requires_grad=True)
    calls = (lambda: layers.linear(x, p), lambda: layers.linear(p, w), lambda: layers.linear(x, w, bias=b),
             lambda: layers.linear(x, p.t()), lambda: layers.linear(x, w, residual=p), lambda: layers.linear(x, w, out=p),
             lambda: layers.linear_q8(x, b, w, b), lambda: layers.linear_backward(x, x, p),
             lambda: layers.linear_backward(x, x, w, dw=p), lambda: layers.rmsnorm(p), lambda: layers.rmsnorm(x, b),
             lambda: layers.rmsnorm_q8(x, b), lambda: layers.rmsnorm_backward(p, x), lambda: layers.rmsnorm_backward(x, x, b))
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):  # the next check
            call()


def test_a_sum_without_a_residual_is_refused():
    # nothing would be written to it (and the C entry point refuses it)
    x = torch.zeros(4, 8)
    for norm in (layers.rmsnorm, layers.rmsnorm_q8):
        with pytest.raises(ValueError, match="residual"):
            norm(x, sum=torch.zeros(4, 8))


def test_an_output_of_another_dtype_is_refused():
    # the call used out's own dtype and said nothing
    x, w, scale = torch.zeros(4, 8), torch.zeros(8, 8), torch.ones(8)
    q = torch.zeros(8, 8).to(torch.float8_e4m3fn)
    for call in (lambda out, dtype: layers.linear(x, w, out=out, out_dtype=dtype),
                 lambda out, dtype: layers.linear_q8(q, scale, q.t(), scale, out=out, out_dtype=dtype)):
        with pytest.raises(TypeError, match="out_dtype"):
            call(torch.zeros(4, 8), torch.bfloat16)
        with pytest.raises(TypeError, match="CUDA"):  # the next check
            call(torch.zeros(4, 8), torch.float32)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    # the call went to the current stream of the tensors' device instead
    from types import SimpleNamespace

    class Stream:
        device = torch.device("cuda:1")

    class OnDevice0(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda:0")

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    x = torch.zeros(4, 8).as_subclass(OnDevice0)
    for call in (lambda: layers.linear(x, x, stream=Stream()), lambda: layers.linear_q8(x, x, x, x, stream=Stream()),
                 lambda: layers.linear_backward(x, x, x, stream=Stream()), lambda: layers.rmsnorm(x, stream=Stream()),
                 lambda: layers.rmsnorm_q8(x, stream=Stream()), lambda: layers.rmsnorm_backward(x, x, stream=Stream())):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    for x in (torch.zeros(4, 8), "x"):
        for stream in (Stream(), 0, SimpleNamespace(cuda_stream=0)):
            with pytest.raises(TypeError):
                layers.rmsnorm(x, stream=stream)
