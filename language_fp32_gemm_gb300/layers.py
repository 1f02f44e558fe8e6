"""Transformer-layer operators on torch tensors: ``include/phobos_layers.h`` bound.

    out = linear(x, w, bias, residual, act="gelu")        act(x w + bias) + residual
    dx, dw, dbias = linear_backward(dout, x, w, z, act="gelu")
    out = linear_q8(xq, x_scale, wq, w_scale, ...)         the same with 8-bit operands
    y, h = rmsnorm(x, weight, residual)                    h = x + residual, y = h / rms(h) * weight
    q, scale, h = rmsnorm_q8(x, weight, residual)          y in 8 bits, one scale per row
    dh, dweight = rmsnorm_backward(dy, h, weight, dsum)

As in the rest of the package, only arguments are marshalled here: every step
runs in the kernels of ``libphobos_gemm.so``, and there is no CPU fallback.  The
marshalling itself is ``csrc/layers_binding.cc``, built beside the library against
the torch in use; without it importing an operator's binding raises.

Tensors are two-dimensional CUDA tensors of one device (``bias``, ``weight`` and
scales one-dimensional).  ``x`` and ``w`` may be transposed views (``w`` is K x N:
pass ``weight.t()`` for a weight stored N x K); the others have unit column stride.
Work is enqueued on ``stream`` (default: torch's current stream); outputs that the
caller does not pass are allocated there.  Wrong arguments raise ``TypeError`` or
``ValueError``, a non-zero status of the library ``PhobosError``.

Autograd does not record these calls.  With gradients enabled, a tensor that requires grad
is refused (``ValueError``): call the operators under ``torch.no_grad()``, or pair each with
its backward pass in a ``torch.autograd.Function``, whose methods run so.
"""
import contextlib

from . import PhobosError, library

LAYERS_ABI_FUNCTIONS = ("phobos_linear", "phobos_linear_backward", "phobos_rmsnorm",
                        "phobos_rmsnorm_backward")
PRODUCTS = {"auto": 0, "ffma": 1, "tensor": 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_binding = None


def _load():
    global _binding
    if _binding is None:
        import ctypes

        import torch  # noqa: F401  (the binding's symbols)
        lib = library()
        try:
            from . import _layers_binding
        except ImportError as e:
            raise ImportError("the torch binding of the layer operators is not built; run "
                              "language_fp32_gemm_gb300.build.build() (%s)" % e) from e
        _layers_binding.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                               for name in LAYERS_ABI_FUNCTIONS))
        _binding = _layers_binding
    return _binding


def _named(table, name, what):
    try:
        return table[name]
    except KeyError:
        raise ValueError("unknown %s %r (one of %s)" % (what, name, ", ".join(table))) from None


@contextlib.contextmanager
def _on(stream, *tensors):
    """Allocate and enqueue on another stream than the current one, of the tensors' device."""
    import torch
    first = tensors[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise TypeError("operands must be CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), first.device)
    elif stream.device != first.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, first.device))
    try:
        with torch.cuda.stream(stream):
            yield
    finally:
        # the caching allocator must not hand these out again before the stream is past them
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)


def _done(result, entry):
    if type(result) is int:
        raise PhobosError(result, entry)
    return result


def linear(x, w, bias=None, residual=None, act="none", out=None, preact=None, save_preact=False,
           out_dtype=None, products="auto", stream=None):
    """act(x w + bias) + residual.

    x: M x K, w: K x N, both float32, float16 or bfloat16.  bias (N), residual, out and
    preact (M x N) have ``out_dtype`` (default: that of ``out``, or x's).  act: "none",
    "relu", "gelu" (exact), "gelu_tanh" or "silu".  With ``save_preact`` returns (out, z) with
    z = x w + bias, which ``linear_backward`` takes; ``preact`` gives its memory.  ``out`` may
    be ``residual``.  products: "auto" chooses by size between "ffma" (CUDA cores, fp32
    products) and "tensor" (see the C header).
    """
    if stream is not None:
        with _on(stream, x, w, bias, residual, out, preact):
            return linear(x, w, bias, residual, act, out, preact, save_preact, out_dtype, products)
    act, products = _named(ACTIVATIONS, act, "activation"), _named(PRODUCTS, products, "products")
    out, preact = _done((_binding or _load()).linear(x, w, None, None, bias, residual, act, out, out_dtype, preact,
                                                     save_preact, products), "phobos_linear")
    return (out, preact) if save_preact else out


def linear_q8(x, x_scale, w, w_scale, bias=None, residual=None, act="none", out=None, preact=None,
              save_preact=False, out_dtype=None, products="auto", stream=None):
    """``linear`` of x_ij = x[i, j] * x_scale[i] and w_jk = w[j, k] * w_scale[k].

    x (M x K) and w (K x N, the transposed view of an N x K tensor) are float8_e4m3fn, the
    scales float32.  ``out_dtype`` defaults to bfloat16.
    """
    if stream is not None:
        with _on(stream, x, w, x_scale, w_scale, bias, residual, out, preact):
            return linear_q8(x, x_scale, w, w_scale, bias, residual, act, out, preact, save_preact, out_dtype, products)
    if x_scale is None or w_scale is None:
        raise TypeError("8-bit operands need x_scale and w_scale")
    act, products = _named(ACTIVATIONS, act, "activation"), _named(PRODUCTS, products, "products")
    if out is None and out_dtype is None:
        import torch
        out_dtype = torch.bfloat16
    out, preact = _done((_binding or _load()).linear(x, w, x_scale, w_scale, bias, residual, act, out, out_dtype, preact,
                                                     save_preact, products), "phobos_linear")
    return (out, preact) if save_preact else out


def linear_backward(dout, x, w, preact=None, act="none", dx=None, dw=None, dbias=None, need_dx=True,
                    need_dw=True, need_dbias=True, grad_dtype=None, accumulate=False, products="auto", stream=None):
    """(dx, dw, dbias) of ``linear``; None in the place of one that is not needed.

    dz = dout * act'(preact), dx = dz w^T, dw = x^T dz, dbias = column sums of dz.  The
    residual's gradient is ``dout``.  dw has w's layout; dw and dbias have ``grad_dtype``
    (default: x's; or float32), and with ``accumulate`` are added to the tensors passed.
    """
    if stream is not None:
        with _on(stream, dout, x, w, preact, dx, dw, dbias):
            return linear_backward(dout, x, w, preact, act, dx, dw, dbias, need_dx, need_dw, need_dbias, grad_dtype,
                                   accumulate, products)
    act, products = _named(ACTIVATIONS, act, "activation"), _named(PRODUCTS, products, "products")
    return _done((_binding or _load()).linear_backward(dout, x, w, preact, act, dx, dw, dbias, need_dx, need_dw,
                                                       need_dbias, grad_dtype, accumulate, products),
                 "phobos_linear_backward")


def rmsnorm(x, weight=None, residual=None, eps=1e-6, out=None, sum=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual.

    Returns y, or (y, h) with a residual; ``out`` and ``sum`` give their memory (``sum``, for
    calls with a residual, may be ``residual`` or ``x``).  All tensors have x's dtype; the
    sum is rounded to it first.
    """
    if stream is not None:
        with _on(stream, x, weight, residual, out, sum):
            return rmsnorm(x, weight, residual, eps, out, sum)
    y, _, h = _done((_binding or _load()).rmsnorm(x, weight, residual, eps, out, sum, False, None), "phobos_rmsnorm")
    return y if residual is None else (y, h)


def rmsnorm_q8(x, weight=None, residual=None, eps=1e-6, out=None, scale=None, sum=None, stream=None):
    """``rmsnorm`` with y in float8_e4m3fn: returns (q, scale) or (q, scale, h), where row i of y
    is q[i] * scale[i] and scale[i] = max |y[i]| / 448."""
    if stream is not None:
        with _on(stream, x, weight, residual, out, scale, sum):
            return rmsnorm_q8(x, weight, residual, eps, out, scale, sum)
    q, scale, h = _done((_binding or _load()).rmsnorm(x, weight, residual, eps, out, sum, True, scale), "phobos_rmsnorm")
    return (q, scale) if residual is None else (q, scale, h)


def rmsnorm_backward(dy, h, weight=None, dsum=None, eps=1e-6, dx=None, dweight=None, need_dweight=True,
                     stream=None):
    """(dx, dweight): the gradients of h (and so of x and of the residual) and of weight.

    ``h`` is what was normalised, ``dsum`` the gradient that reaches h by other ways (dx may
    be its memory).  dweight is None where it is not needed.
    """
    if stream is not None:
        with _on(stream, dy, h, weight, dsum, dx, dweight):
            return rmsnorm_backward(dy, h, weight, dsum, eps, dx, dweight, need_dweight)
    return _done((_binding or _load()).rmsnorm_backward(dy, h, weight, dsum, eps, dx, dweight, need_dweight),
                 "phobos_rmsnorm_backward")
