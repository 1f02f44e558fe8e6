"""The layer operators where their kernels take turns, run long or meet extreme values."""
import pytest

import layers_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from language_fp32_gemm_gb300 import layers  # noqa: E402
import language_fp32_gemm_gb300 as phobos  # noqa: E402
from test_layers_gpu import BF16, E4M3, F16, F32, IDS, TYPES, dev, normal, vector, weight  # noqa: E402, F401


def small_integers(rows, cols, dtype, seed):
    """-1, 0 or 1: sums of up to 256 products are exact in every type."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, (rows, cols), generator=g, device="cuda").to(dtype)


# More tiles than SMs, short contractions, and columns that leave a tile with fewer output blocks
# than a warp has places for: one tile's stores are still on their way when the next one's begin.
# Exact sums, so that a block stored twice, late or over another shows in any element.
@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("preact", [False, True], ids=["out", "out+z"])
@pytest.mark.parametrize("M,N,K", [(40000, 64, 64), (40000, 32, 64), (8192, 192, 64), (64, 60000, 64), (32, 60000, 64),
                                   (16, 60000, 128), (40, 60008, 64), (8192, 4104, 64), (8192, 4128, 128)])
def test_many_tiles_without_a_residual(M, N, K, preact, dtype):
    x, w = small_integers(M, K, dtype, 1), small_integers(N, K, dtype, 2).t()
    want = x.float() @ w.float()
    assert torch.equal(want, want.round()) and want.abs().max() <= K
    for _ in range(5):
        out, z = torch.full_like(want, 7.0, dtype=dtype), torch.full_like(want, 7.0, dtype=dtype)
        if preact:
            layers.linear(x, w, act="relu", out=out, preact=z, save_preact=True, products="tensor")
            assert torch.equal(z.float(), want) and torch.equal(out.float(), want.clamp(min=0))
        else:
            layers.linear(x, w, out=out, products="tensor")
            assert torch.equal(out.float(), want)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_many_tiles_of_gradients(dtype):
    M, N, K = 8192, 64, 4128
    x, w, dout = small_integers(M, K, dtype, 1), small_integers(K, N, dtype, 2), small_integers(M, N, dtype, 3)
    dx_want, dw_want = dout.float() @ w.float().t(), x.float().t() @ dout.float()
    for _ in range(5):
        dx, dw, _ = layers.linear_backward(dout, x, w, need_dbias=False, grad_dtype=F32, products="tensor")
        assert torch.equal(dx.float(), dx_want) and torch.equal(dw, dw_want)


LONG = [(3, 4097), (5, 1000), (400, 1003), (2, 16384), (2, 20001), (2, 33001), (1, 40001)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("over", ["residual", "x"])
@pytest.mark.parametrize("pad_out", [0, 8])
@pytest.mark.parametrize("size", LONG, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_sum_over_an_input(size, pad_out, over, dtype):
    # inputs on 16-byte boundaries, outputs there or not; rows within the registers and beyond them
    rows, cols = size
    x, r = (normal(size, dtype, i, 1.0, pad=-cols % 8) for i in (1, 2))
    w = (1 + 0.1 * vector(cols, F32, 3)).to(dtype)
    h = (x.float() + r.float()).to(dtype)
    want, bound = ref.rmsnorm(h, w, 1e-6)
    y0 = torch.empty(rows, cols + (-cols % 8 if pad_out else 0), dtype=dtype, device="cuda")[:, :cols]
    q0 = torch.empty(rows, cols + (-cols % 16 if pad_out else 0), dtype=E4M3, device="cuda")[:, :cols]
    for eight_bit in (False, True):
        a, b = (torch.empty_strided(t.shape, t.stride(), dtype=dtype, device="cuda").copy_(t) for t in (x, r))
        if eight_bit:
            q, scale, got = layers.rmsnorm_q8(a, w, b, out=q0, sum=b if over == "residual" else a)
            s = ref.f64(scale)[:, None]
            ref.check(ref.f64(q) * s, want, bound + s * (2.0 ** -4 * (want / s).abs() + 2.0 ** -10) * (1 + 2.0 ** -20), "q")
        else:
            y, got = layers.rmsnorm(a, w, b, out=y0, sum=b if over == "residual" else a)
            ref.check(y, want, ref.rounded(bound, want, dtype), "y")
        assert torch.equal(got, h) and got.data_ptr() == (b if over == "residual" else a).data_ptr()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("size", LONG, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_gradient_over_dsum(size, dtype):
    rows, cols = size
    h, dy, ds = (normal(size, dtype, i, 1.0, pad=-cols % 8) for i in (1, 2, 3))
    dx, dw = layers.rmsnorm_backward(dy, h, None, ds)
    over, dw2 = layers.rmsnorm_backward(dy, h, None, ds, dx=ds)
    assert over.data_ptr() == ds.data_ptr() and torch.equal(over, dx) and torch.equal(dw, dw2)


# Tiles cut along the contraction: pieces' sums meet in the workspace.  Exact sums.
@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("residual", [False, True], ids=["", "residual"])
@pytest.mark.parametrize("M,N,K", [(16, 8192, 8192), (5, 300, 16384), (600, 520, 4096), (300, 264, 2080), (3000, 136, 4096)])
def test_pieces_of_tiles(M, N, K, residual, dtype):
    x, w = small_integers(M, K, dtype, 1), small_integers(N, K, dtype, 2).t()
    r = small_integers(M, N, F32, 3) if residual else None
    want = x.float() @ w.float() + (r if residual else 0.0)
    for _ in range(5):
        out = layers.linear(x, w, residual=r, out_dtype=F32, products="tensor")
        assert torch.equal(out, want)


def test_rmsnorm_of_the_longest_row():
    # 2^31 - 1024 columns: a thread's last step passes 2^31.  Ones times two: every sum is exact
    # (2^21 or fewer squares of four a thread), rstd and y are known to the bit in bf16.
    cols = (1 << 31) - 1024
    x = torch.full((1, cols), 2.0, dtype=BF16, device="cuda")
    y = layers.rmsnorm(x)
    assert y.shape == x.shape and (y == 1.0).all()
    del y
    q, scale = layers.rmsnorm_q8(x)
    assert (q.view(torch.uint8) == 0x7E).all() and abs(scale.item() * 448 - 1) < 2.0 ** -20
    del q
    # dy = h: dx = rstd (dy - n mean(dy n)) is h's rounding errors times rstd, dweight = 2 n
    dx, dw = layers.rmsnorm_backward(x, x)
    assert dx.abs().max() <= 2.0 ** -18 and (dw == 2.0).all()
    del x, dx, dw
    phobos.phobos_release()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=IDS.get)
@pytest.mark.parametrize("rows,cols", [(4, 300), (5, 4096), (400, 2048), (3, 1001)])
def test_rmsnorm_q8_of_small_numbers(rows, cols, dtype):
    # rows from 1e-34 down to the smallest normal numbers, with zeros among them: eps decides rstd
    x = normal((rows, cols), F32, 1) * torch.logspace(-34, -38, rows, device="cuda")[:, None]
    x[:, ::3] = 0
    x = x.to(dtype)
    q, scale = layers.rmsnorm_q8(x)
    want, bound = ref.rmsnorm(x, None, 1e-6)
    amax = want.abs().amax(1)
    s = ref.f64(scale)
    exact = (amax / 448).clamp(min=2.0 ** -126)
    assert ((s - exact).abs() <= 2.0 ** -20 * exact).all()
    # below the least scale, q loses what half of e4m3's smallest step leaves: 2^-10 of the scale.
    # Below 2^-126 fp32 products round by up to 2^-150.
    s = s[:, None]
    ref.check(ref.f64(q) * s, want, bound + s * (2.0 ** -4 * (want / s).abs() + 2.0 ** -10) * (1 + 2.0 ** -20) + 2.0 ** -148, "q")
    assert not q[:, ::3].float().any()


# Sums of one sign, where truncation in tensor memory adds up.  The residual takes the sum away
# again, so that the output's own rounding does not hide the error.  Whole tiles (76 pairs of SMs
# have one each), so that each sums all of K.
WHOLE_TILES = 1024, 4864


@pytest.mark.parametrize("dtype", [F16, BF16], ids=IDS.get)
@pytest.mark.parametrize("K", [8192, 16384])
def test_one_large_term_and_many_small_ones(K, dtype):
    # each 16 products after the first add 1.75 2^-24 of the sum: less than its last bit
    M, N = WHOLE_TILES
    x = torch.full((M, K), 64.0, dtype=dtype, device="cuda")
    w = torch.zeros(N, K, dtype=dtype, device="cuda")
    w[:, ::16] = 1.75 * 2.0 ** -20
    w[:, 0] = 16.0
    r = torch.full((M, N), -1024.0, dtype=dtype, device="cuda")
    want, _, bound, _ = ref.linear(x[:1], w.t()[:, :1], None, r[:1, :1])
    out = layers.linear(x, w.t(), residual=r, products="tensor")
    ref.check(out, want.expand(M, N), bound.expand(M, N), "out")


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids={F16: "f16", BF16: "bf16", E4M3: "e4m3"}.get)
@pytest.mark.parametrize("K", [8192, 16384])
def test_sums_of_one_sign(K, dtype):
    M, N = WHOLE_TILES
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.rand(M, K, generator=g, device="cuda").to(dtype)
    w = (torch.rand(N, K, generator=g, device="cuda") * (0.5 if dtype == E4M3 else 2.0 ** -5)).to(dtype)
    rows = [*range(4), *range(M - 4, M)]
    out_dtype = BF16 if dtype == E4M3 else dtype
    scales = (torch.ones(M, device="cuda"), torch.full((N,), 2.0 ** -4, device="cuda")) if dtype == E4M3 else (None, None)
    part = None if dtype != E4M3 else scales[0][rows]
    z = ref.linear(x[rows], w.t(), None, None, "none", part, scales[1], out_dtype)[1]
    r = torch.zeros(M, N, dtype=out_dtype, device="cuda")
    r[rows] = (-z).to(out_dtype).cuda()
    want, _, bound, _ = ref.linear(x[rows], w.t(), None, r[rows], "none", part, scales[1], out_dtype)
    if dtype == E4M3:
        out = layers.linear_q8(x, scales[0], w.t(), scales[1], residual=r, out_dtype=out_dtype, products="tensor")
    else:
        out = layers.linear(x, w.t(), residual=r, products="tensor")
    ref.check(out[rows], want, bound, "out")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("small", ["x", "w"])
@pytest.mark.parametrize("M,N,K", [(40, 64, 300), (300, 600, 1024), (900, 1100, 2048)])
def test_fp32_rows_of_the_smallest_numbers(M, N, K, small, layout):
    # rows of one operand from 2^-90 to 2^-135, below the normal numbers, against large ones: the
    # products are ordinary numbers, and each output keeps its own relative accuracy
    x, w = normal((M, K), F32, 1), normal((K, N), F32, 2)
    down = torch.linspace(-90, -135, M if small == "x" else N, device="cuda", dtype=torch.float64).round()
    if small == "x":
        x, w = (x.double() * torch.exp2(down)[:, None]).float(), w * 2.0 ** 100
    else:
        x, w = x * 2.0 ** 100, (w.double() * torch.exp2(down)[None, :]).float()
    w = w.t().contiguous().t() if layout == "nk" else w
    want, _, bound, _ = ref.linear(x, w)
    ref.check(layers.linear(x, w, products="tensor"), want, bound, "out")
    # both small: nothing is left
    assert not layers.linear(x[:2] * 2.0 ** -126, w * 2.0 ** -126, products="tensor").any()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_slopes_far_from_zero(act, dtype):
    # one where z is large, zero where it is large and negative: up to the type's largest value, and
    # for the infinity that a pre-activation beyond it becomes.  A NaN stays.
    far = torch.tensor([60.0, 104.0, 1e4, 2e19, 1e30, float("inf")])
    far = far[(far <= torch.finfo(dtype).max) | far.isinf()]
    z = torch.cat([far, -far, torch.tensor([float("nan")])]).to(dtype).cuda()[None, :]
    n = len(far)
    dout = torch.ones_like(z)
    x, w = torch.ones(1, 1, dtype=dtype, device="cuda"), torch.ones(1, z.shape[1], dtype=dtype, device="cuda")
    _, _, db = layers.linear_backward(dout, x, w, z, act, need_dx=False, need_dw=False)
    assert (db[:n] == 1).all() and (db[n:2 * n].abs() <= 2.0 ** -40).all()
    assert db[-1].isnan() if act != "relu" else db[-1] == 0


def test_autograd_is_told():
    # refused while gradients are enabled, taken without; a tensor that was written is seen to be
    x, w = normal((40, 64), F32, 1), weight(64, 48, F32, 2, "nk").requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        layers.linear(x, w)
    with torch.no_grad():
        want = layers.linear(x, w)
    assert torch.equal(layers.linear(x, w.detach()), want)
    buf, s, z = torch.ones(40, 48, device="cuda"), torch.ones(40, device="cuda"), torch.ones(40, 64, device="cuda")
    leaf = torch.ones(40, 48, device="cuda", requires_grad=True)
    loss = (leaf * buf).sum()
    layers.linear(x, w.detach(), out=buf)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    for t, call in ((buf, lambda: layers.linear(x, w.detach(), preact=buf, save_preact=True)),
                    (z, lambda: layers.linear_backward(want, x, w.detach(), dx=z)),
                    (s[:8], lambda: layers.linear_backward(want[:, :8], x, w.detach()[:, :8], dbias=s[:8])),
                    (z, lambda: layers.rmsnorm(x, None, x, sum=z)),
                    (s, lambda: layers.rmsnorm_q8(x, scale=s)),
                    (z, lambda: layers.rmsnorm_backward(x, x, dx=z))):
        before = t._version
        call()
        assert t._version > before
    with torch.inference_mode():
        assert torch.equal(layers.linear(x, w, out=torch.empty_like(want)), want)


def test_as_an_autograd_function():
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            out, z = layers.linear(x, w.t(), b, act="gelu", save_preact=True)
            ctx.save_for_backward(x, w, z)
            return out

        @staticmethod
        def backward(ctx, dout):
            x, w, z = ctx.saved_tensors
            dx, dw, db = layers.linear_backward(dout.contiguous(), x, w.t(), z, "gelu")
            return dx, dw.t(), db

    x, w, b = normal((40, 64), F32, 1), normal((48, 64), F32, 2), vector(48, F32, 3)
    dout = normal((40, 48), F32, 4)
    x, w, b = (t.clone().requires_grad_() for t in (x, w, b))
    Linear.apply(x, w, b).backward(dout)
    with torch.no_grad():
        z = layers.linear(x, w.t(), b)
        want = layers.linear_backward(dout, x, w.t(), z, "gelu")
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1].t()) and torch.equal(b.grad, want[2])


def test_per_thread_default_streams_have_their_own_workspaces():
    # one handle, a stream a thread: operands split into the workspace and pieces' sums of two
    # threads at a time, in products and in the GEMM.  Exact sums.
    import ctypes
    import threading

    from test_layers_host import structures
    per_thread = 2  # the handle of the per-thread default stream
    kind = type("args", (ctypes.Structure,), {"_fields_": structures()["phobos_linear_args_t"]})
    linear = phobos.library().phobos_linear
    shapes = [(300, 600, 1024), (40, 520, 4096), (260, 1300, 512), (130, 264, 2080)]
    work = []
    for i, (M, N, K) in enumerate(shapes):
        x, w = small_integers(M, K, F32, 2 * i), small_integers(K, N, F32, 2 * i + 1)
        work.append((x, w, torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda"), x @ w))
    torch.cuda.synchronize()
    wrong, ready = [], threading.Barrier(len(shapes))

    def thread(x, w, out, c, want):
        try:
            (M, K), N = x.shape, w.shape[1]
            args = kind(M=M, N=N, K=K, products=2, x=x.data_ptr(), x_row=K, x_col=1, w=w.data_ptr(), w_row=N, w_col=1,
                        out=out.data_ptr(), out_row=N)
            ready.wait()
            for _ in range(20):
                for _ in range(10):
                    st = linear(ctypes.c_char_p(bytes(args)), ctypes.c_void_p(per_thread))
                    st = st or phobos.phobos_sgemm_ex(M, N, K, 1.0, x.data_ptr(), K, w.data_ptr(), N, 0.0, c.data_ptr(), N,
                                                      per_thread, phobos.PHOBOS_MATH_3XTF32)
                st = st or phobos.phobos_check_device(per_thread)  # waits for this thread's stream
                if st or not torch.equal(out.cpu(), want.cpu()) or not torch.equal(c.cpu(), want.cpu()):
                    wrong.append((tuple(x.shape), st))
        except BaseException as e:  # noqa: B902
            wrong.append(e)

    threads = [threading.Thread(target=thread, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert phobos.phobos_release() == phobos.PHOBOS_OK
