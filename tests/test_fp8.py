"""8-bit block-scaled products and the rounding of their activations, against
their definition in float64.

Tolerances.  The rounding is exact arithmetic and is compared for equality.
Products of small whole numbers, with power-of-two scales, are exact in every
step (each block's 128 products need under 12 bits), so the layout tests ask
for equality too.  With general data the matrix instruction drops what lies
about 2^-14 below a block's largest product, 128 times at random; 2^-12 of the
sum of the products' magnitudes covers it with the float32 sum over the
blocks, and a bf16 result adds half its step, 2^-8 of the value."""

import ctypes as C

import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")


def up(n, m=128):
    return -(-n // m) * m


def ref_round(x):
    """(values, exponents, values * scale) of x by the definition."""
    x = x.double()
    t, k = x.shape
    b = torch.zeros(t, up(k), dtype=torch.float64)
    b[:, :k] = x
    b = b.view(t, -1, 128)
    top = b.abs().amax(2)
    e = torch.full(top.shape, -127.0, dtype=torch.float64)
    pos = top > 0
    guess = torch.ceil(torch.log2(torch.where(pos, top, torch.ones_like(top)) / 448))
    for d in (-1, 0, 1):   # the smallest power that holds the block
        fits = pos & (top <= 448 * torch.exp2(guess + d)) & ~(top <= 448 * torch.exp2(guess + d - 1))
        e = torch.where(fits, guess + d, e)
    e = e.clamp(-127, 127)
    v = b / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    q = torch.round(v / step) * step
    return q.view(t, -1), e, (q * torch.exp2(e)[..., None]).view(t, -1)[:, :k]


def unpack(rows):
    """(values, exponents) of an Fp8Rows."""
    _, off = L.lora_fp8_operand_layout(rows.rows, rows.cols)
    buf, w = rows.buf.cpu(), up(rows.cols)
    q = buf[:rows.rows * w].view(torch.float8_e4m3fn).double().view(rows.rows, w)
    e = buf[off:off + up(rows.rows) * (w // 128)].view(w // 128, up(rows.rows))
    t = torch.arange(rows.rows)
    return q, e[:, t - t % 128 + 8 * (t % 16) + (t // 16) % 8].t().double() - 127


QSHAPES = [(1, 1), (1, 128), (3, 129), (17, 64), (130, 300), (128, 256), (257, 1000), (5, 2560), (2, 9728)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantize_is_the_definition(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, cols, generator=g))
    x[rows // 2] *= 1e-30
    x[0, cols // 2] = 448.0
    x = x.to(dtype)
    wide = torch.full((rows, cols + 3), 5.0, dtype=dtype, device=DEV)
    wide[:, 1:cols + 1] = x.to(DEV)
    for src in (x.to(DEV), wide[:, 1:cols + 1]):   # aligned rows, and odd strides
        out = L.fp8_rows(rows, cols)
        out.buf.fill_(255)
        L.lora_fp8_quantize(src, out)
        q, e = unpack(out)
        rq, re, _ = ref_round(x)
        assert torch.equal(e, re) and torch.equal(q, rq)


@gpu
def test_quantize_edges():
    """Borders of the scale, ties, subnormals, zeros; NaN and infinity in
    their own block only."""
    x = torch.zeros(6, 384)
    x[0, :3] = torch.tensor([448.0, 449.0, -447.0])
    x[0, 128:130] = torch.tensor([0.4375, 0.21875])        # 448 2^-10 exactly
    x[1, :4] = torch.tensor([1e-40, -3e-39, 0.0, 1e-45])
    x[1, 130] = 3.4e38
    x[2, :8] = torch.tensor([17.0, 19.0, 21.0, 23.0, -17.0, 33.0, 35.0, 448.0])   # ties at 16 steps
    x[3, 5], x[3, 6] = float("nan"), 1.0
    x[4, 200], x[4, 201] = float("-inf"), 2.0
    out = L.fp8_rows(6, 384)
    L.lora_fp8_quantize(x.to(DEV), out)
    q, e = unpack(out)
    ok = torch.ones(6, 3, dtype=torch.bool)
    ok[3, 0] = ok[4, 1] = False
    rq, re, _ = ref_round(torch.nan_to_num(x, posinf=0, neginf=0, nan=0))
    assert torch.equal(e[ok], re[ok])
    okc = ok.repeat_interleave(128, 1)
    assert torch.equal(q[okc], rq[okc])
    assert torch.isnan(q[3, 5]) and not torch.isnan(q[3, 6]) and torch.isnan(q[4, 200])


def weight(N, K, seed, whole):
    """(Fp8Weight, float64 values)"""
    g = torch.Generator().manual_seed(seed)
    nb, kb = up(N) // 128, up(K) // 128
    if whole:
        v = torch.randint(-3, 4, (N, K), generator=g).float()
        s = torch.exp2(torch.randint(-3, 3, (nb, kb), generator=g).float())
    else:
        v = torch.randn(N, K, generator=g) * 100
        s = 1e-3 * torch.rand(nb, kb, generator=g) + 1e-4
    q = v.clamp(-448, 448).to(torch.float8_e4m3fn)
    w = q.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return L.fp8_pack(q.to(DEV), s.to(DEV)), w


# Tokens, inputs, outputs: every tile size, splits of the contraction, ragged
# in each direction.
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 2560, 4096), (7, 300, 40), (17, 9728, 260), (32, 260, 520), (33, 640, 264), (40, 4096, 130),
          (128, 1024, 1024), (129, 1000, 257), (200, 136, 2000), (1000, 2056, 1368), (255, 384, 512),
          (600, 256, 1100), (2048, 640, 2560), (2100, 200, 2600), (4096, 128, 4200),
          # whole rounds of the largest tile, then the other columns
          (4096, 2560, 4360), (3000, 2056, 6000)]


@gpu
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_product_of_whole_numbers_is_exact(T, K, N, dx):
    W, w = weight(N, K, T + K, True)
    g = torch.Generator().manual_seed(T)
    x = torch.randint(-3, 4, (T, N if dx else K), generator=g).float()
    x[:, 0] = 3.0
    x = x * torch.exp2(torch.randint(-2, 2, (T, 1), generator=g).float())
    # the reference product in float64 on the GPU (whole numbers: exact)
    wd = w.to(DEV) if dx else w.t().contiguous().to(DEV)
    ref = x.double().to(DEV) @ wd
    q = L.fp8_rows(*x.shape)
    L.lora_fp8_quantize(x.to(DEV), q)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((T * (K if dx else N) + 64,), 7.0, device=DEV, dtype=dt)
        y = out[:T * (K if dx else N)].view(T, -1)
        L.lora_fp8_product(q, W, y, dx=dx)
        assert torch.equal(y, ref.to(dt))
        assert (out[T * (K if dx else N):] == 7.0).all()


@gpu
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("T,K,N", [(1, 2560, 1024), (50, 1000, 700), (300, 2560, 1024), (2048, 1280, 2560)])
def test_product_of_general_data(T, K, N, dx):
    W, w = weight(N, K, 5, False)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, N if dx else K, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    x = x * torch.exp(0.7 * torch.randn(x.shape[1], generator=g))
    xr = ref_round(x)[2].to(DEV)
    wd = w.to(DEV) if dx else w.t().contiguous().to(DEV)
    ref, mag = xr @ wd, xr.abs() @ wd.abs()
    q = L.fp8_rows(*x.shape)
    L.lora_fp8_quantize(x.to(DEV), q)
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty(T, K if dx else N, device=DEV, dtype=dt)
        L.lora_fp8_product(q, W, y, dx=dx)
        tol = 2.0 ** -12 * mag + (2.0 ** -8 * ref.abs() if dt == torch.bfloat16 else 0)
        assert ((y.double() - ref).abs() <= tol).all()


@gpu
def test_non_finite_rows_stay_rows():
    """A NaN in X reaches its own row of Y; a NaN in one row of W its own
    column (one row of the contraction in dX: everything)."""
    T, K, N = 130, 512, 300
    W, w = weight(N, K, 5, True)
    x = torch.ones(T, K)
    x[77, 300] = float("nan")
    q = L.fp8_rows(T, K)
    L.lora_fp8_quantize(x.to(DEV), q)
    y = torch.empty(T, N, device=DEV)
    L.lora_fp8_product(q, W, y)
    bad = torch.isnan(y).cpu()
    assert bad[77].all() and bad.sum() == N
    W.buf[up(K) * 5 + 9] = 0x7f
    q2 = L.fp8_rows(T, K)
    L.lora_fp8_quantize(torch.ones(T, K, device=DEV), q2)
    L.lora_fp8_product(q2, W, y)
    bad = torch.isnan(y).cpu()
    assert bad[:, 5].all() and bad.sum() == T


@gpu
@pytest.mark.parametrize("dx", [False, True])
def test_repeats_streams_and_graph(dx):
    for T, K, N in ((1, 2560, 1024), (300, 1024, 2560)):
        W, _ = weight(N, K, 5, False)
        x = torch.randn(T, N if dx else K, device=DEV)
        q, y = L.fp8_rows(*x.shape), torch.empty(T, K if dx else N, device=DEV, dtype=torch.bfloat16)
        need = L.lora_fp8_product_workspace_bytes(q, W, dx)
        ws = torch.empty(max(16, need), device=DEV, dtype=torch.uint8)

        def work(st=None):
            L.lora_fp8_quantize(x, q, stream=st)
            L.lora_fp8_product(q, W, y, dx=dx, ws=ws, stream=st)

        work()
        torch.cuda.synchronize()
        first = y.clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        work(side)
        torch.cuda.synchronize()
        assert torch.equal(first, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        for k in range(4):
            x.normal_()
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone()
            y.fill_(0)
            ws.fill_(255)
            work()
            torch.cuda.synchronize()
            assert torch.equal(got, y)


# ---------------------------------------------------------------- refusals
@no_device
def test_layouts():
    assert L.lora_fp8_weight_layout(300, 200) == (384 * 256 + 3 * 2 * 4, 384 * 256)
    assert L.lora_fp8_operand_layout(3, 130) == (768 + 256, 768)
    for bad in ((0, 5), (5, 0), (1 << 20, 1 << 20)):
        with pytest.raises(ValueError, match="no 8-bit layout"):
            L.lora_fp8_weight_layout(*bad)
    with pytest.raises(ValueError, match="no 8-bit layout"):
        L.lora_fp8_operand_layout(1, (1 << 22) + 1)


@no_device
def test_invalid_arguments_are_refused():
    lib = L.lib()
    op = lambda rows=4, cols=256, data=256: C.byref(L.LoraFp8Operand(rows, cols, data))
    quant = lambda o, X=256, dt=0, ld=256: lib.lora_fp8_quantize(X, dt, ld, o, None)
    assert quant(None) == -1 and quant(op(), X=None) == -1 and quant(op(data=None)) == -1
    assert quant(op(rows=0)) == -2 and quant(op(cols=-1)) == -2 and quant(op(), ld=255) == -2
    assert quant(op(), dt=2) == -3 and quant(op(data=264)) == -4 and quant(op(), X=258) == -4

    def prod(o, W=256, n=384, k=256, dx=0, out=256, dt=0, ws=256, size=1 << 40):
        return lib.lora_fp8_product(o, W, n, k, dx, out, dt, ws, size, None)

    assert prod(None) == -1 and prod(op(), W=None) == -1 and prod(op(), out=None) == -1
    assert prod(op(data=None)) == -1
    assert prod(op(cols=255)) == -2 and prod(op(), dx=1) == -2 and prod(op(), n=0) == -2
    assert prod(op(cols=1 << 20), n=1 << 20, k=1 << 20) == -2
    assert prod(op(), dt=3) == -3
    assert prod(op(), W=264) == -4 and prod(op(), out=8) == -4 and prod(op(data=8)) == -4
    big = lambda: op(rows=64, cols=9728)
    need = lib.lora_fp8_product_workspace_bytes(big(), 256, 9728, 0)
    assert need > 0
    assert prod(big(), n=256, k=9728, size=need - 1) == -5
    assert prod(big(), n=256, k=9728, ws=None) == -5


def test_binding_refuses_wrong_tensors():
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        L.fp8_pack(torch.zeros(4, 4), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="scales"):
        L.fp8_pack(torch.zeros(4, 4).to(torch.float8_e4m3fn), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        L.Fp8Weight(4, 4, torch.zeros(1 << 20, dtype=torch.uint8))


@gpu
def test_binding_checks_shapes():
    W, _ = weight(300, 200, 1, True)
    q = L.fp8_rows(4, 200)
    with pytest.raises(ValueError, match="columns"):
        L.lora_fp8_product(q, W, torch.empty(4, 200, device=DEV), dx=True)
    with pytest.raises(ValueError, match="the call reads or writes"):
        L.lora_fp8_product(q, W, torch.empty(4, 299, device=DEV))
    with pytest.raises(TypeError):
        L.lora_fp8_product(q, W, torch.empty(4, 300, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="an 8-bit W"):
        L.Fp8Weight(300, 200, torch.zeros(100, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="must be"):
        L.lora_fp8_quantize(torch.zeros(4, 201, device=DEV), q)
