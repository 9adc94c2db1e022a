"""Layer norm and RMS norm, forward and backward, against the formulas in
float64.

Tolerances.  A float32 result carries the rounding of its own few operations
(half a step is 2^-24 relative) and of the sums behind it: a row sum of K
terms in lanes of at most 32 terms followed by a tree of at most 9 levels and
8 waves stays under 64 half steps of the sum of magnitudes, a column sum over
at most 64 rows a block under 64 more.  128 * 2^-24 of the largest value
bounds them with the mean's and rstd's own errors; bf16 results add half a
bf16 step (2^-8 as torch.finfo(bfloat16).eps / 2, relative) of the value."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")
F32_TOL = 128 * 2.0 ** -24


def ref_forward(x, gamma, beta, kind, eps):
    x = x.double()
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=torch.float64)
    var = (x - mean[:, None]).square().mean(1)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * (1.0 if gamma is None else gamma.double())
    if kind == "layer" and beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def ref_backward(x, dys, gamma, stats, kind):
    x, dy = x.double(), sum(d.double() for d in dys)
    mean, rstd = stats.double().unbind(1)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma.double()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd[:, None], (dy * xh).sum(0), dy.sum(0), (dy * xh).abs().sum(0), dy.abs().sum(0)


def close(got, ref, dtype, scale=None):
    """Within F32_TOL of `scale` (the largest value unless given), and half a
    bf16 step of the value itself where the result is bf16."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape
    scale = ref.abs().max() if scale is None else scale
    tol = F32_TOL * scale + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0.0)
    bad = (got - ref).abs() > tol + 1e-30
    assert not bad.any(), ((got - ref).abs() / (tol + 1e-30)).max().item()


def data(rows, dim, n, dtype, seed=0):
    g = torch.Generator().manual_seed(1000 * rows + dim + seed)
    x = torch.randn(rows, dim, generator=g) * torch.exp(torch.randn(rows, 1, generator=g)) + 0.5
    dys = [torch.randn(rows, dim, generator=g) for _ in range(n)]
    return (x.to(dtype), [d.to(dtype) for d in dys], 1 + 0.3 * torch.randn(dim, generator=g),
            0.2 * torch.randn(dim, generator=g))


def test_formula_against_differences():
    """The reference's dx, dgamma and dbeta against central differences."""
    for kind in ("layer", "rms"):
        x, (dy,), gamma, beta = data(3, 7, 1, torch.float64)
        gamma, beta = gamma.double(), beta.double()
        _, mean, rstd = ref_forward(x, gamma, beta, kind, 1e-5)
        dx, dg, db, _, _ = ref_backward(x, [dy], gamma, torch.stack([mean, rstd], 1), kind)
        f = lambda x, g, b: float((ref_forward(x, g, b, kind, 1e-5)[0] * dy).sum())
        h = 1e-6
        for t, grad in ((x, dx), (gamma, dg), (beta, db)):
            if t is beta and kind == "rms":
                continue
            flat, gf = t.view(-1), grad.reshape(-1)
            for i in range(flat.numel()):
                keep = flat[i].item()
                flat[i] = keep + h
                up = f(x, gamma, beta)
                flat[i] = keep - h
                down = f(x, gamma, beta)
                flat[i] = keep
                # the difference's own error: h^2 of the third derivative, 1e-16 / h of rounding
                assert abs((up - down) / (2 * h) - gf[i].item()) < 1e-7 * (1 + gf.abs().max().item())


# Every kernel shape's edge (widths it just holds and the next ones), odd
# widths, one row to more rows than the blocks of a grid.
SHAPES = [(1, 1), (1, 64), (3, 65), (37, 128), (1, 257), (1025, 60), (5, 1024), (33, 1028), (9, 1536),
          (130, 2048), (70, 2560), (65, 2561), (2, 4096), (3, 5120), (4, 8192), (2, 10240), (2, 16384),
          (3, 16383), (2100, 132)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward_and_backward(rows, dim, kind, dtype):
    n = 1 + (rows + dim) % 4
    x, dys, gamma, beta = data(rows, dim, n, dtype)
    xd, dyd, gd, bd = x.to(DEV), [d.to(DEV) for d in dys], gamma.to(DEV), beta.to(DEV)
    nm = L.make_norm(kind, rows, dim, dtype, 1e-5, gd, bd)
    y, stats = torch.empty_like(xd), torch.empty(rows, 2, device=DEV)
    L.lora_norm_forward(nm, xd, y, stats)
    ry, mean, rstd = ref_forward(x, gamma, beta, kind, 1e-5)
    close(y, ry, dtype)
    close(stats[:, 0], mean, torch.float32, x.double().abs().max())
    close(stats[:, 1] / rstd.float().to(DEV), torch.ones(rows), torch.float32)
    layer = kind == "layer"
    dx, dg = torch.empty_like(xd), torch.full((dim,), 7.0, device=DEV)
    db = torch.full((dim,), 5.0, device=DEV) if layer else None
    L.lora_norm_backward(nm, xd, dyd, stats, dx, dg, db)
    rdx, rdg, rdb, adg, adb = ref_backward(x, dys, gamma, stats.cpu(), kind)
    close(dx, rdx, dtype, max(rdx.abs().max(), (n * rstd.max() * gamma.abs().max())))
    close(dg, rdg, torch.float32, adg.max())
    if layer:
        close(db, rdb, torch.float32, adb.max())
    # accumulation, and the gradients without dX
    L.lora_norm_backward(nm, xd, dyd, stats, None, dg, db, accumulate=True)
    close(dg, 2 * rdg, torch.float32, 2 * adg.max())
    if layer:
        close(db, 2 * rdb, torch.float32, 2 * adb.max())
    # dX alone needs no workspace and is the same
    alone = torch.empty_like(xd)
    L.lora_norm_backward(nm, xd, dyd, stats, alone)
    assert torch.equal(alone, dx)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,ld", [(0, 96), (4, 100), (1, 97)])
def test_column_slices_and_no_vectors(off, ld, dtype):
    """Rows inside a wider matrix, aligned and not, without gamma and beta;
    nothing outside the slice is written."""
    rows, dim = 11, 88
    x, dys, _, _ = data(rows, dim, 2, dtype)
    wide = lambda t: torch.full((rows, ld), 9.0, dtype=dtype, device=DEV)[:, off:off + dim].copy_(t)
    xs, ds = wide(x), [wide(d) for d in dys]
    nm = L.make_norm("layer", rows, dim, dtype, 1e-5, ldx=ld, ldy=ld)
    full = torch.full((rows, ld), 9.0, dtype=dtype, device=DEV)
    y, stats = full[:, off:off + dim], torch.empty(rows, 2, device=DEV)
    L.lora_norm_forward(nm, xs, y, stats)
    ry, mean, rstd = ref_forward(x, None, None, "layer", 1e-5)
    close(y, ry, dtype)
    full2 = torch.full((rows, ld), 9.0, dtype=dtype, device=DEV)
    L.lora_norm_backward(nm, xs, ds, stats, full2[:, off:off + dim])
    rdx = ref_backward(x, dys, None, stats.cpu(), "layer")[0]
    close(full2[:, off:off + dim], rdx, dtype, max(rdx.abs().max(), 2 * rstd.max()))
    for f in (full, full2):
        edge = torch.cat([f[:, :off].reshape(-1), f[:, off + dim:].reshape(-1)])
        assert (edge == 9.0).all()


@gpu
def test_forward_in_place_and_inference():
    x, _, gamma, _ = data(300, 2560, 1, torch.float32)
    xd, gd = x.to(DEV), gamma.to(DEV)
    nm = L.make_norm("rms", 300, 2560, torch.float32, 1e-6, gd)
    y = torch.empty_like(xd)
    L.lora_norm_forward(nm, xd, y)
    L.lora_norm_forward(nm, xd, xd)
    assert torch.equal(xd, y)


@gpu
def test_edge_rows():
    """A constant row (variance 0), a zero row, a row of huge values, and rows
    with NaN or infinity, which stay in their own rows."""
    dim = 260
    x = torch.randn(6, dim, generator=torch.Generator().manual_seed(1))
    x[0] = 3.0
    x[1] = 0.0
    x[2] *= 1e15
    x[3, 7] = float("nan")
    x[4, 5] = float("inf")
    for kind in ("layer", "rms"):
        nm = L.make_norm(kind, 6, dim, torch.float32, 1e-5)
        y, st = torch.empty(6, dim, device=DEV), torch.empty(6, 2, device=DEV)
        L.lora_norm_forward(nm, x.to(DEV), y, st)
        ry, _, _ = ref_forward(x, None, None, kind, 1e-5)
        for r in (0, 1, 2, 5):
            close(y[r:r + 1], ry[r:r + 1], torch.float32, max(1.0, ry[r].abs().max()))
        assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
        assert torch.isfinite(y[5]).all()
        dy = torch.ones(6, dim, device=DEV)
        dx = torch.empty(6, dim, device=DEV)
        L.lora_norm_backward(nm, x.to(DEV), [dy], st, dx)
        assert torch.isfinite(dx[[0, 1, 5]]).all() and torch.isnan(dx[3]).all()


@gpu
def test_streams_and_repeats():
    """The same bits on a side stream and on every repeat."""
    x, dys, gamma, beta = data(777, 2560, 3, torch.float32)
    xd, dyd, gd, bd = x.to(DEV), [d.to(DEV) for d in dys], gamma.to(DEV), beta.to(DEV)
    nm = L.make_norm("layer", 777, 2560, torch.float32, 1e-5, gd, bd)
    outs = []
    side = torch.cuda.Stream()
    for st in (None, side, None):
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        y, stats = torch.empty_like(xd), torch.empty(777, 2, device=DEV)
        dx, dg, db = torch.empty_like(xd), torch.empty_like(gd), torch.empty_like(bd)
        ws = torch.empty(L.lora_norm_workspace_bytes(nm), device=DEV, dtype=torch.uint8)
        L.lora_norm_forward(nm, xd, y, stats, stream=st)
        L.lora_norm_backward(nm, xd, dyd, stats, dx, dg, db, ws=ws, stream=st)
        torch.cuda.synchronize()
        outs.append((y, stats, dx, dg, db))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@gpu
def test_captured_in_a_graph():
    """Forward and backward in a HIP graph, replayed on changing inputs with
    eager work between the replays."""
    rows, dim = 515, 2048
    x, dys, gamma, beta = data(rows, dim, 2, torch.float32)
    xd, dyd, gd, bd = x.to(DEV), [d.to(DEV) for d in dys], gamma.to(DEV), beta.to(DEV)
    nm = L.make_norm("layer", rows, dim, torch.float32, 1e-5, gd, bd)
    y, stats = torch.empty_like(xd), torch.empty(rows, 2, device=DEV)
    dx, dg, db = torch.empty_like(xd), torch.empty_like(gd), torch.empty_like(bd)
    ws = torch.empty(L.lora_norm_workspace_bytes(nm), device=DEV, dtype=torch.uint8)

    def work():
        L.lora_norm_forward(nm, xd, y, stats)
        L.lora_norm_backward(nm, xd, dyd, stats, dx, dg, db, ws=ws)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for k in range(4):
        xd.copy_(x.to(DEV) * (k + 1) + 0.1 * k)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, stats, dx, dg, db)]
        for t in (y, stats, dx, dg, db):
            t.fill_(float("nan"))
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, stats, dx, dg, db)))


# ---------------------------------------------------------------- refusals
def _norm(**kw):
    d = dict(rows=4, dim=8, ldx=8, ldy=8, kind=0, dtype=0, gamma=256, beta=256, eps=1e-5)
    d.update(kw)
    return L.LoraNorm(**d)


@no_device
@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), -2), (dict(dim=0), -2), (dict(dim=16388, ldx=16388, ldy=16388), -2),
    (dict(ldx=7), -2), (dict(ldy=7), -2), (dict(kind=2), -1), (dict(dtype=2), -3),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(eps=math.inf), -1), (dict(gamma=258), -4),
    (dict(beta=257), -4),
])
def test_invalid_descriptors_are_refused(kw, status):
    nm = _norm(**kw)
    lib = L.lib()
    assert lib.lora_norm_forward(C.byref(nm), 256, 256, 256, None) == status
    assert lib.lora_norm_workspace_bytes(C.byref(nm)) == 0
    dy = (C.c_void_p * 1)(256)
    assert lib.lora_norm_backward(C.byref(nm), 256, 1, dy, 256, 256, 256, 256, 0, 256, 1 << 20,
                                  None) == status


@no_device
def test_invalid_arguments_are_refused():
    lib, nm = L.lib(), _norm()
    fwd = lambda *a: lib.lora_norm_forward(C.byref(nm), *a, None)
    assert fwd(None, 256, 256) == -1 and fwd(256, None, 256) == -1
    assert fwd(258, 256, 256) == -4 and fwd(256, 257, 256) == -4 and fwd(256, 256, 260) == -4
    assert lib.lora_norm_forward(None, 256, 256, 256, None) == -1
    dy = (C.c_void_p * 4)(256, 256, 256, 256)

    def bwd(n=1, X=256, dys=dy, stats=256, dX=256, dg=256, db=256, ws=256, size=1 << 20, d=nm):
        return lib.lora_norm_backward(C.byref(d), X, n, dys, stats, dX, dg, db, 0, ws, size, None)

    assert bwd(n=0) == -1 and bwd(n=5) == -1 and bwd(X=None) == -1 and bwd(stats=None) == -1
    assert bwd(dys=None) == -1 and bwd(n=2, dys=(C.c_void_p * 2)(256, None)) == -1
    assert bwd(dX=None, dg=None, db=None) == -1
    assert bwd(d=_norm(kind=1)) == -1          # dbeta of an RMS norm
    assert bwd(dX=258) == -4 and bwd(dg=258) == -4 and bwd(stats=260) == -4
    assert bwd(n=2, dys=(C.c_void_p * 2)(256, 257)) == -4
    big = _norm(rows=4096, dim=2560, ldx=2560, ldy=2560)
    need = lib.lora_norm_workspace_bytes(C.byref(big))
    assert need > 0 and need % (2 * 2560 * 4) == 0
    assert bwd(d=big, size=need - 1) == -5 and bwd(d=big, ws=None, size=need) == -5
    assert bwd(d=big, ws=264, size=need) == -5


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError, match="kind"):
        L.make_norm("batch", 4, 8)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        L.make_norm("rms", 4, 8, torch.float16)
    nm = L.make_norm("rms", 4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        L.lora_norm_forward(nm, torch.zeros(4, 8), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="1 to 4"):
        L.lora_norm_backward(nm, torch.zeros(4, 8), [], torch.zeros(4, 2))


@gpu
def test_binding_checks_shapes_and_strides():
    nm = L.make_norm("rms", 4, 8)
    x = torch.zeros(4, 8, device=DEV)
    for bad in (torch.zeros(4, 9, device=DEV), torch.zeros(8, 4, device=DEV).t(),
                torch.zeros(4, 16, device=DEV)[:, :8]):
        with pytest.raises(ValueError):
            L.lora_norm_forward(nm, bad, x.clone())
    with pytest.raises(TypeError):
        L.lora_norm_forward(nm, x.bfloat16(), x.clone())
    with pytest.raises(ValueError, match="stats"):
        L.lora_norm_forward(nm, x, x.clone(), torch.zeros(7, device=DEV))
