"""Newton-Schulz orthogonalisation and the update built on it, against the
iteration as defined (on the matrix itself) in float64.

Tolerances.  lora_orthogonalize sums in float64 and rounds once: half a
float32 step (2^-24) of the value, plus 1e-8 of the largest for the float64
work itself (its 1e-16 errors of G, magnified by at most a^steps / the
smallest singular value that the iteration has not yet lifted).  In
lora_muon_step u carries up to three float32 roundings, 3 * 2^-24 relative to
|g'| + momentum |m|, and the map u / ||u|| -> orth(u) has slope at most
a^steps = 485: 485 * 3 * 2^-24 < 9e-5 of a unit matrix's scale, times rate,
and 2 steps of the parameter's own rounding."""

import ctypes as C
import math

import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")
NS = (3.4445, -4.7750, 2.0315)


def orth(u, steps=5, eps=1e-7, coeffs=NS):
    x = u.double()
    if x.shape[0] > x.shape[1]:
        x = x.t()
    a, b, c = coeffs
    n = x.norm() + eps
    x = x / n if n > 0 else x
    for _ in range(steps):
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x if u.shape[0] <= u.shape[1] else x.t()


def close_orth(got, ref):
    got = got.cpu().double()
    tol = 2.0 ** -24 * ref.abs() + 1e-8 * ref.abs().max()
    assert ((got - ref).abs() <= tol + 1e-30).all(), (got - ref).abs().max().item()


def matrix(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    r = min(rows, cols)
    k = max(1, r // 4)
    low = torch.randn(rows, k, generator=g) @ torch.randn(k, cols, generator=g)
    return 1e-3 * (low + 0.3 * torch.randn(rows, cols, generator=g))


def test_reference_against_singular_values():
    """The iteration maps each singular value by the quintic alone."""
    u = matrix(6, 40, 3).double()
    U, s, V = torch.linalg.svd(u, full_matrices=False)
    s = s / (u.norm() + 1e-7)
    for _ in range(5):
        s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
    assert torch.allclose(U @ torch.diag(s) @ V, orth(u), rtol=0, atol=1e-12)
    assert torch.allclose(orth(u.t()), orth(u).t(), rtol=0, atol=1e-12)


SHAPES = [(1, 1), (1, 300), (300, 1), (3, 5), (5, 3), (4, 64), (64, 4), (8, 2048), (2048, 8), (16, 16),
          (17, 257), (257, 17), (30, 1001), (1001, 30), (32, 520), (64, 2560), (2560, 64), (61, 999),
          (999, 61), (64, 64), (65, 260), (260, 65), (128, 128), (128, 1000), (1000, 128), (127, 771),
          (771, 127)]


@gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols):
    u = matrix(rows, cols, 7 * rows + cols)
    out = torch.full((rows, cols), 9.0, device=DEV)
    L.lora_orthogonalize(u.to(DEV), out, [L.make_matrix_run(0, rows, cols)], L.make_muon(0.1))
    close_orth(out, orth(u))


@gpu
@pytest.mark.parametrize("steps", [1, 2, 7, 10])
def test_orthogonalize_steps_and_coefficients(steps):
    coeffs = (2.0, -1.5, 0.5)
    for rows, cols in ((20, 300), (300, 20), (100, 110)):
        u = matrix(rows, cols, steps)
        out = torch.empty(rows, cols, device=DEV)
        L.lora_orthogonalize(u.to(DEV), out, [L.make_matrix_run(0, rows, cols)],
                             L.make_muon(0.1, coeffs=coeffs, steps=steps, eps=1e-3))
        close_orth(out, orth(u, steps, 1e-3, coeffs))


@gpu
@pytest.mark.parametrize("rows,cols", [(64, 1000), (1000, 64)])
def test_wide_spectrum_keeps_its_small_directions(rows, cols):
    """Singular values over five orders of magnitude: the sums of G in float64
    keep the smallest directions to float32's own accuracy."""
    g = torch.Generator().manual_seed(11)
    r, side = min(rows, cols), max(rows, cols)
    U = torch.linalg.qr(torch.randn(r, r, generator=g, dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(side, r, generator=g, dtype=torch.float64))[0]
    u = (U @ torch.diag(torch.logspace(0, -5, r, dtype=torch.float64)) @ V.t()).float()
    u = u if rows <= cols else u.t().contiguous()
    out = torch.empty(rows, cols, device=DEV)
    L.lora_orthogonalize(u.to(DEV), out, [L.make_matrix_run(0, rows, cols)], L.make_muon(0.1))
    close_orth(out, orth(u))


@gpu
def test_batches_strides_and_mixed_runs():
    """Runs of every padded short side in one call, with gaps between the
    matrices; the gaps keep their values."""
    runs, end = [], 3
    for i, (rows, cols, count, gap) in enumerate([(8, 96, 5, 32), (96, 8, 5, 0), (20, 70, 2, 5),
                                                  (64, 300, 3, 4), (300, 64, 2, 1), (100, 200, 2, 7),
                                                  (1, 9, 4, 2)]):
        runs.append(L.make_matrix_run(end, rows, cols, count, rows * cols + gap))
        end += count * (rows * cols + gap) + 2
    src = torch.randn(end, generator=torch.Generator().manual_seed(1))
    out = torch.full((end,), 9.0, device=DEV)
    L.lora_orthogonalize(src.to(DEV), out, runs, L.make_muon(0.1))
    res, used = out.cpu(), torch.zeros(end, dtype=torch.bool)
    for r in runs:
        for k in range(r.count):
            o = r.offset + k * r.stride
            sl = slice(o, o + r.rows * r.cols)
            used[sl] = True
            close_orth(res[sl].view(r.rows, r.cols), orth(src[sl].view(r.rows, r.cols)))
    assert (res[~used] == 9.0).all()


@gpu
def test_zero_matrices():
    """A zero gradient (A's at the first step, where B is zero) gives a zero
    update, with and without eps."""
    for eps in (1e-7, 0.0):
        g = torch.zeros(2, 8, 64)
        g[1] = matrix(8, 64, 5)
        out = torch.full((2, 8, 64), 9.0, device=DEV)
        L.lora_orthogonalize(g.to(DEV), out, [L.make_matrix_run(0, 8, 64, 2)],
                             L.make_muon(0.1, eps=eps))
        assert (out[0] == 0).all()
        close_orth(out[1], orth(g[1], eps=eps))


@gpu
def test_non_finite_matrix_stays_alone():
    g = torch.stack([matrix(8, 64, i) for i in range(3)])
    g[1, 3, 5] = float("nan")
    out = torch.empty(3, 8, 64, device=DEV)
    L.lora_orthogonalize(g.to(DEV), out, [L.make_matrix_run(0, 8, 64, 3)], L.make_muon(0.1))
    assert torch.isnan(out[1]).all()
    for i in (0, 2):
        close_orth(out[i], orth(g[i]))


def ref_step(p, g, m, sc, hp, rows, cols, kind):
    g = g.double() * sc
    m = hp.momentum * m.double() + g
    u = g + hp.momentum * m if hp.nesterov else m
    f = 0.2 * math.sqrt(max(rows, cols)) if hp.adjust else math.sqrt(max(1.0, rows / cols))
    rate = hp.lr * f * (hp.plus_ratio if kind == L.KIND_B else 1.0)
    decay = hp.lr * hp.weight_decay if kind == L.KIND_A else 0.0
    p = p.double()
    return p - rate * orth(u, hp.steps, hp.eps) - decay * p, m, rate


@gpu
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("adjust", ["shape", "rms"])
@pytest.mark.parametrize("rows,cols,kind", [(8, 2048, 0), (256, 8, 1), (64, 640, 0), (1001, 30, 1),
                                            (100, 300, 0), (500, 128, 1), (5, 7, 0)])
def test_muon_steps(rows, cols, kind, adjust, nesterov):
    """Three updates of two matrices from the same start, momentum carried."""
    g0 = torch.Generator().manual_seed(rows + cols)
    p = 0.02 * torch.randn(2, rows, cols, generator=g0)
    m = torch.zeros(2, rows, cols)
    hp = L.make_muon(0.02, 0.9, 0.1, 4.0, nesterov=nesterov, adjust=adjust)
    run = [L.make_matrix_run(0, rows, cols, 2, kind=kind)]
    pd, md = p.to(DEV), m.to(DEV)
    scale = torch.full((1,), 0.25, device=DEV)
    for k in range(3):
        g = torch.stack([matrix(rows, cols, 10 * k + i) for i in range(2)])
        pd0, md0 = pd.cpu(), md.cpu()
        L.lora_muon_step(pd, g.to(DEV), md, run, hp, scale)
        for i in range(2):
            rp, rm, rate = ref_step(pd0[i], g[i], md0[i], 0.25, hp, rows, cols, kind)
            tm = 2.0 ** -23 * (0.25 * g[i].double().abs() + md0[i].double().abs())
            assert ((md[i].cpu().double() - rm).abs() <= tm + 1e-30).all()
            tp = 9e-5 * rate + 2.0 ** -23 * (rp.abs() + pd0[i].double().abs())
            assert ((pd[i].cpu().double() - rp).abs() <= tp).all()


@gpu
def test_veto_changes_nothing():
    for bad in (float("nan"), float("inf"), float("-inf")):
        p, g, m = (torch.randn(100, 300, device=DEV) for _ in range(3))
        before = p.clone(), m.clone()
        L.lora_muon_step(p, g, m, [L.make_matrix_run(0, 100, 300)], L.make_muon(0.1),
                         torch.full((1,), bad, device=DEV))
        assert torch.equal(p, before[0]) and torch.equal(m, before[1])


@gpu
def test_repeats_streams_and_graph():
    """The same bits again, on a side stream, and from a graph replayed with
    eager work between the replays."""
    runs = [L.make_matrix_run(0, 64, 2560, 3), L.make_matrix_run(3 * 64 * 2560, 1024, 64, 2, kind=1)]
    n = 3 * 64 * 2560 + 2 * 1024 * 64
    g, hp = torch.randn(n, device=DEV), L.make_muon(0.02)
    scale = torch.ones(1, device=DEV)
    ws = torch.empty(L.lora_muon_workspace_bytes(runs), device=DEV, dtype=torch.uint8)
    p0, m0 = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    p, m = p0.clone(), m0.clone()
    L.lora_muon_step(p, g, m, runs, hp, scale, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ps, ms = p0.clone(), m0.clone()
    torch.cuda.synchronize()
    ws.fill_(255)
    side.wait_stream(torch.cuda.current_stream())
    L.lora_muon_step(ps, g, ms, runs, hp, scale, ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(p, ps) and torch.equal(m, ms)
    pg, mg = p0.clone(), m0.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        L.lora_muon_step(pg, g, mg, runs, hp, scale, ws)
    p, m = p0.clone(), m0.clone()
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        ws2 = torch.empty_like(ws)
        L.lora_muon_step(p, g, m, runs, hp, scale, ws2)
        torch.cuda.synchronize()
        assert torch.equal(pg, p) and torch.equal(mg, m)


# ---------------------------------------------------------------- refusals
def _call(runs, hp, **kw):
    d = dict(P=256, G=256, M=256, scale=256, ws=256, size=1 << 40)
    d.update(kw)
    arr = (L.LoraMatrixRun * max(1, len(runs)))(*runs)
    n = d.get("n", len(runs))
    h = C.byref(hp) if hp is not None else None
    step = L.lib().lora_muon_step(d["P"], d["G"], d["M"], arr, n, h, d["scale"], d["ws"], d["size"],
                                  None)
    return step


RUN = (0, 8, 64)


@no_device
@pytest.mark.parametrize("run,status", [
    ((0, 0, 64), -2), ((0, 8, -1), -2), ((0, 129, 200), -2), ((0, 8, (1 << 22) + 1), -2),
    ((0, 8, 64, 0), -2), ((0, 8, 64, 2, 511), -1), ((-1, 8, 64), -1), ((0, 8, 64, 1, None, 2), -1),
    ((0, 8, 64, 1 << 21), -2),
])
def test_invalid_runs_are_refused(run, status):
    r = L.make_matrix_run(*run)
    assert _call([r], L.make_muon(0.1)) == status
    assert _call([L.make_matrix_run(*RUN), r], L.make_muon(0.1)) == status
    arr = (L.LoraMatrixRun * 1)(r)
    assert L.lib().lora_muon_workspace_bytes(arr, 1) == 0
    assert L.lib().lora_orthogonalize(256, 512, arr, 1, C.byref(L.make_muon(0.1)), 256, 1 << 40,
                                      None) == status


@no_device
def test_invalid_hyper_parameters_and_buffers_are_refused():
    ok = [L.make_matrix_run(*RUN)]
    for kw in (dict(lr=math.nan), dict(lr=0.1, momentum=1.0), dict(lr=0.1, momentum=-0.1),
               dict(lr=0.1, eps=-1.0), dict(lr=0.1, steps=0), dict(lr=0.1, steps=11),
               dict(lr=0.1, weight_decay=math.inf), dict(lr=0.1, coeffs=(math.nan, 0, 0))):
        assert _call(ok, L.make_muon(**kw)) == -1
    bad = L.make_muon(0.1)
    bad.adjust = 2
    assert _call(ok, bad) == -1 and _call(ok, None) == -1
    hp = L.make_muon(0.1)
    assert _call([], hp) == -1 and _call(ok, hp, n=33) == -1
    for name in ("P", "G", "M"):
        assert _call(ok, hp, **{name: None}) == -1 and _call(ok, hp, **{name: 264}) == -4
    assert _call(ok, hp, scale=None) == -1 and _call(ok, hp, scale=258) == -4
    need = L.lora_muon_workspace_bytes(ok)
    assert need > 0
    assert _call(ok, hp, size=need - 1) == -5 and _call(ok, hp, ws=None) == -5
    assert _call(ok, hp, ws=264) == -4
    with pytest.raises(ValueError, match="adjust"):
        L.make_muon(0.1, adjust="none")


@gpu
def test_binding_checks_the_arena_length():
    t = torch.zeros(8 * 64, device=DEV)
    runs = [L.make_matrix_run(4, 8, 64)]
    with pytest.raises(ValueError, match="the call reads or writes"):
        L.lora_orthogonalize(t, torch.empty(8 * 64 + 4, device=DEV), runs, L.make_muon(0.1))
