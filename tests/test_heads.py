"""Norm and rotation of heads, forward and backward, against the formulas in
float64.

Tolerances.  A float32 result carries the roundings (2^-24 of the value each)
of about ten operations after the norm, of a sum of at most 256 squares in
lanes of eight and a tree, and of sine and cosine (two steps, 2^-22, and the
remainder's rounding, 2^-24 of pi): under 64 * 2^-24 of the pair's magnitudes.
dx's two sums over the head add as much again.  dgamma sums at most 64 terms a
lane and 64 more down its tree: 128 * 2^-24 of the sum of magnitudes.  bf16
results add half a bf16 step, 2^-8 of the value."""

import ctypes as C
import math

import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")
STEP = 2.0 ** -24


def pairs(rot, inter):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def turn(z, pos, freqs, inter, sign=1):
    """z [tokens, heads, dim] turned, and the magnitudes behind each value."""
    out, mag = z.clone(), z.abs()
    rot = 2 * freqs.numel()
    a, b = pairs(rot, inter)
    phi = pos.double()[:, None, None] * freqs
    co, si = torch.cos(phi), sign * torch.sin(phi)
    out[..., a] = z[..., a] * co - z[..., b] * si
    out[..., b] = z[..., b] * co + z[..., a] * si
    mag[..., a] = mag[..., b] = z[..., a].abs() + z[..., b].abs()
    return out, mag


def reference(x, dy, pos, gamma, freqs, inter, norm, eps):
    """y, dx, dgamma and the magnitudes that their errors scale with."""
    x, dy = x.double(), dy.double()
    dim = x.shape[-1]
    gamma = torch.ones(dim, dtype=torch.float64) if gamma is None else gamma.double()
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt() if norm else torch.ones_like(x[..., :1])
    xh = x * rstd
    y, ymag = turn(xh * gamma if norm else x, pos, freqs, inter)
    dz, zmag = turn(dy, pos, freqs, inter, -1)
    if not norm:
        return y, ymag, dz, zmag, None, None
    g = dz * gamma
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    gm = zmag * gamma.abs()
    dmag = 2 * rstd * (gm + xh.abs() * (gm * xh.abs()).mean(-1, keepdim=True))
    return y, ymag, dx, dmag, (dz * xh).sum((0, 1)), (zmag * xh.abs()).sum((0, 1))


def close(got, ref, mag, dtype, steps=64):
    tol = steps * STEP * mag + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0.0) + 1e-30
    err = (got.detach().cpu().double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()


def data(tokens, heads, dim, xt, yt, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * tokens + 131 * heads + dim)
    x = torch.randn(tokens, heads, dim, generator=g) * torch.exp(torch.randn(tokens, heads, 1, generator=g))
    dy = torch.randn(tokens, heads, dim, generator=g)
    return x.to(xt), dy.to(yt), 1 + 0.3 * torch.randn(dim, generator=g)


def test_formula_against_differences():
    x, dy, gamma = data(2, 2, 6, torch.float64, torch.float64)
    gamma = gamma.double()
    pos, freqs = torch.tensor([3, -5]), torch.tensor([0.7, 0.05], dtype=torch.float64)
    for inter in (False, True):
        ref = reference(x, dy, pos, gamma, freqs, inter, True, 1e-3)
        f = lambda: float((reference(x, dy, pos, gamma, freqs, inter, True, 1e-3)[0] * dy).sum())
        h = 1e-6
        for t, grad in ((x, ref[2]), (gamma, ref[4])):
            flat, gf = t.view(-1), grad.reshape(-1)
            for i in range(flat.numel()):
                keep = flat[i].item()
                flat[i] = keep + h
                up = f()
                flat[i] = keep - h
                down = f()
                flat[i] = keep
                # h^2 of the third derivative and 1e-16 / h of rounding
                assert abs((up - down) / (2 * h) - gf[i].item()) < 1e-7 * (1 + gf.abs().max().item())


# (tokens, heads of each set, head_dim, rot_dim, interleaved, norm)
CASES = [
    (1, (32, 8), 128, 128, False, True), (1, (1,), 64, 64, True, False), (37, (4, 2, 2), 64, 64, False, True),
    (5, (3,), 128, 64, False, True), (9, (12, 4), 80, 80, True, True), (130, (7, 1), 96, 32, True, True),
    (3, (5,), 256, 256, False, True), (17, (2,), 8, 8, False, True), (2, (65,), 32, 16, False, False),
    (11, (3, 3), 33, 20, False, True), (4, (2,), 7, 6, True, True), (6, (5,), 100, 50, False, True),
    (3, (1,), 1, 0, False, True), (600, (8, 8, 8, 8), 64, 64, False, True), (21, (16,), 128, 0, False, False),
    (5, (2,), 250, 250, True, True), (2100, (3,), 40, 40, False, True),
]
TYPES = [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32)]


@gpu
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case, xt, yt):
    tokens, sets, dim, rot, inter, norm = case
    pos = (torch.arange(tokens) * 9973 + 100003) % 131072 - 17
    freqs = L.rope_freqs(rot, 1e4, "cpu") if rot else torch.zeros(0, dtype=torch.float64)
    hs, X, DY, refs = [], [], [], []
    for i, n in enumerate(sets):
        x, dy, gamma = data(tokens, n, dim, xt, yt, i)
        gm = gamma if norm and i != 1 else None
        refs.append(reference(x, dy, pos, gm, freqs, inter, norm, 1e-5))
        hs.append(L.make_heads(tokens, n, dim, xt, yt, norm, 1e-5, None if gm is None else gm.to(DEV),
                               freqs=freqs.to(DEV) if rot else None, interleaved=inter))
        X.append(x.to(DEV))
        DY.append(dy.to(DEV))
    pd = pos.int().to(DEV)
    Y = [torch.empty(x.shape, device=DEV, dtype=yt) for x in X]
    DX = [torch.empty_like(x) for x in X]
    DG = [torch.full((dim,), 3.0, device=DEV) if norm else None for _ in X]
    L.lora_heads_forward(hs, X, Y, pd)
    L.lora_heads_backward(hs, X, DY, DX, DG, pd)
    for (y, ymag, dx, dmag, dg, gmag), gy, gx, gg in zip(refs, Y, DX, DG):
        close(gy, y, ymag, yt)
        close(gx, dx, dmag, xt)
        if norm:
            close(gg, dg, gmag, torch.float32, 128 + 64)
    if norm:   # added to what is there; gradients alone
        again = [g.clone() for g in DG]
        L.lora_heads_backward(hs, X, DY, None, again, pd, accumulate=True)
        for g, a in zip(DG, again):
            assert torch.allclose(a, 2 * g, rtol=2.0 ** -22, atol=1e-30)


@gpu
def test_strides_either_order_and_in_place():
    """[heads, tokens, dim] outputs, inputs inside wider rows, unaligned rows,
    and Y in X's place: the values of the plain layout, and nothing else written."""
    t, n, d = 23, 6, 64
    x, dy, gamma = data(t, n, d, torch.float32, torch.float32)
    pos, freqs = torch.arange(t).int().to(DEV), L.rope_freqs(d)
    kw = dict(eps=1e-6, gamma=gamma.to(DEV), freqs=freqs)
    plain = L.make_heads(t, n, d, **kw)
    xd, y = x.to(DEV), torch.empty(t, n, d, device=DEV)
    L.lora_heads_forward([plain], [xd], [y], pos)
    near = lambda got: close(got, y.cpu().double(), y.abs().cpu().double() + y.abs().max().item(), torch.float32)
    for extra in (40, 37):   # the second's rows are off 16 bytes: element accesses, which sum in another order
        wide = torch.full((t, n * d + extra), 5.0, device=DEV)
        wide[:, :n * d] = xd.view(t, n * d)
        out = torch.full((n, t, d), 9.0, device=DEV)
        h = L.make_heads(t, n, d, ldx=n * d + extra, ldy=d, hy=t * d, **kw)
        L.lora_heads_forward([h], [wide[:, :n * d]], [out.transpose(0, 1)], pos)
        near(out.transpose(0, 1))
        assert (wide[:, n * d:] == 5).all() and (extra == 37 or torch.equal(out.transpose(0, 1), y))
    odd = torch.full((t * n * d + 1,), 0.0, device=DEV)   # rows 4 bytes off: element accesses
    odd[1:] = xd.flatten()
    y2 = torch.empty_like(y)
    L.lora_heads_forward([plain], [odd[1:].view(t, n, d)], [y2], pos)
    near(y2)
    L.lora_heads_forward([plain], [xd], [xd], pos)
    assert torch.equal(xd, y)


@gpu
def test_a_call_that_only_converts():
    v = torch.randn(50, 4, 80, device=DEV)
    v[3, 1, 5], v[4, 0, 0] = math.inf, math.nan
    h = L.make_heads(50, 4, 80, torch.float32, torch.bfloat16, norm=False)
    out = torch.empty(50, 4, 80, device=DEV, dtype=torch.bfloat16)
    L.lora_heads_forward([h], [v], [out])
    assert torch.equal(out.nan_to_num(7), v.bfloat16().nan_to_num(7)) and out[4, 0, 0].isnan()
    back = torch.empty_like(v)
    L.lora_heads_backward([h], None, [out], [back])
    assert torch.equal(back.nan_to_num(7), out.float().nan_to_num(7))


@gpu
def test_infinities_stay_in_their_pair():
    """Without a norm, an infinity past rot_dim is passed on and one inside it
    reaches its own pair only."""
    x = torch.ones(1, 1, 64, device=DEV)
    x[0, 0, 60], x[0, 0, 2] = math.inf, math.inf
    h = L.make_heads(1, 1, 64, norm=False, freqs=L.rope_freqs(32))
    y = torch.empty_like(x)
    L.lora_heads_forward([h], [x], [y], torch.tensor([1], device=DEV, dtype=torch.int32))
    bad = ~torch.isfinite(y[0, 0])
    assert bad.nonzero().flatten().tolist() == [2, 18, 60] and y[0, 0, 60] == math.inf


@gpu
def test_replayed_graph_and_other_stream():
    t, n, d = 300, 8, 128
    x, dy, gamma = data(t, n, d, torch.float32, torch.float32)
    h = [L.make_heads(t, n, d, gamma=gamma.to(DEV), freqs=L.rope_freqs(d))]
    pos = torch.arange(t, device=DEV).int()
    xd, dyd = x.to(DEV), dy.to(DEV)
    y, dx, dg = torch.empty_like(xd), torch.empty_like(xd), torch.empty(d, device=DEV)
    ws = torch.empty(L.lora_heads_workspace_bytes(h), device=DEV, dtype=torch.uint8)

    def call(stream=None):
        L.lora_heads_forward(h, [xd], [y], pos, stream=stream)
        L.lora_heads_backward(h, [xd], [dyd], [dx], [dg], pos, ws=ws, stream=stream)
    call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        xd.copy_(x * (k + 1))
        call()
        torch.cuda.synchronize()
        ref = [v.clone() for v in (y, dx, dg)]
        for v in (y, dx, dg):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (y, dx, dg)))


def _h(**kw):
    d = dict(tokens=4, heads=2, head_dim=64, rot_dim=64, ldx=128, hx=64, ldy=128, hy=64, x_dtype=L.F32,
             y_dtype=L.F32, norm=1, interleaved=0, gamma=256, freqs=256, eps=1e-6)
    d.update(kw)
    return L.LoraHeads(**d)


@no_device
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), -2), (dict(heads=0), -2), (dict(head_dim=0), -2), (dict(head_dim=264, ldx=528, hx=264), -2),
    (dict(rot_dim=66), -2), (dict(rot_dim=63), -2), (dict(rot_dim=-2), -2), (dict(ldx=63), -2), (dict(hy=32), -2),
    (dict(ldx=127), -2), (dict(ldy=64, hy=192), -2), (dict(x_dtype=2), -3), (dict(y_dtype=8), -3),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(freqs=None), -1), (dict(norm=0), -1),
    (dict(gamma=258), -4), (dict(freqs=260), -4),
])
def test_invalid_heads_are_refused(kw, status):
    arr = (L.LoraHeads * 2)(_h(), _h(**kw))
    ptr = (C.c_void_p * 2)(256, 256)
    assert L.lib().lora_heads_forward(2, arr, ptr, ptr, 256, None) == status
    assert L.lib().lora_heads_backward(2, arr, ptr, ptr, ptr, None, 256, 0, None, 0, None) == status
    assert L.lib().lora_heads_workspace_bytes(2, arr) == 0


@no_device
def test_invalid_calls_are_refused():
    lib = L.lib()
    arr, ptr = (L.LoraHeads * 2)(_h(tokens=4000), _h(tokens=4000)), (C.c_void_p * 2)(256, 256)
    fwd = lambda n=2, a=arr, x=ptr, y=ptr, pos=256: lib.lora_heads_forward(n, a, x, y, pos, None)
    assert fwd(n=0) == fwd(n=5) == fwd(a=None) == fwd(x=None) == fwd(y=None) == fwd(pos=None) == -1
    assert fwd(x=(C.c_void_p * 2)(256, None)) == -1 and fwd(y=(C.c_void_p * 2)(256, 258)) == -4
    assert fwd(pos=258) == -4
    assert fwd(a=(L.LoraHeads * 2)(_h(), _h(tokens=5))) == -2
    need = lib.lora_heads_workspace_bytes(2, arr)
    assert need > 0
    bwd = lambda x=ptr, dy=ptr, dx=ptr, dg=ptr, ws=256, nb=need, a=arr: lib.lora_heads_backward(
        2, a, x, dy, dx, dg, 256, 0, ws, nb, None)
    assert bwd(x=None) == bwd(dy=None) == bwd(dx=None, dg=None) == -1
    assert bwd(dx=None, dg=(C.c_void_p * 2)(256, None)) == -1
    assert bwd(ws=None) == bwd(nb=need - 1) == bwd(ws=264) == -5
    assert bwd(dg=(C.c_void_p * 2)(258, 256)) == -4
    plain = (L.LoraHeads * 2)(_h(norm=0, gamma=None), _h())
    assert bwd(a=plain) == -1   # a dgamma without a norm


def test_binding_refuses_wrong_tensors():
    h = L.make_heads(4, 2, 8, norm=False)
    with pytest.raises(ValueError, match="GPU tensor"):
        L.lora_heads_forward([h], [torch.zeros(4, 2, 8)], [torch.zeros(4, 2, 8)])
    with pytest.raises(TypeError):
        L.make_heads(4, 2, 8, torch.float16)


@gpu
def test_binding_checks_tensors():
    h = L.make_heads(4, 2, 8, norm=False)
    ok = torch.zeros(4, 2, 8, device=DEV)
    for bad in (torch.zeros(4, 3, 8, device=DEV), torch.zeros(4, 2, 16, device=DEV)[..., ::2],
                torch.zeros(2, 4, 8, device=DEV).transpose(0, 1)):
        with pytest.raises(ValueError):
            L.lora_heads_forward([h], [bad], [ok])
    with pytest.raises(TypeError):
        L.lora_heads_forward([h], [ok.bfloat16()], [ok])
    with pytest.raises(ValueError):
        L.lora_heads_forward([h, h], [ok], [ok])


@no_device
@pytest.mark.parametrize("kw", [dict(y_dtype=L.BF16), dict(ldy=256), dict(ldy=64, hy=256)])
def test_in_place_with_other_rows_is_refused(kw):
    arr, ptr, ws = (L.LoraHeads * 1)(_h(**kw)), (C.c_void_p * 1)(256), 1 << 20
    assert L.lib().lora_heads_forward(1, arr, ptr, ptr, 256, None) == -1
    assert L.lib().lora_heads_backward(1, arr, (C.c_void_p * 1)(512), ptr, ptr, None, 256, 0, 256, ws, None) == -1
