"""The adapted linear over an 8-bit W, and the trainer's update with 8-bit
weights, norms before the groups and the orthogonalised update.

Tolerances.  The frozen product as in test_fp8 (2^-12 of its magnitudes).  The
LoRA term's factors are rounded to bf16 (half a step, 2^-8 relative, each):
2^-7 of its magnitudes and a little for their product, 2^-6.9.  U, dA and dB
come from the float32 kernels, 1e-4 of the largest value as elsewhere in this
suite."""

import ctypes as C
import dataclasses

import pytest
import torch

from bwd_adamw_amd import fp8_step as F
from bwd_adamw_amd import lora as L
from bwd_adamw_amd import step as S
from bwd_adamw_amd import workloads as WL
from helpers import rel_err
from test_fp8 import ref_round

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")


def make(T, K, N, r, seed=0):
    g = torch.Generator().manual_seed(seed + T + K + N)
    q, s = WL.fp8_weight(0.02 * torch.randn(N, K, generator=g))
    w = q.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    rnd = lambda *sh: torch.randn(*sh, generator=g)
    return (L.fp8_pack(q.to(DEV), s.to(DEV)), w, 0.05 * rnd(r, K), 0.1 * rnd(N, r), rnd(T, K),
            0.1 * rnd(T, N))


SHAPES = [(1, 64, 64, 4), (33, 200, 132, 8), (128, 640, 264, 12), (300, 1024, 512, 32),
          (512, 512, 2560, 64), (257, 260, 300, 128)]


@gpu
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("T,K,N,r", SHAPES)
def test_forward_and_backward(T, K, N, r, p):
    W, w, A, B, X, dY = make(T, K, N, r)
    s = 1.7
    Ad, Bd = A.to(DEV), B.to(DEV)   # the descriptor holds only their addresses
    lin = L.make_linear(W, Ad, Bd, s, T)
    drop = L.make_dropout(5, 1, 0, 0, 2, p) if p else None
    keep = torch.ones(T, K)
    if p:
        mask = torch.empty(T * K, device=DEV, dtype=torch.uint8)
        L.lora_dropout_mask(drop, T, K, mask)
        keep = mask.cpu().view(T, K).float() / (1 - p)
    ws = torch.empty(max(16, L.lora_workspace_bytes(lin)), device=DEV, dtype=torch.uint8)
    Xd, dYd = X.to(DEV), dY.to(DEV)
    Y, Z, U = (torch.empty(T, n, device=DEV) for n in (N, N, r))
    L.lora_forward(lin, Xd, Y, U, Z, drop, ws)
    u = (X.double() * keep.double()) @ A.double().t()
    assert rel_err(U, u) <= 1e-4
    xq = ref_round(X)[2]
    ref = xq @ w.t() + s * u @ B.double().t()
    tol = 2.0 ** -12 * (xq.abs() @ w.abs().t()) + 2.0 ** -6.9 * s * (u.abs() @ B.double().abs().t())
    assert ((Y.cpu().double() - ref).abs() <= tol + 1e-12).all()
    assert torch.equal(Y, Z)
    dX, dA, dB = torch.empty(T, K, device=DEV), torch.empty(r, K, device=DEV), torch.empty(N, r, device=DEV)
    L.lora_backward(lin, Xd, dYd, U, None, dX, dA, dB, drop=drop, ws=ws)
    v = dY.double() @ B.double()
    gq = ref_round(dY)[2]
    ref = gq @ w + s * (v @ A.double()) * keep.double()
    tol = 2.0 ** -12 * (gq.abs() @ w.abs()) + 2.0 ** -6.9 * s * (v.abs() @ A.double().abs()) * keep.double()
    assert ((dX.cpu().double() - ref).abs() <= tol + 1e-12).all()
    assert rel_err(dB, s * dY.double().t() @ u) <= 1e-4
    assert rel_err(dA, s * v.t() @ (X.double() * keep.double())) <= 1e-4


@gpu
def test_group_equals_separate_calls():
    """A group with one float32 and two 8-bit linears over one X (which the
    8-bit ones share rounded) gives the separate calls' bits."""
    T, K, r = 256, 512, 16
    lins = []
    X = torch.randn(T, K, device=DEV)
    for i, N in enumerate((512, 256, 384)):
        W, w, A, B, _, _ = make(T, K, N, r, i)
        if i == 1:
            W = w.float().to(DEV)
        lins.append((W, A.to(DEV), B.to(DEV), 0, N))
    ds = [L.make_linear(W, A, B, 0.5, T) for W, A, B, _, _ in lins]
    ws = torch.empty(L.lora_group_workspace_bytes(ds), device=DEV, dtype=torch.uint8)
    Y = [torch.empty(T, l[4], device=DEV) for l in lins]
    U = [torch.empty(T, r, device=DEV) for _ in lins]
    L.lora_forward_group(ds, X, Y, U, ws=ws)
    dY = [torch.randn(T, l[4], device=DEV) for l in lins]
    dX, dA, dB = ([torch.empty(*sh, device=DEV) for l in lins for sh in [f(l)]]
                  for f in (lambda l: (T, K), lambda l: (r, K), lambda l: (l[4], r)))
    L.lora_backward_group(ds, X, dY, U, None, dX, dA, dB, ws=ws)
    for i, d in enumerate(ds):
        w1 = torch.empty(max(16, L.lora_workspace_bytes(d)), device=DEV, dtype=torch.uint8)
        y, u = torch.empty_like(Y[i]), torch.empty_like(U[i])
        L.lora_forward(d, X, y, u, ws=w1)
        a, b, x = torch.empty_like(dA[i]), torch.empty_like(dB[i]), torch.empty_like(dX[i])
        L.lora_backward(d, X, dY[i], u, None, x, a, b, ws=w1)
        assert all(torch.equal(p, q) for p, q in
                   ((y, Y[i]), (u, U[i]), (x, dX[i]), (a, dA[i]), (b, dB[i])))


@gpu
def test_trainer_step_is_its_calls():
    """The trainer's update (four streams) over two layers with norms, 8-bit
    weights and the orthogonalised update, against the same library calls in
    sequence on one stream."""
    proj = (WL.Projection("wq", 0, 256, 384, 0), WL.Projection("wv", 2, 256, 128, 0),
            WL.Projection("wo", 3, 384, 256, 1), WL.Projection("wgate", 4, 256, 512, 2))
    cfg = WL.LoraConfig(4, "two-bf16-layers", 2, proj, tokens=96, rank=8, dropout=0.1, dy_std=1e-2,
                        weight_decay=0.1, plus_ratio=4.0)
    trainer, slot, chunks = F.build(cfg)
    _, ref, _ = F.build(cfg)
    cfg, model, T = trainer.cfg, trainer.model, trainer.T
    assert len(slot.runs) == 8 and all(r.count == 2 for r in slot.runs)
    m = torch.zeros_like(ref.params)
    scale, stats = torch.zeros(1, device=DEV), torch.zeros(2, device=DEV, dtype=torch.float64)
    pw = torch.empty(L.lora_grad_prepare_workspace_bytes(ref.n), device=DEV, dtype=torch.uint8)
    for k in range(2):
        st = trainer.step(slot, chunks)
        assert not st.vetoed
        dH = {}
        for group in trainer.groups:
            key = group[0]
            lay, xg = key[0], next(p.x_group for p in proj if p.ordinal == key[1])
            H = X = chunks[0][key][0]
            nm = None
            if (lay, xg) in model.norms:
                kind, eps, gamma, beta = model.norms[(lay, xg)]
                nm = L.make_norm(kind, T, H.shape[1], torch.float32, eps, gamma, beta)
                X, rs = torch.empty_like(H), torch.empty(T, 2, device=DEV)
                L.lora_norm_forward(nm, H, X, rs)
            dXs = []
            for kk in group:
                W = model.W[kk]
                lin = L.make_linear(W, ref.A[kk], ref.B[kk], trainer.scale, T)
                drop = L.make_dropout(ref.seed, k, 0, kk[0], kk[1], cfg.dropout)
                ws = torch.empty(L.lora_workspace_bytes(lin), device=DEV, dtype=torch.uint8)
                Y, U = torch.empty(T, W.out_dim, device=DEV), torch.empty(T, cfg.rank, device=DEV)
                L.lora_forward(lin, X, Y, U, None, drop, ws)
                assert torch.equal(Y, trainer.Y[kk])
                dXs.append(torch.empty(T, W.in_dim, device=DEV))
                L.lora_backward(lin, X, chunks[0][kk][1], U, None, dXs[-1], ref.gA[kk], ref.gB[kk],
                                drop=drop, ws=ws)
            if nm is not None:
                dh = torch.empty_like(H)
                L.lora_norm_backward(nm, H, dXs, rs, dh)
                dH[(lay, xg)] = dh
        assert torch.equal(ref.grads, slot.grads)
        assert set(dH) == set(trainer.dH) and len(dH) == 4
        assert all(torch.equal(dH[x], trainer.dH[x]) for x in dH)
        L.lora_grad_prepare(ref.grads, T, cfg.max_norm, scale, stats, True, pw)
        hp = L.make_muon(cfg.lr, cfg.momentum, cfg.weight_decay, cfg.plus_ratio, adjust="rms")
        L.lora_muon_step(ref.params, ref.grads, m, ref.runs, hp, scale)
        assert torch.equal(ref.params, slot.params) and torch.equal(m, slot.m)


@gpu
def test_muon_with_dora_updates_the_magnitudes_by_adamw():
    cfg = dataclasses.replace(WL.get_config(1), dora=True, optimizer="muon")
    pj = cfg.projections[0]
    inp = WL.linear_inputs(cfg, 0, pj)
    key = (0, pj.ordinal)
    model = S.FrozenModel(cfg, {key: inp["W"].cuda()})
    tr = S.Trainer(cfg, model)
    slot = S.Slot(cfg, model, {key: inp["A"].cuda()}, {key: inp["B"].cuda()}, 1)
    tr.init_dora(slot)
    mag = slot.mag[key].clone()
    tr.step(slot, [{key: (inp["X"][0].cuda(), inp["dY"][0].cuda())}])
    # AdamW's first step moves each magnitude by lr.
    assert torch.allclose((slot.mag[key] - mag).abs(), torch.full_like(mag, cfg.lr), rtol=0.02)


@no_device
def test_refusals():
    lib = L.lib()
    lin = lambda **kw: L.LoraLinear(**{**dict(tokens=8, in_dim=16, out_dim=16, rank=4, w_dtype=L.FP8,
                                              scale=2.0, W=256, A=256, B=256, dora_mag=None,
                                              dora_norm=None), **kw})
    ok = lin()
    assert lib.lora_workspace_bytes(C.byref(ok)) > 0
    for bad, rc in ((lin(in_dim=18), -4), (lin(dora_mag=256, dora_norm=256), -3),
                    (lin(in_dim=1 << 20, out_dim=1 << 20), -2), (lin(W=264), -4)):
        assert lib.lora_workspace_bytes(C.byref(bad)) == 0
        assert lib.lora_forward(C.byref(bad), 256, 256, 256, None, None, 256, 1 << 40, None) == rc
    need = lib.lora_workspace_bytes(C.byref(ok))
    assert lib.lora_forward(C.byref(ok), 256, 256, 256, None, None, 256, 16, None) == -5
    assert need > 16
    assert lib.lora_dora_row_norms(C.byref(ok), 256, None, 0, None) == -3
    with pytest.raises(ValueError, match="optimizer"):
        cfg = dataclasses.replace(WL.get_config(1), optimizer="sgd")
        S.Trainer(cfg, S.FrozenModel(cfg, {}), device="cpu")
