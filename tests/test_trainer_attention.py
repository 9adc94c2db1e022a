"""Attention between wq, wk, wv and wo in the trainer: what wo reads, and the
gradients that wq, wk and wv get, against the formulas in float64.

Tolerances.  The trainer's own Y and dX are taken as the inputs.  Values, queries
and keys are rounded to bf16 (2^-8 relative, half a step), and so are the weights
p (the gradient's ds and dO too): each output is off by a few such steps of the
magnitudes behind it.  Scores are off by 2^-7 of theirs (q and k rounded), which
moves p by as much times the score; scores here stay under 12 (unit heads, scale
1, 1.1 times 1.1 ...), softened by what the row sums take out.  16 * 2^-8 of the
largest magnitude of an output's rows bounds them; float32 products stay within
2^-14 of it."""

import pytest
import torch

from bwd_adamw_amd import fp8_step as F
from bwd_adamw_amd import lora as L
from bwd_adamw_amd import step as S
from bwd_adamw_amd import workloads as WL

gpu = pytest.mark.gpu
H, KV, D, T = 4, 2, 32, 96
PROJ = (WL.Projection("wq", 0, 128, H * D, 0), WL.Projection("wk", 1, 128, KV * D, 0),
        WL.Projection("wv", 2, 128, KV * D, 0), WL.Projection("wo", 3, H * D, 128, 1))


def setup(w_dtype="bf16", layers=2, dtype=torch.bfloat16, device="cuda", chunks=1, offsets=None, proj=PROJ, qk_norm=True,
          **kw):
    cfg = WL.LoraConfig(4, "attention", layers, proj, tokens=T, rank=8, w_dtype=w_dtype, dy_std=1e-2, chunks=chunks)
    weights, A, B, data = {}, {}, {}, [{} for _ in range(chunks)]
    for l in range(layers):
        for pj in proj:
            inp, key = WL.linear_inputs(cfg, l, pj, device=device), (l, pj.ordinal)
            weights[key] = inp["W"].bfloat16() if w_dtype == "bf16" else inp["W"] * 3
            A[key], B[key] = inp["A"], inp["B"]
            for c in range(chunks):
                x, dy = inp["X"][c], inp["dY"][c]
                data[c][key] = (None if pj.ordinal == 3 else x, dy if pj.ordinal == 3 else None)
                if offsets is not None:
                    data[c]["offsets"] = offsets
    g = torch.Generator().manual_seed(3)
    gam = lambda: (1 + 0.1 * torch.randn(D, generator=g)).to(device) if qk_norm else None
    spec = S.AttentionSpec(H, KV, D, L.rope_freqs(D, 1e4, device), qk_norm, gam(), gam(), dtype=dtype)
    model = S.FrozenModel(cfg, weights, attention={l: spec for l in range(layers)})
    trainer = S.Trainer(cfg, model, device=device, **kw)
    return trainer, S.Slot(cfg, model, A, B, 1, device), data, spec


def attend(y, spec, offsets):
    """wo's input from [Yq, Yk, Yv] in float64 (differentiable)."""
    pos = torch.cat([torch.arange(b - a) for a, b in zip(offsets, offsets[1:])]).double()
    phi = pos[:, None] * spec.freqs.cpu()
    co, si = phi.cos()[:, None], phi.sin()[:, None]

    def head(x, n, gamma):
        z = x.view(T, n, D)
        if spec.qk_norm:
            z = z * (z.square().mean(-1, keepdim=True) + spec.eps).rsqrt() * gamma.cpu().double()
        a, b = z[..., :D // 2], z[..., D // 2:]
        return torch.cat([a * co - b * si, b * co + a * si], -1)
    q, k, v = head(y[0], H, spec.q_gamma), head(y[1], KV, spec.k_gamma), y[2].view(T, KV, D)
    out = []
    for a, b in zip(offsets, offsets[1:]):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(H // KV, 1)) * D ** -0.5
        s = s.masked_fill(torch.ones(b - a, b - a).triu(1).bool(), float("-inf"))
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[a:b].repeat_interleave(H // KV, 1)))
    return torch.cat(out).reshape(T, H * D)


def close(got, ref, tol):
    assert (got.detach().cpu().double() - ref).abs().max() <= tol * ref.abs().max()


@gpu
@pytest.mark.parametrize("offsets", [None, [0, 1, 40, 40, T]])
@pytest.mark.parametrize("dtype,qk_norm", [(torch.bfloat16, True), (torch.float32, True), (torch.float32, False)])
def test_forward_and_gradients(dtype, qk_norm, offsets):
    trainer, slot, chunks, spec = setup("f32" if dtype == torch.float32 else "bf16", dtype=dtype, offsets=offsets,
                                        qk_norm=qk_norm)
    trainer.forward_backward(slot, chunks)
    torch.cuda.synchronize()
    tol = 2.0 ** -14 if dtype == torch.float32 else 16 * 2.0 ** -8
    for l, at in trainer.attention.items():
        y = [trainer.Y[(l, o)].cpu().double().requires_grad_() for o in range(3)]
        o = attend(y, spec, offsets or [0, T])
        close(at.O, o.detach(), tol)
        o.backward(trainer.dX[(l, 3)].cpu().double())
        for t, dy, key in zip(y, at.dY, [(l, o) for o in range(3)]):
            close(dy, t.grad, tol)
            # and that is what the projection's gradients come from
            gb = trainer.scale * dy.cpu().double().T @ trainer.U[key].cpu().double()
            close(slot.gB[key], gb, 2.0 ** -7)
        gb = trainer.scale * chunks[0][(l, 3)][1].cpu().double().T @ trainer.U[(l, 3)].cpu().double()
        close(slot.gB[(l, 3)], gb, 2.0 ** -7)
        u = at.O.cpu().double() @ slot.A[(l, 3)].cpu().double().T
        close(trainer.U[(l, 3)], u, 2.0 ** -7)


@gpu
def test_streams_chunks_and_slots():
    """Four streams as one; two chunks add up; two slots take turns."""
    one, slot1, chunks, _ = setup(layers=3, chunks=2, offsets=[0, 50, T], streams=1)
    four, slot4, _, _ = setup(layers=3, chunks=2, offsets=[0, 50, T])
    one.step(slot1, chunks)
    four.step(slot4, chunks)
    assert torch.equal(slot1.grads, slot4.grads) and torch.equal(slot1.params, slot4.params)
    first, second = (setup(layers=3, chunks=2, offsets=[0, 50, T]) for _ in range(2))
    first[0].forward_backward(first[1], chunks[:1])
    second[0].forward_backward(second[1], chunks[1:])
    tot = first[1].grads + second[1].grads
    assert (tot - slot1.grads).abs().max() <= 2.0 ** -22 * (first[1].grads.abs() + second[1].grads.abs()).max()
    both = S.Trainer(one.cfg, one.model, slots=2)
    a, b = setup(layers=3, chunks=2)[1], setup(layers=3, chunks=2)[1]
    both.step_slots([a, b], [chunks, chunks])
    assert not both.stack_slots and torch.equal(a.params, slot1.params) and torch.equal(b.params, slot1.params)


@gpu
def test_offsets_are_checked():
    trainer, slot, chunks, _ = setup()
    for bad in ([0, 10], [1, T], [0, 60, 50, T], [0]):
        chunks[0]["offsets"] = bad
        with pytest.raises(ValueError, match="offsets"):
            trainer.forward_backward(slot, chunks)


@gpu
@pytest.mark.parametrize("change,match", [
    ({0: WL.Projection("wq", 0, 128, 2 * H * D, 0)}, "projection"),
    ({3: WL.Projection("wo", 3, 2 * H * D, 128, 1)}, "projection"),
    ({3: None}, "no projection"),
    ({3: WL.Projection("wo", 3, H * D, 128, 0)}, "to itself"),
])
def test_projections_that_do_not_fit(change, match):
    proj = tuple(p for p in (change.get(p.ordinal, p) for p in PROJ) if p is not None)
    with pytest.raises(ValueError, match=match):
        setup(proj=proj)


@gpu
def test_8_bit_step_with_norms_and_attention():
    """The whole step of the command, small: it runs, updates every factor, and
    does the same twice."""
    proj = (WL.Projection("wq", 0, 256, 1024, 0), WL.Projection("wk", 1, 256, 1024, 0),
            WL.Projection("wv", 2, 256, 1024, 0), WL.Projection("wo", 3, 1024, 256, 1))
    cfg = WL.LoraConfig(4, "small", 2, proj, tokens=64, rank=8, dy_std=1e-2)
    out = []
    for _ in range(2):
        trainer, slot, chunks = F.build(cfg, sequences=3)
        before = slot.params.clone()
        for _ in range(2):
            st = trainer.step(slot, chunks)
        assert not st.vetoed and st.norm > 0
        assert all((slot.A[k] != before[:slot.A[k].numel()].view_as(slot.A[k])).any() for k in slot.keys[:1])
        out.append(slot.params.clone())
    assert torch.equal(*out) and set(trainer.attention) == {0, 1}
