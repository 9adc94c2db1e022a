"""Norms before the groups in the trainer: one that several groups of
projections read, and two slots.

A group holds at most four projections and neighbours in key order, so one X
can have several groups; the gradient of its norm's input is over all of them.

Tolerance: as in test_norm, 128 * 2^-24 of the largest value of each group's
result, and half a step of each addition of the groups' results."""

import pytest
import torch

from bwd_adamw_amd import fp8_step as F
from bwd_adamw_amd import step as S
from bwd_adamw_amd import workloads as WL

gpu = pytest.mark.gpu


def proj(ordinals_and_groups):
    return tuple(WL.Projection(f"p{o}", o, 256, 128 + 64 * (o % 3), g) for o, g in ordinals_and_groups)


@gpu
@pytest.mark.parametrize("projections", [
    [(0, 0), (1, 0), (2, 0), (3, 0), (4, 0)],                       # more than one group holds
    [(0, 0), (1, 2), (2, 0), (3, 2)],                               # not neighbours in key order
    [(k, 0) for k in range(9)] + [(9, 2)],                          # three groups of one norm
])
@pytest.mark.parametrize("streams", [1, 4])
def test_gradient_of_a_shared_norms_input(projections, streams):
    cfg = WL.LoraConfig(4, "shared-norm", 2, proj(projections), tokens=96, rank=8, dy_std=1e-2)
    trainer, slot, chunks = F.build(cfg, streams=streams)
    trainer.forward_backward(slot, chunks)
    torch.cuda.synchronize()
    assert set(trainer.dH) == {(l, g) for l in range(2) for g in {g for _, g in projections} & {0, 2}}
    for (layer, g), dH in trainer.dH.items():
        keys = [(layer, o) for o, xg in projections if xg == g]
        X = chunks[0][keys[0]][0].double()
        dy = sum(trainer.dX[k].double() for k in keys)
        rstd = 1 / (X.square().mean(1, keepdim=True) + 1e-6).sqrt()
        xh = X * rstd
        ref = rstd * (dy - xh * (dy * xh).mean(1, keepdim=True))
        mag = rstd * sum(trainer.dX[k].double().abs() for k in keys)
        tol = (128 + len(projections)) * 2.0 ** -24 * mag.max()
        assert ((dH.double() - ref).abs() <= tol).all()


def two_slots(device, **kw):
    """(trainer of `kw`, slots, chunks) over bf16 weights, norms before the X."""
    cfg = WL.LoraConfig(4, "two-slots", 1, proj([(0, 0), (1, 0)]), tokens=256, rank=8, w_dtype="bf16",
                        dy_std=1e-2)
    weights, chunk, A, B = {}, {}, {}, {}
    for pj in cfg.projections:
        inp = WL.linear_inputs(cfg, 0, pj, chunks=1, device=device)
        key = (0, pj.ordinal)
        weights[key], A[key], B[key] = inp["W"].bfloat16(), inp["A"], inp["B"]
        chunk[key] = (inp["X"][0], inp["dY"][0])
    model = S.FrozenModel(cfg, weights, {(0, 0): ("rms", 1e-6, None, None)})
    slots = [S.Slot(cfg, model, A, B, seed, device) for seed in (1, 2)]
    return S.Trainer(cfg, model, device=device, **kw), slots, [chunk]


def test_slots_with_norms_are_not_stacked():
    trainer, _, _ = two_slots("cpu", slots=2, streams=1)
    assert not trainer.stack_slots and list(trainer.dH) == [(0, 0)]


@gpu
def test_two_slots_with_norms():
    """Together as each alone."""
    together, slots, chunks = two_slots("cuda", slots=2)
    alone, refs, _ = two_slots("cuda")
    together.step_slots(slots, [chunks, chunks])
    for ref, slot in zip(refs, slots):
        alone.step(ref, chunks)
        assert torch.equal(ref.grads, slot.grads) and torch.equal(ref.params, slot.params)
    assert torch.equal(alone.dH[(0, 0)], together.dH[(0, 0)])
