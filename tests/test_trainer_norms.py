"""A norm that several groups of projections read, in the trainer.

A group holds at most four projections and neighbours in key order, so one X
can have several groups; the gradient of its norm's input is over all of them.

Tolerance: as in test_norm, 128 * 2^-24 of the largest value of each group's
result, and half a step of each addition of the groups' results."""

import pytest
import torch

from bwd_adamw_amd import fp8_step as F
from bwd_adamw_amd import workloads as WL

pytestmark = pytest.mark.gpu


def proj(ordinals_and_groups):
    return tuple(WL.Projection(f"p{o}", o, 256, 128 + 64 * (o % 3), g) for o, g in ordinals_and_groups)


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
