"""Vetoed updates and non-finite matrices on every kernel of the
orthogonalised update: each padded short side (16, 32, 64, 128) wide and tall,
and at 16 both the one-block kernel (long sides up to 512) and the pair of
passes.  Tolerances as in test_muon."""

import pytest
import torch

from bwd_adamw_amd import lora as L
from test_muon import close_orth, matrix, orth

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [(8, 64), (64, 8), (16, 512), (512, 16), (8, 516), (2048, 8), (1, 700), (24, 640), (640, 24),
          (32, 2560), (60, 640), (1001, 61), (64, 64), (100, 300), (300, 100), (128, 1000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_veto_changes_nothing(rows, cols, bad):
    p, g, m = (torch.randn(3, rows, cols, device=DEV) for _ in range(3))
    before = p.clone(), m.clone(), g.clone()
    run = [L.make_matrix_run(0, rows, cols, 3)]
    L.lora_muon_step(p, g, m, run, L.make_muon(0.1, weight_decay=0.1), torch.full((1,), bad, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip((p, m, g), before))
    L.lora_muon_step(p, g, m, run, L.make_muon(0.1), torch.ones(1, device=DEV))
    assert not torch.equal(p, before[0]) and not torch.equal(m, before[1])


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_matrix_stays_alone(rows, cols, bad):
    g = torch.stack([matrix(rows, cols, i) for i in range(3)])
    g[1, rows // 2, cols // 3] = bad
    runs, hp = [L.make_matrix_run(0, rows, cols, 3)], L.make_muon(0.1)
    out = torch.empty(3, rows, cols, device=DEV)
    L.lora_orthogonalize(g.to(DEV), out, runs, hp)
    assert torch.isnan(out[1]).all()
    for i in (0, 2):
        close_orth(out[i], orth(g[i]))
    p, m = torch.zeros(3, rows, cols, device=DEV), torch.zeros(3, rows, cols, device=DEV)
    L.lora_muon_step(p, g.to(DEV), m, runs, hp, torch.ones(1, device=DEV))
    assert torch.isnan(p[1]).all() and torch.isfinite(p[[0, 2]]).all()
    assert torch.isfinite(m[[0, 2]]).all() and (~torch.isfinite(m[1])).sum() == 1
