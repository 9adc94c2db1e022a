"""A norm's descriptor keeps the vectors whose addresses it holds."""

import gc
import weakref

import torch

from bwd_adamw_amd import lora as L


def test_the_descriptor_keeps_gamma_and_beta(monkeypatch):
    monkeypatch.setattr(L, "_sized", lambda t, name, need, dtype=None: t.data_ptr())
    gamma, beta = torch.ones(512), torch.zeros(512)
    refs, at = [weakref.ref(t) for t in (gamma, beta)], (gamma.data_ptr(), beta.data_ptr())
    nm = L.make_norm("layer", 600, 512, gamma=gamma, beta=beta)
    del gamma, beta
    gc.collect()
    assert all(r() is not None for r in refs) and (nm.gamma, nm.beta) == at
    del nm
    gc.collect()
    assert all(r() is None for r in refs)
