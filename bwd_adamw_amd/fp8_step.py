"""An optimizer update over an 8-bit base, with the norms before its layers.

    python -m bwd_adamw_amd.fp8_step [--layers 36] [--tokens 4096] [--steps 5]

Adapters on Qwen3-4B-shaped layers whose frozen weights are e4m3 with a scale
for each 128 x 128 block: an RMS norm before each group of projections that
read the residual stream, the groups' forward and backward on 8-bit products,
the norms' backward over the summed gradients of their projections, and the
orthogonalised update of the factors.  Inputs are seeded and synthetic.
"""

from __future__ import annotations

import argparse
import dataclasses
import time

import torch

from . import lora as L
from . import step as S
from . import workloads as WL

#: Groups of a layer that read a norm's output (wq, wk, wv; wgate, wup).
NORMED = (0, 2)


def build(cfg, device="cuda", **kw):
    """(trainer, slot, chunks) of `cfg` with 8-bit weights and norms."""
    cfg = dataclasses.replace(cfg, w_dtype="fp8", optimizer="muon",
                              name=cfg.name.replace("bf16", "fp8"))
    weights, A, B, chunk = {}, {}, {}, {}
    for l in range(cfg.layers):
        xs = {}
        for pj in cfg.projections:
            inp = WL.linear_inputs(cfg, l, pj, chunks=1, device=device)
            key = (l, pj.ordinal)
            weights[key] = L.fp8_pack(*WL.fp8_weight(inp["W"]), device=device)
            A[key], B[key] = inp["A"], inp["B"]
            chunk[key] = (xs.setdefault(pj.x_group, inp["X"][0]), inp["dY"][0])
    dims = {pj.x_group: pj.in_dim for pj in cfg.projections}
    norms = {(l, g): ("rms", 1e-6, torch.ones(dims[g], device=device), None)
             for l in range(cfg.layers) for g in NORMED if g in dims}
    model = S.FrozenModel(cfg, weights, norms)
    slot = S.Slot(cfg, model, A, B, cfg.seeds[0], device)
    return S.Trainer(cfg, model, device=device, **kw), slot, [chunk]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=36)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    args = ap.parse_args()
    cfg = WL.get_config(4).shrink(layers=args.layers, tokens=args.tokens)
    trainer, slot, chunks = build(cfg)
    for k in range(2 + args.steps):
        if k == 2:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        st = trainer.step(slot, chunks)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / args.steps * 1e3
    print(f"{trainer.cfg.name}, {args.layers} layers, {args.tokens} tokens: {ms:.2f} ms/step, "
          f"{args.tokens / ms * 1e3:.0f} tokens/s, gradient norm {st.norm:.4g}")


if __name__ == "__main__":
    main()
