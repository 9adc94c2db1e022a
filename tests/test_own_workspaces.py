"""Calls that take their workspace from torch's allocator, on another stream
than the current one: the memory may not be handed out again while the call is
still waiting or running there."""

import pytest
import torch

from bwd_adamw_amd import lora as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


def norm_backward():
    nm = L.make_norm("layer", 600, 512, gamma=torch.randn(512, device=DEV))
    x, dy, st = (torch.randn(*s, device=DEV) for s in ((600, 512), (600, 512), (600, 2)))
    out = [torch.zeros(512, device=DEV), torch.zeros(512, device=DEV)]
    return out, L.lora_norm_workspace_bytes(nm), lambda s: L.lora_norm_backward(nm, x, [dy], st, None,
                                                                                *out, stream=s)


def product():
    w = torch.randn(256, 4096, device=DEV).mul_(50).to(torch.float8_e4m3fn)
    W = L.fp8_pack(w, torch.ones(2, 32, device=DEV))
    q, y = L.fp8_rows(64, 4096), torch.zeros(64, 256, device=DEV)
    L.lora_fp8_quantize(torch.randn(64, 4096, device=DEV), q)
    need = L.lora_fp8_product_workspace_bytes(q, W)
    return [y], need, lambda s: L.lora_fp8_product(q, W, y, stream=s)


def orthogonalize():
    g, o = torch.randn(3, 32, 1024, device=DEV), torch.zeros(3, 32, 1024, device=DEV)
    runs, hp = [L.make_matrix_run(0, 32, 1024, 3)], L.make_muon(0.1)
    need = L.lora_muon_workspace_bytes(runs)
    return [o], need, lambda s: L.lora_orthogonalize(g, o, runs, hp, stream=s)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("case", [norm_backward, product, orthogonalize])
def test_workspace_stays_until_the_other_stream_is_done(case, handle):
    torch.manual_seed(1)
    out, need, call = case()
    assert need > 0
    call(None)
    torch.cuda.synchronize()
    ref = [t.clone() for t in out]
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):   # a few milliseconds ahead of the call
            busy = busy @ busy * 1e-3
    call(side.cuda_stream if handle else side)
    # what the current stream is given now, and writes at once
    junk = [torch.full((need,), 255, device=DEV, dtype=torch.uint8) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    del junk
