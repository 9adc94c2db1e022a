"""Infinities in the factors of an adapted linear over an 8-bit W reach the
results that the formula says, with its sign, at ranks that leave part of a
contraction step empty: 0 * infinity there would make them NaN."""

import pytest
import torch

from bwd_adamw_amd import lora as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,K,N", [(5, 128, 132), (300, 256, 512), (512, 512, 2560)])
@pytest.mark.parametrize("r", [4, 12, 32, 40])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_factor(T, K, N, r, sign):
    g = torch.Generator().manual_seed(r)
    W = L.fp8_pack(torch.ones(N, K).to(torch.float8_e4m3fn).to(DEV), torch.full((-(-N // 128), -(-K // 128)), 0.01).to(DEV))
    A = (0.5 + torch.rand(r, K, generator=g)) * torch.where(torch.rand(r, K, generator=g) < 0.5, -1.0, 1.0)
    A[1] = A[1].abs()
    A, B = A.to(DEV), (0.5 + torch.rand(N, r, generator=g)).to(DEV)
    B[3, 1] = sign * float("inf")
    lin = L.make_linear(W, A, B, 1.0, T)
    ws = torch.empty(L.lora_workspace_bytes(lin), device=DEV, dtype=torch.uint8)
    X, Y, U = torch.ones(T, K, device=DEV), torch.empty(T, N, device=DEV), torch.empty(T, r, device=DEV)
    L.lora_forward(lin, X, Y, U, ws=ws)
    others = torch.arange(N, device=DEV) != 3
    assert torch.isfinite(Y[:, others]).all()
    assert (Y[:, 3] == sign * float("inf")).all()     # U[:, 1] > 0
    dX, dA, dB = torch.empty(T, K, device=DEV), torch.empty_like(A), torch.empty_like(B)
    dY = torch.ones(T, N, device=DEV)
    L.lora_backward(lin, X, dY, U, None, dX, dA, dB, ws=ws)
    assert (dX == sign * float("inf") * A[1].sign()).all()   # V[:, 1] is infinite
