"""The 8-bit products' sums keep 32 bits.

Whole numbers, of which one pair of every row cancels: the products reach
448 * 448 = 200704, whole rows sum to little, and the magnitudes of all products
of a row stay below 2^24.  Every partial sum, in whatever order, is then a
whole number that float32 holds, so the results have to be equal to the exact
ones: with sums of 32 bits or more each addition is exact, and a sum that drops
bits below its largest term loses the small products beside the large ones.
Scales are powers of two, which change no digit."""

import pytest
import torch

from bwd_adamw_amd import lora as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cancelling(T, K, N, seed):
    """x [T, K] and w [N, K], whole numbers: in every other block of 128 of the
    contraction two neighbours hold 448 and the weights +-448."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-3, 4, (T, K), generator=g).double()
    w = torch.randint(-3, 4, (N, K), generator=g).double()
    for b in range(0, -(-K // 128), 2):
        room = min(127, K - b * 128 - 1)   # places for a pair
        if room < 1:
            continue
        i = b * 128 + int(torch.randint(0, room, (1,), generator=g))
        x[:, i:i + 2] = 448
        w[:, i] = 448
        w[:, i + 1] = -448
    assert (x.abs() @ w.abs().t()).max() < 2 ** 24
    return x, w


def weight(w, scale):
    N, K = w.shape
    s = torch.full((-(-N // 128), -(-K // 128)), scale)
    return L.fp8_pack(w.float().to(torch.float8_e4m3fn).to(DEV), s.to(DEV))


# Few tokens, each tile size, splits of the contraction, ragged sizes.
SHAPES = [(1, 128, 64), (1, 2560, 1024), (9, 300, 130), (16, 9728, 264), (40, 4096, 130), (130, 1000, 257),
          (200, 640, 2000), (300, 2560, 1024), (1000, 2056, 1368), (2048, 1280, 2560), (4096, 256, 4360)]


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_small_products_beside_large_ones(T, K, N, dx):
    a, b = cancelling(T, N if dx else K, K if dx else N, T + K)
    W = weight(b.t().contiguous() if dx else b, 0.25)
    ref = 0.5 * (a @ b.t())
    q = L.fp8_rows(*a.shape)
    L.lora_fp8_quantize((2 * a).float().to(DEV), q)
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty(T, K if dx else N, device=DEV, dtype=dt)
        L.lora_fp8_product(q, W, y, dx=dx)
        assert torch.equal(y.cpu(), ref.to(dt))


@pytest.mark.parametrize("T,K,N", [(1, 2560, 1024), (96, 512, 260), (512, 1280, 2560), (4096, 256, 4360)])
def test_small_products_beside_large_ones_in_an_adapted_linear(T, K, N):
    """Forward and dX with a zero adapter, which adds exactly nothing."""
    r = 8
    A, B = torch.zeros(r, K, device=DEV), torch.zeros(N, r, device=DEV)
    for dx in (False, True):
        a, b = cancelling(T, N if dx else K, K if dx else N, T)
        W = weight(b.t().contiguous() if dx else b, 1.0)
        lin = L.make_linear(W, A, B, 2.0, T)
        ws = torch.empty(L.lora_workspace_bytes(lin), device=DEV, dtype=torch.uint8)
        U = torch.zeros(T, r, device=DEV)
        src, out = a.float().to(DEV), torch.empty(T, K if dx else N, device=DEV)
        if dx:
            L.lora_backward(lin, torch.ones(T, K, device=DEV), src, U, None, out, torch.empty_like(A),
                            torch.empty_like(B), ws=ws)
        else:
            L.lora_forward(lin, src, out, U, ws=ws)
        assert torch.equal(out.cpu().double(), a @ b.t())


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("power", [-126, -110, -100, -60, 60, 100, 115])
def test_blocks_of_every_size(T, power):
    """Rows of 2^power: the results are 2^power times those of whole numbers,
    with W's scale bringing them back to the range of normal numbers."""
    K, N = 256, 132
    g = torch.Generator().manual_seed(power + 200)
    x = torch.randint(-3, 4, (T, K), generator=g).double()
    w = torch.randint(-3, 4, (N, K), generator=g).double()
    W = weight(w, 2.0 ** max(-120, min(120, -power)))
    q = L.fp8_rows(T, K)
    L.lora_fp8_quantize((x * 2.0 ** power).float().to(DEV), q)
    y = torch.empty(T, N, device=DEV)
    L.lora_fp8_product(q, W, y)
    assert torch.equal(y.cpu().double(), (x @ w.t()) * 2.0 ** (power + max(-120, min(120, -power))))
