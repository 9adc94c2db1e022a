"""The norm backward's sums over many rows.

A lane adds the rows of its block that it holds one after another in float32,
at most rows / 256 + 16 of them; the block's lanes and the blocks follow, the
latter in float64.  Each addition rounds by half a step of the running sum,
which the sum of magnitudes bounds, and each term carries three roundings:
(rows / 256 + 24) * 2^-24 of the sum of magnitudes."""

import pytest
import torch

from bwd_adamw_amd import lora as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,dim,kind,dtype", [
    (300007, 64, "layer", torch.float32), (200003, 132, "rms", torch.float32),
    (150000, 257, "layer", torch.bfloat16), (60001, 2052, "layer", torch.float32),
    (20000, 10244, "rms", torch.bfloat16)])
def test_column_sums_of_many_rows(rows, dim, kind, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, dim, device=DEV, generator=g).to(dtype)
    dy = (torch.randn(rows, dim, device=DEV, generator=g) + 0.5).to(dtype)   # sums that grow
    stats = torch.stack([0.1 * torch.randn(rows, device=DEV, generator=g),
                         0.5 + torch.rand(rows, device=DEV, generator=g)], 1)
    if kind == "rms":
        stats[:, 0] = 0
    nm = L.make_norm(kind, rows, dim, dtype)
    dg, db = torch.empty(dim, device=DEV), torch.empty(dim, device=DEV) if kind == "layer" else None
    L.lora_norm_backward(nm, x, [dy], stats, None, dg, db)
    s, ref, mag, refb, magb = stats.double(), 0, 0, 0, 0
    for a in range(0, rows, 20000):
        d = dy[a:a + 20000].double()
        t = d * (x[a:a + 20000].double() - s[a:a + 20000, :1]) * s[a:a + 20000, 1:]
        # the centring's own rounding is relative to the larger of x and the mean
        big = d.abs() * (x[a:a + 20000].double().abs() + s[a:a + 20000, :1].abs()) * s[a:a + 20000, 1:]
        ref, mag, refb, magb = ref + t.sum(0), mag + big.sum(0), refb + d.sum(0), magb + d.abs().sum(0)
    tol = (rows / 256 + 24) * 2.0 ** -24
    assert ((dg.double() - ref).abs() <= tol * mag).all()
    if db is not None:
        assert ((db.double() - refb).abs() <= tol * magb).all()
