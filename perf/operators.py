"""Cases of the operators around the adapted linear: the norm before it, the
8-bit block-scaled frozen product, and the orthogonalised update of its
factors.

  norm_fwd  y = (x - mean) rstd gamma + beta per row (layer norm), or
            y = x rstd gamma (RMS norm), with the row statistics
  norm_bwd  dx, dgamma, dbeta from one to four gradients of y, one for each
            projection that read y
  fp8_fwd   Y = Q(X) W^T in bf16, where Q rounds each 128-wide block of a row
            to e4m3 with a power-of-two scale and W is e4m3 with a float32
            scale for each 128 x 128 block
  fp8_dx    dX = Q(dY) W, the same W read in its own layout
  orth      Newton-Schulz orthogonalisation of a batch of matrices
  muon      momentum, orthogonalisation and the update of the parameters

`own` selects the calls of the framework's kernels; otherwise `run` computes
the operators from elementary torch operations in 32 bits.
"""

import math

import torch

own = False

#: Coefficients of the quintic step X <- a X + (b G + c G^2) X, G = X X^T.
NS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
LR, MOMENTUM, DECAY = 2e-3, 0.95, 0.01


def listed():
    return [
        # The input of the 64-wide single linear: nothing but latency.
        {"name": "norm fwd 32x64", "op": "norm_fwd", "kind": "layer", "rows": 32, "dim": 64, "dtype": "f32"},
        # The hidden state before a Qwen3-4B-shaped layer's projections, one chunk.
        {"name": "norm fwd 4096x2560 rms", "op": "norm_fwd", "kind": "rms", "rows": 4096, "dim": 2560, "dtype": "f32"},
        # An odd number of rows of an odd width, bf16 activations.
        {"name": "norm bwd 1537x4100 bf16", "op": "norm_bwd", "kind": "layer", "rows": 1537, "dim": 4100, "dtype": "bf16", "grads": 1},
        # The backward before wq, wk and wv: three gradients of one y.
        {"name": "norm bwd 4096x2560 rms", "op": "norm_bwd", "kind": "rms", "rows": 4096, "dim": 2560, "dtype": "f32", "grads": 3},
        # One token through a query projection: the weight's bytes are the cost.
        {"name": "fp8 fwd 1x2560x4096", "op": "fp8_fwd", "tokens": 1, "in_dim": 2560, "out_dim": 4096, "dtype": "f32"},
        # A ragged chunk through a ragged weight, bf16 activations.
        {"name": "fp8 fwd 1000x2056x1368", "op": "fp8_fwd", "tokens": 1000, "in_dim": 2056, "out_dim": 1368, "dtype": "bf16"},
        # The widest frozen product of a Qwen3-4B-shaped layer, one chunk.
        {"name": "fp8 fwd 4096x2560x9728", "op": "fp8_fwd", "tokens": 4096, "in_dim": 2560, "out_dim": 9728, "dtype": "f32"},
        # Its gradient, over a chunk of the two-slot workload.
        {"name": "fp8 dx 2048x2560x9728", "op": "fp8_dx", "tokens": 2048, "in_dim": 2560, "out_dim": 9728, "dtype": "f32"},
        # The factor of the 64-wide single linear.
        {"name": "muon 1x64x4", "op": "muon", "count": 1, "rows": 64, "cols": 4},
        # The A factors of the TinyLlama-shaped query projections.
        {"name": "muon 22x8x2048", "op": "muon", "count": 22, "rows": 8, "cols": 2048},
        # The gradients of 36 A factors of rank 64, orthogonalised alone.
        {"name": "orth 36x64x2560", "op": "orth", "count": 36, "rows": 64, "cols": 2560},
        # The B factors of 36 gate and 36 up projections of rank 64.
        {"name": "muon 72x9728x64", "op": "muon", "count": 72, "rows": 9728, "cols": 64},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "fp8_fwd", "fp8_dx", "orth", "muon"])
    if op.startswith("norm"):
        c = {"op": op, "kind": rng.choice(["layer", "rms"]), "rows": _log(rng, 1, 4096), "dim": _log(rng, 32, 10240),
             "dtype": rng.choice(["f32", "bf16"])}
        c["rows"] = min(c["rows"], 4096 * 2560 // c["dim"])
        if op == "norm_bwd":
            c["grads"] = rng.randint(1, 3)
        return c
    if op.startswith("fp8"):
        c = {"op": op, "tokens": _log(rng, 1, 4096), "in_dim": _log(rng, 64, 9728, 8), "out_dim": _log(rng, 64, 9728, 8),
             "dtype": rng.choice(["f32", "bf16"])}
        c["tokens"] = max(1, min(c["tokens"], 4096 * 2560 * 9728 // (c["in_dim"] * c["out_dim"])))
        return c
    rank, side = _log(rng, 3, 128), _log(rng, 128, 9728)
    count = max(1, min(_log(rng, 1, 72), 72 * 9728 * 64 * 64 // (rank * rank * side)))
    rows, cols = (rank, side) if rng.random() < 0.5 else (side, rank)
    return {"op": op, "count": count, "rows": rows, "cols": cols}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _activations(g, rows, dim):
    """Rows of different sizes, with some wide columns, as hidden states have."""
    x = _rand(g, rows, dim) * torch.exp(0.5 * _rand(g, rows, 1))
    return x * torch.exp(0.7 * _rand(g, dim)) + 0.1 * _rand(g, dim)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        rows, dim = case["rows"], case["dim"]
        s = {"case": case, "eps": 1e-6 if case["kind"] == "rms" else 1e-5,
             "x": _activations(g, rows, dim).to(_type(case)), "gamma": 1 + 0.2 * _rand(g, dim),
             "beta": 0.1 * _rand(g, dim) if case["kind"] == "layer" else None}
        if op == "norm_bwd":
            s["dy"] = [(1e-2 * _rand(g, rows, dim)).to(_type(case)) for _ in range(case["grads"])]
            x = s["x"].double()
            mean = x.mean(1) if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
            var = (x - mean[:, None]).square().mean(1)
            s["stats"] = torch.stack([mean, (var + s["eps"]).rsqrt()], 1).float()
        return s
    if op in ("fp8_fwd", "fp8_dx"):
        t, k, n = case["tokens"], case["in_dim"], case["out_dim"]
        # e4m3 values with zeros up to whole 128 x 128 blocks, then the scales,
        # in one buffer: what a program keeps of a frozen 8-bit weight.
        nb, kb = -(-n // 128), -(-k // 128)
        w = torch.zeros(nb * 128, kb * 128, device="cuda")
        w[:n, :k] = 0.02 * _rand(g, n, k) * torch.exp(0.3 * _rand(g, n, 1))
        tiles = w.view(nb, 128, kb, 128)
        scale = tiles.abs().amax((1, 3)) / 448
        q = (tiles / scale[:, None, :, None]).view(nb * 128, kb * 128).to(torch.float8_e4m3fn)
        buf = torch.cat([q.view(torch.uint8).flatten(), scale.flatten().view(torch.uint8)])
        x = _activations(g, t, k) if op == "fp8_fwd" else 1e-2 * torch.exp(0.5 * _rand(g, t, 1)) * _rand(g, t, n)
        return {"case": case, "x": x.to(_type(case)), "w": buf}
    # Gradients of a low-rank factor: a few strong directions over noise.
    b, m, n = case["count"], case["rows"], case["cols"]
    r = min(m, n)
    grad = 0.3 * _rand(g, b, m, n) + torch.bmm(_rand(g, b, m, max(1, r // 4)), _rand(g, b, max(1, r // 4), n))
    s = {"case": case, "g": 1e-3 * grad}
    if op == "muon":
        s["p"] = 0.02 * _rand(g, b, m, n)
        s["m"] = 5e-3 * _rand(g, b, m, n)
        s["scale"] = torch.full((1,), 0.5, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _norm_fwd(s):
    x = s["x"].float()
    layer = s["case"]["kind"] == "layer"
    mean = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + s["eps"])
    y = xc * rstd * s["gamma"]
    if layer:
        y = y + s["beta"]
    return y.to(s["x"].dtype), torch.cat([mean, rstd], 1)


def _norm_bwd(s):
    x, rstd = s["x"].float(), s["stats"][:, 1:]
    layer = s["case"]["kind"] == "layer"
    dy = torch.stack([d.float() for d in s["dy"]]).sum(0)
    xh = (x - s["stats"][:, :1]) * rstd
    gdy = dy * s["gamma"]
    dx = gdy - xh * (gdy * xh).mean(1, keepdim=True)
    if layer:
        dx = dx - gdy.mean(1, keepdim=True)
    return (dx * rstd).to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0) if layer else None


def _weight(s):
    """The frozen weight's values in float32."""
    k, n = s["case"]["in_dim"], s["case"]["out_dim"]
    nb, kb = -(-n // 128), -(-k // 128)
    q = s["w"][:nb * kb * 16384].view(torch.float8_e4m3fn).float().view(nb, 128, kb, 128)
    scale = s["w"][nb * kb * 16384:].view(torch.float32).view(nb, 1, kb, 1)
    return (q * scale).view(nb * 128, kb * 128)[:n, :k]


def _rounded(x):
    """x with each 128-wide block of a row rounded to e4m3 times the smallest
    power of two that holds the block's largest value."""
    t, k = x.shape
    b = torch.nn.functional.pad(x, (0, -k % 128)).view(t, -1, 128)
    frac, exp = torch.frexp(b.abs().amax(2, keepdim=True))
    exp = torch.where(frac > 0.875, exp - 8, exp - 9).clamp(-127, 127)
    q = torch.ldexp(b, -exp).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, exp).view(t, -1)[:, :k]


def _fp8(s):
    w = _weight(s)
    y = torch.matmul(_rounded(s["x"].float()), w.t() if s["case"]["op"] == "fp8_fwd" else w)
    return y.to(torch.bfloat16)


def _ns_step(x):
    gram = torch.bmm(x, x.transpose(1, 2))
    return NS[0] * x + torch.bmm(NS[1] * gram + NS[2] * torch.bmm(gram, gram), x)


def _orth(u):
    wide = u.shape[1] <= u.shape[2]
    x = u if wide else u.transpose(1, 2).contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    x = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(x)))))
    return x if wide else x.transpose(1, 2).contiguous()


def _factor(case):
    return math.sqrt(max(1.0, case["rows"] / case["cols"]))


def _muon(s):
    g = s["g"] * s["scale"]
    s["m"].copy_(MOMENTUM * s["m"] + g)
    update = _orth(g + MOMENTUM * s["m"])
    s["p"].copy_(s["p"] - LR * _factor(s["case"]) * update - LR * DECAY * s["p"])
    return s["p"], s["m"]


# ------------------------------------------------------ the framework's calls
def _own(s):
    from bwd_adamw_amd import lora as L

    case, op = s["case"], s["case"]["op"]
    if op in ("norm_fwd", "norm_bwd"):
        x = s["x"]
        nm = L.make_norm(case["kind"], case["rows"], case["dim"], x.dtype, s["eps"], s["gamma"], s["beta"])
        if op == "norm_fwd":
            y, stats = torch.empty_like(x), torch.empty(case["rows"], 2, device="cuda")
            L.lora_norm_forward(nm, x, y, stats)
            return y, stats
        dx, dgamma = torch.empty_like(x), torch.empty_like(s["gamma"])
        dbeta = torch.empty_like(s["beta"]) if s["beta"] is not None else None
        L.lora_norm_backward(nm, x, s["dy"], s["stats"], dx, dgamma, dbeta)
        return dx, dgamma, dbeta
    if op in ("fp8_fwd", "fp8_dx"):
        w = L.Fp8Weight(case["out_dim"], case["in_dim"], s["w"])
        q = L.fp8_rows(*s["x"].shape)
        L.lora_fp8_quantize(s["x"], q)
        y = torch.empty(case["tokens"], case["out_dim"] if op == "fp8_fwd" else case["in_dim"], device="cuda", dtype=torch.bfloat16)
        L.lora_fp8_product(q, w, y, dx=op == "fp8_dx")
        return y
    runs = [L.make_matrix_run(0, case["rows"], case["cols"], case["count"])]
    hp = L.make_muon(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, eps=NS_EPS, coeffs=NS, steps=5)
    if op == "orth":
        out = torch.empty_like(s["g"])
        L.lora_orthogonalize(s["g"], out, runs, hp)
        return out
    L.lora_muon_step(s["p"], s["g"], s["m"], runs, hp, s["scale"])
    return s["p"], s["m"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm_fwd":
        return _norm_fwd(state)
    if op == "norm_bwd":
        return _norm_bwd(state)
    if op in ("fp8_fwd", "fp8_dx"):
        return _fp8(state)
    return _orth(state["g"]) if op == "orth" else _muon(state)


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        rows, dim, e = case["rows"], case["dim"], 2 if case["dtype"] == "bf16" else 4
        vectors = 4 * dim * (2 if case["kind"] == "layer" else 1)
        if op == "norm_fwd":
            return {"bytes": 2 * e * rows * dim + 8 * rows + vectors, "flops": 8 * rows * dim}
        return {"bytes": (2 + case["grads"]) * e * rows * dim + 8 * rows + vectors + 4 * dim, "flops": 14 * rows * dim}
    if op in ("fp8_fwd", "fp8_dx"):
        t, k, n = case["tokens"], case["in_dim"], case["out_dim"]
        rd, wr = (k, n) if op == "fp8_fwd" else (n, k)
        scales = 4 * -(-k // 128) * -(-n // 128)
        return {"bytes": (2 if case["dtype"] == "bf16" else 4) * t * rd + k * n + scales + 2 * t * wr, "flops": 2 * t * k * n}
    size, r = case["count"] * case["rows"] * case["cols"], min(case["rows"], case["cols"])
    # Two products with the matrix (its Gram matrix, half of it by symmetry,
    # and the polynomial times it) and the polynomial's small ones.
    flops = 3 * r * size + case["count"] * 5 * 4 * r ** 3
    return {"bytes": 4 * size * (2 if op == "orth" else 5), "flops": flops}


# ------------------------------------------------------------ in 64 bits
def _exact_norm(case, s):
    x, gamma = s["x"].double(), s["gamma"].double()
    layer = case["kind"] == "layer"
    if case["op"] == "norm_fwd":
        mean = x.sum(1) / case["dim"] if layer else torch.zeros(case["rows"], device=x.device, dtype=x.dtype)
        second = (x * x).sum(1) / case["dim"]
        var = second - mean * mean
        rstd = (var + s["eps"]) ** -0.5
        y = (x - mean[:, None]) * (rstd[:, None] * gamma)
        return (y + s["beta"].double() if layer else y), torch.stack([mean, rstd], 1)
    mean, rstd = s["stats"].double().unbind(1)
    dy = sum(d.double() for d in s["dy"])
    xhat = (x - mean[:, None]) * rstd[:, None]
    dxhat = dy * gamma
    along = (dxhat * xhat).sum(1) / case["dim"]
    level = dxhat.sum(1) / case["dim"] if layer else torch.zeros_like(along)
    dx = rstd[:, None] * (dxhat - level[:, None] - xhat * along[:, None])
    return dx, torch.einsum("td,td->d", dy, xhat), dy.sum(0) if layer else None


def _exact_fp8(case, s):
    k, n = case["in_dim"], case["out_dim"]
    nb, kb = -(-n // 128), -(-k // 128)
    values, scales = s["w"][:nb * kb * 16384], s["w"][nb * kb * 16384:]
    w = values.view(torch.float8_e4m3fn).double().view(nb * 128, kb * 128)
    w = w * scales.view(torch.float32).double().view(nb, kb).repeat_interleave(128, 0).repeat_interleave(128, 1)
    x = s["x"].double()
    rows, cols = x.shape
    pad = torch.zeros(rows, -(-cols // 128) * 128, device=x.device, dtype=x.dtype)
    pad[:, :cols] = x
    blocks = pad.view(rows, -1, 128)
    top = blocks.abs().amax(2, keepdim=True)
    power = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
    power = power + (top > 448 * torch.exp2(power)).double() - (top <= 448 * torch.exp2(power - 1)).double()
    scale = torch.exp2(power.clamp(-127, 127))
    v = blocks / scale
    # e4m3: three bits after the leading one, down to steps of 2^-9.
    octave = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(octave.clamp_min(-6) - 3)
    rounded = torch.round(v / step) * step * scale
    rounded = rounded.view(rows, -1)[:, :cols].contiguous()
    return rounded @ (w[:n, :k].t().contiguous() if case["op"] == "fp8_fwd" else w[:n, :k].contiguous())


def _exact_orth(u):
    b, m, n = u.shape
    x = u if m <= n else u.transpose(1, 2)
    x = (x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + NS_EPS)).contiguous()
    a, b2, c = NS
    eye = torch.eye(min(m, n), device=u.device, dtype=u.dtype)
    for _ in range(5):
        gram = x @ x.transpose(1, 2).contiguous()
        x = (a * eye + b2 * gram + c * (gram @ gram)) @ x
    return x if m <= n else x.transpose(1, 2).contiguous()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s)
    if op in ("fp8_fwd", "fp8_dx"):
        return _exact_fp8(case, s)
    if op == "orth":
        return _exact_orth(s["g"].double())
    g = s["g"].double() * s["scale"].double()
    m = MOMENTUM * s["m"].double() + g
    o = _exact_orth(g + MOMENTUM * m)
    p = s["p"].double()
    return p * (1 - LR * DECAY) - LR * max(1.0, case["rows"] / case["cols"]) ** 0.5 * o, m
