"""Cases of the operators between a layer's projections: the norm and rotation
of query and key heads, and causal attention over packed sequences.

  heads_fwd  y = rot(x rstd gamma) for each head of queries and of keys, rstd
             of the head's own values (or no norm), rot by the token's position
  heads_bwd  dx and dgamma of the same
  attn_fwd   o = softmax(scale q k^T) v in each sequence, with the log-sum of
             every row; a row sees the keys up to its own, several query heads
             share a key head, keys may reach back before the queries
  attn_bwd   dq, dk and dv from do, with o and the log-sums of the forward

`own` selects the calls of the framework's kernels; otherwise `run` computes
the operators from elementary torch operations in 32 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # A decoded token's queries and keys: nothing but latency.
        {"name": "heads fwd 1x(32+8)x128", "op": "heads_fwd", "tokens": 1, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "norm": True, "interleaved": False, "x": "bf16", "y": "bf16", "start": 30011},
        # wq's and wk's outputs in a Qwen3-4B-shaped layer, one chunk, rounded for the attention.
        {"name": "heads fwd 4096x(32+8)x128", "op": "heads_fwd", "tokens": 4096, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "norm": True, "interleaved": False, "x": "f32", "y": "bf16", "start": 0},
        # TinyLlama-shaped heads, an odd number of tokens, neighbours rotated, no norm.
        {"name": "heads fwd 1537x(32+4)x64", "op": "heads_fwd", "tokens": 1537, "heads": 32, "kv_heads": 4, "head_dim": 64,
         "norm": False, "interleaved": True, "x": "bf16", "y": "bf16", "start": 500},
        # The gradients of wq's and wk's outputs and of both gammas, a chunk of the two-slot workload.
        {"name": "heads bwd 2048x(32+8)x128", "op": "heads_bwd", "tokens": 2048, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "norm": True, "interleaved": False, "x": "f32", "y": "f32", "start": 0},
        # The TinyLlama-shaped step's four chunks of 128 tokens, float32.
        {"name": "attn fwd 4x128 32/4x64 f32", "op": "attn_fwd", "tokens": 512, "seqs": 4, "even": True, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 4, "head_dim": 64, "dtype": "f32"},
        # One new token of 32 requests over their caches, 8 to 4096 keys long.
        {"name": "attn fwd 32x1 over 4096", "op": "attn_fwd", "tokens": 32, "seqs": 32, "even": True, "prefix": 4095, "capacity": 4096,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16"},
        # One chunk of a Qwen3-4B-shaped layer as a single sequence.
        {"name": "attn fwd 4096 32/8x128", "op": "attn_fwd", "tokens": 4096, "seqs": 1, "even": True, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16"},
        # A packed batch of conversations of different lengths.
        {"name": "attn fwd 9 in 4001 32/8x128", "op": "attn_fwd", "tokens": 4001, "seqs": 9, "even": False, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16"},
        # A long prompt.
        {"name": "attn fwd 8192 32/8x128", "op": "attn_fwd", "tokens": 8192, "seqs": 1, "even": True, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16"},
        # A chunk of the two-slot workload.
        {"name": "attn bwd 2048 32/8x128", "op": "attn_bwd", "tokens": 2048, "seqs": 1, "even": True, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16"},
        # A packed batch through TinyLlama-shaped heads.
        {"name": "attn bwd 7 in 4001 32/4x64", "op": "attn_bwd", "tokens": 4001, "seqs": 7, "even": False, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 4, "head_dim": 64, "dtype": "bf16"},
        # The TinyLlama-shaped step's backward, float32.
        {"name": "attn bwd 4x128 32/4x64 f32", "op": "attn_bwd", "tokens": 512, "seqs": 4, "even": True, "prefix": 0, "capacity": 0,
         "heads": 32, "kv_heads": 4, "head_dim": 64, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["heads_fwd", "heads_bwd", "attn_fwd", "attn_fwd", "attn_bwd"])
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 16), (12, 4), (8, 1)])
    c = {"op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": rng.choice([64, 80, 128])}
    if op.startswith("heads"):
        x = rng.choice(["f32", "bf16"])
        c |= {"tokens": _log(rng, 1, 4096 if op == "heads_fwd" else 2048), "norm": rng.random() < 0.7,
              "interleaved": rng.random() < 0.3, "x": x, "y": rng.choice([x, "bf16"]), "start": rng.choice([0, _log(rng, 1, 40000)])}
        return c
    c["dtype"] = "f32" if rng.random() < 0.25 else "bf16"
    if op == "attn_fwd" and rng.random() < 0.3:
        # A few new tokens of several requests over their caches.
        seqs = _log(rng, 1, 32)
        new, prefix = rng.choice([1, 1, rng.randint(2, 5)]), _log(rng, 1, 4000)
        return c | {"tokens": seqs * new, "seqs": seqs, "even": True, "prefix": prefix, "capacity": prefix + new}
    most = 1024 if c["dtype"] == "f32" else 8192 if op == "attn_fwd" else 4096
    tokens = _log(rng, 1, most)
    seqs = min(tokens, _log(rng, 1, 16))
    return c | {"tokens": tokens, "seqs": seqs, "even": tokens % seqs == 0,
                "prefix": rng.randint(1, 1024) if rng.random() < 0.3 and seqs < 4 else 0, "capacity": 0}


def _lengths(case):
    """Queries and keys of each sequence."""
    n, tokens = case["seqs"], case["tokens"]
    rng = random.Random(tokens * 1000 + n)
    if case["even"]:
        lq = [tokens // n] * n
    else:
        cuts = sorted(rng.sample(range(1, tokens), n - 1))
        lq = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    if case["capacity"]:   # caches filled to different lengths, the last one whole
        back = [rng.randint(min(8, case["prefix"]), case["prefix"]) for _ in range(n - 1)] + [case["prefix"]]
    else:
        back = [case["prefix"]] * n
    return lq, [a + b for a, b in zip(lq, back)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _offsets(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    if op.startswith("heads"):
        t = case["tokens"]
        s = {"case": case, "x": [], "gamma": [], "positions": torch.arange(case["start"], case["start"] + t, device="cuda").int(),
             "freqs": 1e6 ** (-torch.arange(0, d, 2, device="cuda").double() / d)}
        for n in (h, kv):
            x = _rand(g, t, n, d) * torch.exp(0.5 * _rand(g, t, 1, 1)) * torch.exp(0.5 * _rand(g, 1, n, d))
            s["x"].append(x.view(t, n * d).to(_type(case["x"])))
            s["gamma"].append(1 + 0.2 * _rand(g, d) if case["norm"] else None)
        if op == "heads_bwd":
            s["dy"] = [(1e-2 * _rand(g, t, n * d)).to(_type(case["y"])) for n in (h, kv)]
        return s
    lq, lk = _lengths(case)
    dt, tq = _type(case["dtype"]), sum(lq)
    qo = _offsets(lq)
    if case["capacity"]:
        ko = torch.arange(len(lq) + 1, device="cuda").int() * case["capacity"]
        lens, tk = torch.tensor(lk, device="cuda").int(), len(lq) * case["capacity"]
    else:
        ko, lens, tk = _offsets(lk), None, sum(lk)
    # Normed heads with a common direction, so that some keys take much of a row.
    along = _rand(g, 1, kv, 1, d)
    q = _unit(_rand(g, tq, kv, h // kv, d) + 0.5 * along).view(tq, h, d) * (1.3 + 0.2 * _rand(g, d))
    k = _unit(_rand(g, tk, kv, d) + 0.5 * _rand(g, tk, 1, 1) * along[:, :, 0]) * (1.3 + 0.2 * _rand(g, d))
    v = _rand(g, tk, kv, d) * torch.exp(0.3 * _rand(g, tk, 1, 1))
    s = {"case": case, "q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "scale": d ** -0.5, "q_offsets": qo, "k_offsets": ko,
         "k_lens": lens, "max_q": max(lq), "max_k": max(lk)}
    if op == "attn_bwd":
        s["o"], s["lse"] = _attend(s)
        s["do"] = (1e-2 * _rand(g, tq, h, d)).to(dt)
    return s


# ------------------------------------------------------------- plain forms
def _angles(s):
    phi = s["positions"].double()[:, None] * s["freqs"]
    return torch.cos(phi).float()[:, None], torch.sin(phi).float()[:, None]


def _pairs(case, z):
    return (z[..., 0::2], z[..., 1::2]) if case["interleaved"] else z.chunk(2, -1)


def _joined(case, a, b):
    return torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)


def _heads_fwd(s, x, gamma):
    case = s["case"]
    cos, sin = _angles(s)
    z = x.float().view(x.shape[0], -1, case["head_dim"])
    if gamma is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS) * gamma
    a, b = _pairs(case, z)
    return _joined(case, a * cos - b * sin, b * cos + a * sin).flatten(1).to(_type(case["y"]))


def _heads_bwd(s, x, gamma, dy):
    case = s["case"]
    cos, sin = _angles(s)
    x = x.float().view(x.shape[0], -1, case["head_dim"])
    a, b = _pairs(case, dy.float().view(x.shape))
    dz = _joined(case, a * cos + b * sin, b * cos - a * sin)
    if gamma is None:
        return dz.flatten(1).to(_type(case["x"])), None
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh, gz = x * rstd, dz * gamma
    dx = rstd * (gz - xh * (gz * xh).mean(-1, keepdim=True))
    return dx.flatten(1).to(_type(case["x"])), (dz * xh).sum((0, 1))


def _rows(offsets, lens, most):
    """Row numbers [sequences, most] of a padded batch, and which are there."""
    at = torch.arange(most, device=offsets.device)
    there = at < lens[:, None]
    return torch.where(there, offsets[:-1, None] + at, 0), there


def _padded(s):
    """q [B, KV, G maxq, D], k and v [B, KV, maxk, D] in float32, the mask
    [B, 1, 1, maxq, maxk], and the rows of the padded batch."""
    h, kv, d = s["case"]["heads"], s["case"]["kv_heads"], s["case"]["head_dim"]
    qo, ko = s["q_offsets"].long(), s["k_offsets"].long()
    lq = qo.diff()
    lk = ko.diff() if s["k_lens"] is None else s["k_lens"].long()
    qr, qin = _rows(qo, lq, s["max_q"])
    kr, kin = _rows(ko, lk, s["max_k"])
    q = s["q"].float()[qr].view(len(lq), -1, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(len(lq), kv, -1, d)
    k, v = (s[n].float()[kr].transpose(1, 2).contiguous() for n in "kv")
    i, j = torch.arange(s["max_q"], device=lq.device), torch.arange(s["max_k"], device=lq.device)
    sees = (j <= i[:, None] + (lk - lq)[:, None, None]) & kin[:, None] & qin[:, :, None]
    return q, k, v, sees[:, None, None], (qr, qin, kr, kin)


def _scores(s, q, k, sees):
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    b, kv = x.shape[:2]
    return x.view(b, kv, -1, s["max_q"], s["max_k"]).masked_fill_(~sees, -math.inf)


def _unpadded(x, there):
    """[B, KV, N maxq, ...] of a padded batch to [rows, KV N, ...] of its sequences."""
    b, kv, most = x.shape[0], x.shape[1], there.shape[1]
    x = x.reshape(b, kv, -1, most, *x.shape[3:]).flatten(1, 2).transpose(1, 2)
    return x[there]


def _attend(s):
    q, k, v, sees, (_, qin, _, _) = _padded(s)
    x = _scores(s, q, k, sees)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / total.clamp_min(1e-30)).flatten(2, 3), v)
    lse = _unpadded((top + torch.log(total)).flatten(2, 3), qin)[..., 0].t().contiguous()
    return _unpadded(o, qin).to(s["q"].dtype), lse


def _attn_bwd(s):
    q, k, v, sees, (qr, qin, _, kin) = _padded(s)
    h, kv, d = s["case"]["heads"], s["case"]["kv_heads"], s["case"]["head_dim"]
    b, dt = q.shape[0], s["q"].dtype
    group = lambda t: t[qr].view(b, -1, kv, h // kv, t.shape[2]).permute(0, 2, 3, 1, 4)
    lse = group(s["lse"].t()[..., None])
    do = group(s["do"].float())
    delta = (do * group(s["o"].float())).sum(-1, keepdim=True)
    p = torch.exp(_scores(s, q, k, sees) - lse)
    do = do.reshape(q.shape)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous()).view(p.shape)
    ds = (p * (dp - delta)).flatten(2, 3) * s["scale"]
    dv = torch.matmul(p.flatten(2, 3).transpose(2, 3).contiguous(), do)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    dq = torch.matmul(ds, k)
    keys = lambda t: t.transpose(1, 2)[kin].to(dt)
    return _unpadded(dq, qin).to(dt), keys(dk), keys(dv)


# ------------------------------------------------------ the framework's calls
def _own(s):
    from bwd_adamw_amd import lora as L

    case, op = s["case"], s["case"]["op"]
    if op.startswith("heads"):
        both = [L.make_heads(case["tokens"], n, case["head_dim"], _type(case["x"]), _type(case["y"]), norm=case["norm"], eps=EPS,
                             gamma=g, freqs=s["freqs"], interleaved=case["interleaved"])
                for n, g in zip((case["heads"], case["kv_heads"]), s["gamma"])]
        if op == "heads_fwd":
            y = [torch.empty(x.shape, device="cuda", dtype=_type(case["y"])) for x in s["x"]]
            L.lora_heads_forward(both, s["x"], y, s["positions"])
            return y
        dx = [torch.empty_like(x) for x in s["x"]]
        dg = [None if g is None else torch.empty_like(g) for g in s["gamma"]]
        L.lora_heads_backward(both, s["x"], s["dy"], dx, dg, s["positions"])
        return [(dx[0], dg[0]), (dx[1], dg[1])]
    q, k, v = s["q"], s["k"], s["v"]
    at = L.make_attention(q.shape[0], k.shape[0], case["heads"], case["kv_heads"], case["head_dim"], s["q_offsets"], s["k_offsets"],
                          k_lens=s["k_lens"], dtype=q.dtype, scale=s["scale"], causal=True)
    if op == "attn_fwd":
        o, lse = torch.empty_like(q), torch.empty(case["heads"], q.shape[0], device="cuda")
        L.lora_attention_forward(at, q, k, v, o, lse)
        return o, lse
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    L.lora_attention_backward(at, q, k, v, s["o"], s["do"], s["lse"], dq, dk, dv)
    return dq, dk, dv


def run(state):
    if own:
        return _own(state)
    s, op = state, state["case"]["op"]
    if op == "heads_fwd":
        return [_heads_fwd(s, s["x"][0], s["gamma"][0]), _heads_fwd(s, s["x"][1], s["gamma"][1])]
    if op == "heads_bwd":
        return [_heads_bwd(s, s["x"][0], s["gamma"][0], s["dy"][0]), _heads_bwd(s, s["x"][1], s["gamma"][1], s["dy"][1])]
    return _attend(s) if op == "attn_fwd" else _attn_bwd(s)


def work(case):
    op, h, kv, d = case["op"], case["heads"], case["kv_heads"], case["head_dim"]
    size = lambda n: 2 if n == "bf16" else 4
    if op.startswith("heads"):
        n = case["tokens"] * (h + kv) * d
        if op == "heads_fwd":
            return {"bytes": n * (size(case["x"]) + size(case["y"])) + 4 * case["tokens"], "flops": 8 * n}
        return {"bytes": n * (2 * size(case["x"]) + size(case["y"])) + 4 * case["tokens"], "flops": 16 * n}
    lq, lk = _lengths(case)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
    e, tq, tk = size(case["dtype"]), sum(lq), sum(lk)
    rows, keys = e * tq * h * d, e * tk * kv * d
    if op == "attn_fwd":
        return {"bytes": 2 * rows + 2 * keys + 4 * h * tq, "flops": 4 * d * h * pairs}
    return {"bytes": 4 * rows + 4 * keys + 4 * h * tq, "flops": 10 * d * h * pairs}


# ------------------------------------------------------------ in 64 bits
def _turned(case, z, phi):
    """Rotation of the last axis of z by phi, as complex products."""
    half = case["head_dim"] // 2
    pair = z.unflatten(-1, (half, 2)) if case["interleaved"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
    w = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(phi), phi)[:, None]
    w = torch.view_as_real(w)
    return (w if case["interleaved"] else w.transpose(-1, -2)).flatten(-2)


def _exact_heads(case, s):
    phi, out = torch.outer(s["positions"].double(), s["freqs"]), []
    for n in range(2):
        x = s["x"][n].double().unflatten(1, (-1, case["head_dim"]))
        gamma = s["gamma"][n].double() if case["norm"] else None
        rstd = (x.square().sum(-1, keepdim=True) / case["head_dim"] + EPS) ** -0.5
        if case["op"] == "heads_fwd":
            out.append(_turned(case, x if gamma is None else x * rstd * gamma, phi).flatten(1))
            continue
        dz = _turned(case, s["dy"][n].double().view(x.shape), -phi)
        if gamma is None:
            out.append((dz.flatten(1), None))
            continue
        along = (dz * gamma * x).sum(-1, keepdim=True) / case["head_dim"]
        dx = rstd * dz * gamma - rstd ** 3 * x * along
        out.append((dx.flatten(1), torch.einsum("thd,thd->d", dz, x * rstd)))
    return out


def _exact_attn(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    lq, lk = _lengths(case)
    group, fwd = h // kv, case["op"] == "attn_fwd"
    qo, ko = s["q_offsets"].tolist(), s["k_offsets"].tolist()
    full = lambda like: torch.zeros(like.shape, device=like.device, dtype=torch.float64)
    if fwd:
        o, lse = full(s["q"]), torch.zeros(h, s["q"].shape[0], device="cuda", dtype=torch.float64)
    else:
        dq, dk, dv = full(s["q"]), full(s["k"]), full(s["v"])
    for b, (m, n) in enumerate(zip(lq, lk)):
        hidden = torch.ones(m, n, device="cuda", dtype=torch.bool).triu(n - m + 1)
        for a in range(h):
            qs, ks = slice(qo[b], qo[b] + m), slice(ko[b], ko[b] + n)
            q, k, v = s["q"][qs, a].double(), s["k"][ks, a // group].double(), s["v"][ks, a // group].double()
            x = s["scale"] * (q @ k.t().contiguous())
            x[hidden] = -math.inf
            if fwd:
                lse[a, qs] = torch.logsumexp(x, 1)
                o[qs, a] = torch.softmax(x, 1) @ v
                continue
            p = torch.exp(x - s["lse"][a, qs].double()[:, None])
            do = s["do"][qs, a].double()
            dp = do @ v.t().contiguous() - (do * s["o"][qs, a].double()).sum(1, keepdim=True)
            ds = s["scale"] * p * dp
            dq[qs, a] = ds @ k
            dk[ks, a // group] += ds.t().contiguous() @ q
            dv[ks, a // group] += p.t().contiguous() @ do
    return (o, lse) if fwd else (dq, dk, dv)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_heads(case, s) if case["op"].startswith("heads") else _exact_attn(case, s)
