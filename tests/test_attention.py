"""Attention over packed sequences, forward and backward, against the formulas
in float64.

Tolerances, beside the reference: every operation's rounding (2^-24 of its
result) is carried through to the outputs with magnitudes in place of values.
A score's sum of D products is off by (D + 8) 2^-24 of its magnitudes, and so
is its exponential, in relative terms, with two steps of the hardware's exp2
and the roundings of s c - max (2^-23 of both); sums over n keys or rows add
(n + 16) 2^-24 of their magnitudes; bf16 operands p and ds add half a step, 2^-8,
of their own magnitudes, as does a float32 dO rounded to bf16; bf16 results add
2^-8 of their value."""

import ctypes as C
import math

import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"
gpu = pytest.mark.gpu
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder-pointer tests run only on GPU-less hosts")
STEP, HALF = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16


def sees(lq, lk, causal):
    j = torch.arange(lk)
    i = torch.arange(lq)[:, None]
    return (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)


def forward_ref(q, k, v, qo, ko, lens, causal, scale, dtype=torch.float64):
    """o, its tolerance before rounding, lse and its tolerance; q [T, H, D] ..."""
    H, KV, D = q.shape[1], k.shape[1], q.shape[2]
    q, k, v = q.double(), k.double(), v.double()
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse, ltol = torch.full((H, q.shape[0]), -math.inf, dtype=torch.float64), torch.zeros(H, q.shape[0], dtype=torch.float64)
    half = HALF if dtype == BF16 else 0.0
    for b in range(len(qo) - 1):
        qs = slice(qo[b], qo[b + 1])
        n = ko[b + 1] - ko[b] if lens is None else lens[b]
        ks = slice(ko[b], ko[b] + n)
        if qo[b + 1] == qo[b] or n == 0:
            continue
        ok = sees(qo[b + 1] - qo[b], n, causal)
        for h in range(H):
            g = h // (H // KV)
            s = scale * (q[qs, h] @ k[ks, g].T)
            mag = scale * (q[qs, h].abs() @ k[ks, g].abs().T)
            s = s.masked_fill(~ok, -math.inf)
            top = s.amax(1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            p = torch.exp(s - top)
            total = p.sum(1, keepdim=True)
            w = torch.where(total > 0, p / total, 0.0)
            off = (D + 8) * STEP * mag.masked_fill(~ok, 0).amax(1, keepdim=True) * 2 + 2.0 ** -21 + \
                2.0 ** -22 * top.abs()
            o[qs, h] = w @ v[ks, g]
            tol[qs, h] = (off + (n + 16) * STEP + half) * (w @ v[ks, g].abs()) * 2
            lse[h, qs] = (top + torch.log(total))[:, 0]
            ltol[h, qs] = (off + (n + 16) * STEP)[:, 0] + 4 * STEP * lse[h, qs].abs().nan_to_num(0, 0, 0)
    return o, tol, lse, ltol


def backward_ref(q, k, v, o, do, lse, qo, ko, lens, causal, scale, dtype, do_rounded):
    """(dq, tol), (dk, tol), (dv, tol) for the given o and lse."""
    H, KV, D = q.shape[1], k.shape[1], q.shape[2]
    q, k, v, o, do, lse = (t.double() for t in (q, k, v, o, do, lse))
    zero = lambda t: [torch.zeros_like(t), torch.zeros_like(t)]
    dq, dk, dv = zero(q), zero(k), zero(v)
    half = HALF if dtype == BF16 else 0.0
    dhalf = HALF if do_rounded else 0.0
    for b in range(len(qo) - 1):
        qs = slice(qo[b], qo[b + 1])
        m = qo[b + 1] - qo[b]
        n = ko[b + 1] - ko[b] if lens is None else lens[b]
        ks = slice(ko[b], ko[b] + n)
        if m == 0 or n == 0:
            continue
        ok = sees(m, n, causal)
        for h in range(H):
            g = h // (H // KV)
            s = scale * (q[qs, h] @ k[ks, g].T)
            mag = scale * (q[qs, h].abs() @ k[ks, g].abs().T)
            row = torch.where(lse[h, qs] == -math.inf, 0.0, lse[h, qs])[:, None]
            p = torch.where(ok, torch.exp(s - row), 0.0)
            poff = (D + 8) * STEP * mag + 2.0 ** -21 + 2.0 ** -22 * (row.abs() + s.abs())
            dp, dpm = do[qs, h] @ v[ks, g].T, do[qs, h].abs() @ v[ks, g].abs().T
            delta = (do[qs, h] * o[qs, h]).sum(1, keepdim=True)
            dem = (do[qs, h] * o[qs, h]).abs().sum(1, keepdim=True)
            ds = p * (dp - delta)
            dsoff = poff * ds.abs() + p * (((D + 8) * STEP + dhalf) * dpm + (D + 8) * STEP * dem) + half * ds.abs()
            dq[0][qs, h] = scale * (ds @ k[ks, g])
            dq[1][qs, h] = scale * 2 * (dsoff @ k[ks, g].abs() + (n + 16) * STEP * (ds.abs() @ k[ks, g].abs()))
            rows = (m + 16) * STEP * (H // KV)
            dk[0][ks, g] += scale * (ds.T @ q[qs, h])
            dk[1][ks, g] += scale * 2 * (dsoff.T @ q[qs, h].abs() + rows * (ds.abs().T @ q[qs, h].abs()))
            dv[0][ks, g] += p.T @ do[qs, h]
            dv[1][ks, g] += 2 * ((p * (poff + half + dhalf)).T @ do[qs, h].abs() + rows * (p.T @ do[qs, h].abs()))
    return dq, dk, dv


def close(got, ref, tol, dtype, what):
    got = got.detach().cpu().double()
    tol = tol + (HALF * (ref.abs() + tol) if dtype == BF16 else STEP * ref.abs()) + 1e-30
    err = (got - ref).abs()
    err = torch.where(got == ref, 0.0, err)   # equal infinities
    assert (err <= tol).all(), (what, (err / tol).nan_to_num(1e9).max().item())


def offsets(lens, gap=0):
    out = [0]
    for n in lens:
        out.append(out[-1] + n + gap)
    return out


def data(tq, tk, H, KV, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(tq, H, D, generator=g) * 1.5
    k, v = torch.randn(tk, KV, D, generator=g) * 1.5, torch.randn(tk, KV, D, generator=g)
    return q.to(dtype), k.to(dtype), v.to(dtype), torch.randn(tq, H, D, generator=g)


def dints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def check(lq, lk, H, KV, D, causal, dtype, out, lens=None, tail=3, scale=None):
    """Forward and backward of sequences lq, lk (lens: keys used of each room),
    with `tail` rows behind the last one that nothing may touch."""
    scale = D ** -0.5 if scale is None else scale
    qo, ko = offsets(lq), offsets(lk)
    tq, tk = qo[-1] + tail, ko[-1] + tail
    q, k, v, do = data(tq, tk, H, KV, D, dtype, 17 * tq + tk + D + H)
    do = do.to(out)
    # outside the sequences: values that would show
    q[qo[-1]:], do[qo[-1]:] = math.nan, math.nan
    k[ko[-1]:], v[ko[-1]:] = math.nan, math.inf
    for b, n in enumerate(lens or []):
        k[ko[b] + n:ko[b + 1]], v[ko[b] + n:ko[b + 1]] = math.nan, math.nan
    dev = [t.to(DEV) for t in (q, k, v, do)]
    at = L.make_attention(tq, tk, H, KV, D, dints(qo), dints(ko), None if lens is None else dints(lens), dtype,
                          out, scale, causal)
    o = torch.full((tq, H, D), 77.0, device=DEV, dtype=out)
    lse = torch.full((H, tq), 77.0, device=DEV)
    print("forward", lq, lk, H, KV, D, causal, dtype, out, flush=True)
    L.lora_attention_forward(at, *dev[:3], o, lse)
    torch.cuda.synchronize()
    ro, otol, rlse, ltol = forward_ref(q, k, v, qo, ko, lens, causal, scale, dtype)
    rows = slice(0, qo[-1])
    close(o[rows], ro[rows], otol[rows], out, "o")
    close(lse[:, rows], rlse[:, rows], ltol[:, rows], F32, "lse")
    assert (o[qo[-1]:] == 77).all() and (lse[:, qo[-1]:] == 77).all()
    no_lse = torch.full_like(o, 77.0)
    L.lora_attention_forward(at, *dev[:3], no_lse)
    assert torch.equal(no_lse, o)
    # the backward on the reference's o and log-sums
    o0, lse0 = ro.to(out), rlse.float()
    dq, dk, dv = (torch.full(t.shape, 55.0, device=DEV, dtype=out) for t in (q, k, v))
    print("backward", flush=True)
    L.lora_attention_backward(at, *dev[:3], o0.to(DEV), dev[3], lse0.to(DEV), dq, dk, dv)
    torch.cuda.synchronize()
    refs = backward_ref(q, k, v, o0, do, lse0, qo, ko, lens, causal, scale, dtype, out == F32 and dtype == BF16)
    used = torch.zeros(tk, dtype=torch.bool)
    for b in range(len(lk)):
        used[ko[b]:ko[b] + (lk[b] if lens is None else lens[b])] = True
    for got, (ref, tol), there, what in ((dq, refs[0], torch.arange(tq) < qo[-1], "dq"), (dk, refs[1], used, "dk"),
                                         (dv, refs[2], used, "dv")):
        close(got[there.to(DEV)], ref[there], tol[there], out, what)
        assert (got[~there.to(DEV)] == 55).all()
    return at, dev, o, lse


def test_formula_against_differences():
    """The reference's dq, dk and dv against central differences."""
    qo, ko = [0, 3, 5], [0, 4, 9]
    q, k, v, do = (t.double() for t in data(5, 9, 4, 2, 6, torch.float64, 3))
    for causal in (True, False):
        f = lambda: float((forward_ref(q, k, v, qo, ko, None, causal, 0.4)[0] * do).sum())
        o, _, lse, _ = forward_ref(q, k, v, qo, ko, None, causal, 0.4)
        refs = backward_ref(q, k, v, o, do, lse, qo, ko, None, causal, 0.4, torch.float64, False)
        h = 1e-5
        for t, (grad, _) in ((q, refs[0]), (k, refs[1]), (v, refs[2])):
            flat, gf = t.view(-1), grad.reshape(-1)
            for i in range(0, flat.numel(), 3):
                keep = flat[i].item()
                flat[i] = keep + h
                up = f()
                flat[i] = keep - h
                down = f()
                flat[i] = keep
                # h^2 of the third derivative and 1e-15 / h of rounding
                assert abs((up - down) / (2 * h) - gf[i].item()) < 1e-7 * (1 + gf.abs().max().item())


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
CASES = [
    # queries, keys of each sequence; heads, key heads, head_dim
    ([1], [1], 1, 1, 8), ([1], [1], 4, 2, 64), ([1], [300], 8, 2, 128), ([1, 1, 1, 1], [5, 130, 64, 257], 4, 1, 64),
    ([33], [33], 2, 2, 64), ([130], [130], 4, 1, 128), ([257], [257], 3, 1, 40), ([64, 64], [64, 64], 8, 2, 128),
    ([7, 0, 50, 1], [7, 0, 50, 1], 4, 2, 80), ([5, 20], [0, 20], 2, 1, 64), ([0, 20], [31, 20], 2, 2, 128),
    ([40, 3], [16, 70], 6, 2, 64),            # more queries than keys: rows that see none
    ([31, 90], [131, 90], 4, 4, 96),          # keys that reach back before the queries
    ([2, 3, 4], [70, 200, 129], 12, 4, 128), ([100], [517], 16, 1, 128), ([600], [600], 2, 1, 64),
    ([1] * 70, [1 + i % 40 for i in range(70)], 2, 1, 32), ([150] * 3, [150] * 3, 7, 7, 24),
]


@gpu
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c).replace(" ", "")[:60])
def test_forward_and_backward(case, causal, dtype, out):
    check(*case, causal, dtype, out)


@gpu
@pytest.mark.parametrize("dtype,out", TYPES)
def test_caches_in_use_up_to_a_length(dtype, out):
    """Rooms of keys filled to different lengths; what lies behind a length
    (NaN here) is neither read into a result nor written."""
    check([1, 1, 2, 1], [100, 100, 100, 100], 8, 2, 128, True, dtype, out, lens=[37, 100, 2, 0])
    check([9, 30], [64, 200], 4, 4, 64, True, dtype, out, lens=[64, 129])


@gpu
def test_many_sequences():
    """More sequences than one round of the search over offsets takes."""
    lq = [(i * 7) % 3 for i in range(5000)]
    check(lq, lq, 1, 1, 8, True, BF16, BF16)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    """Scores far past where exp overflows, rows with one dominant key."""
    check([70], [70], 2, 1, 64, True, dtype, dtype, scale=40.0)


def run(at, q, k, v, do, shape_k, out):
    o, lse = torch.empty(q.shape, device=DEV, dtype=out), torch.empty(q.shape[1], q.shape[0], device=DEV)
    L.lora_attention_forward(at, q, k, v, o, lse)
    dq, dk, dv = torch.empty_like(o), torch.empty(shape_k, device=DEV, dtype=out), torch.empty(shape_k, device=DEV, dtype=out)
    L.lora_attention_backward(at, q, k, v, o, do, lse, dq, dk, dv)
    return o, lse, dq, dk, dv


@gpu
def test_non_finite_rows_stay_in_their_sequence():
    q, k, v, do = (t.to(DEV) for t in data(90, 90, 4, 2, 64, BF16, 5))
    do = do.bfloat16()
    at = L.make_attention(90, 90, 4, 2, 64, dints([0, 30, 60, 90]), dints([0, 30, 60, 90]))
    clean = run(at, q, k, v, do, k.shape, BF16)
    for t in (q, k, v, do):
        t[35], t[40] = math.nan, math.inf
    bad = run(at, q, k, v, do, k.shape, BF16)
    for a, b in zip(clean, bad):
        a, b = (a.T, b.T) if a.dim() == 2 else (a, b)
        assert torch.equal(a[:30], b[:30]) and torch.equal(a[60:], b[60:])
    assert bad[0][41:60].isnan().any()


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    """[heads, tokens, dim] tensors, and heads inside wider rows: bitwise the
    plain layout's results, and nothing else written."""
    H, KV, D, T = 6, 2, 64, 75
    q, k, v, do = (t.to(DEV) for t in data(T, T, H, KV, D, dtype, 9))
    do = do.to(dtype)
    off = dints([0, 20, 75])
    at = L.make_attention(T, T, H, KV, D, off, off, dtype=dtype)
    ref = run(at, q, k, v, do, k.shape, dtype)
    swapped = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    room = torch.full((T, (H + 2 * KV) * D + 16), 3.0, device=DEV, dtype=dtype)
    ld = room.shape[1]
    qw, kw, vw = (room[:, a * D:b * D].view(T, -1, D) for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
    for dst, src in ((qw, q), (kw, k), (vw, v)):
        dst.copy_(src)
    for st, ten in (((T, D), [swapped(t) for t in (q, k, v)]), ((ld, D), [qw, kw, vw])):
        st = (D, T * D) if st == (T, D) else st
        kinds = dict(q_strides=st, k_strides=st, v_strides=st)
        at2 = L.make_attention(T, T, H, KV, D, off, off, dtype=dtype, o_strides=(D, T * D), **kinds)
        o = torch.empty(H, T, D, device=DEV, dtype=dtype).transpose(0, 1)
        lse = torch.empty(H, T, device=DEV)
        L.lora_attention_forward(at2, *ten, o, lse)
        grads = [torch.empty_strided(t.shape, t.stride(), device=DEV, dtype=dtype).fill_(1) for t in ten]
        L.lora_attention_backward(at2, *ten, o, swapped(do), lse, *grads)
        for a, b in zip(ref, (o, lse, *grads)):
            assert torch.equal(a, b)
    assert (room[:, -16:] == 3).all()


@gpu
def test_offsets_that_pass_32_bits():
    """Keys past 2^31 elements (4 GiB of bf16) into their buffer."""
    KV, D, T = 8, 128, 2_200_000
    k, v = (torch.empty(T, KV, D, device=DEV, dtype=BF16) for _ in range(2))
    q, ks, vs, do = data(40, 300, 8, KV, D, BF16, 4)
    k[T - 300:], v[T - 300:] = ks.to(DEV), vs.to(DEV)
    at = L.make_attention(40, T, 8, KV, D, dints([0, 40]), dints([T - 300, T]))
    near = L.make_attention(40, 300, 8, KV, D, dints([0, 40]), dints([0, 300]))
    far = [torch.empty(40, 8, D, device=DEV, dtype=BF16), torch.empty(8, 40, device=DEV)]
    qd, dod = q.to(DEV), do.bfloat16().to(DEV)
    L.lora_attention_forward(at, qd, k, v, *far)
    ref = run(near, qd, ks.to(DEV), vs.to(DEV), dod, ks.shape, BF16)
    for a, b in zip(ref, far):
        assert torch.allclose(a, b, rtol=2 * HALF, atol=2 * HALF)   # the keys may be split otherwise
    dq, dk, dv = torch.empty_like(qd), torch.empty_like(k), torch.empty_like(v)
    L.lora_attention_backward(at, qd, k, v, ref[0], dod, ref[1], dq, dk, dv)
    for a, b in zip(ref[2:], (dq, dk[T - 300:], dv[T - 300:])):
        assert torch.allclose(a, b, rtol=2 * HALF, atol=2 * HALF * a.abs().max().item())


@gpu
def test_offsets_outside_the_buffers_are_cut():
    q, k, v, do = (t.to(DEV) for t in data(50, 60, 2, 1, 64, BF16, 8))
    do = do.bfloat16()
    at = L.make_attention(50, 60, 2, 1, 64, dints([-5, 20, 500]), dints([-9, 30, 99999]))
    cut = L.make_attention(50, 60, 2, 1, 64, dints([0, 20, 50]), dints([0, 30, 60]))
    for a, b in zip(run(at, q, k, v, do, k.shape, BF16), run(cut, q, k, v, do, k.shape, BF16)):
        assert torch.equal(a, b)


@gpu
def test_twice_the_same_and_on_another_stream_and_replayed():
    """Equal inputs give bitwise equal outputs: again, on another stream (with
    workspaces of its own), and from a graph whose inputs change."""
    T, H, KV, D = 333, 8, 2, 128
    q, k, v, do = (t.to(DEV) for t in data(T, T, H, KV, D, BF16, 12))
    do = do.bfloat16()
    off = dints([0, 1, 130, T])
    at = L.make_attention(T, T, H, KV, D, off, off)
    ref = run(at, q, k, v, do, k.shape, BF16)
    assert all(torch.equal(a, b) for a, b in zip(ref, run(at, q, k, v, do, k.shape, BF16)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = run(at, q, k, v, do, k.shape, BF16)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    ws = [torch.empty(max(16, L.lora_attention_workspace_bytes(at, b)), device=DEV, dtype=torch.uint8) for b in (0, 1)]
    out = [torch.empty_like(t) for t in ref]

    def call():
        L.lora_attention_forward(at, q, k, v, out[0], out[1], ws=ws[0])
        L.lora_attention_backward(at, q, k, v, out[0], do, out[1], *out[2:], ws=ws[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    base = q.clone()
    for n in range(3):
        q.copy_(base * (1 + 0.25 * n))
        off.copy_(dints([[0, 1, 130, T], [0, 200, 201, T], [5, 5, 300, T]][n]))
        for t in out:
            t.zero_()
        call()
        torch.cuda.synchronize()
        eager = [t.clone() for t in out]
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))


def _at(**kw):
    d = dict(q_tokens=8, k_tokens=8, heads=4, kv_heads=2, head_dim=64, seqs=2, ldq=256, hq=64, ldk=128, hk=64,
             ldv=128, hv=64, ldo=256, ho=64, dtype=L.BF16, out_dtype=L.BF16, causal=1, scale=0.1, q_offsets=256,
             k_offsets=256, k_lens=None)
    d.update(kw)
    return L.LoraAttention(**d)


@no_device
@pytest.mark.parametrize("kw,status", [
    (dict(q_tokens=0), -2), (dict(k_tokens=0), -2), (dict(heads=0), -2), (dict(kv_heads=0), -2), (dict(seqs=0), -2),
    (dict(heads=3, kv_heads=2), -2), (dict(head_dim=136, hq=136, hk=136, hv=136, ho=136), -2), (dict(head_dim=0), -2),
    (dict(q_tokens=1 << 29), -2), (dict(k_tokens=1 << 30), -2), (dict(seqs=1 << 29), -2), (dict(heads=1 << 17), -2),
    (dict(ldq=248), -2), (dict(hk=32), -2), (dict(ldo=8), -2), (dict(ldk=(1 << 22) + 8), -2),
    (dict(dtype=2), -3), (dict(out_dtype=8), -3), (dict(dtype=L.F32), -3),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
    (dict(q_offsets=None), -1), (dict(k_offsets=None), -1),
    (dict(head_dim=60), -4), (dict(ldq=260), -4), (dict(hv=68, ldv=136), -4), (dict(k_lens=258), -4),
])
def test_invalid_descriptor_is_refused(kw, status):
    at, lib = _at(**kw), L.lib()
    assert lib.lora_attention_workspace_bytes(C.byref(at), 0) == lib.lora_attention_workspace_bytes(C.byref(at), 1) == 0
    assert lib.lora_attention_forward(C.byref(at), 256, 256, 256, 256, 256, 256, 1 << 30, None) == status
    assert lib.lora_attention_backward(C.byref(at), *[256] * 10, 1 << 30, None) == status


@no_device
def test_invalid_calls_are_refused():
    lib, at = L.lib(), _at()
    fwd = lambda i, p: lib.lora_attention_forward(C.byref(at), *[p if j == i else 256 for j in range(5)], 256, 1 << 30, None)
    bwd = lambda i, p: lib.lora_attention_backward(C.byref(at), *[p if j == i else 256 for j in range(9)], 256, 1 << 30, None)
    assert lib.lora_attention_forward(None, *[256] * 6, 1 << 30, None) == -1
    for i in range(4):
        assert fwd(i, None) == -1 and fwd(i, 264) == -4
    assert fwd(4, 258) == -4
    for i in range(9):
        assert bwd(i, None) == -1 and bwd(i, 258) == -4
    need = lib.lora_attention_workspace_bytes(C.byref(at), 1)
    assert need > 0
    for ws, n in ((None, need), (256, need - 1), (264, need)):
        assert lib.lora_attention_backward(C.byref(at), *[256] * 9, ws, n, None) == -5


@gpu
def test_binding_checks_tensors():
    off = dints([0, 8])
    at = L.make_attention(8, 8, 4, 2, 64, off, off)
    q, k = torch.zeros(8, 4, 64, device=DEV, dtype=BF16), torch.zeros(8, 2, 64, device=DEV, dtype=BF16)
    L.lora_attention_forward(at, q.view(8, 256), k, k, q.clone())
    for bad in (k, q.float(), q[:7], q.transpose(0, 1).contiguous().transpose(0, 1), q.cpu()):
        with pytest.raises((ValueError, TypeError)):
            L.lora_attention_forward(at, bad, k, k, q.clone())
    with pytest.raises(ValueError):
        L.lora_attention_forward(at, q, k, k, q.clone(), torch.zeros(31, device=DEV))
    with pytest.raises(TypeError):
        L.make_attention(8, 8, 4, 2, 64, off.long(), off)
    with pytest.raises(ValueError):
        L.make_attention(8, 8, 4, 2, 64, off, dints([0]))
