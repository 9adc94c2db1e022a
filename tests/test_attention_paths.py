"""The attention's other kernels: batches large enough for four row tiles a block,
calls that overlap on two streams, workspaces that the binding takes, and a run of
heads, attention and their gradients as they are used together.  Formulas and
tolerances are test_attention's."""

import math

import pytest
import torch

from bwd_adamw_amd import lora as L
from test_attention import BF16, DEV, F32, HALF, TYPES, check, close, data, dints, run

pytestmark = pytest.mark.gpu


# 256 blocks of 128 rows and more over the key heads; the last has heads in
# threes (stages that do not begin at a token's first head) and keys before the queries
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [([600], [600], 64, 64, 64), ([300, 0, 340], [300, 9, 340], 64, 16, 128),
                                  ([520, 100], [700, 90], 48, 16, 40)], ids=str)
def test_large_batches(case, causal, dtype, out):
    check(*case, causal, dtype, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_caches_of_a_large_batch(dtype):
    check([70] * 12, [100] * 12, 32, 32, 64, True, dtype, dtype, lens=[100, 70, 75, 99, 71, 70, 80, 90, 73, 74, 100, 0])


# three rounds of blocks of 128 rows and more, where float32 takes four row tiles a block too
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [([200, 130], [200, 140], 256, 256, 64), ([200, 130], [190, 130], 256, 128, 128)], ids=str)
def test_larger_batches_in_float32(case, causal):
    check(*case, causal, F32, F32)


# one long sequence in up to two rounds of blocks: two row tiles a block, in bf16 too
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("case", [([1100], [1100], 34, 34, 64), ([1030], [1100], 36, 36, 128)], ids=str)
def test_long_sequences_of_few_blocks(case, dtype, out):
    check(*case, True, dtype, out)


# more sequences than a wave has lanes, each long enough for its key tiles to be shared
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_shared_key_tiles_of_many_sequences(D, dtype, out):
    lens = [40 + (i * 11) % 31 for i in range(66)]
    check(lens, [n + i % 2 for i, n in enumerate(lens)], 8, 1, D, True, dtype, out)


def both(at, q, k, v, do, out):
    """A call on any stream with everything it writes made beforehand."""
    o, lse, dq, dk, dv = out
    def call(ws, stream=None):
        L.lora_attention_forward(at, q, k, v, o, lse, ws=ws and ws[0], stream=stream)
        L.lora_attention_backward(at, q, k, v, o, do, lse, dq, dk, dv, ws=ws and ws[1], stream=stream)
    return call


def problem(seed, lens=(200, 57), H=8, KV=2, D=128):
    T = sum(lens)
    q, k, v, do = (t.to(DEV) for t in data(T, T, H, KV, D, BF16, seed))
    off = dints([0, lens[0], T])
    at = L.make_attention(T, T, H, KV, D, off, off)
    out = [torch.empty_like(q), torch.empty(H, T, device=DEV), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
    ref = [t.clone() for t in run(at, q, k, v, do.bfloat16(), k.shape, BF16)]
    return at, both(at, q, k, v, do.bfloat16(), out), out, ref


def test_two_calls_at_once():
    """Two streams, each with a workspace: each as alone."""
    probs = [problem(s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in probs]
    wss = [[torch.empty(max(16, L.lora_attention_workspace_bytes(p[0], b)), device=DEV, dtype=torch.uint8)
            for b in (False, True)] for p in probs]
    torch.cuda.synchronize()
    for _ in range(4):
        for (_, call, _, _), st, ws in zip(probs, streams, wss):
            call(ws, st)
    torch.cuda.synchronize()
    for _, _, out, ref in probs:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("handle", [False, True])
def test_workspace_stays_until_the_other_stream_is_done(handle):
    at, call, out, ref = problem(3)
    need = L.lora_attention_workspace_bytes(at, True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):   # a few milliseconds ahead of the call
            busy = busy @ busy * 1e-3
    call(None, side.cuda_stream if handle else side)
    # what the current stream is given now, and writes at once
    junk = [torch.full((need,), 255, device=DEV, dtype=torch.uint8) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    del junk


def test_workspace_is_as_asked():
    """Nothing is written behind the bytes that a call asks for."""
    for lens, H, KV, D, dt, out in (((1, 1), 8, 2, 128, BF16, BF16), ((300, 20), 8, 2, 128, BF16, F32),
                                    ((300, 20), 4, 4, 64, F32, F32)):
        T, Tk = sum(lens), sum(lens) + 2000
        q, k, v, do = (t.to(DEV) for t in data(T, Tk, H, KV, D, dt, 7))
        at = L.make_attention(T, Tk, H, KV, D, dints([0, lens[0], T]), dints([0, lens[0] + 1000, Tk]), dtype=dt, out_dtype=out)
        o, lse = torch.empty(q.shape, device=DEV, dtype=out), torch.empty(H, T, device=DEV)
        grads = [torch.empty(t.shape, device=DEV, dtype=out) for t in (q, k, v)]
        for bwd in (False, True):
            need = L.lora_attention_workspace_bytes(at, bwd)
            ws = torch.full((need + 4096,), 165, device=DEV, dtype=torch.uint8)
            part = ws[:need] if need else None
            if bwd:
                L.lora_attention_backward(at, q, k, v, o, do.to(out), lse, *grads, ws=part)
            else:
                L.lora_attention_forward(at, q, k, v, o, lse, ws=part)
            torch.cuda.synchronize()
            assert (ws[need:] == 165).all()


def test_heads_then_attention_and_back():
    """Projections' outputs in float32 to wo's input and back, as a layer runs
    them, against float64 derivatives of the whole.  Tolerance: the bf16 steps of
    q, k, v, p, ds and dO (half a step each, 2^-8 of the magnitudes behind them) and
    a score's shift from q and k, 2^-7 of scores under 10: 16 * 2^-8 of an output's
    largest value."""
    T, H, KV, D = 150, 4, 2, 64
    offs = [0, 40, 41, T]
    g = torch.Generator().manual_seed(11)
    ys = [torch.randn(T, n * D, generator=g) for n in (H, KV, KV)]
    do = torch.randn(T, H * D, generator=g)
    gam = [1 + 0.1 * torch.randn(D, generator=g) for _ in range(2)]
    freqs = L.rope_freqs(D, 1e4, "cpu")
    pos = torch.cat([torch.arange(b - a) for a, b in zip(offs, offs[1:])])
    # float64
    yr = [y.double().requires_grad_() for y in ys]
    gr = [x.double().requires_grad_() for x in gam]
    phi = pos.double()[:, None, None] * freqs

    def turned(x, n, gamma):
        z = x.view(T, n, D)
        z = z * (z.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma
        a, b = z[..., :D // 2], z[..., D // 2:]
        return torch.cat([a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin()], -1)
    qr, kr, vr = turned(yr[0], H, gr[0]), turned(yr[1], KV, gr[1]), yr[2].view(T, KV, D)
    parts = []
    for a, b in zip(offs, offs[1:]):
        s = torch.einsum("ihd,jhd->hij", qr[a:b], kr[a:b].repeat_interleave(H // KV, 1)) * D ** -0.5
        s = s.masked_fill(torch.ones(b - a, b - a).triu(1).bool(), -math.inf)
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), vr[a:b].repeat_interleave(H // KV, 1)))
    orf = torch.cat(parts).reshape(T, H * D)
    orf.backward(do.double())
    # the framework's calls
    yd, fd, pd = [y.to(DEV) for y in ys], freqs.to(DEV), pos.int().to(DEV)
    gd = [x.to(DEV) for x in gam]
    q, k, v = (torch.empty(T, n * D, device=DEV, dtype=BF16) for n in (H, KV, KV))
    sets = [L.make_heads(T, n, D, F32, BF16, gamma=x, freqs=fd) for n, x in zip((H, KV), gd)]
    L.lora_heads_forward(sets + [L.make_heads(T, KV, D, F32, BF16, norm=False)], yd, [q, k, v], pd)
    at = L.make_attention(T, T, H, KV, D, dints(offs), dints(offs), out_dtype=F32)
    o, lse = torch.empty(T, H * D, device=DEV), torch.empty(H, T, device=DEV)
    L.lora_attention_forward(at, q, k, v, o, lse)
    dy = [torch.empty_like(y) for y in yd]
    L.lora_attention_backward(at, q, k, v, o, do.to(DEV), lse, *dy)
    back = [L.make_heads(T, n, D, F32, F32, gamma=x, freqs=fd) for n, x in zip((H, KV), gd)]
    dg = [torch.empty(D, device=DEV) for _ in range(2)]
    L.lora_heads_backward(back, yd[:2], dy[:2], dy[:2], dg, pd)
    for got, ref in [(o, orf)] + list(zip(dy, [y.grad for y in yr])) + list(zip(dg, [x.grad for x in gr])):
        ref = ref.detach()
        assert (got.cpu().double() - ref).abs().max() <= 16 * HALF * ref.abs().max()


@pytest.mark.gpu
def test_calls_on_another_device_than_the_current_one_are_refused(monkeypatch):
    """Kernels are launched on the current device: tensors (and streams) of
    another are refused before anything is."""
    bf = torch.bfloat16
    x = torch.randn(4, 2, 64, device="cuda", dtype=bf)
    off = torch.tensor([0, 4], device="cuda", dtype=torch.int32)
    heads = [L.make_heads(4, 2, 64, bf, bf)]
    at = L.make_attention(4, 4, 2, 2, 64, off, off)
    y, lse, stream = torch.full_like(x, 7.0), torch.zeros(2, 4, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for s in (None, stream):
        for call in (lambda: L.lora_heads_forward(heads, [x], [y], stream=s),
                     lambda: L.lora_heads_backward(heads, [x], [x], [y], stream=s),
                     lambda: L.lora_attention_forward(at, x, x, x, y, stream=s),
                     lambda: L.lora_attention_backward(at, x, x, x, x, x, lse, y, y, y, stream=s)):
            with pytest.raises(ValueError, match="GPU 0, the current one is 1"):
                call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert (y == 7.0).all()


def test_an_output_in_place_of_an_input_is_refused():
    bf = torch.bfloat16
    off = dints([0, 4])
    at = L.make_attention(4, 4, 2, 2, 64, off, off)
    q, k, v, o, do, dq, dk, dv = (torch.ones(4, 2, 64, device=DEV, dtype=bf) for _ in range(8))
    lse = torch.zeros(2, 4, device=DEV)
    for t in (q, k, v):
        with pytest.raises(L.LoraError):
            L.lora_attention_forward(at, q, k, v, t, lse)
    for i in range(3):
        for t in (q, k, v, o, do, *[g for j, g in enumerate((dq, dk, dv)) if j != i]):
            grads = [dq, dk, dv]
            grads[i] = t
            with pytest.raises(L.LoraError):
                L.lora_attention_backward(at, q, k, v, o, do, lse, *grads)
    torch.cuda.synchronize()
    assert all((t == 1).all() for t in (q, k, v, o, do, dq, dk, dv))
