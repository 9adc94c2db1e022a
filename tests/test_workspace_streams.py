"""A workspace that the binding takes for a call belongs to the call's stream.

A block of another stream's pool may still be in use by work queued there when
torch hands it out again: only work of that stream is ordered behind it."""

import contextlib
import types

import pytest
import torch

from bwd_adamw_amd import lora as L

DEV = "cuda"


class Side:
    def __init__(self, handle=7):
        self.cuda_stream = handle


@pytest.mark.parametrize("stream,under", [(None, None), (Side(7), 7), (9, 9), (0, 0)])
def test_the_workspace_is_taken_under_the_calls_stream(monkeypatch, stream, under):
    now, taken = [None], []

    @contextlib.contextmanager
    def entered(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    def empty(need, device, dtype):
        taken.append((need, now[-1]))
        return types.SimpleNamespace(record_stream=lambda s: None)

    monkeypatch.setattr(L, "torch", types.SimpleNamespace(
        empty=empty, uint8=torch.uint8,
        cuda=types.SimpleNamespace(Stream=Side, stream=entered, default_stream=lambda d: Side(0),
                                   ExternalStream=lambda h, device: Side(h))))
    L._own_ws(48, DEV, stream)
    assert taken == [(48, under)]


class Taken(Exception):
    pass


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: GPU-less hosts only")
def test_every_call_takes_its_workspace_there(monkeypatch):
    def own(need, device, stream):
        assert need > 0
        raise Taken(stream)

    monkeypatch.setattr(L, "_own_ws", own)
    monkeypatch.setattr(L, "_ptr", lambda t, name, dtype=None: None if t is None else 256)
    lin = L.LoraLinear(64, 512, 1024, 8, L.F32, 2.0, 256, 256, 256, None, None)
    t = torch.zeros(1 << 21)
    W = types.SimpleNamespace(out_dim=256, in_dim=4096, buf=t)
    rows = types.SimpleNamespace(rows=64, cols=4096, desc=L.LoraFp8Operand(64, 4096, 256))
    runs, hp = [L.make_matrix_run(0, 32, 1024, 3)], L.make_muon(0.1)
    nm, x = L.LoraNorm(600, 512, 512, 512, 0, 0, None, None, 1e-5), torch.zeros(600, 512)
    calls = (
        lambda s: L.lora_dora_row_norms(lin, t, stream=s),
        lambda s: L.lora_dora_row_norms_batch([lin, lin], [t, t], stream=s),
        lambda s: L.lora_merge(lin, t.bfloat16(), rmse=t.double(), stream=s),
        lambda s: L.lora_fp8_product(rows, W, t, stream=s),
        lambda s: L.lora_orthogonalize(t, t, runs, hp, stream=s),
        lambda s: L.lora_muon_step(t, t, t, runs, hp, t, stream=s),
        lambda s: L.lora_norm_backward(nm, x, [x], t, None, t, stream=s),
    )
    monkeypatch.setattr(L, "_rows_ptr", lambda *a: 256)
    for call in calls:
        with pytest.raises(Taken) as e:
            call(9)
        assert e.value.args == (9,)


def norm_backward(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    nm = L.make_norm("layer", 600, 512)
    x, dy, st = rnd(600, 512), rnd(600, 512), rnd(600, 2)
    out = [torch.zeros(512, device=DEV), torch.zeros(512, device=DEV)]
    return out, lambda s: L.lora_norm_backward(nm, x, [dy], st, None, *out, stream=s)


def product(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(256, 4096, device=DEV, generator=g).mul_(50).to(torch.float8_e4m3fn)
    W = L.fp8_pack(w, torch.ones(2, 32, device=DEV))
    q, y = L.fp8_rows(64, 4096), torch.zeros(64, 256, device=DEV)
    L.lora_fp8_quantize(torch.randn(64, 4096, device=DEV, generator=g), q)
    assert L.lora_fp8_product_workspace_bytes(q, W) > 0
    return [y], lambda s: L.lora_fp8_product(q, W, y, stream=s)


def muon_step(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda: torch.randn(3, 32, 1024, device=DEV, generator=g)
    p, gr, m, scale = rnd(), rnd(), rnd(), torch.ones(1, device=DEV)
    runs, hp = [L.make_matrix_run(0, 32, 1024, 3)], L.make_muon(0.1)
    return [p, m], lambda s: L.lora_muon_step(p, gr, m, runs, hp, scale, stream=s)


def row_norms(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    W, A, B, out = rnd(256, 4096), rnd(8, 4096), rnd(256, 8), torch.zeros(256, device=DEV)
    lin = L.make_linear(W, A, B, 2.0, 32)
    assert L.lora_dora_row_norms_workspace_bytes(lin) > 0
    return [out], lambda s, keep=(W, A, B): L.lora_dora_row_norms(lin, out, stream=s)


def merge(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    W, A, B = rnd(256, 4096), rnd(8, 4096), rnd(256, 8)
    out, rmse = torch.zeros(256, 4096, device=DEV, dtype=torch.bfloat16), torch.zeros(1, device=DEV, dtype=torch.float64)
    lin = L.make_linear(W, A, B, 2.0, 32)
    return [out, rmse], lambda s, keep=(W, A, B): L.lora_merge(lin, out, rmse, stream=s)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("case", [norm_backward, product, muon_step, row_norms, merge])
def test_calls_on_two_streams_share_no_workspace(case, handle):
    """A call that waits on the busy current stream, then at once the same
    operator on a side stream with other operands: both as if alone."""
    refs = []
    for seed in (1, 2):
        out, call = case(seed)
        call(None)
        torch.cuda.synchronize()
        refs.append([t.clone() for t in out])
    (out1, call1), (out2, call2) = case(1), case(2)
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(8):   # a few milliseconds ahead of the first call
        busy = busy @ busy * 1e-3
    call1(None)
    call2(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    for out, ref in ((out1, refs[0]), (out2, refs[1])):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
