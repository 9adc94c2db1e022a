"""Thin ctypes binding of liblora (include/lora.h).

Argument marshalling only: every function here checks tensor placement and
dtype, turns tensors into device pointers and calls the C entry point of the
same name.  All computation happens in the HIP kernels behind the C ABI.
There is no fallback: if liblora.so is missing or the device is not a GPU,
the call raises.
"""

from __future__ import annotations

import ctypes as C
import functools
import os

import torch

__all__ = [
    "LoraError", "lib", "LoraLinear", "LoraDropout", "LoraSegment", "LoraAdamwHparams",
    "F32", "BF16", "KIND_A", "KIND_B", "KIND_MAG",
    "lora_workspace_bytes", "lora_forward", "lora_backward",
    "lora_grad_prepare_workspace_bytes", "lora_grad_prepare", "lora_adamw_step",
    "lora_dropout_mask", "lora_dora_row_norms_workspace_bytes", "lora_dora_row_norms",
    "lora_merge_workspace_bytes", "lora_merge", "lora_scaling", "lora_lr_at",
    "lora_status_string", "lora_profile_begin", "lora_profile_end", "lora_set_bf16_config",
    "lora_group_workspace_bytes", "lora_forward_group", "lora_backward_group",
    "lora_slots_workspace_bytes", "lora_forward_slots", "lora_backward_slots",
    "lora_qweight_layout", "lora_grad_prepare_noalloc",
    "lora_dora_row_norms_batch_workspace_bytes", "lora_dora_row_norms_batch", "QWeight", "qweight_pack", "Q_FORMATS", "EXPORTS", "GroupCall",
    "LoraNorm", "make_norm", "lora_norm_forward", "lora_norm_workspace_bytes",
    "lora_norm_backward", "LoraMatrixRun", "LoraMuonHparams", "make_matrix_run", "make_muon",
    "lora_muon_workspace_bytes", "lora_orthogonalize", "lora_muon_step",
    "Fp8Weight", "fp8_pack", "Fp8Rows", "fp8_rows", "lora_fp8_weight_layout",
    "lora_fp8_operand_layout", "lora_fp8_quantize", "lora_fp8_product_workspace_bytes",
    "lora_fp8_product",
    "LoraHeads", "make_heads", "rope_freqs", "lora_heads_forward", "lora_heads_workspace_bytes",
    "lora_heads_backward", "LoraAttention", "make_attention", "lora_attention_workspace_bytes",
    "lora_attention_forward", "lora_attention_backward",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblora.so")

F32, BF16, FP8 = 0, 1, 8
# Block-quantized W formats (lora_dtype): code and plane names in layout order.
Q_FORMATS = {"q8_0": (2, ("qs", "d")), "q4_0": (3, ("qs", "d")),
             "q4_k": (4, ("qs", "sm", "dm")), "q6_k": (5, ("ql", "qh", "sc", "d"))}
KIND_A, KIND_B, KIND_MAG = 0, 1, 2
LORA_E_NONFINITE = -6

# Every symbol include/lora.h declares.
EXPORTS = (
    "lora_workspace_bytes", "lora_forward", "lora_backward",
    "lora_grad_prepare_workspace_bytes", "lora_grad_prepare", "lora_adamw_step",
    "lora_dropout_mask", "lora_dora_row_norms_workspace_bytes", "lora_dora_row_norms",
    "lora_merge_workspace_bytes", "lora_merge", "lora_scaling", "lora_lr_at",
    "lora_status_string", "lora_profile_begin", "lora_profile_end", "lora_set_bf16_config",
    "lora_group_workspace_bytes", "lora_forward_group", "lora_backward_group",
    "lora_slots_workspace_bytes", "lora_forward_slots", "lora_backward_slots",
    "lora_qweight_layout", "lora_grad_prepare_noalloc",
    "lora_dora_row_norms_batch_workspace_bytes", "lora_dora_row_norms_batch",
    "lora_norm_forward", "lora_norm_workspace_bytes", "lora_norm_backward",
    "lora_muon_workspace_bytes", "lora_orthogonalize", "lora_muon_step",
    "lora_fp8_weight_layout", "lora_fp8_operand_layout", "lora_fp8_quantize",
    "lora_fp8_product_workspace_bytes", "lora_fp8_product",
    "lora_heads_forward", "lora_heads_workspace_bytes", "lora_heads_backward",
    "lora_attention_workspace_bytes", "lora_attention_forward", "lora_attention_backward",
)


class LoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {lora_status_string(status)} (status {status})")


class LoraDropout(C.Structure):
    _fields_ = [("seed", C.c_uint64), ("step", C.c_int64), ("ordinal", C.c_int32),
                ("layer", C.c_int32), ("proj", C.c_int32), ("p", C.c_float)]


class LoraLinear(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("in_dim", C.c_int64), ("out_dim", C.c_int64),
                ("rank", C.c_int64), ("w_dtype", C.c_int32), ("scale", C.c_float),
                ("W", C.c_void_p), ("A", C.c_void_p), ("B", C.c_void_p),
                ("dora_mag", C.c_void_p), ("dora_norm", C.c_void_p), ("dora_from_y", C.c_int32)]


class LoraProfileEntry(C.Structure):
    _fields_ = [("kernel", C.c_char_p), ("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64),
                ("launches", C.c_int64), ("total_ms", C.c_double), ("flops", C.c_double),
                ("bytes", C.c_double)]


class LoraSegment(C.Structure):
    _fields_ = [("offset", C.c_int64), ("count", C.c_int64), ("kind", C.c_int32)]


class LoraAdamwHparams(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("weight_decay", C.c_double), ("plus_ratio", C.c_double),
                ("t", C.c_int64)]


class LoraNorm(C.Structure):
    _fields_ = [("rows", C.c_int64), ("dim", C.c_int64), ("ldx", C.c_int64), ("ldy", C.c_int64),
                ("kind", C.c_int32), ("dtype", C.c_int32), ("gamma", C.c_void_p),
                ("beta", C.c_void_p), ("eps", C.c_float)]


class LoraHeads(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("heads", C.c_int64), ("head_dim", C.c_int64),
                ("rot_dim", C.c_int64), ("ldx", C.c_int64), ("hx", C.c_int64), ("ldy", C.c_int64),
                ("hy", C.c_int64), ("x_dtype", C.c_int32), ("y_dtype", C.c_int32),
                ("norm", C.c_int32), ("interleaved", C.c_int32), ("gamma", C.c_void_p),
                ("freqs", C.c_void_p), ("eps", C.c_float)]


class LoraAttention(C.Structure):
    _fields_ = [("q_tokens", C.c_int64), ("k_tokens", C.c_int64), ("heads", C.c_int64),
                ("kv_heads", C.c_int64), ("head_dim", C.c_int64), ("seqs", C.c_int64),
                ("ldq", C.c_int64), ("hq", C.c_int64), ("ldk", C.c_int64), ("hk", C.c_int64),
                ("ldv", C.c_int64), ("hv", C.c_int64), ("ldo", C.c_int64), ("ho", C.c_int64),
                ("dtype", C.c_int32), ("out_dtype", C.c_int32), ("causal", C.c_int32),
                ("scale", C.c_float), ("q_offsets", C.c_void_p), ("k_offsets", C.c_void_p),
                ("k_lens", C.c_void_p)]


class LoraFp8Operand(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("data", C.c_void_p)]


class LoraMatrixRun(C.Structure):
    _fields_ = [("offset", C.c_int64), ("stride", C.c_int64), ("count", C.c_int64),
                ("rows", C.c_int64), ("cols", C.c_int64), ("kind", C.c_int32)]


class LoraMuonHparams(C.Structure):
    _fields_ = [("lr", C.c_double), ("momentum", C.c_double), ("weight_decay", C.c_double),
                ("plus_ratio", C.c_double), ("eps", C.c_double), ("a", C.c_double),
                ("b", C.c_double), ("c", C.c_double), ("steps", C.c_int32),
                ("nesterov", C.c_int32), ("adjust", C.c_int32)]


_LIB = None


def lib() -> C.CDLL:
    """Load liblora.so once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bwd_adamw_amd.build`")
        L = C.CDLL(LIB_PATH)
        P, I64, I32, F, SZ = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_size_t
        sig = {
            "lora_workspace_bytes": (SZ, [P]),
            "lora_forward": (I32, [P, P, P, P, P, P, P, SZ, P]),
            "lora_backward": (I32, [P, P, P, P, P, P, P, P, P, I32, P, P, SZ, P]),
            "lora_grad_prepare_workspace_bytes": (SZ, [I64]),
            "lora_grad_prepare": (I32, [P, I64, I64, F, P, P, P, P, SZ, P]),
            "lora_grad_prepare_noalloc": (I32, [P, I64, I64, F, P, P, P, P]),
            "lora_adamw_step": (I32, [P, P, P, P, P, I32, P, P, P]),
            "lora_dropout_mask": (I32, [P, I64, I64, P, P]),
            "lora_dora_row_norms_workspace_bytes": (SZ, [P]),
            "lora_dora_row_norms": (I32, [P, P, P, SZ, P]),
            "lora_merge_workspace_bytes": (SZ, [P]),
            "lora_merge": (I32, [P, P, I32, P, P, SZ, P]),
            "lora_scaling": (C.c_double, [C.c_double, I64, I32]),
            "lora_lr_at": (C.c_double, [I64, C.c_double, I32, I64, I64, C.c_double]),
            "lora_status_string": (C.c_char_p, [I32]),
            "lora_profile_begin": (I32, [I32]),
            "lora_profile_end": (I32, [P, I32]),
            "lora_set_bf16_config": (I32, [I32]),
            "lora_group_workspace_bytes": (SZ, [I32, P]),
            "lora_forward_group": (I32, [I32, P, P, P, P, P, P, P, SZ, P]),
            "lora_backward_group": (I32, [I32, P, P, P, P, P, P, P, P, P, I32, P, P, SZ, P]),
            "lora_slots_workspace_bytes": (SZ, [I32, P]),
            "lora_forward_slots": (I32, [I32, P, P, P, P, P, P, P, SZ, P]),
            "lora_backward_slots": (I32, [I32, P, P, P, P, P, P, P, P, P, I32, P, P, SZ, P]),
            "lora_qweight_layout": (SZ, [I32, I64, I64, P]),
            "lora_dora_row_norms_batch_workspace_bytes": (SZ, [I32, P]),
            "lora_dora_row_norms_batch": (I32, [I32, P, P, P, SZ, P]),
            "lora_fp8_weight_layout": (SZ, [I64, I64, P]),
            "lora_fp8_operand_layout": (SZ, [I64, I64, P]),
            "lora_fp8_quantize": (I32, [P, I32, I64, P, P]),
            "lora_fp8_product_workspace_bytes": (SZ, [P, I64, I64, I32]),
            "lora_fp8_product": (I32, [P, P, I64, I64, I32, P, I32, P, SZ, P]),
            "lora_muon_workspace_bytes": (SZ, [P, I32]),
            "lora_orthogonalize": (I32, [P, P, P, I32, P, P, SZ, P]),
            "lora_muon_step": (I32, [P, P, P, P, I32, P, P, P, SZ, P]),
            "lora_norm_forward": (I32, [P, P, P, P, P]),
            "lora_norm_workspace_bytes": (SZ, [P]),
            "lora_norm_backward": (I32, [P, P, I32, P, P, P, P, P, I32, P, SZ, P]),
            "lora_heads_forward": (I32, [I32, P, P, P, P, P]),
            "lora_heads_workspace_bytes": (SZ, [I32, P]),
            "lora_heads_backward": (I32, [I32, P, P, P, P, P, P, I32, P, SZ, P]),
            "lora_attention_workspace_bytes": (SZ, [P, I32]),
            "lora_attention_forward": (I32, [P, P, P, P, P, P, P, SZ, P]),
            "lora_attention_backward": (I32, [P, P, P, P, P, P, P, P, P, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


# ------------------------------------------------------------------ helpers
def _ptr(t, name, dtype=torch.float32):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _sized(t, name, need, dtype=torch.float32):
    """_ptr that also refuses a tensor with fewer than `need` elements: the
    kernels address every buffer from the linear's sizes alone."""
    p = _ptr(t, name, dtype)
    if p is not None and t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} elements, the call reads or writes {need}")
    return p


# The handle of the current stream.  torch.cuda.current_stream() builds a Stream
# object on every call (2.8 us, as much as a launch); torch's own compiled code
# asks for the bare handle (0.3 us with the device lookup).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _own_ws(need, device, stream):
    """A workspace from torch's allocator for a call on `stream` (None: the
    current one), taken under that stream: what used the block before and what
    gets it after the call returns is then ordered with the call's kernels.  A
    block of the current stream's pool may still be in use by work queued there,
    which a call on another stream does not wait for."""
    if stream is None:
        return torch.empty(need, device=device, dtype=torch.uint8)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(need, device=device, dtype=torch.uint8)


def _check(fn, rc):
    if rc != 0:
        raise LoraError(fn, rc)


def lora_qweight_layout(fmt: str, out_dim: int, in_dim: int):
    """(total bytes, [offset of each plane]) of a block-quantized W."""
    code, names = Q_FORMATS[fmt]
    off = (C.c_size_t * 4)()
    total = int(lib().lora_qweight_layout(code, int(out_dim), int(in_dim), off))
    if total == 0:
        raise ValueError(f"{fmt} cannot hold a [{out_dim}, {in_dim}] weight")
    return total, [int(o) for o in off[: len(names)]]


class QWeight:
    """A block-quantized W [out_dim, in_dim] in the library's layout: one
    uint8 device buffer holding the format's planes (include/lora.h)."""

    def __init__(self, fmt: str, out_dim: int, in_dim: int, buf: torch.Tensor):
        self.fmt, self.out_dim, self.in_dim, self.buf = fmt, int(out_dim), int(in_dim), buf
        self.code = Q_FORMATS[fmt][0]

    @property
    def shape(self):
        return (self.out_dim, self.in_dim)


def _plane_row_bytes(fmt, K):
    return {"q8_0": (K, K // 16), "q4_0": (K // 2, K // 16),
            "q4_k": (K // 2, K // 16, K // 64),
            "q6_k": (K // 2, K // 4, K // 16, K // 128)}[fmt]


def qweight_pack(fmt: str, out_dim: int, in_dim: int, planes: dict, device="cuda") -> QWeight:
    """Copy the planes (tensors of any dtype, by their bytes, row-major) into
    one device buffer laid out by lora_qweight_layout."""
    total, offs = lora_qweight_layout(fmt, out_dim, in_dim)
    names = Q_FORMATS[fmt][1]
    buf = torch.zeros(total, dtype=torch.uint8, device=device)
    for name, off, rb in zip(names, offs, _plane_row_bytes(fmt, int(in_dim))):
        raw = planes[name].contiguous().view(torch.uint8).reshape(-1)
        if raw.numel() != rb * out_dim:
            raise ValueError(f"{fmt} plane {name} holds {raw.numel()} bytes, the layout "
                             f"needs {rb * out_dim}")
        buf[off:off + raw.numel()].copy_(raw)
    return QWeight(fmt, out_dim, in_dim, buf)


def make_linear(W, A, B, scale, tokens, dora_mag=None, dora_norm=None,
                dora_from_y=False) -> LoraLinear:
    """Descriptor of one adapted linear: W [N,K] (float32 or bfloat16, a
    QWeight or an Fp8Weight), A [r,K], B [N,r] float32, optional DoRA magnitude and norm [N].
    dora_from_y (DoRA only): the backward takes the forward's Y where it
    would take Z, so the forward need not write Z."""
    if isinstance(W, (QWeight, Fp8Weight)):
        wd = W.code
    elif W.dtype in (torch.float32, torch.bfloat16):
        wd = F32 if W.dtype == torch.float32 else BF16
    else:
        raise TypeError(f"W must be float32, bfloat16, a QWeight or an Fp8Weight, got {W.dtype}")
    N, K = W.shape
    r = A.shape[0] if A is not None else 0
    if A is not None and tuple(A.shape) != (r, K):
        raise ValueError(f"A must be [{r}, {K}], got {list(A.shape)}")
    if B is not None and tuple(B.shape) != (N, r):
        raise ValueError(f"B must be [{N}, {r}], got {list(B.shape)}")
    for t, nm in ((dora_mag, "dora_mag"), (dora_norm, "dora_norm")):
        if t is not None and t.numel() != N:
            raise ValueError(f"{nm} must hold {N} elements, got {t.numel()}")
    wptr = (_ptr(W.buf, "W", torch.uint8) if isinstance(W, (QWeight, Fp8Weight))
            else _ptr(W, "W", None))
    return LoraLinear(int(tokens), int(K), int(N), int(r), wd, float(scale), wptr,
                      _ptr(A, "A"), _ptr(B, "B"), _ptr(dora_mag, "dora_mag"),
                      _ptr(dora_norm, "dora_norm"), 1 if dora_from_y else 0)


def make_dropout(seed, step, ordinal, layer, proj, p) -> LoraDropout:
    return LoraDropout(int(seed), int(step), int(ordinal), int(layer), int(proj), float(p))


def _ref(s):
    return None if s is None else C.byref(s)


# ------------------------------------------------------------ entry points
def lora_status_string(status: int) -> str:
    return lib().lora_status_string(int(status)).decode()


def lora_scaling(alpha: float, rank: int, rslora: bool = False) -> float:
    return lib().lora_scaling(float(alpha), int(rank), 1 if rslora else 0)


def lora_lr_at(k: int, lr: float, schedule: int = 0, warmup: int = 0, total: int = 100,
               lr_min: float = 0.0) -> float:
    return lib().lora_lr_at(int(k), float(lr), int(schedule), int(warmup), int(total), float(lr_min))


def lora_workspace_bytes(lin: LoraLinear) -> int:
    return int(lib().lora_workspace_bytes(C.byref(lin)))


def lora_forward(lin, X, Y, U, Z=None, drop=None, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    T, K, N, r = lin.tokens, lin.in_dim, lin.out_dim, lin.rank
    rc = lib().lora_forward(C.byref(lin), _sized(X, "X", T * K), _sized(Y, "Y", T * N),
                            _sized(U, "U", T * r), _sized(Z, "Z", T * N), _ref(drop),
                            _ptr(ws, "ws", None), ws_bytes, _stream(stream))
    _check("lora_forward", rc)


def lora_backward(lin, X, dY, U, Z, dX, dA, dB, dMag=None, accumulate=False, drop=None,
                  ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    T, K, N, r = lin.tokens, lin.in_dim, lin.out_dim, lin.rank
    rc = lib().lora_backward(C.byref(lin), _sized(X, "X", T * K), _sized(dY, "dY", T * N),
                             _sized(U, "U", T * r), _sized(Z, "Z", T * N), _sized(dX, "dX", T * K),
                             _sized(dA, "dA", r * K), _sized(dB, "dB", N * r),
                             _sized(dMag, "dMag", N), 1 if accumulate else 0, _ref(drop),
                             _ptr(ws, "ws", None), ws_bytes, _stream(stream))
    _check("lora_backward", rc)


MAX_GROUP = 4
MAX_SLOTS = 4
MAX_RUNS = 32


def _linears(lins):
    arr = (LoraLinear * len(lins))(*lins)
    return arr


# Elements of each per-linear tensor argument, from a linear's sizes.
_NEED = {
    "X": lambda l: l.tokens * l.in_dim, "dX": lambda l: l.tokens * l.in_dim,
    "Y": lambda l: l.tokens * l.out_dim, "Z": lambda l: l.tokens * l.out_dim,
    "dY": lambda l: l.tokens * l.out_dim, "U": lambda l: l.tokens * l.rank,
    "dA": lambda l: l.rank * l.in_dim, "dB": lambda l: l.out_dim * l.rank,
    "dMag": lambda l: l.out_dim, "out_norm": lambda l: l.out_dim,
}


def _ptrs(ts, name, lins, optional=False):
    """Array of device pointers, one per linear of `lins`, each checked
    against that linear's sizes; None when every entry is None and the
    argument is optional."""
    if ts is None or (optional and all(t is None for t in ts)):
        if not optional:
            raise ValueError(f"{name} is required")
        return None
    if len(ts) != len(lins):
        raise ValueError(f"{name} has {len(ts)} entries for {len(lins)} linears")
    return (C.c_void_p * len(ts))(*[_sized(t, f"{name}[{i}]", _NEED[name](l))
                                    for i, (t, l) in enumerate(zip(ts, lins))])


def _drops(drops, n):
    if drops is None or all(d is None for d in drops):
        return None
    zero = LoraDropout(0, 0, 0, 0, 0, 0.0)
    return (LoraDropout * n)(*[zero if d is None else d for d in drops])


def lora_group_workspace_bytes(lins) -> int:
    return int(lib().lora_group_workspace_bytes(len(lins), _linears(lins)))


def lora_forward_group(lins, X, Y, U, Z=None, drops=None, ws=None, stream=None):
    """Forward of the linears `lins` that read one X; Y, U (and Z) are lists
    with one tensor per linear."""
    n = len(lins)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_forward_group(n, _linears(lins), _sized(X, "X", _NEED["X"](lins[0])),
                                  _ptrs(Y, "Y", lins), _ptrs(U, "U", lins),
                                  _ptrs(Z, "Z", lins, True), _drops(drops, n), _ptr(ws, "ws", None),
                                  ws_bytes, _stream(stream))
    _check("lora_forward_group", rc)


def lora_backward_group(lins, X, dY, U, Z, dX, dA, dB, dMag=None, accumulate=False, drops=None,
                        ws=None, stream=None):
    """Backward of the linears `lins` that read one X; every other tensor
    argument is a list with one entry per linear."""
    n = len(lins)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_backward_group(n, _linears(lins), _sized(X, "X", _NEED["X"](lins[0])),
                                   _ptrs(dY, "dY", lins), _ptrs(U, "U", lins),
                                   _ptrs(Z, "Z", lins, True), _ptrs(dX, "dX", lins, True),
                                   _ptrs(dA, "dA", lins), _ptrs(dB, "dB", lins),
                                   _ptrs(dMag, "dMag", lins, True),
                                   1 if accumulate else 0, _drops(drops, n), _ptr(ws, "ws", None),
                                   ws_bytes, _stream(stream))
    _check("lora_backward_group", rc)


class GroupCall:
    """Marshalled arguments of lora_forward_group / lora_backward_group for
    one group of linears whose descriptors and trainer-owned buffers stay
    put across calls (Y, U, Z, dX, the gradients, the workspace, the
    stream): they are checked and marshalled once, here.  Each call checks
    and marshals only its own inputs (X, dY, dropout keys); an X or dY list
    whose tensors are the ones of the previous call reuses their pointers."""

    def __init__(self, lins, Y, U, Z=None, dX=None, dA=None, dB=None, dMag=None, ws=None,
                 stream=None):
        self.n = len(lins)
        self.lins = list(lins)
        self.arr = _linears(self.lins)
        self.Y, self.U = _ptrs(Y, "Y", lins), _ptrs(U, "U", lins)
        self.Z = _ptrs(Z, "Z", lins, True)
        # DoRA linears with dora_from_y: the forward writes no Z and the
        # backward reads Y in its place.
        self.from_y = any(l.dora_from_y for l in lins)
        if self.from_y and not all(l.dora_from_y for l in lins):
            raise ValueError("dora_from_y must be set for all linears of a group call or none")
        self.Zf = None if self.from_y else self.Z
        self.Zb = self.Y if self.from_y else self.Z
        self.dX = _ptrs(dX, "dX", lins, True)
        self.dA = None if dA is None else _ptrs(dA, "dA", lins)
        self.dB = None if dB is None else _ptrs(dB, "dB", lins)
        self.dMag = _ptrs(dMag, "dMag", lins, True)
        self.ws = _ptr(ws, "ws", None)
        self.ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
        self.stream = _stream(stream)
        self._held = (Y, U, Z, dX, dA, dB, dMag, ws, stream)   # the marshalled buffers stay alive
        self._x = self._xp = None
        self._dy = self._dyp = None

    def _x_ptr(self, X):
        if X is not self._x:
            self._xp = _sized(X, "X", _NEED["X"](self.lins[0]))
            self._x = X
        return self._xp

    def _dy_ptrs(self, dY):
        if self._dy is None or len(dY) != len(self._dy) or any(a is not b for a, b in zip(dY, self._dy)):
            self._dyp = _ptrs(dY, "dY", self.lins)
            self._dy = list(dY)
        return self._dyp

    def dropouts(self, drops):
        """The marshalled dropout keys (one LoraDropout or None per linear),
        to pass to forward and backward of the same chunk."""
        return _drops(drops, self.n)

    def _d(self, drops):
        return drops if drops is None or isinstance(drops, C.Array) else _drops(drops, self.n)

    def forward(self, X, drops=None):
        rc = lib().lora_forward_group(self.n, self.arr, self._x_ptr(X), self.Y, self.U, self.Zf,
                                      self._d(drops), self.ws, self.ws_bytes, self.stream)
        _check("lora_forward_group", rc)

    def backward(self, X, dY, accumulate=False, drops=None):
        if self.dA is None or self.dB is None:
            raise ValueError("this GroupCall was prepared without gradients")
        rc = lib().lora_backward_group(self.n, self.arr, self._x_ptr(X), self._dy_ptrs(dY),
                                       self.U, self.Zb, self.dX, self.dA, self.dB, self.dMag,
                                       1 if accumulate else 0, self._d(drops), self.ws,
                                       self.ws_bytes, self.stream)
        _check("lora_backward_group", rc)


def lora_slots_workspace_bytes(lins) -> int:
    return int(lib().lora_slots_workspace_bytes(len(lins), _linears(lins)))


def lora_forward_slots(lins, X, Y, U, Z=None, drops=None, ws=None, stream=None):
    """Forward of adapter slots over one W: every tensor argument is a list
    with one entry per slot."""
    n = len(lins)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_forward_slots(n, _linears(lins), _ptrs(X, "X", lins), _ptrs(Y, "Y", lins),
                                  _ptrs(U, "U", lins), _ptrs(Z, "Z", lins, True),
                                  _drops(drops, n), _ptr(ws, "ws", None),
                                  ws_bytes, _stream(stream))
    _check("lora_forward_slots", rc)


def lora_backward_slots(lins, X, dY, U, Z, dX, dA, dB, dMag=None, accumulate=False, drops=None,
                        ws=None, stream=None):
    """Backward of adapter slots over one W: every tensor argument is a list
    with one entry per slot."""
    n = len(lins)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_backward_slots(n, _linears(lins), _ptrs(X, "X", lins), _ptrs(dY, "dY", lins),
                                   _ptrs(U, "U", lins), _ptrs(Z, "Z", lins, True),
                                   _ptrs(dX, "dX", lins, True), _ptrs(dA, "dA", lins),
                                   _ptrs(dB, "dB", lins), _ptrs(dMag, "dMag", lins, True),
                                   1 if accumulate else 0, _drops(drops, n), _ptr(ws, "ws", None),
                                   ws_bytes, _stream(stream))
    _check("lora_backward_slots", rc)


def lora_grad_prepare_workspace_bytes(n: int) -> int:
    return int(lib().lora_grad_prepare_workspace_bytes(int(n)))


def lora_grad_prepare(grads, n_pred_tokens, max_norm, d_scale, d_stats=None, sync=True,
                      ws=None, stream=None):
    """Returns the norm (host float) when sync is True, else None.  A vetoed
    (non-finite) update raises LoraError with status LORA_E_NONFINITE when
    sync is True; otherwise the veto travels in d_scale (NaN)."""
    n = grads.numel()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    h = C.c_double(0.0)
    rc = lib().lora_grad_prepare(_ptr(grads, "grads"), n, int(n_pred_tokens), float(max_norm),
                                 _ptr(d_scale, "d_scale"), _ptr(d_stats, "d_stats", torch.float64),
                                 C.byref(h) if sync else None, _ptr(ws, "ws", None), ws_bytes,
                                 _stream(stream))
    _check("lora_grad_prepare", rc)
    return h.value if sync else None


def lora_grad_prepare_noalloc(grads, n_pred_tokens, max_norm, d_scale, d_stats=None, sync=True,
                              stream=None):
    """lora_grad_prepare with the library's static device scratch in place of
    a workspace (nothing is allocated); same returns and errors."""
    h = C.c_double(0.0)
    rc = lib().lora_grad_prepare_noalloc(_ptr(grads, "grads"), grads.numel(), int(n_pred_tokens),
                                         float(max_norm), _ptr(d_scale, "d_scale"),
                                         _ptr(d_stats, "d_stats", torch.float64),
                                         C.byref(h) if sync else None, _stream(stream))
    _check("lora_grad_prepare_noalloc", rc)
    return h.value if sync else None


def lora_adamw_step(params, grads, m, v, segments, hp: LoraAdamwHparams, d_scale, stream=None):
    segs = (LoraSegment * len(segments))(*[LoraSegment(int(o), int(c), int(k)) for o, c, k in segments])
    end = max((int(o) + int(c) for o, c, _ in segments), default=0)
    rc = lib().lora_adamw_step(_sized(params, "params", end), _sized(grads, "grads", end),
                               _sized(m, "m", end), _sized(v, "v", end), segs, len(segments),
                               C.byref(hp), _sized(d_scale, "d_scale", 1), _stream(stream))
    _check("lora_adamw_step", rc)


def lora_dropout_mask(drop: LoraDropout, tokens, in_dim, mask, stream=None):
    rc = lib().lora_dropout_mask(C.byref(drop), int(tokens), int(in_dim),
                                 _sized(mask, "mask", int(tokens) * int(in_dim), torch.uint8),
                                 _stream(stream))
    _check("lora_dropout_mask", rc)


def lora_dora_row_norms_workspace_bytes(lin: LoraLinear) -> int:
    return int(lib().lora_dora_row_norms_workspace_bytes(C.byref(lin)))


def lora_dora_row_norms(lin: LoraLinear, out_norm, ws=None, stream=None, split=True):
    """Row norms of W + s B A into out_norm.  `ws` is a device uint8 tensor of
    at least lora_dora_row_norms_workspace_bytes(lin) bytes; when it is None
    one is taken from torch's allocator (split=False passes none at all)."""
    if ws is None and split:
        need = lora_dora_row_norms_workspace_bytes(lin)
        if need:
            ws = _own_ws(need, out_norm.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_dora_row_norms(C.byref(lin), _sized(out_norm, "out_norm", lin.out_dim),
                                   _ptr(ws, "ws", None), ws_bytes, _stream(stream))
    _check("lora_dora_row_norms", rc)


def lora_dora_row_norms_batch_workspace_bytes(lins) -> int:
    return int(lib().lora_dora_row_norms_batch_workspace_bytes(len(lins), _linears(lins)))


def lora_dora_row_norms_batch(lins, out_norms, ws=None, stream=None):
    """Row norms of W + s B A for every linear of `lins` into the matching
    entry of `out_norms`; `ws` as lora_dora_row_norms_batch_workspace_bytes
    asks (taken from torch's allocator when None)."""
    if len(lins) == 0:
        return
    if ws is None:
        need = lora_dora_row_norms_batch_workspace_bytes(lins)
        if need:
            ws = _own_ws(need, out_norms[0].device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_dora_row_norms_batch(len(lins), _linears(lins),
                                         _ptrs(out_norms, "out_norm", lins), _ptr(ws, "ws", None),
                                         ws_bytes, _stream(stream))
    _check("lora_dora_row_norms_batch", rc)


def lora_merge_workspace_bytes(lin: LoraLinear) -> int:
    return int(lib().lora_merge_workspace_bytes(C.byref(lin)))


def lora_merge(lin: LoraLinear, W_out, rmse=None, ws=None, stream=None):
    """W_out = c (W + s B A) (c = mag/norm for DoRA) as float32 or bfloat16
    (W_out's dtype).  `rmse` is a device float64 tensor of one element or
    None; bf16 output needs `ws` (taken from torch's allocator when None)."""
    if W_out.dtype == torch.float32:
        od = F32
    elif W_out.dtype == torch.bfloat16:
        od = BF16
    else:
        raise TypeError(f"W_out must be float32 or bfloat16, got {W_out.dtype}")
    if rmse is not None and ws is None and od == BF16:
        ws = _own_ws(max(8, lora_merge_workspace_bytes(lin)), W_out.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_merge(C.byref(lin), _sized(W_out, "W_out", lin.out_dim * lin.in_dim, None), od,
                          _sized(rmse, "rmse", 1, torch.float64), _ptr(ws, "ws", None), ws_bytes,
                          _stream(stream))
    _check("lora_merge", rc)


# ------------------------------------------------------------ 8-bit products
@functools.lru_cache(maxsize=256)   # a pure function of the sizes
def _fp8_layout(fn, what, rows, cols):
    off = C.c_size_t()
    total = int(getattr(lib(), fn)(int(rows), int(cols), C.byref(off)))
    if total == 0:
        raise ValueError(f"no 8-bit layout for {what} [{rows}, {cols}]")
    return total, int(off.value)


def lora_fp8_weight_layout(out_dim, in_dim):
    """(bytes, offset of the scales) of an 8-bit W [out_dim, in_dim]."""
    return _fp8_layout("lora_fp8_weight_layout", "a weight", out_dim, in_dim)


def lora_fp8_operand_layout(rows, cols):
    """(bytes, offset of the exponents) of 8-bit activations [rows, cols]."""
    return _fp8_layout("lora_fp8_operand_layout", "activations", rows, cols)


class Fp8Weight:
    """An 8-bit W [out_dim, in_dim] in the library's layout (include/lora.h):
    one uint8 device buffer, e4m3 values in whole 128 x 128 blocks, then the
    blocks' float32 scales."""

    code = FP8

    def __init__(self, out_dim: int, in_dim: int, buf: torch.Tensor):
        total, _ = lora_fp8_weight_layout(out_dim, in_dim)
        _sized(buf, "an 8-bit W", total, torch.uint8)
        self.out_dim, self.in_dim, self.buf = int(out_dim), int(in_dim), buf

    @property
    def shape(self):
        return (self.out_dim, self.in_dim)


def fp8_pack(values, scales, device="cuda") -> Fp8Weight:
    """Lay out e4m3 values [N, K] (float8_e4m3fn) and block scales
    [ceil(N/128), ceil(K/128)] in one device buffer."""
    N, K = values.shape
    nb, kb = -(-N // 128), -(-K // 128)
    if values.dtype != torch.float8_e4m3fn:
        raise TypeError(f"values must be float8_e4m3fn, got {values.dtype}")
    if tuple(scales.shape) != (nb, kb):
        raise ValueError(f"scales must be [{nb}, {kb}], got {list(scales.shape)}")
    total, off = lora_fp8_weight_layout(N, K)
    buf = torch.zeros(total, dtype=torch.uint8, device=device)
    buf[:nb * 128 * kb * 128].view(nb * 128, kb * 128)[:N, :K].copy_(values.view(torch.uint8))
    buf[off:off + 4 * nb * kb].copy_(scales.float().contiguous().view(torch.uint8).flatten())
    return Fp8Weight(N, K, buf)


class Fp8Rows:
    """8-bit activations [rows, cols] with a power-of-two scale for each
    128-wide block of a row, as lora_fp8_quantize leaves them."""

    def __init__(self, rows: int, cols: int, buf: torch.Tensor):
        self.rows, self.cols, self.buf = int(rows), int(cols), buf
        total, _ = lora_fp8_operand_layout(rows, cols)
        self.desc = LoraFp8Operand(self.rows, self.cols,
                                   _sized(buf, "8-bit activations", total, torch.uint8))


def fp8_rows(rows, cols, device="cuda") -> Fp8Rows:
    """Room for 8-bit activations [rows, cols], from torch's allocator."""
    return Fp8Rows(rows, cols, torch.empty(lora_fp8_operand_layout(rows, cols)[0], device=device,
                                           dtype=torch.uint8))


def lora_fp8_quantize(X, out: Fp8Rows, stream=None):
    """Round X [rows, cols] (float32 or bfloat16, rows any distance apart)
    into `out`."""
    ld = X.stride(0) if isinstance(X, torch.Tensor) and X.dim() == 2 and out.rows > 1 else out.cols
    dt = _act(X.dtype)
    rc = lib().lora_fp8_quantize(_rows_ptr(X, "X", out.rows, out.cols, ld, dt), dt, ld,
                                 C.byref(out.desc), _stream(stream))
    _check("lora_fp8_quantize", rc)


def lora_fp8_product_workspace_bytes(x: Fp8Rows, W: Fp8Weight, dx=False) -> int:
    return int(lib().lora_fp8_product_workspace_bytes(C.byref(x.desc), W.out_dim, W.in_dim,
                                                      1 if dx else 0))


def lora_fp8_product(x: Fp8Rows, W: Fp8Weight, out, dx=False, ws=None, stream=None):
    """out = x W^T, or x W with dx (x the rounded X or dY); out is float32 or
    bfloat16, `ws` is taken from torch's allocator when None."""
    if x.cols != (W.out_dim if dx else W.in_dim):
        raise ValueError(f"x has {x.cols} columns for W [{W.out_dim}, {W.in_dim}], dx={dx}")
    if ws is None:
        need = lora_fp8_product_workspace_bytes(x, W, dx)
        if need:
            ws = _own_ws(need, out.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_fp8_product(C.byref(x.desc), W.buf.data_ptr(), W.out_dim, W.in_dim,
                                1 if dx else 0,
                                _sized(out, "out", x.rows * (W.in_dim if dx else W.out_dim), None),
                                _act(out.dtype), _ptr(ws, "ws", None), ws_bytes, _stream(stream))
    _check("lora_fp8_product", rc)


# ------------------------------------------------------ orthogonalised update
MUON_ADJUST = {"shape": 0, "rms": 1}


def make_matrix_run(offset, rows, cols, count=1, stride=None, kind=KIND_A) -> LoraMatrixRun:
    """`count` matrices [rows, cols] of an arena, the first at element
    `offset`, `stride` elements apart (default: one after another)."""
    return LoraMatrixRun(int(offset), int(rows * cols if stride is None else stride), int(count),
                         int(rows), int(cols), int(kind))


def make_muon(lr, momentum=0.95, weight_decay=0.0, plus_ratio=1.0, eps=1e-7,
              coeffs=(3.4445, -4.7750, 2.0315), steps=5, nesterov=True,
              adjust="shape") -> LoraMuonHparams:
    """Hyper-parameters of lora_muon_step (and, without the step itself, of
    lora_orthogonalize)."""
    if adjust not in MUON_ADJUST:
        raise ValueError(f"adjust must be one of {sorted(MUON_ADJUST)}, got {adjust!r}")
    a, b, c = coeffs
    return LoraMuonHparams(float(lr), float(momentum), float(weight_decay), float(plus_ratio),
                           float(eps), float(a), float(b), float(c), int(steps),
                           1 if nesterov else 0, MUON_ADJUST[adjust])


def _runs(runs):
    """The marshalled runs and the arena length that they reach."""
    end = max((r.offset + (r.count - 1) * r.stride + r.rows * r.cols for r in runs), default=0)
    return (LoraMatrixRun * len(runs))(*runs), end


def lora_muon_workspace_bytes(runs) -> int:
    return int(lib().lora_muon_workspace_bytes(_runs(runs)[0], len(runs)))


def _muon_ws(arr, n, ws, device, stream):
    if ws is None:
        ws = _own_ws(max(16, int(lib().lora_muon_workspace_bytes(arr, n))), device, stream)
    return ws


def lora_orthogonalize(G, O, runs, hp: LoraMuonHparams, ws=None, stream=None):
    """O = the orthogonalised matrices of the arena G; `ws` is
    taken from torch's allocator when None."""
    arr, end = _runs(runs)
    g, o = _sized(G, "G", end), _sized(O, "O", end)
    ws = _muon_ws(arr, len(runs), ws, G.device, stream)
    rc = lib().lora_orthogonalize(g, o, arr, len(runs), C.byref(hp), _ptr(ws, "ws", None),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check("lora_orthogonalize", rc)


def lora_muon_step(params, grads, m, runs, hp: LoraMuonHparams, d_scale, ws=None, stream=None):
    """Momentum, orthogonalisation and update of the matrices of `runs`;
    `ws` is taken from torch's allocator when None."""
    arr, end = _runs(runs)
    p, g, mo = _sized(params, "params", end), _sized(grads, "grads", end), _sized(m, "m", end)
    ws = _muon_ws(arr, len(runs), ws, params.device, stream)
    rc = lib().lora_muon_step(p, g, mo, arr, len(runs), C.byref(hp), _sized(d_scale, "d_scale", 1),
                              _ptr(ws, "ws", None), ws.numel() * ws.element_size(),
                              _stream(stream))
    _check("lora_muon_step", rc)


# --------------------------------------------------------------- row norms
NORM_KINDS = {"layer": 0, "rms": 1}
_ACT_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _act(dtype) -> int:
    if dtype not in _ACT_DTYPES:
        raise TypeError(f"activations must be float32 or bfloat16, got {dtype}")
    return _ACT_DTYPES[dtype]


def make_norm(kind, rows, dim, dtype=torch.float32, eps=1e-5, gamma=None, beta=None, ldx=None,
              ldy=None) -> LoraNorm:
    """Descriptor of a row norm ("layer" or "rms") over X [rows, dim]; ldx and
    ldy are the elements between rows of X, dX and of Y, dY (default dim).  The
    descriptor keeps gamma and beta alive."""
    if kind not in NORM_KINDS:
        raise ValueError(f"norm kind must be one of {sorted(NORM_KINDS)}, got {kind!r}")
    dt = _act(dtype)
    norm = LoraNorm(int(rows), int(dim), int(dim if ldx is None else ldx),
                    int(dim if ldy is None else ldy), NORM_KINDS[kind], dt,
                    _sized(gamma, "gamma", int(dim)), _sized(beta, "beta", int(dim)), float(eps))
    norm.vectors = (gamma, beta)   # the structure itself holds only their addresses
    return norm


def _rows_ptr(t, name, rows, dim, ld, dtype):
    """Device pointer of a [rows, dim] tensor whose rows are ld elements
    apart (a column slice of a wider matrix, say)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if _act(t.dtype) != dtype:
        raise TypeError(f"{name} must be {'float32' if dtype == F32 else 'bfloat16'}, got {t.dtype}")
    if tuple(t.shape) != (rows, dim):
        raise ValueError(f"{name} must be [{rows}, {dim}], got {list(t.shape)}")
    if (dim > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) != ld):
        raise ValueError(f"{name} must have strides [{ld}, 1], got {list(t.stride())}")
    return t.data_ptr()


def lora_norm_forward(norm: LoraNorm, X, Y, stats=None, stream=None):
    """Y = norm(X); stats [rows, 2] float32 receives each row's mean and rstd."""
    r, d = norm.rows, norm.dim
    rc = lib().lora_norm_forward(C.byref(norm), _rows_ptr(X, "X", r, d, norm.ldx, norm.dtype),
                                 _rows_ptr(Y, "Y", r, d, norm.ldy, norm.dtype),
                                 _sized(stats, "stats", 2 * r), _stream(stream))
    _check("lora_norm_forward", rc)


def lora_norm_workspace_bytes(norm: LoraNorm) -> int:
    return int(lib().lora_norm_workspace_bytes(C.byref(norm)))


def lora_norm_backward(norm: LoraNorm, X, dY, stats, dX=None, dgamma=None, dbeta=None,
                       accumulate=False, ws=None, stream=None):
    """Gradients of lora_norm_forward from the gradients of Y in the list dY
    (one to four, summed).  A workspace is taken from torch's allocator when
    dgamma or dbeta is wanted and `ws` is None."""
    r, d, dt = norm.rows, norm.dim, norm.dtype
    if not 1 <= len(dY) <= MAX_GROUP:
        raise ValueError(f"dY must hold 1 to {MAX_GROUP} gradients, got {len(dY)}")
    dys = (C.c_void_p * len(dY))(*[_rows_ptr(t, f"dY[{i}]", r, d, norm.ldy, dt)
                                   for i, t in enumerate(dY)])
    if ws is None and (dgamma is not None or dbeta is not None):
        need = lora_norm_workspace_bytes(norm)
        if need:
            ws = _own_ws(need, X.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().lora_norm_backward(C.byref(norm), _rows_ptr(X, "X", r, d, norm.ldx, dt), len(dY),
                                  dys, _sized(stats, "stats", 2 * r),
                                  _rows_ptr(dX, "dX", r, d, norm.ldx, dt),
                                  _sized(dgamma, "dgamma", d), _sized(dbeta, "dbeta", d),
                                  1 if accumulate else 0, _ptr(ws, "ws", None), ws_bytes,
                                  _stream(stream))
    _check("lora_norm_backward", rc)


# ------------------------------------------------------ heads and attention
def rope_freqs(rot_dim, base=10000.0, device="cuda"):
    """base^(-2i/rot_dim) for the pairs i < rot_dim / 2, in float64: radians a
    position."""
    i = torch.arange(0, int(rot_dim), 2, dtype=torch.float64)
    return (float(base) ** (-i / int(rot_dim))).to(device)


def _device_ints(t, name, need):
    return _sized(t, name, need, torch.int32)


def _here(stream):
    """The current device, on which a call's kernels are launched (-2: none;
    -1 is what CPU tensors are on)."""
    try:
        here = torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != here:
        raise ValueError(f"the stream is of GPU {stream.device_index}, the current one is {here}")
    return here


def _stream_on(stream, here):
    """_stream, with the current device known."""
    return _raw_stream(here) if stream is None and _raw_stream is not None and here >= 0 else _stream(stream)


def _all_here(here, *ts):
    for t in ts:
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor of the call is on GPU {t.get_device()}, the current one is {here}")


def make_heads(tokens, heads, head_dim, x_dtype=torch.float32, y_dtype=None, norm=True, eps=1e-6, gamma=None,
               rot_dim=None, freqs=None, interleaved=False, ldx=None, hx=None, ldy=None,
               hy=None) -> LoraHeads:
    """Descriptor of a set of heads: norm (RMS over the head; gamma None: ones)
    and rotation by `freqs` [rot_dim / 2] float64 (rope_freqs; None: no
    rotation).  ldx and hx (X, dX), ldy and hy (Y, dY) are the elements between
    tokens and between heads, by default those of [tokens, heads, head_dim].
    y_dtype (default x_dtype) is the type of Y and of dY.  The descriptor keeps
    gamma and freqs alive."""
    rot = (0 if freqs is None else 2 * freqs.numel()) if rot_dim is None else int(rot_dim)
    t, h, d = int(tokens), int(heads), int(head_dim)
    hx, hy = int(d if hx is None else hx), int(d if hy is None else hy)
    ldx, ldy = int(h * d if ldx is None else ldx), int(h * d if ldy is None else ldy)
    out = LoraHeads(t, h, d, rot, ldx, hx, ldy, hy, _act(x_dtype), _act(y_dtype or x_dtype),
                    1 if norm else 0, 1 if interleaved else 0, _sized(gamma, "gamma", d),
                    _sized(freqs, "freqs", rot // 2, torch.float64), float(eps))
    out.vectors = (gamma, freqs)
    return out


def _strided(t, name, i, tokens, heads, dim, ld, h, dtype, here):
    """Device pointer, on GPU `here`, of heads whose tokens are ld and heads h
    elements apart: a [tokens, heads, dim] tensor of those strides, or (where
    the heads of a token lie together) [tokens, heads * dim]."""
    if t is None:
        return None
    name = name if i is None else f"{name}[{i}]"
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    _all_here(here, t)
    if _act(t.dtype) != dtype:
        raise TypeError(f"{name} must be {'float32' if dtype == F32 else 'bfloat16'}, got {t.dtype}")
    if t.dim() == 2 and tuple(t.shape) == (tokens, heads * dim) and (h == dim or heads == 1):
        shape, want = (tokens, heads * dim), (ld, 1)
    else:
        shape, want = (tokens, heads, dim), (ld, h, 1)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}], got {list(t.shape)}")
    if any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), want)):
        raise ValueError(f"{name} must have strides {list(want)}, got {list(t.stride())}")
    return t.data_ptr()


def _head_ptr(t, name, i, tokens, heads, dim, ld, h, dtype, here):
    """_strided, in few steps for the usual tensors (a token's call is host
    time: the checks above take 2 us a tensor)."""
    if type(t) is torch.Tensor and t.get_device() == here and _ACT_DTYPES.get(t.dtype) == dtype:
        shape, st = t.shape, t.stride()
        if (shape == (tokens, heads, dim) and st == (ld, h, 1)) or \
                (h == dim and shape == (tokens, heads * dim) and st == (ld, 1)):
            return t.data_ptr()
    return _strided(t, name, i, tokens, heads, dim, ld, h, dtype, here)


def _head_ptrs(heads, ts, name, x, here):
    if ts is None:
        return None
    if len(ts) != len(heads):
        raise ValueError(f"{name} has {len(ts)} entries for {len(heads)} sets of heads")
    out = (C.c_void_p * len(ts))()
    for i, d in enumerate(heads):
        out[i] = _head_ptr(ts[i], name, i, d.tokens, d.heads, d.head_dim,
                           *((d.ldx, d.hx, d.x_dtype) if x else (d.ldy, d.hy, d.y_dtype)), here)
    return out


def lora_heads_forward(heads, X, Y, positions=None, stream=None):
    """Y[i] = the heads X[i], normed and rotated, for each set of `heads` (one
    to four of the same tokens); positions [tokens] int32."""
    arr = (LoraHeads * len(heads))(*heads)
    here = _here(stream)
    px, py = _head_ptrs(heads, X, "X", True, here), _head_ptrs(heads, Y, "Y", False, here)
    pos = _device_ints(positions, "positions", heads[0].tokens if len(heads) else 0)
    _all_here(here, positions, *[t for d in heads for t in getattr(d, "vectors", ())])
    rc = lib().lora_heads_forward(len(heads), arr, px, py, pos, _stream_on(stream, here))
    _check("lora_heads_forward", rc)


def lora_heads_workspace_bytes(heads) -> int:
    return int(lib().lora_heads_workspace_bytes(len(heads), (LoraHeads * len(heads))(*heads)))


def lora_heads_backward(heads, X, dY, dX=None, dgamma=None, positions=None, accumulate=False, ws=None,
                        stream=None):
    """Gradients of lora_heads_forward; dX and dgamma are lists (entries may be
    None).  `ws` is taken from torch's allocator when a dgamma is wanted and it
    is None."""
    arr = (LoraHeads * len(heads))(*heads)
    if dgamma is not None and len(dgamma) != len(heads):
        raise ValueError(f"dgamma has {len(dgamma)} entries for {len(heads)} sets of heads")
    dg = None if dgamma is None else (C.c_void_p * len(heads))(
        *[_sized(t, f"dgamma[{i}]", h.head_dim) for i, (t, h) in enumerate(zip(dgamma, heads))])
    here = _here(stream)
    px, py = _head_ptrs(heads, X, "X", True, here), _head_ptrs(heads, dY, "dY", False, here)
    pdx = _head_ptrs(heads, dX, "dX", True, here)
    pos = _device_ints(positions, "positions", heads[0].tokens if len(heads) else 0)
    _all_here(here, positions, ws, *(dgamma or ()), *[t for d in heads for t in getattr(d, "vectors", ())])
    if ws is None and dgamma is not None and any(t is not None for t in dgamma):
        need = int(lib().lora_heads_workspace_bytes(len(heads), arr))
        if need:
            ws = _own_ws(need, dY[0].device, stream)
    rc = lib().lora_heads_backward(len(heads), arr, px, py, pdx, dg, pos, 1 if accumulate else 0, _ptr(ws, "ws", None),
                                   0 if ws is None else ws.numel() * ws.element_size(), _stream_on(stream, here))
    _check("lora_heads_backward", rc)


def make_attention(q_tokens, k_tokens, heads, kv_heads, head_dim, q_offsets, k_offsets, k_lens=None,
                   dtype=torch.bfloat16, out_dtype=None, scale=None, causal=True, q_strides=None, k_strides=None,
                   v_strides=None, o_strides=None) -> LoraAttention:
    """Descriptor of attention over the packed sequences of q_offsets and
    k_offsets [sequences + 1] (k_lens [sequences]: the keys in use of each
    sequence's room), int32 on the GPU.  Strides are (elements between tokens,
    between heads), by default those of [tokens, heads, head_dim].  out_dtype
    (default dtype) is the type of O and of all gradients; scale defaults to
    head_dim^-1/2.  The descriptor keeps the offsets alive."""
    d, seqs = int(head_dim), int(q_offsets.numel()) - 1
    st = lambda given, n: (int(n) * d, d) if given is None else tuple(map(int, given))
    at = LoraAttention(int(q_tokens), int(k_tokens), int(heads), int(kv_heads), d, seqs, *st(q_strides, heads),
                       *st(k_strides, kv_heads), *st(v_strides, kv_heads), *st(o_strides, heads), _act(dtype),
                       _act(out_dtype or dtype), 1 if causal else 0, float(d ** -0.5 if scale is None else scale),
                       _device_ints(q_offsets, "q_offsets", 1), _device_ints(k_offsets, "k_offsets", seqs + 1),
                       _device_ints(k_lens, "k_lens", seqs))
    at.vectors = (q_offsets, k_offsets, k_lens)
    return at


def lora_attention_workspace_bytes(at: LoraAttention, backward=False) -> int:
    return int(lib().lora_attention_workspace_bytes(C.byref(at), 1 if backward else 0))


def _attn_ptrs(at, ts, here):
    """Device pointers of tensors laid out like Q, K, V or O: (tensor, name,
    whose strides, whether of out_dtype)."""
    q, k, d, io = (at.q_tokens, at.heads), (at.k_tokens, at.kv_heads), at.head_dim, (at.dtype, at.out_dtype)
    lay = {"q": (*q, d, at.ldq, at.hq), "k": (*k, d, at.ldk, at.hk), "v": (*k, d, at.ldv, at.hv),
           "o": (*q, d, at.ldo, at.ho)}
    return [_head_ptr(t, name, None, *lay[of], io[out], here) for t, name, of, out in ts]


def lora_attention_forward(at: LoraAttention, Q, K, V, O, lse=None, ws=None, stream=None):
    """O = attention of Q over K and V; lse [heads, q_tokens] float32 receives
    what the backward needs.  `ws` is taken from torch's allocator when one is
    needed and it is None."""
    here = _here(stream)
    ptrs = _attn_ptrs(at, ((Q, "Q", "q", 0), (K, "K", "k", 0), (V, "V", "v", 0), (O, "O", "o", 1)), here)
    ptrs.append(_sized(lse, "lse", at.heads * at.q_tokens))
    _all_here(here, lse, ws, *getattr(at, "vectors", ()))
    if ws is None:
        need = int(lib().lora_attention_workspace_bytes(C.byref(at), 0))
        if need:
            ws = _own_ws(need, O.device, stream)
    rc = lib().lora_attention_forward(C.byref(at), *ptrs, _ptr(ws, "ws", None),
                                      0 if ws is None else ws.numel() * ws.element_size(), _stream_on(stream, here))
    _check("lora_attention_forward", rc)


def lora_attention_backward(at: LoraAttention, Q, K, V, O, dO, lse, dQ, dK, dV, ws=None, stream=None):
    """Gradients of lora_attention_forward from dO; `ws` is taken from torch's
    allocator when None."""
    here = _here(stream)
    ptrs = _attn_ptrs(at, ((Q, "Q", "q", 0), (K, "K", "k", 0), (V, "V", "v", 0), (O, "O", "o", 1), (dO, "dO", "o", 1),
                           (dQ, "dQ", "q", 1), (dK, "dK", "k", 1), (dV, "dV", "v", 1)), here)
    ptrs.insert(5, _sized(lse, "lse", at.heads * at.q_tokens))
    _all_here(here, lse, ws, *getattr(at, "vectors", ()))
    if ws is None:
        ws = _own_ws(max(16, int(lib().lora_attention_workspace_bytes(C.byref(at), 1))), dQ.device, stream)
    rc = lib().lora_attention_backward(C.byref(at), *ptrs, _ptr(ws, "ws", None), ws.numel() * ws.element_size(),
                                       _stream_on(stream, here))
    _check("lora_attention_backward", rc)


def lora_set_bf16_config(cfg: int):
    """Pin the tile configuration of the bf16-W products (-1: the planner
    chooses per product).  Process-wide; size workspaces after setting it."""
    _check("lora_set_bf16_config", lib().lora_set_bf16_config(int(cfg)))


def lora_profile_begin(max_launches: int = 100000):
    _check("lora_profile_begin", lib().lora_profile_begin(int(max_launches)))


def lora_profile_end(max_entries: int = 512) -> list:
    """Close the profile; returns dicts with kernel, M, N, K, launches,
    total_ms, avg_ms, flops and bytes (per launch)."""
    buf = (LoraProfileEntry * max_entries)()
    n = lib().lora_profile_end(buf, max_entries)
    if n < 0:
        raise LoraError("lora_profile_end", n)
    out = []
    for e in buf[:n]:
        out.append(dict(kernel=e.kernel.decode(), M=e.M, N=e.N, K=e.K, launches=e.launches,
                        total_ms=e.total_ms, avg_ms=e.total_ms / max(1, e.launches),
                        flops=e.flops, bytes=e.bytes))
    return out
