"""ctypes binding of libmoe_mxfp4.so (argument marshalling only).

Each function has the name of the C entry point it calls and takes torch
tensors that live on the GPU; it checks dtypes, shapes and contiguity, passes
raw device pointers and the current HIP stream, and raises MoeError on a
non-OK status.  No step of the layer runs here: every one runs in the HIP
library.  If the library is missing, load() raises instead of falling back to
anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mxfp4.so")

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_MISALIGNED", 4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_HIP"}

EXPORTS = ("moe_route", "moe_build_bitmatrix", "moe_expert_offsets", "moe_route_and_group",
           "moe_grouped_ffn_mxfp4", "moe_combine", "moe_workspace_bytes", "moe_status_string",
           "moe_route_scored", "moe_route_scored_and_group", "moe_quantize_fp8", "moe_gemm_fp8",
           "moe_gemm_fp8_workspace_bytes", "moe_grouped_ffn_fp8", "moe_fp8_workspace_bytes",
           "moe_rms_norm", "moe_rms_norm_grad", "moe_rms_norm_grad_workspace_bytes",
           "moe_balance_loss", "moe_balance_loss_grad", "moe_balance_loss_workspace_bytes",
           "moe_lora_group", "moe_lora_add", "moe_lora_add_workspace_bytes")


# bf16 buffers may be given as bfloat16 tensors or as int16 tensors of bit patterns
BF16 = (torch.bfloat16, torch.int16)


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SIG = {
    "moe_route": [_P, _I64, _I32, _I32, _P, _P, _P],
    "moe_build_bitmatrix": [_P, _I64, _I32, _I32, _P, _P],
    "moe_expert_offsets": [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_route_and_group": [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                            _P],
    "moe_grouped_ffn_mxfp4": [_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                              ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
    "moe_combine": [_P, _P, _P, _I64, _I32, _I32, _P, _P],
    "moe_forward_mxfp4": [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_float,
                          _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_forward_mxfp4_noalloc": [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                  ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "moe_forward_mxfp4_timed": [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P, _P],
    "moe_read_probe": [_P, ctypes.c_size_t, _P, _P],
    "moe_route_scored": [_P, _I32, _I64, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32,
                         ctypes.c_float, _P, _P, _P],
    "moe_route_scored_and_group": [_P, _I32, _I64, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32,
                                   ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P],
    "moe_quantize_fp8": [_P, _I64, _I32, _P, _P, _P],
    "moe_gemm_fp8": [_P, _P, _I64, _I32, _I32, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P],
    "moe_gemm_fp8_workspace_bytes": [_I64, _I32, _I32],
    "moe_grouped_ffn_fp8": [_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                            ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
    "moe_fp8_workspace_bytes": [_I64, _I32, _I32, _I32, _I32],
    "moe_rms_norm": [_P, _I64, _P, _I64, _I32, _I32, _P, ctypes.c_float, _P, _P, _P, _P, _P],
    "moe_rms_norm_grad": [_P, _I64, _I64, _I32, _I32, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                          ctypes.c_size_t, _P],
    "moe_rms_norm_grad_workspace_bytes": [_I64, _I32],
    "moe_balance_loss": [_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P, _P, _P,
                         ctypes.c_size_t, _P],
    "moe_balance_loss_grad": [_P, _I32, _I64, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P],
    "moe_balance_loss_workspace_bytes": [_I64, _I32, _I32],
    "moe_lora_group": [_P, _I64, _I32, _P, _P, _P],
    "moe_lora_add": [_P, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I32, _P, _I64, _P,
                     _I64, _P, ctypes.c_size_t, _P],
    "moe_lora_add_workspace_bytes": [_I64, _I32, _I32, _I32, _I32],
    "moe_workspace_bytes": [_I64, _I32, _I32, _I32, _I32],
    "moe_status_string": [ctypes.c_int],
}


def load(path: str = LIB_PATH):
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build it with `python -m "
                           "mxfp4_routed_expert_route_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    for name, args in _SIG.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("moe_workspace_bytes", "moe_gemm_fp8_workspace_bytes", "moe_fp8_workspace_bytes",
                 "moe_rms_norm_grad_workspace_bytes", "moe_balance_loss_workspace_bytes",
                 "moe_lora_add_workspace_bytes"):
        getattr(lib, name).restype = ctypes.c_size_t
    lib.moe_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor") -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None:
        ok = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
        if not ok:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, code: int):
    if code != 0:
        raise MoeError(fn, code)


def moe_workspace_bytes(T: int, E: int, k: int, H: int, I: int) -> int:
    return int(load().moe_workspace_bytes(T, E, k, H, I))


def moe_status_string(code: int) -> str:
    return load().moe_status_string(code).decode()


def moe_route(logits, k: int, topk_ids, topk_weights, stream=None):
    T, E = logits.shape
    _check("moe_route", load().moe_route(
        _ptr(logits, torch.float32, "logits"), T, E, k, _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_weights, torch.float32, "topk_weights"), _stream(stream)))


def moe_build_bitmatrix(topk_ids, E: int, bitmatrix, stream=None):
    T, k = topk_ids.shape
    _check("moe_build_bitmatrix", load().moe_build_bitmatrix(
        _ptr(topk_ids, torch.int32, "topk_ids"), T, E, k,
        _ptr(bitmatrix, torch.int32, "bitmatrix"), _stream(stream)))


def moe_expert_offsets(bitmatrix, topk_ids, E: int, counts, offsets, gather, scatter, ws,
                       stream=None):
    T, k = topk_ids.shape
    _check("moe_expert_offsets", load().moe_expert_offsets(
        _ptr(bitmatrix, torch.int32, "bitmatrix"), _ptr(topk_ids, torch.int32, "topk_ids"), T, E, k,
        _ptr(counts, torch.int32, "counts"), _ptr(offsets, torch.int32, "offsets"),
        _ptr(gather, torch.int32, "gather"), _ptr(scatter, torch.int32, "scatter"),
        _ptr(ws, torch.uint8, "ws"), ws.numel() if ws is not None else 0, _stream(stream)))


def moe_route_and_group(logits, k: int, topk_ids, topk_weights, bitmatrix, counts, offsets,
                        gather, scatter, ws, stream=None):
    T, E = logits.shape
    _check("moe_route_and_group", load().moe_route_and_group(
        _ptr(logits, torch.float32, "logits"), T, E, k, _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(bitmatrix, torch.int32, "bitmatrix"),
        _ptr(counts, torch.int32, "counts"), _ptr(offsets, torch.int32, "offsets"),
        _ptr(gather, torch.int32, "gather"), _ptr(scatter, torch.int32, "scatter"),
        _ptr(ws, torch.uint8, "ws"), ws.numel() if ws is not None else 0, _stream(stream)))


def moe_grouped_ffn_mxfp4(x, k: int, w1, w1_scale, w2, w2_scale, counts, offsets, gather,
                          swiglu_limit: float, y_sorted, ws, stream=None):
    T, H = x.shape
    E, two_i, _ = w1.shape
    _check("moe_grouped_ffn_mxfp4", load().moe_grouped_ffn_mxfp4(
        _ptr(x, BF16, "x"), T, H, two_i // 2, E, k, _ptr(w1, torch.uint8, "w1"),
        _ptr(w1_scale, torch.uint8, "w1_scale"), _ptr(w2, torch.uint8, "w2"),
        _ptr(w2_scale, torch.uint8, "w2_scale"), _ptr(counts, torch.int32, "counts"),
        _ptr(offsets, torch.int32, "offsets"), _ptr(gather, torch.int32, "gather"),
        float(swiglu_limit), _ptr(y_sorted, BF16, "y_sorted"), _ptr(ws, torch.uint8, "ws"),
        ws.numel() if ws is not None else 0, _stream(stream)))


def moe_combine(y_sorted, topk_weights, scatter, y, stream=None):
    T, k = topk_weights.shape
    H = y.shape[1]
    # on y's GPU, like the scored-routing and FP8 calls whose rows it sums
    _run("moe_combine", y.get_device(), stream,
         _ptr(y_sorted, BF16, "y_sorted"), _ptr(topk_weights, torch.float32, "topk_weights"),
         _ptr(scatter, torch.int32, "scatter"), T, H, k, _ptr(y, BF16, "y"))


def moe_forward_mxfp4(logits, x, k: int, w1, w1_scale, w2, w2_scale, swiglu_limit: float,
                      topk_ids, topk_weights, bitmatrix, counts, offsets, gather, scatter,
                      y_sorted, y, ws, stream=None):
    T, E = logits.shape
    H = x.shape[1]
    two_i = w1.shape[1]
    _check("moe_forward_mxfp4", load().moe_forward_mxfp4(
        _ptr(logits, torch.float32, "logits"), _ptr(x, BF16, "x"), T, H, two_i // 2, E, k,
        _ptr(w1, torch.uint8, "w1"), _ptr(w1_scale, torch.uint8, "w1_scale"),
        _ptr(w2, torch.uint8, "w2"), _ptr(w2_scale, torch.uint8, "w2_scale"),
        float(swiglu_limit), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(bitmatrix, torch.int32, "bitmatrix"), _ptr(counts, torch.int32, "counts"),
        _ptr(offsets, torch.int32, "offsets"), _ptr(gather, torch.int32, "gather"),
        _ptr(scatter, torch.int32, "scatter"), _ptr(y_sorted, BF16, "y_sorted"),
        _ptr(y, BF16, "y"), _ptr(ws, torch.uint8, "ws"), ws.numel() if ws is not None else 0,
        _stream(stream)))


def moe_forward_mxfp4_timed(logits, x, k: int, w1, w1_scale, w2, w2_scale, swiglu_limit: float,
                            topk_ids, topk_weights, bitmatrix, counts, offsets, gather, scatter,
                            y_sorted, y, ws, events, stream=None):
    """moe_forward_mxfp4 plus three HIP events recorded around its W1 and W2
    kernels; `events` holds three hipEvent_t handles (ints) created by the caller."""
    T, E = logits.shape
    H = x.shape[1]
    two_i = w1.shape[1]
    ev = None
    if events is not None:
        if len(events) != 3:
            raise ValueError("events must hold three hipEvent_t handles")
        ev = (ctypes.c_void_p * 3)(*events)
    _check("moe_forward_mxfp4_timed", load().moe_forward_mxfp4_timed(
        _ptr(logits, torch.float32, "logits"), _ptr(x, BF16, "x"), T, H, two_i // 2, E, k,
        _ptr(w1, torch.uint8, "w1"), _ptr(w1_scale, torch.uint8, "w1_scale"),
        _ptr(w2, torch.uint8, "w2"), _ptr(w2_scale, torch.uint8, "w2_scale"),
        float(swiglu_limit), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(bitmatrix, torch.int32, "bitmatrix"), _ptr(counts, torch.int32, "counts"),
        _ptr(offsets, torch.int32, "offsets"), _ptr(gather, torch.int32, "gather"),
        _ptr(scatter, torch.int32, "scatter"), _ptr(y_sorted, BF16, "y_sorted"),
        _ptr(y, BF16, "y"), _ptr(ws, torch.uint8, "ws"), ws.numel() if ws is not None else 0,
        ev, _stream(stream)))


# moe_forward_mxfp4_noalloc's static device scratch (MOE_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 128 << 20


def moe_forward_mxfp4_noalloc(logits, x, k: int, w1, w1_scale, w2, w2_scale,
                              swiglu_limit: float, topk_ids, topk_weights, bitmatrix, counts,
                              offsets, gather, scatter, y_sorted, y, stream=None):
    T, E = logits.shape
    H = x.shape[1]
    two_i = w1.shape[1]
    _check("moe_forward_mxfp4_noalloc", load().moe_forward_mxfp4_noalloc(
        _ptr(logits, torch.float32, "logits"), _ptr(x, BF16, "x"), T, H, two_i // 2, E, k,
        _ptr(w1, torch.uint8, "w1"), _ptr(w1_scale, torch.uint8, "w1_scale"),
        _ptr(w2, torch.uint8, "w2"), _ptr(w2_scale, torch.uint8, "w2_scale"),
        float(swiglu_limit), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(bitmatrix, torch.int32, "bitmatrix"), _ptr(counts, torch.int32, "counts"),
        _ptr(offsets, torch.int32, "offsets"), _ptr(gather, torch.int32, "gather"),
        _ptr(scatter, torch.int32, "scatter"), _ptr(y_sorted, BF16, "y_sorted"),
        _ptr(y, BF16, "y"), _stream(stream)))


READ_PROBE_SINK_WORDS = 8192


def moe_read_probe(buf, sink, stream=None):
    """Streaming read of every byte of `buf` (a contiguous device tensor, 16-byte
    aligned, size a multiple of 16); `sink` is an int32 device tensor of
    READ_PROBE_SINK_WORDS entries that receives the per-workgroup XORs."""
    if not buf.is_contiguous():
        raise ValueError("buf must be contiguous")
    if sink.dtype != torch.int32 or sink.numel() < READ_PROBE_SINK_WORDS:
        raise ValueError(f"sink must be int32 with >= {READ_PROBE_SINK_WORDS} entries")
    _check("moe_read_probe", load().moe_read_probe(
        _ptr(buf, None, "buf"), buf.numel() * buf.element_size(), _ptr(sink, torch.int32, "sink"),
        _stream(stream)))


# ------------------------------------------------------------ scored routing, block-scaled FP8
#
# These calls also check shapes, and that every tensor is on one GPU; they run on that GPU's
# current stream (or the one given).

# E4M3 buffers may be given as float8_e4m3fn tensors or as uint8 tensors of codes
E4M3 = (torch.float8_e4m3fn, torch.uint8)
SCORES = {"softmax": 0, "sigmoid": 1}
LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_LOGITS = tuple(LOGIT_TYPES)
FP8_BLOCK = 128


_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_several = None   # more than one GPU is visible
_fns = {}


def _arg(t, dtypes, shape, dev, name):
    """Pointer of a tensor on GPU `dev`, checked: dtype, shape, contiguity.  The checks cost
    about as much as a call's own launch, so a right tensor passes in one expression."""
    if t is not None and t.dtype in dtypes and t.shape == shape and t.get_device() == dev >= 0 and t.is_contiguous():
        return t.data_ptr()
    if t is None or t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {None if t is None else t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another GPU than the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


try:   # the same checks natively (csrc/marshal.cc), 0.1 us a tensor instead of 0.45
    from . import _marshal
except ImportError:   # not built, or for another PyTorch
    pass
else:
    _refuse = _arg
    _marshal.set_refuse(_refuse)
    _arg = _marshal.arg


def _ws(t, dev):
    return (None, 0) if t is None else (_arg(t, _U8, t.shape, dev, "ws"), t.numel())


def _run(fn: str, dev: int, stream, *args):
    """Calls entry point `fn` on `dev`'s current stream, or the stream given."""
    global _several
    if stream is None:
        handle = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    else:
        handle = _stream(stream)
    call = _fns.get(fn)
    if call is None:
        call = _fns[fn] = getattr(load(), fn)
        _several = torch.cuda.device_count() > 1
    if not _several or dev == torch.cuda.current_device():
        code = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = call(*args, handle)
    if code:
        raise MoeError(fn, code)


def _runs(n: int) -> int:
    return -(-n // FP8_BLOCK)


_END32 = 2 ** 31   # ctypes cuts a number to the C type's bits without a word


def _refuse_past_32_bits(**numbers):
    for name, v in numbers.items():
        if not -_END32 <= v < _END32:
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def _sizes(rows: int, *sizes: int) -> bool:
    """Whether a row count and sizes arrive as they are (64 and 32 bits)."""
    return rows < 2 ** 63 and all(v < _END32 for v in sizes) and min(rows, *sizes) >= 0


def _scored(logits, k, topk_ids, topk_weights, score, bias, groups, topk_groups, group_top,
            renormalize, scale):
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    kind = LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if not (E < _END32 and -_END32 <= k < _END32 and -_END32 <= groups < _END32
            and -_END32 <= topk_groups < _END32 and -_END32 <= group_top < _END32):
        _refuse_past_32_bits(E=E, k=k, groups=groups, topk_groups=topk_groups, group_top=group_top)
    dev = logits.get_device()
    return (_arg(logits, _LOGITS, (T, E), dev, "logits"), kind, T, E, k, SCORES[score],
            None if bias is None else _arg(bias, _F32, (E,), dev, "bias"),
            groups, topk_groups, group_top, 1 if renormalize else 0, scale,
            _arg(topk_ids, _I32, (T, k), dev, "topk_ids"),
            _arg(topk_weights, _F32, (T, k), dev, "topk_weights"))


def moe_route_scored(logits, k: int, topk_ids, topk_weights, *, score: str = "softmax", bias=None,
                     groups: int = 1, topk_groups: int = 1, group_top: int = 2,
                     renormalize: bool = True, scale: float = 1.0, stream=None):
    """Top-k over softmax or sigmoid scores plus a balance bias, within the best expert groups;
    weights are the chosen scores, renormalised or not, times `scale`."""
    how = _scored(logits, k, topk_ids, topk_weights, score, bias, groups, topk_groups, group_top,
                  renormalize, scale)
    _run("moe_route_scored", logits.get_device(), stream, *how)


def moe_route_scored_and_group(logits, k: int, topk_ids, topk_weights, bitmatrix, counts, offsets,
                               gather, scatter, ws, *, score: str = "softmax", bias=None,
                               groups: int = 1, topk_groups: int = 1, group_top: int = 2,
                               renormalize: bool = True, scale: float = 1.0, stream=None):
    """moe_route_scored, moe_build_bitmatrix and moe_expert_offsets in one call."""
    how = _scored(logits, k, topk_ids, topk_weights, score, bias, groups, topk_groups, group_top,
                  renormalize, scale)
    T, E = logits.shape
    dev = logits.get_device()
    _run("moe_route_scored_and_group", dev, stream, *how,
         _arg(bitmatrix, _I32, (T, (E + 31) // 32), dev, "bitmatrix"),
         _arg(counts, _I32, (E,), dev, "counts"), _arg(offsets, _I32, (E + 1,), dev, "offsets"),
         _arg(gather, _I32, (T * k,), dev, "gather"), _arg(scatter, _I32, (T * k,), dev, "scatter"),
         *_ws(ws, dev))


def moe_quantize_fp8(x, q, scale, stream=None):
    """bf16 rows [rows, K] to E4M3 codes q [rows, K] with scale [rows, ceil(K / 128)]."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    rows, K = x.shape
    if K >= _END32:
        _refuse_past_32_bits(K=K)
    dev = x.get_device()
    _run("moe_quantize_fp8", dev, stream, _arg(x, BF16, (rows, K), dev, "x"), rows, K,
         _arg(q, E4M3, (rows, K), dev, "q"),
         _arg(scale, _F32, (rows, _runs(K)), dev, "scale"))


def moe_gemm_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    """0 at every size."""
    if not _sizes(M, N, K):
        return 0
    return int(load().moe_gemm_fp8_workspace_bytes(M, N, K))


def moe_gemm_fp8(xq, x_scale, w, w_scale, y, ws=None, stream=None):
    """y [M, N] (bf16 or fp32) = X W^T of block-scaled E4M3 xq [M, K] and w [N, K].  No size
    needs a workspace (moe_gemm_fp8_workspace_bytes is 0)."""
    if xq.dim() != 2 or w.dim() != 2:
        raise ValueError("xq must be [M, K] and w [N, K]")
    M, K = xq.shape
    N = w.shape[0]
    if K >= _END32 or N >= _END32:
        _refuse_past_32_bits(K=K, N=N)
    dev, nk = xq.get_device(), _runs(K)
    kind = 0 if y.dtype is torch.float32 else 1
    _run("moe_gemm_fp8", dev, stream, _arg(xq, E4M3, (M, K), dev, "xq"),
         _arg(x_scale, _F32, (M, nk), dev, "x_scale"), M, N, K,
         _arg(w, E4M3, (N, K), dev, "w"), _arg(w_scale, _F32, (_runs(N), nk), dev, "w_scale"),
         kind, _arg(y, BF16 if kind else _F32, (M, N), dev, "y"), *_ws(ws, dev))


def moe_fp8_workspace_bytes(T: int, E: int, k: int, H: int, I: int) -> int:
    if not _sizes(T, E, k, H, I):
        return 0
    return int(load().moe_fp8_workspace_bytes(T, E, k, H, I))


def moe_grouped_ffn_fp8(x, k: int, w1, w1_scale, w2, w2_scale, counts, offsets, gather,
                        swiglu_limit: float, y_sorted, ws, stream=None):
    """The grouped expert FFN over block-scaled E4M3 weights w1 [E, 2I, H] (gate rows, then up
    rows) and w2 [E, H, I]; ws holds moe_fp8_workspace_bytes(T, E, k, H, I) bytes."""
    if x.dim() != 2 or w1.dim() != 3 or w1.shape[1] % 2:
        raise ValueError("x must be [T, H] and w1 [E, 2I, H]")
    T, H = x.shape
    E, I = w1.shape[0], w1.shape[1] // 2
    if not (H < _END32 and I < _END32 and E < _END32 and -_END32 <= k < _END32):
        _refuse_past_32_bits(H=H, I=I, E=E, k=k)
    dev = x.get_device()
    _run("moe_grouped_ffn_fp8", dev, stream, _arg(x, BF16, (T, H), dev, "x"), T, H, I, E, k,
         _arg(w1, E4M3, (E, 2 * I, H), dev, "w1"),
         _arg(w1_scale, _F32, (E, _runs(2 * I), _runs(H)), dev, "w1_scale"),
         _arg(w2, E4M3, (E, H, I), dev, "w2"),
         _arg(w2_scale, _F32, (E, _runs(H), _runs(I)), dev, "w2_scale"),
         _arg(counts, _I32, (E,), dev, "counts"), _arg(offsets, _I32, (E + 1,), dev, "offsets"),
         _arg(gather, _I32, (T * k,), dev, "gather"), swiglu_limit,
         _arg(y_sorted, BF16, (T * k, H), dev, "y_sorted"), *_ws(ws, dev))


# ------------------------------------------------------------ around the routed layer

_FLOATS = {torch.float32: 0, torch.bfloat16: 1, torch.int16: 1}


def _kind(t, name):
    kind = None if t is None else _FLOATS.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {None if t is None else t.dtype}")
    return kind


def _of_kind(kind):
    return BF16 if kind else _F32


def _rows(t, dtypes, shape, dev, name):
    """Pointer and row stride of a matrix whose rows are contiguous, checked like _arg's."""
    if t is None or t.is_contiguous() or t.dim() != 2 or t.stride(1) != 1 or t.shape != shape:
        return _arg(t, dtypes, shape, dev, name), shape[1]
    if t.dtype not in dtypes or t.get_device() != dev or dev < 0:
        _arg(t, dtypes, shape, dev, name)   # raises
    return t.data_ptr(), t.stride(0)


def _opt(t, dtypes, shape, dev, name):
    return None if t is None else _arg(t, dtypes, shape, dev, name)


def moe_rms_norm(x, weight, eps: float, *, residual=None, sum=None, y=None, q=None, scale=None,
                 stream=None):
    """RMS norm of s = bf16(x + residual) (or x), bf16 rows x [rows, H] (their stride may be more than
    H): y [rows, H] in bf16, or q [rows, H] in E4M3 with scale [rows, ceil(H / 128)], or both; s goes
    to sum.  weight [H] is fp32 or bf16."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, H]")
    rows, H = x.shape
    if H >= _END32:
        _refuse_past_32_bits(H=H)
    dev, kind = x.get_device(), _kind(weight, "weight")
    ptr, stride = _rows(x, BF16, (rows, H), dev, "x")
    _run("moe_rms_norm", dev, stream, ptr, stride, _opt(residual, BF16, (rows, H), dev, "residual"),
         rows, H, kind, _arg(weight, _of_kind(kind), (H,), dev, "weight"), eps,
         _opt(sum, BF16, (rows, H), dev, "sum"), _opt(y, BF16, (rows, H), dev, "y"),
         _opt(q, E4M3, (rows, H), dev, "q"), _opt(scale, _F32, (rows, _runs(H)), dev, "scale"))


def moe_rms_norm_grad_workspace_bytes(rows: int, H: int) -> int:
    if not _sizes(rows, H):
        return 0
    return int(load().moe_rms_norm_grad_workspace_bytes(rows, H))


def moe_rms_norm_grad(s, weight, eps: float, dy, dx, dweight, ws, *, dsum=None, stream=None):
    """Gradient of moe_rms_norm's y: dx [rows, H] bf16 by s (moe_rms_norm's sum, or x without a
    residual), with the gradient dsum that reaches s beside the norm, and dweight [H] fp32.  Either
    of dx and dweight may be None; ws holds moe_rms_norm_grad_workspace_bytes(rows, H) bytes."""
    if s.dim() != 2:
        raise ValueError("s must be [rows, H]")
    rows, H = s.shape
    if H >= _END32:
        _refuse_past_32_bits(H=H)
    dev, kind = s.get_device(), _kind(weight, "weight")
    ptr, stride = _rows(s, BF16, (rows, H), dev, "s")
    _run("moe_rms_norm_grad", dev, stream, ptr, stride, rows, H, kind,
         _arg(weight, _of_kind(kind), (H,), dev, "weight"), eps, _arg(dy, BF16, (rows, H), dev, "dy"),
         _opt(dsum, BF16, (rows, H), dev, "dsum"), _opt(dx, BF16, (rows, H), dev, "dx"),
         _opt(dweight, _F32, (H,), dev, "dweight"), *_ws(ws, dev))


def _balance(logits, k, score, seq_offsets, n_seqs):
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    kind = LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if not (E < _END32 and -_END32 <= k < _END32 and n_seqs < _END32):
        _refuse_past_32_bits(E=E, k=k, n_seqs=n_seqs)
    dev = logits.get_device()
    return (T, E, dev, (logits.dtype,), (_arg(logits, _LOGITS, (T, E), dev, "logits"), kind, T, E, k, SCORES[score]),
            _opt(seq_offsets, _I32, (n_seqs + 1,), dev, "seq_offsets"))


def moe_balance_loss_workspace_bytes(T: int, E: int, n_seqs: int = 1) -> int:
    if not _sizes(T, E, n_seqs):
        return 0
    return int(load().moe_balance_loss_workspace_bytes(T, E, n_seqs))


def moe_balance_loss(logits, topk_ids, loss, counts, ws, *, score: str = "softmax", seq_offsets=None,
                     dloss=None, dlogits=None, add_to=None, stream=None):
    """The balance loss [n_seqs] of router logits [T, E] and their chosen topk_ids [T, k] over packed
    sequences (seq_offsets [n_seqs + 1]; None: one of all tokens), and the experts' counts
    [n_seqs, E]; with dlogits, in the same pass, its gradient times dloss [n_seqs], plus add_to.
    ws holds moe_balance_loss_workspace_bytes(T, E, n_seqs) bytes."""
    if topk_ids.dim() != 2 or loss.dim() != 1:
        raise ValueError("topk_ids must be [T, k] and loss [n_seqs]")
    k, S = topk_ids.shape[1], loss.shape[0]
    T, E, dev, of, how, offsets = _balance(logits, k, score, seq_offsets, S)
    _run("moe_balance_loss", dev, stream, *how, _arg(topk_ids, _I32, (T, k), dev, "topk_ids"), offsets, S,
         _arg(loss, _F32, (S,), dev, "loss"), _arg(counts, _I32, (S, E), dev, "counts"),
         _opt(dloss, _F32, (S,), dev, "dloss"), _opt(add_to, of, (T, E), dev, "add_to"),
         _opt(dlogits, of, (T, E), dev, "dlogits"), *_ws(ws, dev))


def moe_balance_loss_grad(logits, k: int, counts, dloss, dlogits, *, score: str = "softmax",
                          seq_offsets=None, add_to=None, stream=None):
    """moe_balance_loss's dlogits alone, from its counts."""
    if dloss.dim() != 1:
        raise ValueError("dloss must be [n_seqs]")
    S = dloss.shape[0]
    T, E, dev, of, how, offsets = _balance(logits, k, score, seq_offsets, S)
    _run("moe_balance_loss_grad", dev, stream, *how, offsets, S, _arg(counts, _I32, (S, E), dev, "counts"),
         _arg(dloss, _F32, (S,), dev, "dloss"), _opt(add_to, of, (T, E), dev, "add_to"),
         _arg(dlogits, of, (T, E), dev, "dlogits"))


def moe_lora_group(adapter, L: int, offsets, rows, stream=None):
    """The rows of a batch in their adapters' order: adapter [M] is each row's adapter (outside
    0 .. L-1: none); rows [M], with adapter a's from offsets[a] to offsets[a + 1]."""
    if adapter.dim() != 1:
        raise ValueError("adapter must be [M]")
    M = adapter.shape[0]
    if not -_END32 <= L < _END32:
        _refuse_past_32_bits(L=L)
    dev = adapter.get_device()
    _run("moe_lora_group", dev, stream, _arg(adapter, _I32, (M,), dev, "adapter"), M, L,
         _arg(offsets, _I32, (L + 1,), dev, "offsets"), _arg(rows, _I32, (M,), dev, "rows"))


def moe_lora_add_workspace_bytes(M: int, N: int, K: int, R: int, L: int) -> int:
    if not _sizes(M, N, K, R, L):
        return 0
    return int(load().moe_lora_add_workspace_bytes(M, N, K, R, L))


def moe_lora_add(x, a, b, scaling, offsets, rows, base, y, ws, stream=None):
    """y [M, N] (bf16 or fp32) = base + scaling[l] (x A_l^T) B_l^T for the rows of each adapter l, base
    for the others; x [M, K], a [L, R, K] and b [L, N, R] are bf16, scaling [L] fp32 or None (1),
    offsets and rows moe_lora_group's.  base may be None (0), or y itself.  x, base and y may have row
    strides of their own; ws holds moe_lora_add_workspace_bytes(M, N, K, R, L) bytes."""
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [M, K], a [L, R, K] and b [L, N, R]")
    M, K = x.shape
    L, R, _ = a.shape
    N = b.shape[1]
    if not (K < _END32 and N < _END32 and R < _END32 and L < _END32):
        _refuse_past_32_bits(K=K, N=N, R=R, L=L)
    dev, kind = x.get_device(), _kind(y, "y")
    xp, xs = _rows(x, BF16, (M, K), dev, "x")
    bp, bs = (None, 0) if base is None else _rows(base, _of_kind(kind), (M, N), dev, "base")
    yp, ys = _rows(y, _of_kind(kind), (M, N), dev, "y")
    _run("moe_lora_add", dev, stream, xp, xs, M, K, N, R, L, _arg(a, BF16, (L, R, K), dev, "a"),
         _arg(b, BF16, (L, N, R), dev, "b"), _opt(scaling, _F32, (L,), dev, "scaling"),
         _arg(offsets, _I32, (L + 1,), dev, "offsets"), _arg(rows, _I32, (M,), dev, "rows"), kind, bp, bs,
         yp, ys, *_ws(ws, dev))
