"""NVFP4 W4A4 linear layer for GB300 (sm_103a): Python binding of ``include/nvfp4.h``.

The functions below carry the C entry points' names and arguments and do
argument marshalling only (tensor -> device pointer, current CUDA stream);
every step of the computation runs in the CUDA library
``libnvfp4_gb300.so``.  There is no fallback: if the library is missing or the
device is not compute capability 10.3, calls raise.

Tensors: bf16 activations/weights/bias/outputs are ``torch.bfloat16`` CUDA
tensors (or any dtype viewed as raw 16-bit storage), packed FP4 and scales are
``torch.uint8``, global scales and alpha are 1-element ``torch.float32``
device tensors.  Row strides are taken from the tensors (``stride(0)``) and the
innermost stride must be 1.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

__all__ = [
    "NVFP4_OK", "Nvfp4Error", "library_path", "load_library", "build",
    "nvfp4_abi_version", "nvfp4_is_supported", "nvfp4_last_error_string", "nvfp4_device_error",
    "nvfp4_packed_bytes", "nvfp4_scale_bytes", "nvfp4_linear_workspace_bytes",
    "nvfp4_prepare_weight", "nvfp4_quant_act", "nvfp4_quant_act_export_y", "nvfp4_act_global_scale", "nvfp4_mxfp4_scale_bytes", "nvfp4_mxfp4_quant_act",
    "nvfp4_mxfp4_gemm", "nvfp4_mxfp4_linear_workspace_bytes", "nvfp4_mxfp4_linear", "mxfp4_linear",
    "nvfp4_gemm", "nvfp4_gemm_ex", "nvfp4_grouped_gemm", "nvfp4_linear", "nvfp4_linear_noalloc",
    "nvfp4_gemm_act", "nvfp4_linear_act", "nvfp4_mxfp4_gemm_act", "nvfp4_mxfp4_linear_act", "nvfp4_grouped_gemm_act",
    "nvfp4_mxfp8_bytes", "nvfp4_add_rmsnorm_quant", "nvfp4_moe_rows", "nvfp4_moe_sort_workspace_bytes",
    "nvfp4_moe_sort", "nvfp4_moe_dispatch", "nvfp4_moe_dispatch_quant", "nvfp4_moe_combine",
    "nvfp4_moe_combine_backward", "ACTIVATIONS", "NVFP4_FORMAT_NVFP4", "NVFP4_FORMAT_MXFP4", "NVFP4_FORMAT_MXFP8",
    "interleave_gate_up", "add_rmsnorm_quant", "moe_sort", "moe_dispatch", "moe_dispatch_quant", "moe_combine",
    "moe_combine_backward",
    "nvfp4_moe_route", "nvfp4_moe_route_backward", "nvfp4_act_checkpoint", "nvfp4_act_checkpoint_backward",
    "nvfp4_checkpoint_wgrad", "nvfp4_checkpoint_wgrad_workspace_bytes", "SCORES", "NVFP4_TYPE_F32", "NVFP4_TYPE_BF16",
    "moe_route", "moe_route_backward", "act_checkpoint", "act_checkpoint_backward", "checkpoint_wgrad",
    "padded_k", "scale_shape", "quant_act", "quant_act_mx", "prepare_weight", "linear", "act_global_scale",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libnvfp4_gb300.so")
_lock = threading.Lock()
_lib = None

NVFP4_OK = 0
STATUS_NAMES = {0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_UNSUPPORTED_DEVICE",
                3: "NVFP4_ERR_ALIGNMENT", 4: "NVFP4_ERR_ALIAS", 5: "NVFP4_ERR_CUDA", 6: "NVFP4_ERR_TIMEOUT",
                7: "NVFP4_ERR_WORKSPACE"}

# Values of nvfp4_activation (gated ones halve the columns) and nvfp4_format.
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4, "geglu": 5}
GATED_ACTIVATIONS = ("swiglu", "geglu")
NVFP4_FORMAT_NVFP4, NVFP4_FORMAT_MXFP4, NVFP4_FORMAT_MXFP8 = 0, 1, 2
# Values of nvfp4_score and nvfp4_type.
SCORES = {"softmax": 0, "sigmoid": 1}
NVFP4_TYPE_F32, NVFP4_TYPE_BF16 = 0, 1

# (name, restype, argtypes) of every exported symbol of include/nvfp4.h
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
EXPORTS = [
    ("nvfp4_abi_version", _I32, []),
    ("nvfp4_is_supported", _I32, [_I32, ctypes.c_char_p, _SZ]),
    ("nvfp4_last_error_string", ctypes.c_char_p, []),
    ("nvfp4_device_error", _I32, [_I32]),
    ("nvfp4_packed_bytes", _SZ, [_I64, _I64]),
    ("nvfp4_scale_bytes", _SZ, [_I64, _I64]),
    ("nvfp4_linear_workspace_bytes", _SZ, [_I64, _I64, _I64]),
    ("nvfp4_prepare_weight", _I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P]),
    ("nvfp4_quant_act", _I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _P]),
    ("nvfp4_quant_act_export_y", _I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _P, _P]),
    ("nvfp4_act_global_scale", _I32, [_P, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _P]),
    ("nvfp4_mxfp4_scale_bytes", _SZ, [_I64, _I64]),
    ("nvfp4_mxfp4_quant_act", _I32, [_P, _I64, _I64, _I64, _P, _P, _P]),
    ("nvfp4_mxfp4_gemm", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _I64, _P]),
    ("nvfp4_mxfp4_linear_workspace_bytes", _SZ, [_I64, _I64, _I64]),
    ("nvfp4_mxfp4_linear", _I32, [_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _P, _SZ, _P]),
    ("nvfp4_gemm", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _P]),
    ("nvfp4_grouped_gemm", _I32, [_P, _P, _I64, _P, _I32, _P, _P, _I64, _I64, _P, _P, _P, _I64, _P]),
    ("nvfp4_gemm_ex", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _I32, ctypes.c_uint64, _I32,
                             _P]),
    ("nvfp4_linear", _I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I64, _I64, _P, _P, _P, _I64,
                            _P, _SZ, _P]),
    ("nvfp4_linear_noalloc", _I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I64, _I64, _P, _P, _P, _I64,
                                    _P]),
    ("nvfp4_gemm_act", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _P, _I64, _P, _I64, _P]),
    ("nvfp4_linear_act", _I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I64, _I64, _P, _P, _I32, _P, _I64, _P,
                                _I64, _P, _SZ, _P]),
    ("nvfp4_mxfp4_gemm_act", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P, _I64, _P, _I64, _P]),
    ("nvfp4_mxfp4_linear_act", _I32, [_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _P, _I32, _P, _I64, _P, _I64, _P, _SZ,
                                      _P]),
    ("nvfp4_grouped_gemm_act", _I32, [_P, _P, _I64, _P, _I32, _P, _P, _I64, _I64, _P, _P, _I32, _P, _I64, _P]),
    ("nvfp4_mxfp8_bytes", _SZ, [_I64, _I64]),
    ("nvfp4_add_rmsnorm_quant", _I32, [_P, _I64, _P, _I64, _P, ctypes.c_float, _I64, _I64, _I32, _P, _P, _I64, _P, _P,
                                       _P]),
    ("nvfp4_moe_rows", _I64, [_I64, _I32, _I32]),
    ("nvfp4_moe_sort_workspace_bytes", _SZ, [_I64, _I32, _I32]),
    ("nvfp4_moe_sort", _I32, [_P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    ("nvfp4_moe_dispatch", _I32, [_P, _I64, _P, _I64, _I32, _I64, _I64, _P, _P, _I32, _P, _I64, _P]),
    ("nvfp4_moe_dispatch_quant", _I32, [_P, _I64, _P, _P, _I64, _I32, _I64, _I64, _P, _P, _P]),
    ("nvfp4_moe_combine", _I32, [_P, _I64, _P, _P, _I64, _I32, _I64, _I64, _P, _I64, _P, _I64, _P]),
    ("nvfp4_moe_combine_backward", _I32, [_P, _I64, _P, _I64, _P, _P, _I64, _I32, _I64, _I64, _P, _P, _I32, _P, _I64,
                                          _P, _P]),
    ("nvfp4_moe_route", _I32, [_P, _I32, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _P,
                               _P]),
    ("nvfp4_moe_route_backward", _I32, [_P, _P, _P, _I32, _I64, _I64, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _I64, _P]),
    ("nvfp4_act_checkpoint", _I32, [_P, _I64, _I64, _I64, _I32, _P, _P, _I32, _P, _I64, _P, _P, _P]),
    ("nvfp4_act_checkpoint_backward", _I32, [_P, _I64, _P, _P, _I64, _I64, _I32, _P, _P, _I32, _P, _I64, _P, _P, _P]),
    ("nvfp4_checkpoint_wgrad_workspace_bytes", _SZ, [_I64, _I64, _I64, _I32]),
    ("nvfp4_checkpoint_wgrad", _I32, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32, _P, _I64, _P, _SZ, _P]),
]


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def build(force: bool = False) -> str:
    """Compile the CUDA library in-tree (nvcc, sm_103a)."""
    from . import _build
    return _build.build(force=force)


def load_library():
    """Load ``libnvfp4_gb300.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:                 # every call passes here: no lock once loaded
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"NVFP4 CUDA library not built ({_LIB_PATH} missing); "
                               "run nvfp4_quantized_linear_gb300.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, res, args in EXPORTS:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(status: int):
    if status != NVFP4_OK:
        raise Nvfp4Error(status, load_library().nvfp4_last_error_string().decode())


def _ptr(t):
    """Device pointer of a tensor (None -> NULL)."""
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None                   # () -> handle of torch's current stream


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            # the handle itself where torch has the call: a Stream object per launch costs 2 us
            _current_stream = (lambda: raw(dev())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ld(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit inner stride")
    return t.stride(0)


# What the tensor-level helpers check before they hand a pointer on: the library sees
# addresses only, and would read a tensor of another type or shape past its end.  (A raw
# address in place of a vector or scalar goes through unchecked.)

def _require_dtype(t, name, dtype):
    """`dtype`, by name; raw 16-bit storage passes for bfloat16."""
    got = str(t.dtype)[len("torch."):]
    if got != dtype and not (dtype == "bfloat16" and got in ("int16", "uint16")):
        raise ValueError(f"{name} must be {dtype}, got {got}")


def _rows_of(t, name, rows, cols):
    """Row stride of a 2-D bf16 tensor that holds rows x cols elements."""
    ld = _ld(t, name)
    _require_dtype(t, name, "bfloat16")
    if t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{name} must hold {rows} x {cols} elements, got {tuple(t.shape)}")
    return ld


def _flat(t, name, dtype, count):
    """A contiguous tensor of at least `count` elements."""
    if t is None or isinstance(t, int):
        return
    _require_dtype(t, name, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < count:
        raise ValueError(f"{name} must have {count} elements, got {tuple(t.shape)}")


def _routing(dest, group_offsets=None, group_counts=None, weights=None):
    """(tokens, topk) of moe_sort's outputs and the weights that go with them."""
    if dest.dim() != 2:
        raise ValueError(f"dest must be [tokens, topk], got {tuple(dest.shape)}")
    _flat(dest, "dest", "int32", 0)
    if group_counts is not None:
        _flat(group_counts, "group_counts", "int32", 1)
        _flat(group_offsets, "group_offsets", "int32", group_counts.numel() + 1)
    if weights is not None:
        _flat(weights, "weights", "float32", 0)
        if weights.shape != dest.shape and (weights.dim() != 1 or weights.numel() != dest.numel()):
            raise ValueError(f"weights must be {tuple(dest.shape)} like dest, got {tuple(weights.shape)}")
    return dest.shape


def _on_gpu(**tensors):
    device = None
    for name, t in tensors.items():
        if t is None or isinstance(t, int):
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise ValueError(f"{name} is on another device than the tensors before it")


def _on_current_gpu(**tensors):
    """_on_gpu, and the device is the current one, whose stream the call goes to."""
    _on_gpu(**tensors)
    import torch
    for name, t in tensors.items():
        if t is not None and not isinstance(t, int) and t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{torch.cuda.current_device()}")


def _tensors_of(stream):
    """Context in which new tensors belong to the stream that a call goes to: memory that another
    stream's kernels may still use, or may take next, is not theirs."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _check_linear(x, k, n_out, bias, act, residual, out, **operands):
    """The checks of linear() and mxfp4_linear(); returns (ldx, activation code, ldr, ldo)."""
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}, not one of {', '.join(ACTIVATIONS)}")
    m = x.shape[0]
    ldx = _rows_of(x, "x", m, k)
    _flat(bias, "bias", "bfloat16", 2 * n_out if act in GATED_ACTIVATIONS else n_out)
    ldr = _rows_of(residual, "residual", m, n_out) if residual is not None else 0
    ldo = _rows_of(out, "out", m, n_out) if out is not None else n_out
    _on_gpu(x=x, **operands, bias=bias, residual=residual, out=out)
    return ldx, ACTIVATIONS[act], ldr, ldo


# ------------------------------------------------------------- queries ----

def padded_k(k: int) -> int:
    return (k + 31) // 32 * 32


def scale_shape(rows: int, k: int) -> tuple[int, int]:
    """(padded rows, padded scale columns) of a tiled scale tensor."""
    return (rows + 127) // 128 * 128, (padded_k(k) // 16 + 3) // 4 * 4


def nvfp4_abi_version() -> int:
    return load_library().nvfp4_abi_version()


def nvfp4_is_supported(device: int = 0) -> tuple[bool, str | None]:
    buf = ctypes.create_string_buffer(256)
    st = load_library().nvfp4_is_supported(device, buf, 256)
    return (st == NVFP4_OK, None if st == NVFP4_OK else buf.value.decode())


def nvfp4_last_error_string() -> str:
    return load_library().nvfp4_last_error_string().decode()


def nvfp4_device_error(clear: bool = True) -> None:
    _check(load_library().nvfp4_device_error(1 if clear else 0))


def nvfp4_packed_bytes(rows: int, k: int) -> int:
    return load_library().nvfp4_packed_bytes(rows, k)


def nvfp4_scale_bytes(rows: int, k: int) -> int:
    return load_library().nvfp4_scale_bytes(rows, k)


def nvfp4_linear_workspace_bytes(m: int, k: int, n_w: int) -> int:
    return load_library().nvfp4_linear_workspace_bytes(m, k, n_w)


# ---------------------------------------------------------- operations ----

def nvfp4_prepare_weight(w, n: int, k: int, ldw: int, w_gs, w_fp4, w_sf, stream=None) -> None:
    _check(load_library().nvfp4_prepare_weight(_ptr(w), n, k, ldw, _ptr(w_gs), _ptr(w_fp4), _ptr(w_sf),
                                               _stream(stream)))


def nvfp4_quant_act(x, m: int, k: int, ldx: int, gs, transform, bs: int, x_fp4, x_sf, stream=None) -> None:
    _check(load_library().nvfp4_quant_act(_ptr(x), m, k, ldx, _ptr(gs), _ptr(transform), bs, _ptr(x_fp4),
                                          _ptr(x_sf), _stream(stream)))


def nvfp4_quant_act_export_y(x, m: int, k: int, ldx: int, gs, transform, bs: int, x_fp4, x_sf, y,
                             stream=None) -> None:
    _check(load_library().nvfp4_quant_act_export_y(_ptr(x), m, k, ldx, _ptr(gs), _ptr(transform), bs, _ptr(x_fp4),
                                                   _ptr(x_sf), _ptr(y), _stream(stream)))


def nvfp4_act_global_scale(x, m: int, k: int, ldx: int, transform, bs: int, w_gs, gs_out, alpha_out,
                           stream=None) -> None:
    _check(load_library().nvfp4_act_global_scale(_ptr(x), m, k, ldx, _ptr(transform), bs, _ptr(w_gs),
                                                 _ptr(gs_out), _ptr(alpha_out), _stream(stream)))


def nvfp4_mxfp4_scale_bytes(rows: int, k: int) -> int:
    return load_library().nvfp4_mxfp4_scale_bytes(rows, k)


def nvfp4_mxfp4_quant_act(x, m: int, k: int, ldx: int, x_fp4, x_sf, stream=None) -> None:
    _check(load_library().nvfp4_mxfp4_quant_act(_ptr(x), m, k, ldx, _ptr(x_fp4), _ptr(x_sf), _stream(stream)))


def nvfp4_mxfp4_gemm(a_fp4, a_sf, m: int, w_fp4, w_sf, n_w: int, n_out: int, k: int, bias, out, ldo: int,
                     stream=None) -> None:
    _check(load_library().nvfp4_mxfp4_gemm(_ptr(a_fp4), _ptr(a_sf), m, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, k,
                                           _ptr(bias), _ptr(out), ldo, _stream(stream)))


def nvfp4_mxfp4_linear_workspace_bytes(m: int, k: int, n_w: int) -> int:
    return load_library().nvfp4_mxfp4_linear_workspace_bytes(m, k, n_w)


def nvfp4_mxfp4_linear(x, m: int, k: int, ldx: int, w_fp4, w_sf, n_w: int, n_out: int, bias, out, ldo: int,
                       workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().nvfp4_mxfp4_linear(_ptr(x), m, k, ldx, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, _ptr(bias),
                                             _ptr(out), ldo, _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_gemm(a_fp4, a_sf, m: int, w_fp4, w_sf, n_w: int, n_out: int, k: int, alpha, bias, out, ldo: int,
               stream=None) -> None:
    _check(load_library().nvfp4_gemm(_ptr(a_fp4), _ptr(a_sf), m, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, k,
                                     _ptr(alpha), _ptr(bias), _ptr(out), ldo, _stream(stream)))


def nvfp4_grouped_gemm(a_fp4, a_sf, rows: int, group_offsets, num_groups: int, w_fp4, w_sf, n: int, k: int, alpha,
                       bias, out, ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_grouped_gemm(_ptr(a_fp4), _ptr(a_sf), rows, _ptr(group_offsets), num_groups,
                                             _ptr(w_fp4), _ptr(w_sf), n, k, _ptr(alpha), _ptr(bias), _ptr(out), ldo,
                                             _stream(stream)))


def nvfp4_gemm_ex(a_fp4, a_sf, m: int, w_fp4, w_sf, n_w: int, n_out: int, k: int, alpha, bias, out, ldo: int,
                  kernel: int = 0, wait_limit_ns: int = 0, drill: int = 0, stream=None) -> None:
    _check(load_library().nvfp4_gemm_ex(_ptr(a_fp4), _ptr(a_sf), m, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, k,
                                        _ptr(alpha), _ptr(bias), _ptr(out), ldo, kernel, wait_limit_ns, drill,
                                        _stream(stream)))


def nvfp4_linear(x, m: int, k: int, ldx: int, gs, transform, bs: int, w_fp4, w_sf, n_w: int, n_out: int,
                 alpha, bias, out, ldo: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().nvfp4_linear(_ptr(x), m, k, ldx, _ptr(gs), _ptr(transform), bs, _ptr(w_fp4),
                                       _ptr(w_sf), n_w, n_out, _ptr(alpha), _ptr(bias), _ptr(out), ldo,
                                       _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_linear_noalloc(x, m: int, k: int, ldx: int, gs, transform, bs: int, w_fp4, w_sf, n_w: int, n_out: int,
                         alpha, bias, out, ldo: int, stream=None) -> None:
    """nvfp4_linear with the library's built-in 16 MiB scratch instead of a
    workspace, for callers that cannot allocate device memory (see the C
    header for the limit and the sharing rules)."""
    _check(load_library().nvfp4_linear_noalloc(_ptr(x), m, k, ldx, _ptr(gs), _ptr(transform), bs, _ptr(w_fp4),
                                               _ptr(w_sf), n_w, n_out, _ptr(alpha), _ptr(bias), _ptr(out), ldo,
                                               _stream(stream)))


def nvfp4_gemm_act(a_fp4, a_sf, m: int, w_fp4, w_sf, n_w: int, n_out: int, k: int, alpha, bias, act: int, residual,
                   ldr: int, out, ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_gemm_act(_ptr(a_fp4), _ptr(a_sf), m, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, k,
                                         _ptr(alpha), _ptr(bias), act, _ptr(residual), ldr, _ptr(out), ldo,
                                         _stream(stream)))


def nvfp4_linear_act(x, m: int, k: int, ldx: int, gs, transform, bs: int, w_fp4, w_sf, n_w: int, n_out: int, alpha,
                     bias, act: int, residual, ldr: int, out, ldo: int, workspace, workspace_bytes: int,
                     stream=None) -> None:
    _check(load_library().nvfp4_linear_act(_ptr(x), m, k, ldx, _ptr(gs), _ptr(transform), bs, _ptr(w_fp4), _ptr(w_sf),
                                           n_w, n_out, _ptr(alpha), _ptr(bias), act, _ptr(residual), ldr, _ptr(out),
                                           ldo, _ptr(workspace), workspace_bytes, _stream(stream)))


def nvfp4_mxfp4_gemm_act(a_fp4, a_sf, m: int, w_fp4, w_sf, n_w: int, n_out: int, k: int, bias, act: int, residual,
                         ldr: int, out, ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_mxfp4_gemm_act(_ptr(a_fp4), _ptr(a_sf), m, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, k,
                                               _ptr(bias), act, _ptr(residual), ldr, _ptr(out), ldo, _stream(stream)))


def nvfp4_mxfp4_linear_act(x, m: int, k: int, ldx: int, w_fp4, w_sf, n_w: int, n_out: int, bias, act: int, residual,
                           ldr: int, out, ldo: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().nvfp4_mxfp4_linear_act(_ptr(x), m, k, ldx, _ptr(w_fp4), _ptr(w_sf), n_w, n_out, _ptr(bias),
                                                 act, _ptr(residual), ldr, _ptr(out), ldo, _ptr(workspace),
                                                 workspace_bytes, _stream(stream)))


def nvfp4_grouped_gemm_act(a_fp4, a_sf, rows: int, group_offsets, num_groups: int, w_fp4, w_sf, n: int, k: int, alpha,
                           bias, act: int, out, ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_grouped_gemm_act(_ptr(a_fp4), _ptr(a_sf), rows, _ptr(group_offsets), num_groups,
                                                 _ptr(w_fp4), _ptr(w_sf), n, k, _ptr(alpha), _ptr(bias), act,
                                                 _ptr(out), ldo, _stream(stream)))


def nvfp4_mxfp8_bytes(rows: int, k: int) -> int:
    return load_library().nvfp4_mxfp8_bytes(rows, k)


def nvfp4_add_rmsnorm_quant(x, ldx: int, residual, ldr: int, gamma, eps: float, m: int, k: int, fmt: int, gs, h,
                            ldh: int, x_q, x_sf, stream=None) -> None:
    _check(load_library().nvfp4_add_rmsnorm_quant(_ptr(x), ldx, _ptr(residual), ldr, _ptr(gamma), eps, m, k, fmt,
                                                  _ptr(gs), _ptr(h), ldh, _ptr(x_q), _ptr(x_sf), _stream(stream)))


def nvfp4_moe_rows(tokens: int, topk: int, experts: int) -> int:
    return load_library().nvfp4_moe_rows(tokens, topk, experts)


def nvfp4_moe_sort_workspace_bytes(tokens: int, topk: int, experts: int) -> int:
    return load_library().nvfp4_moe_sort_workspace_bytes(tokens, topk, experts)


def nvfp4_moe_sort(expert_ids, id_bytes: int, tokens: int, topk: int, experts: int, group_offsets, group_counts, dest,
                   workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().nvfp4_moe_sort(_ptr(expert_ids), id_bytes, tokens, topk, experts, _ptr(group_offsets),
                                         _ptr(group_counts), _ptr(dest), _ptr(workspace), workspace_bytes,
                                         _stream(stream)))


def nvfp4_moe_dispatch(x, ldx: int, dest, tokens: int, topk: int, rows: int, h: int, group_offsets, group_counts,
                       experts: int, out, ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_moe_dispatch(_ptr(x), ldx, _ptr(dest), tokens, topk, rows, h, _ptr(group_offsets),
                                             _ptr(group_counts), experts, _ptr(out), ldo, _stream(stream)))


def nvfp4_moe_dispatch_quant(x, ldx: int, gs, dest, tokens: int, topk: int, rows: int, h: int, x_fp4, x_sf,
                             stream=None) -> None:
    _check(load_library().nvfp4_moe_dispatch_quant(_ptr(x), ldx, _ptr(gs), _ptr(dest), tokens, topk, rows, h,
                                                   _ptr(x_fp4), _ptr(x_sf), _stream(stream)))


def nvfp4_moe_combine(y, ldy: int, weights, dest, tokens: int, topk: int, rows: int, h: int, residual, ldr: int, out,
                      ldo: int, stream=None) -> None:
    _check(load_library().nvfp4_moe_combine(_ptr(y), ldy, _ptr(weights), _ptr(dest), tokens, topk, rows, h,
                                            _ptr(residual), ldr, _ptr(out), ldo, _stream(stream)))


def nvfp4_moe_combine_backward(dout, ldd: int, y, ldy: int, weights, dest, tokens: int, topk: int, rows: int, h: int,
                               group_offsets, group_counts, experts: int, dy, lddy: int, dweights,
                               stream=None) -> None:
    _check(load_library().nvfp4_moe_combine_backward(_ptr(dout), ldd, _ptr(y), ldy, _ptr(weights), _ptr(dest), tokens,
                                                     topk, rows, h, _ptr(group_offsets), _ptr(group_counts), experts,
                                                     _ptr(dy), lddy, _ptr(dweights), _stream(stream)))


def nvfp4_moe_route(logits, type: int, ldl: int, bias, tokens: int, experts: int, score: int, topk: int, groups: int,
                    group_top: int, topk_groups: int, renormalize: bool, scale: float, expert_ids, weights,
                    stream=None) -> None:
    _check(load_library().nvfp4_moe_route(_ptr(logits), type, ldl, _ptr(bias), tokens, experts, score, topk, groups,
                                          group_top, topk_groups, renormalize, scale, _ptr(expert_ids), _ptr(weights),
                                          _stream(stream)))


def nvfp4_moe_route_backward(dweights, expert_ids, logits, type: int, ldl: int, tokens: int, experts: int, score: int,
                             topk: int, renormalize: bool, scale: float, dlogits, ldd: int, stream=None) -> None:
    _check(load_library().nvfp4_moe_route_backward(_ptr(dweights), _ptr(expert_ids), _ptr(logits), type, ldl, tokens,
                                                   experts, score, topk, renormalize, scale, _ptr(dlogits), ldd,
                                                   _stream(stream)))


def nvfp4_act_checkpoint(x, ldx: int, m: int, n_out: int, act: int, group_offsets, group_counts, num_groups: int, out,
                         ldo: int, q, sf, stream=None) -> None:
    _check(load_library().nvfp4_act_checkpoint(_ptr(x), ldx, m, n_out, act, _ptr(group_offsets), _ptr(group_counts),
                                               num_groups, _ptr(out), ldo, _ptr(q), _ptr(sf), _stream(stream)))


def nvfp4_act_checkpoint_backward(dout, ldd: int, q, sf, m: int, n_out: int, act: int, group_offsets, group_counts,
                                  num_groups: int, dx, ldx: int, act_q, act_sf, stream=None) -> None:
    _check(load_library().nvfp4_act_checkpoint_backward(_ptr(dout), ldd, _ptr(q), _ptr(sf), m, n_out, act,
                                                        _ptr(group_offsets), _ptr(group_counts), num_groups, _ptr(dx), ldx,
                                                        _ptr(act_q), _ptr(act_sf), _stream(stream)))


def nvfp4_checkpoint_wgrad_workspace_bytes(m: int, n: int, k: int, num_groups: int = 0) -> int:
    return load_library().nvfp4_checkpoint_wgrad_workspace_bytes(m, n, k, num_groups)


def nvfp4_checkpoint_wgrad(dy, ldd: int, q, sf, m: int, n: int, k: int, group_offsets, group_counts, num_groups: int,
                           type: int, accumulate: bool, dw, ldw: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().nvfp4_checkpoint_wgrad(_ptr(dy), ldd, _ptr(q), _ptr(sf), m, n, k, _ptr(group_offsets),
                                                 _ptr(group_counts), num_groups, type, accumulate, _ptr(dw), ldw,
                                                 _ptr(workspace), workspace_bytes, _stream(stream)))


# --------------------------------------------- tensor-level conveniences ----
# Thin helpers that allocate the caller-owned outputs with torch and call the
# entry points above; they add no computation.

def quant_act(x, gs, transform=None, bs: int = 0, stream=None):
    """Quantize a [m, k] bf16 CUDA tensor; returns (x_fp4 [m, Kp/2], x_sf flat)."""
    import torch
    m, k = x.shape
    x_fp4 = torch.empty((m, padded_k(k) // 2), dtype=torch.uint8, device=x.device)
    x_sf = torch.empty(max(nvfp4_scale_bytes(m, k), 1), dtype=torch.uint8, device=x.device)
    nvfp4_quant_act(x, m, k, _ld(x, "x"), gs, transform, bs if transform is not None else 0, x_fp4, x_sf, stream)
    return x_fp4, x_sf


def act_global_scale(x, transform=None, bs: int = 0, w_gs=None, stream=None):
    """Dynamic scale of a [m, k] bf16 CUDA tensor; returns (gs, alpha) as
    1-element fp32 device tensors (alpha is None without w_gs)."""
    import torch
    m, k = x.shape
    gs = torch.empty(1, dtype=torch.float32, device=x.device)
    alpha = torch.empty(1, dtype=torch.float32, device=x.device) if w_gs is not None else None
    nvfp4_act_global_scale(x, m, k, _ld(x, "x"), transform, bs if transform is not None else 0, w_gs, gs, alpha,
                           stream)
    return gs, alpha


def quant_act_mx(x, stream=None):
    """MXFP4-quantize a [m, k] bf16 CUDA tensor; returns (x_fp4 [m, Kp/2], x_sf flat E8M0 codes)."""
    import torch
    m, k = x.shape
    x_fp4 = torch.empty((m, padded_k(k) // 2), dtype=torch.uint8, device=x.device)
    x_sf = torch.empty(max(nvfp4_mxfp4_scale_bytes(m, k), 1), dtype=torch.uint8, device=x.device)
    nvfp4_mxfp4_quant_act(x, m, k, _ld(x, "x"), x_fp4, x_sf, stream)
    return x_fp4, x_sf


def mxfp4_linear(x, w_fp4, w_sf, k: int, n_out: int, bias=None, out=None, workspace=None, act: str = "none",
                 residual=None, stream=None):
    """out[m, n_out] = MXFP4 linear of a [m, k] bf16 CUDA tensor against a weight
    quantized by quant_act_mx, with the epilogue of linear() (allocates
    out/workspace if not given)."""
    import torch
    m = x.shape[0]
    n_w = w_fp4.shape[0]
    ldx, code, ldr, ldo = _check_linear(x, k, n_out, bias, act, residual, out, w_fp4=w_fp4, w_sf=w_sf)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(nvfp4_mxfp4_linear_workspace_bytes(m, k, n_w), 1), dtype=torch.uint8,
                                device=x.device)
    if act == "none" and residual is None:
        nvfp4_mxfp4_linear(x, m, k, ldx, w_fp4, w_sf, n_w, n_out, bias, out, ldo, workspace, workspace.numel(), stream)
        return out
    nvfp4_mxfp4_linear_act(x, m, k, ldx, w_fp4, w_sf, n_w, n_out, bias, code, residual, ldr, out, ldo, workspace,
                           workspace.numel(), stream)
    return out


def prepare_weight(w, w_gs, stream=None):
    """Prepare a [n, k] bf16 CUDA weight; returns (w_fp4 [n, Kp/2], w_sf flat)."""
    import torch
    n, k = w.shape
    w_fp4 = torch.empty((n, padded_k(k) // 2), dtype=torch.uint8, device=w.device)
    w_sf = torch.empty(max(nvfp4_scale_bytes(n, k), 1), dtype=torch.uint8, device=w.device)
    nvfp4_prepare_weight(w, n, k, _ld(w, "w"), w_gs, w_fp4, w_sf, stream)
    return w_fp4, w_sf


def linear(x, w_fp4, w_sf, k: int, n_out: int, gs, alpha, bias=None, transform=None, bs: int = 0,
           out=None, workspace=None, act: str = "none", residual=None, stream=None):
    """out[m, n_out] = act(NVFP4 linear of a [m, k] bf16 CUDA tensor + bias) + residual
    (allocates out/workspace if not given).  act is a key of ACTIVATIONS; the
    gated ones take a weight of interleave_gate_up."""
    import torch
    m = x.shape[0]
    n_w = w_fp4.shape[0]
    _flat(gs, "gs", "float32", 1)
    _flat(alpha, "alpha", "float32", 1)
    ldx, code, ldr, ldo = _check_linear(x, k, n_out, bias, act, residual, out, w_fp4=w_fp4, w_sf=w_sf, gs=gs,
                                        alpha=alpha, transform=transform)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.bfloat16, device=x.device)
    need = nvfp4_linear_workspace_bytes(m, k, n_w)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if act == "none" and residual is None:
        nvfp4_linear(x, m, k, ldx, gs, transform, bs if transform is not None else 0, w_fp4, w_sf, n_w, n_out, alpha,
                     bias, out, ldo, workspace, workspace.numel(), stream)
        return out
    nvfp4_linear_act(x, m, k, ldx, gs, transform, bs if transform is not None else 0, w_fp4, w_sf, n_w, n_out, alpha,
                     bias, code, residual, ldr, out, ldo, workspace, workspace.numel(), stream)
    return out


def interleave_gate_up(gate, up):
    """[2n, ...] with rows gate[0], up[0], gate[1], up[1], ...: the weight (or bias)
    order of the gated activations."""
    import torch
    return torch.stack((gate, up), dim=1).reshape(2 * gate.shape[0], *gate.shape[1:])


def add_rmsnorm_quant(x, gamma, eps: float, residual=None, gs=None, fmt: int = NVFP4_FORMAT_NVFP4, h=None,
                      stream=None):
    """Residual addition + RMS norm + quantization of a [m, k] bf16 CUDA tensor;
    returns (x_q, flat x_sf, h).  h (the updated residual stream, None without a
    residual) is allocated unless given; pass residual itself to update it in place."""
    import torch
    ldx = _rows_of(x, "x", 0, 0)
    m, k = x.shape
    ldr = _rows_of(residual, "residual", m, k) if residual is not None else 0
    if h is not None:
        _rows_of(h, "h", m, k)
    _flat(gamma, "gamma", "bfloat16", k)
    _flat(gs, "gs", "float32", 1)
    _on_gpu(x=x, gamma=gamma, residual=residual, gs=gs, h=h)
    cols = padded_k(k) if fmt == NVFP4_FORMAT_MXFP8 else padded_k(k) // 2
    n_sf = nvfp4_scale_bytes(m, k) if fmt == NVFP4_FORMAT_NVFP4 else nvfp4_mxfp4_scale_bytes(m, k)
    x_q = torch.empty((m, cols), dtype=torch.uint8, device=x.device)
    x_sf = torch.empty(max(n_sf, 1), dtype=torch.uint8, device=x.device)
    if h is None and residual is not None:
        h = torch.empty((m, k), dtype=torch.bfloat16, device=x.device)
    nvfp4_add_rmsnorm_quant(x, ldx, residual, ldr, gamma, eps, m, k, fmt, gs, h, h.stride(0) if h is not None else 0, x_q,
                            x_sf, stream)
    return x_q, x_sf, h


def moe_sort(expert_ids, experts: int, stream=None):
    """Sort [tokens, topk] int32/int64 expert ids (contiguous, CUDA); returns
    (group_offsets, group_counts, dest), int32."""
    import torch
    tokens, topk = expert_ids.shape
    if not expert_ids.is_contiguous() or expert_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("expert_ids must be a contiguous int32 or int64 tensor")
    _on_gpu(expert_ids=expert_ids)
    new = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=expert_ids.device)  # noqa: E731
    offsets, counts, dest = new(experts + 1), new(experts), new(tokens, topk)
    ws = new(nvfp4_moe_sort_workspace_bytes(tokens, topk, experts), dtype=torch.uint8)
    nvfp4_moe_sort(expert_ids, expert_ids.element_size(), tokens, topk, experts, offsets, counts, dest, ws, ws.numel(),
                   stream)
    return offsets, counts, dest


def moe_dispatch(x, dest, group_offsets, group_counts, out=None, stream=None):
    """Rows of a [tokens, h] bf16 CUDA tensor in the order of moe_sort, [nvfp4_moe_rows, h]."""
    import torch
    tokens, topk = _routing(dest, group_offsets, group_counts)
    ldx = _rows_of(x, "x", tokens, 0)
    experts, h = group_counts.numel(), x.shape[1]
    if out is not None:
        _rows_of(out, "out", 0, h)                           # (its rows: the library's check)
    _on_gpu(x=x, dest=dest, group_offsets=group_offsets, group_counts=group_counts, out=out)
    if out is None:
        out = torch.empty((nvfp4_moe_rows(tokens, topk, experts), h), dtype=torch.bfloat16, device=x.device)
    nvfp4_moe_dispatch(x, ldx, dest, tokens, topk, out.shape[0], h, group_offsets, group_counts, experts, out,
                       out.stride(0), stream)
    return out


def moe_dispatch_quant(x, gs, dest, experts: int, stream=None):
    """The same as the NVFP4 operand of nvfp4_grouped_gemm; returns (x_fp4, flat x_sf)."""
    import torch
    tokens, topk = _routing(dest)
    ldx = _rows_of(x, "x", tokens, 0)
    _flat(gs, "gs", "float32", 1)
    _on_gpu(x=x, gs=gs, dest=dest)
    h = x.shape[1]
    rows = nvfp4_moe_rows(tokens, topk, experts)
    x_fp4 = torch.empty((rows, padded_k(h) // 2), dtype=torch.uint8, device=x.device)
    x_sf = torch.empty(max(nvfp4_scale_bytes(rows, h), 1), dtype=torch.uint8, device=x.device)
    nvfp4_moe_dispatch_quant(x, ldx, gs, dest, tokens, topk, rows, h, x_fp4, x_sf, stream)
    return x_fp4, x_sf


def moe_combine(y, dest, weights=None, residual=None, out=None, stream=None):
    """[tokens, h] bf16: each token's expert rows, weighted (fp32 [tokens, topk]) and summed,
    plus residual."""
    import torch
    tokens, topk = _routing(dest, weights=weights)
    ldy = _rows_of(y, "y", 0, 0)
    h = y.shape[1]
    ldr = _rows_of(residual, "residual", tokens, h) if residual is not None else 0
    if out is not None:
        _rows_of(out, "out", tokens, h)
    _on_gpu(y=y, dest=dest, weights=weights, residual=residual, out=out)
    if out is None:
        out = torch.empty((tokens, h), dtype=torch.bfloat16, device=y.device)
    nvfp4_moe_combine(y, ldy, weights, dest, tokens, topk, y.shape[0], h, residual, ldr, out, out.stride(0), stream)
    return out


def moe_combine_backward(dout, y, weights, dest, group_offsets, group_counts, dy=None, stream=None):
    """Gradients (dy [rows, h] bf16, dweights [tokens, topk] fp32) of moe_combine."""
    import torch
    tokens, topk = _routing(dest, group_offsets, group_counts, weights)
    ldy = _rows_of(y, "y", 0, 0)
    rows, h = y.shape
    ldd = _rows_of(dout, "dout", tokens, h)
    if dy is not None:
        _rows_of(dy, "dy", rows, h)
    _on_gpu(dout=dout, y=y, weights=weights, dest=dest, group_offsets=group_offsets, group_counts=group_counts, dy=dy)
    if dy is None:
        dy = torch.empty((rows, h), dtype=torch.bfloat16, device=y.device)
    dweights = torch.empty((tokens, topk), dtype=torch.float32, device=y.device)
    nvfp4_moe_combine_backward(dout, ldd, y, ldy, weights, dest, tokens, topk, rows, h, group_offsets, group_counts,
                               group_counts.numel(), dy, dy.stride(0), dweights, stream)
    return dy, dweights


def _logits(logits, score):
    """(type, row stride, tokens, experts, score code) of a router's logits."""
    if score not in SCORES:
        raise ValueError(f"unknown score {score!r}, not one of {', '.join(SCORES)}")
    ld = _ld(logits, "logits")
    got = str(logits.dtype)[len("torch."):]
    if got not in ("float32", "bfloat16"):
        raise ValueError(f"logits must be float32 or bfloat16, got {got}")
    tokens, experts = logits.shape
    if tokens <= 1:
        ld = max(ld, experts)                                # (a stride that nothing is read by)
    elif ld < experts:
        raise ValueError(f"logits has overlapping rows: row stride {ld}, {experts} experts")
    return NVFP4_TYPE_F32 if got == "float32" else NVFP4_TYPE_BF16, ld, tokens, experts, SCORES[score]


def moe_route(logits, topk: int, score: str = "softmax", bias=None, groups: int = 1, group_top: int = 1,
              topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
    """Experts of [tokens, experts] fp32 or bf16 router logits; returns (expert_ids int32, weights
    fp32), both [tokens, topk], as moe_sort and moe_combine take them.  bias (fp32 [experts])
    takes part in the choice only; score is a key of SCORES."""
    import torch
    kind, ld, tokens, experts, code = _logits(logits, score)
    _flat(bias, "bias", "float32", experts)
    _on_current_gpu(logits=logits, bias=bias)
    with _tensors_of(stream):
        ids = torch.empty((tokens, topk), dtype=torch.int32, device=logits.device)
        weights = torch.empty((tokens, topk), dtype=torch.float32, device=logits.device)
    nvfp4_moe_route(logits, kind, ld, bias, tokens, experts, code, topk, groups, group_top, topk_groups, renormalize, scale,
                    ids, weights, stream)
    return ids, weights


def moe_route_backward(dweights, expert_ids, logits, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                       stream=None):
    """Gradient of moe_route's weights: dlogits, of the logits' shape and type."""
    import torch
    if expert_ids.dim() != 2:
        raise ValueError(f"expert_ids must be [tokens, topk], got {tuple(expert_ids.shape)}")
    topk = expert_ids.shape[1]
    kind, ld, tokens, experts, code = _logits(logits, score)
    _flat(expert_ids, "expert_ids", "int32", 0)
    _flat(dweights, "dweights", "float32", 0)
    if expert_ids.shape[0] != tokens:
        raise ValueError(f"expert_ids must have a row per token ({tokens}), got {tuple(expert_ids.shape)}")
    if dweights.shape != expert_ids.shape:
        raise ValueError(f"dweights must be {tuple(expert_ids.shape)} like expert_ids, got {tuple(dweights.shape)}")
    _on_current_gpu(logits=logits, expert_ids=expert_ids, dweights=dweights)
    with _tensors_of(stream):
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    nvfp4_moe_route_backward(dweights, expert_ids, logits, kind, ld, tokens, experts, code, topk, renormalize, scale, dlogits,
                             experts, stream)
    return dlogits


def _group_rows(group_offsets, group_counts):
    """num_groups of a pair of group tensors of moe_sort (0 without them)."""
    if (group_offsets is None) != (group_counts is None):
        raise ValueError("group_offsets and group_counts go together")
    if group_counts is None:
        return 0
    _flat(group_counts, "group_counts", "int32", 1)
    _flat(group_offsets, "group_offsets", "int32", group_counts.numel() + 1)
    return group_counts.numel()


def _mxfp8(q, sf, rows, cols, names=("q", "sf")):
    """An MXFP8 operand of rows x cols, as act_checkpoint returns it."""
    _flat(q, names[0], "uint8", rows * padded_k(cols))
    _flat(sf, names[1], "uint8", nvfp4_mxfp4_scale_bytes(rows, cols))


def _new_mxfp8(rows, cols, device):
    import torch
    return (torch.empty((rows, padded_k(cols)), dtype=torch.uint8, device=device),
            torch.empty(max(nvfp4_mxfp4_scale_bytes(rows, cols), 1), dtype=torch.uint8, device=device))


def _new_rows(rows, cols, dtype, device):
    """[rows, cols], rows on 16-byte boundaries (a slice costs a call 3 us: only where it is one)."""
    import torch
    t = torch.empty((rows, (cols + 7) // 8 * 8), dtype=dtype, device=device)
    return t if cols % 8 == 0 else t[:, :cols]


def _act_columns(columns, act):
    """(activation code, output columns) of an activation over `columns`."""
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}, not one of {', '.join(ACTIVATIONS)}")
    if act in GATED_ACTIVATIONS and columns % 2:
        raise ValueError(f"{act} needs gate and up columns, got {columns}")
    return ACTIVATIONS[act], columns // 2 if act in GATED_ACTIVATIONS else columns


def act_checkpoint(x, act: str = "none", group_offsets=None, group_counts=None, out=None, stream=None):
    """Activation of a [m, k] bf16 CUDA tensor and its checkpoint; returns (out bf16, q [m, Kp], flat
    sf), q and sf being x in MXFP8.  act "none" without out: the checkpoint alone (out is None).  With
    group_offsets and group_counts (of moe_sort) x holds sorted expert rows; other rows of
    the results are then not written."""
    import torch
    ldx = _rows_of(x, "x", 0, 0)
    m, k = x.shape
    code, n = _act_columns(k, act)
    groups = _group_rows(group_offsets, group_counts)
    if out is not None:
        _rows_of(out, "out", m, n)
    _on_current_gpu(x=x, group_offsets=group_offsets, group_counts=group_counts, out=out)
    with _tensors_of(stream):
        if out is None and act != "none":
            out = _new_rows(m, n, torch.bfloat16, x.device)
        q, sf = _new_mxfp8(m, k, x.device)
    nvfp4_act_checkpoint(x, ldx, m, n, code, group_offsets, group_counts, groups, out,
                         out.stride(0) if out is not None else 0, q, sf, stream)
    return out, q, sf


def act_checkpoint_backward(dout, q, sf, act: str = "none", group_offsets=None, group_counts=None, dx=None,
                            recompute: bool = False, stream=None):
    """Gradient of act_checkpoint's activation from its checkpoint; returns (dx bf16, act_q, act_sf), the
    latter two, act(x) in MXFP8, None unless recompute."""
    import torch
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}, not one of {', '.join(ACTIVATIONS)}")
    ldd = _rows_of(dout, "dout", 0, 0)
    m, n = dout.shape
    k = 2 * n if act in GATED_ACTIVATIONS else n
    groups = _group_rows(group_offsets, group_counts)
    _mxfp8(q, sf, m, k)
    if dx is not None:
        _rows_of(dx, "dx", m, k)
    _on_current_gpu(dout=dout, q=q, sf=sf, group_offsets=group_offsets, group_counts=group_counts, dx=dx)
    with _tensors_of(stream):
        if dx is None:
            dx = _new_rows(m, k, torch.bfloat16, dout.device)
        act_q, act_sf = _new_mxfp8(m, n, dout.device) if recompute else (None, None)
    nvfp4_act_checkpoint_backward(dout, ldd, q, sf, m, n, ACTIVATIONS[act], group_offsets, group_counts, groups, dx,
                                  dx.stride(0), act_q, act_sf, stream)
    return dx, act_q, act_sf


def checkpoint_wgrad(dy, q, sf, k: int, group_offsets=None, group_counts=None, dw=None, accumulate: bool = False,
                     dtype=None, workspace=None, stream=None):
    """Weight gradient dY^T X of a [m, n] bf16 CUDA tensor dy and x [m, k] in MXFP8: [n, k], with groups
    [num_groups * n, k].  dw gives the output (fp32 or bf16; accumulate adds to an fp32 one), else one
    of `dtype` (default torch.float32) is allocated."""
    import torch
    ldd = _rows_of(dy, "dy", 0, 0)
    m, n = dy.shape
    groups = _group_rows(group_offsets, group_counts)
    _mxfp8(q, sf, m, k)
    if accumulate and dw is None:
        raise ValueError("accumulate adds to dw: it needs one")
    if dw is not None:
        kind = str(dw.dtype)[len("torch."):]
        if kind not in ("float32", "bfloat16"):
            raise ValueError(f"dw must be float32 or bfloat16, got {kind}")
        _ld(dw, "dw")
        if dw.shape[0] < max(1, groups) * n or dw.shape[1] < k:
            raise ValueError(f"dw must hold {max(1, groups) * n} x {k} elements, got {tuple(dw.shape)}")
    elif dtype not in (None, torch.float32, torch.bfloat16):
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    _flat(workspace, "workspace", "uint8", 0)
    _on_current_gpu(dy=dy, q=q, sf=sf, group_offsets=group_offsets, group_counts=group_counts, dw=dw, workspace=workspace)
    with _tensors_of(stream):
        if dw is None:
            dw = _new_rows(max(1, groups) * n, k, dtype or torch.float32, dy.device)
        if workspace is None:
            workspace = torch.empty(nvfp4_checkpoint_wgrad_workspace_bytes(m, n, k, groups), dtype=torch.uint8,
                                    device=dy.device)
    kind = NVFP4_TYPE_F32 if dw.dtype == torch.float32 else NVFP4_TYPE_BF16
    nvfp4_checkpoint_wgrad(dy, ldd, q, sf, m, n, k, group_offsets, group_counts, groups, kind, accumulate, dw, dw.stride(0),
                           workspace, workspace.numel(), stream)
    return dw
