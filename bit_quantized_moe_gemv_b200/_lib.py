"""ctypes binding of libmoe_b200.so (include/moe.h).

Argument marshalling only: every function takes torch tensors (device
memory) or plain integers, checks what the C ABI cannot see (each tensor is
on a CUDA device, contiguous, of the element type the header names and large
enough for the call), passes addresses and sizes to the C ABI and turns a
non-zero status into a MoeError. No step of the MoE computation runs
here. If the library is missing this module raises at import: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

c_i32, c_i64, c_sz, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE_TOO_SMALL",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_FAULT", 6: "MOE_ERR_TIMEOUT"}

# Every symbol include/moe.h declares (checked by the CPU test suite).
EXPORTS = ("moe_workspace_size", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine", "moe_layer",
           "moe_layer_decode_noalloc", "moe_reset_status", "moe_get_status", "moe_launch_count",
           "moe_set_wait_cycles", "moe_status_string", "moe_permute", "moe_permute_grad", "moe_unpermute",
           "moe_unpermute_grad", "moe_mxfp_scale_stride", "moe_mxfp_quantize", "moe_mxfp_dequantize",
           "moe_mxfp_matmul")


class QMatrixC(ctypes.Structure):
    _fields_ = [("qtype", c_i32), ("rows", c_i32), ("cols", c_i32), ("group", c_i32),
                ("codes", c_vp), ("scales", c_vp), ("mins", c_vp)]


class ExpertC(ctypes.Structure):
    _fields_ = [("gate", QMatrixC), ("up", QMatrixC), ("down", QMatrixC)]


class OptionsC(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("shared_gate", c_vp), ("heat", c_vp)]


MOE_BIAS_SELECTION_ONLY = 1


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}: {status_string(status)}")


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m bit_quantized_moe_gemv_b200.build` "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    sig = {
        "moe_workspace_size": (c_sz, [c_i32] * 5),
        "moe_route": (c_i32, [c_vp, c_i32, c_i32, c_vp, c_i32, c_vp, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz,
                              c_vp]),
        "moe_dispatch": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "moe_expert_ffn": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz,
                                   c_vp]),
        "moe_combine": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz,
                                c_vp]),
        "moe_layer": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp,
                              c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "moe_layer_decode_noalloc": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_i64, c_vp,
                                             c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
        "moe_reset_status": (c_i32, [c_vp, c_vp]),
        "moe_get_status": (c_i32, [c_vp, c_vp, ctypes.POINTER(c_i32)]),
        "moe_launch_count": (ctypes.c_uint64, []),
        "moe_set_wait_cycles": (c_i64, [c_i64]),
        "moe_status_string": (ctypes.c_char_p, [c_i32]),
        "moe_permute": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "moe_permute_grad": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "moe_unpermute": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
        "moe_unpermute_grad": (c_i32, [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz,
                                       c_vp]),
        "moe_mxfp_scale_stride": (c_i32, [c_i32, c_i32]),
        "moe_mxfp_quantize": (c_i32, [c_vp, c_i32, c_i64, c_i32, c_i32, ctypes.c_uint32, c_vp, c_vp, c_vp, c_vp,
                                      c_vp]),
        "moe_mxfp_dequantize": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp]),
        "moe_mxfp_matmul": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_i32, c_vp,
                                    c_i32, c_vp, c_sz, c_vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


LIB = _load()


def launch_count() -> int:
    """Kernels this library has launched in this process (host-side count)."""
    return int(LIB.moe_launch_count())


def set_wait_cycles(cycles: int) -> int:
    """Budget of every bounded wait of later fused decode launches (testing
    the failure path); negative restores the default. Returns the previous."""
    return int(LIB.moe_set_wait_cycles(int(cycles)))


def status_string(st: int) -> str:
    return LIB.moe_status_string(int(st)).decode()


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st)


# Device-tensor arguments must live on a CUDA device (a CPU test of these
# checks turns this off; no call reaches the library that way).
REQUIRE_CUDA = True

_KINDS = {  # element kind in include/moe.h -> accepted torch dtype names
    "bf16": ("bfloat16", "int16", "uint16"),  # bf16 bit patterns
    "f32": ("float32",),
    "i32": ("int32",),
    "u8": ("uint8",),
}


def _dev(t, name, kind, numel=0, optional=False):
    """Address of a device-tensor argument after the checks the C ABI cannot
    make: a CUDA tensor, contiguous, of the element type the header names and
    holding at least the `numel` elements the call touches. None is passed as
    NULL only where the header allows it."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name}: required (the call takes no NULL here)")
    if REQUIRE_CUDA and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor, got one on {t.device}")
    if str(t.dtype).replace("torch.", "") not in _KINDS[kind]:
        raise TypeError(f"{name}: dtype {t.dtype} where the call takes {kind}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _table(t, name, n, optional=False):
    """A device array of n moe_expert descriptors (uint8 bytes)."""
    return _dev(t, name, "u8", n * ctypes.sizeof(ExpertC), optional)


def _ws(ws):
    return _dev(ws, "ws", "u8")


def _bias(bias, T, E, stride):
    if stride < 0 or (stride > 0 and stride < E):
        raise ValueError(f"bias_row_stride {stride}: 0 (one row for all tokens) or at least E = {E}")
    return _dev(bias, "bias", "f32", E if stride == 0 or T == 0 else (T - 1) * stride + E, optional=True)


def _shape2(t, name, cols=None):
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [rows, {cols if cols is not None else 'cols'}]")
    return t.shape


def _opts(H, bias_selection_only=False, shared_gate=None, heat=None, E=0):
    """The moe_options of a call (None = the defaults: NULL). shared_gate is a
    device fp32 [H] tensor, heat a device int32/uint32 [E] counter tensor the
    call adds its picks to; the struct is read on the host during the call."""
    if not bias_selection_only and shared_gate is None and heat is None:
        return None
    g = _dev(shared_gate, "shared_gate", "f32", H, optional=True)
    hp = _dev(heat, "heat", "i32", E, optional=True)
    return ctypes.byref(OptionsC(MOE_BIAS_SELECTION_ONLY if bias_selection_only else 0, g, hp))


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def workspace_size(T, H, I, E, k) -> int:
    return int(LIB.moe_workspace_size(T, H, I, E, k))


def new_workspace(T, H, I, E, k, device="cuda"):
    """Allocate a workspace (torch uint8) and clear its status word."""
    import torch
    n = workspace_size(T, H, I, E, k)
    if n == 0:
        raise MoeError("moe_workspace_size", 1)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    reset_status(ws)
    return ws


def route(x, w_router, bias, bias_row_stride, k, topk_idx, topk_w, ws, logits=None, stream=None,
          bias_selection_only=False, heat=None):
    T, H = _shape2(x, "x")
    E = _shape2(w_router, "w_router", H)[0]
    _check("moe_route", LIB.moe_route(_dev(x, "x", "bf16"), T, H, _dev(w_router, "w_router", "f32"), E,
                                      _bias(bias, T, E, bias_row_stride), bias_row_stride, k,
                                      _dev(topk_idx, "topk_idx", "i32", T * k), _dev(topk_w, "topk_w", "f32", T * k),
                                      _dev(logits, "logits", "f32", T * E, optional=True),
                                      _opts(H, bias_selection_only, heat=heat, E=E), _ws(ws), ws.numel(),
                                      _stream(stream)))


def dispatch(topk_idx, E, counts, offsets, perm_src, inv_perm, ws, stream=None):
    T, k = _shape2(topk_idx, "topk_idx")
    _check("moe_dispatch", LIB.moe_dispatch(_dev(topk_idx, "topk_idx", "i32"), T, k, E,
                                            _dev(counts, "counts", "i32", E), _dev(offsets, "offsets", "i32", E + 1),
                                            _dev(perm_src, "perm_src", "i32", T * k),
                                            _dev(inv_perm, "inv_perm", "i32", T * k), _ws(ws), ws.numel(),
                                            _stream(stream)))


def expert_ffn(x, I, k, E, perm_src, offsets, counts, experts_table, y_perm, ws, stream=None):
    T, H = _shape2(x, "x")
    _check("moe_expert_ffn", LIB.moe_expert_ffn(_dev(x, "x", "bf16"), T, H, I, k, E,
                                                _dev(perm_src, "perm_src", "i32", T * k),
                                                _dev(offsets, "offsets", "i32", E + 1), _dev(counts, "counts", "i32", E),
                                                _table(experts_table, "experts_table", E),
                                                _dev(y_perm, "y_perm", "bf16", T * k * H), _ws(ws), ws.numel(),
                                                _stream(stream)))


def combine(y_perm, inv_perm, topk_w, I, x, shared_table, out, ws, stream=None, shared_gate=None):
    T, k = _shape2(topk_w, "topk_w")
    H = _shape2(out, "out")[1]
    _check("moe_combine", LIB.moe_combine(_dev(y_perm, "y_perm", "bf16", T * k * H),
                                          _dev(inv_perm, "inv_perm", "i32", T * k), _dev(topk_w, "topk_w", "f32"),
                                          T, H, I, k, _dev(x, "x", "bf16", T * H, optional=shared_table is None),
                                          _table(shared_table, "shared_table", 1, optional=True),
                                          _dev(out, "out", "bf16", T * H), _opts(H, shared_gate=shared_gate), _ws(ws),
                                          ws.numel(), _stream(stream)))


def layer(x, I, E, k, w_router, bias, bias_row_stride, experts_table, shared_table, topk_idx, topk_w, out, ws,
          stream=None, logits=None, bias_selection_only=False, shared_gate=None, heat=None):
    T, H = _shape2(x, "x")
    _shape2(w_router, "w_router", H)
    _check("moe_layer", LIB.moe_layer(_dev(x, "x", "bf16"), T, H, I, E, k, _dev(w_router, "w_router", "f32", E * H),
                                      _bias(bias, T, E, bias_row_stride), bias_row_stride,
                                      _table(experts_table, "experts_table", E),
                                      _table(shared_table, "shared_table", 1, optional=True),
                                      _dev(topk_idx, "topk_idx", "i32", T * k), _dev(topk_w, "topk_w", "f32", T * k),
                                      _dev(logits, "logits", "f32", T * E, optional=True),
                                      _dev(out, "out", "bf16", T * H),
                                      _opts(H, bias_selection_only, shared_gate, heat, E), _ws(ws), ws.numel(),
                                      _stream(stream)))


def layer_decode_noalloc(x, I, E, k, w_router, bias, bias_row_stride, experts_table, shared_table, topk_idx,
                         topk_w, out, stream=None, logits=None, bias_selection_only=False, shared_gate=None,
                         heat=None):
    """moe_layer_decode_noalloc: the fused decode step without a workspace."""
    T, H = _shape2(x, "x")
    _shape2(w_router, "w_router", H)
    _check("moe_layer_decode_noalloc",
           LIB.moe_layer_decode_noalloc(_dev(x, "x", "bf16"), T, H, I, E, k, _dev(w_router, "w_router", "f32", E * H),
                                        _bias(bias, T, E, bias_row_stride), bias_row_stride,
                                        _table(experts_table, "experts_table", E),
                                        _table(shared_table, "shared_table", 1, optional=True),
                                        _dev(topk_idx, "topk_idx", "i32", T * k),
                                        _dev(topk_w, "topk_w", "f32", T * k),
                                        _dev(logits, "logits", "f32", T * E, optional=True),
                                        _dev(out, "out", "bf16", T * H),
                                        _opts(H, bias_selection_only, shared_gate, heat, E), _stream(stream)))


def reset_status(ws, stream=None):
    _check("moe_reset_status", LIB.moe_reset_status(_ws(ws), _stream(stream)))


def get_status(ws, stream=None) -> int:
    v = c_i32(0)
    _check("moe_get_status", LIB.moe_get_status(_ws(ws), _stream(stream), ctypes.byref(v)))
    return int(v.value)


# ------------------------------------------------ operators around the step

MOE_STATUS_BYTES = 8704
FORMATS = {"mx": 1, "nv": 2}  # MOE_FP_MX, MOE_FP_NV
_FP_BLOCK = {"mx": 32, "nv": 16}
MOE_FP_SWIGLU = 1
_DTYPES = {"bfloat16": 1, "float16": 2, "float32": 3, "uint8": 4}
_dtype_codes = {}  # torch.dtype -> MOE_DT_*, filled on first use


def new_status_workspace(device="cuda"):
    """The smallest workspace: the status word of the calls below, cleared."""
    import torch
    return torch.zeros(MOE_STATUS_BYTES, dtype=torch.uint8, device=device)


def _dtype(t, name, bytes_ok=False):
    d = t.dtype
    c = _dtype_codes.get(d)
    if c is None:
        c = _dtype_codes[d] = _DTYPES.get(str(d).replace("torch.", ""), 0)
    if c == 0 or (c == 4 and not bytes_ok):
        raise TypeError(f"{name}: dtype {d} where the call takes bf16, fp16 or fp32{' or uint8' if bytes_ok else ''}")
    return c


class _Call:
    """The tensor arguments of one call: all on the current CUDA device (its
    stream is the one the kernels run on), contiguous, of the expected type and
    exactly the expected shape."""

    __slots__ = ("device",)

    def __init__(self):
        if REQUIRE_CUDA:
            import torch
            self.device = torch.cuda.current_device()

    def ptr(self, t, name, shape=None, dtype=None):
        """Address of `t`; `dtype` is a MOE_DT_* code, or the name of a torch
        dtype the header fixes."""
        if t is None:
            raise ValueError(f"{name}: required (the call takes no NULL here)")
        if REQUIRE_CUDA and t.get_device() != self.device:
            raise ValueError(f"{name}: must be a CUDA tensor on the current device {self.device}, got {t.device}")
        if isinstance(dtype, int):
            if _dtype(t, name, True) != dtype:
                raise TypeError(f"{name}: dtype {t.dtype} differs from the call's other rows")
        elif dtype is not None and _type_names(t) != dtype:
            raise TypeError(f"{name}: dtype {t.dtype} where the call takes {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        return t.data_ptr()

    def opt(self, t, name, shape, dtype):
        return None if t is None else self.ptr(t, name, shape, dtype)

    def count(self, t, name):
        """A device int32 scalar (or one-element slice), or None."""
        return None if t is None else self.ptr(t.reshape(-1), name, (1,), "int32")

    def ws(self, t):
        return self.ptr(t, "ws", None, "uint8"), t.numel()

    def stream(self, stream):
        if stream is None:
            import torch
            return torch.cuda.current_stream().cuda_stream
        d = getattr(stream, "device", None)
        if REQUIRE_CUDA and d is not None and d.index is not None and d.index != self.device:
            raise ValueError(f"stream: on device {d.index}, the tensors are on {self.device}")
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_names = {}  # torch.dtype -> its name without "torch."


def _type_names(t):
    d = t.dtype
    n = _names.get(d)
    if n is None:
        n = _names[d] = str(d).replace("torch.", "")
    return n


def _pairs(inv_perm, T):
    """k of an inv_perm [T*k] (or [T, k])."""
    n = inv_perm.numel()
    if T == 0 or n % T or n == 0:
        raise ValueError(f"inv_perm: {n} pairs for {T} tokens")
    return n // T


def permute(x, inv_perm, x_perm, ws, stream=None):
    """moe_permute: x [T, H] to the rows x_perm [T*k, H] sorted by expert."""
    c = _Call()
    T, H = _shape2(x, "x")
    if T == 0:
        return
    k, dt = _pairs(inv_perm, T), _dtype(x, "x", True)
    w, n = c.ws(ws)
    _check("moe_permute", LIB.moe_permute(c.ptr(x, "x"), dt, T, H, k, c.ptr(inv_perm, "inv_perm", None, "int32"),
                                          c.ptr(x_perm, "x_perm", (T * k, H), dt), w, n, c.stream(stream)))


def permute_grad(dx_perm, inv_perm, dx, ws, stream=None):
    """moe_permute_grad: dx [T, H], the sum of each token's rows of dx_perm."""
    c = _Call()
    T, H = _shape2(dx, "dx")
    if T == 0:
        return
    k, dt = _pairs(inv_perm, T), _dtype(dx, "dx")
    w, n = c.ws(ws)
    _check("moe_permute_grad", LIB.moe_permute_grad(c.ptr(dx_perm, "dx_perm", (T * k, H), dt), dt, T, H, k,
                                                    c.ptr(inv_perm, "inv_perm", None, "int32"), c.ptr(dx, "dx"), w, n,
                                                    c.stream(stream)))


def unpermute(y_perm, inv_perm, topk_w, out, ws, stream=None):
    """moe_unpermute: out [T, H], each token's rows weighted by topk_w [T, k]."""
    c = _Call()
    T, H = _shape2(out, "out")
    if T == 0:
        return
    k, dt = _pairs(inv_perm, T), _dtype(out, "out")
    w, n = c.ws(ws)
    _check("moe_unpermute", LIB.moe_unpermute(c.ptr(y_perm, "y_perm", (T * k, H), dt), dt, T, H, k,
                                              c.ptr(inv_perm, "inv_perm", None, "int32"),
                                              c.ptr(topk_w, "topk_w", (T, k), "float32"), c.ptr(out, "out"), w, n,
                                              c.stream(stream)))


def unpermute_grad(dout, y_perm, inv_perm, topk_w, dy_perm, dtopk_w, ws, stream=None):
    """moe_unpermute_grad: the gradients of y_perm and topk_w from dout [T, H]."""
    c = _Call()
    T, H = _shape2(dout, "dout")
    if T == 0:
        return
    k, dt = _pairs(inv_perm, T), _dtype(dout, "dout")
    w, n = c.ws(ws)
    _check("moe_unpermute_grad",
           LIB.moe_unpermute_grad(c.ptr(dout, "dout"), c.ptr(y_perm, "y_perm", (T * k, H), dt), dt, T, H, k,
                                  c.ptr(inv_perm, "inv_perm", None, "int32"),
                                  c.ptr(topk_w, "topk_w", (T, k), "float32"),
                                  c.ptr(dy_perm, "dy_perm", (T * k, H), dt),
                                  c.ptr(dtopk_w, "dtopk_w", (T, k), "float32"), w, n, c.stream(stream)))


def _format(fmt):
    f = FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"format {fmt!r}: one of {', '.join(FORMATS)}")
    return f


def mxfp_scale_stride(cols, fmt) -> int:
    """Scale bytes per row of a [*, cols] matrix in format "mx" or "nv"."""
    s = int(LIB.moe_mxfp_scale_stride(cols, _format(fmt)))
    if s == 0:
        raise MoeError("moe_mxfp_scale_stride", 1)
    return s


def _stride(cols, fmt):  # moe_mxfp_scale_stride without a call
    return (cols // _FP_BLOCK[fmt] + 15) // 16 * 16


def mxfp_quantize(x, codes, scales, fmt, tensor_scale=None, swiglu=False, rows_dev=None, stream=None):
    """moe_mxfp_quantize: x [rows, cols] (with swiglu: gate | up [rows, 2*cols])
    to codes [rows, cols/2] and scales [rows, mxfp_scale_stride(cols, fmt)]."""
    c, f = _Call(), _format(fmt)
    rows, cols = _shape2(x, "x")
    if swiglu:
        if cols % 2:
            raise ValueError(f"x: {cols} columns are no gate and up halves")
        cols //= 2
    _check("moe_mxfp_quantize",
           LIB.moe_mxfp_quantize(c.ptr(x, "x"), _dtype(x, "x"), rows, cols, f, MOE_FP_SWIGLU if swiglu else 0,
                                 c.opt(tensor_scale, "tensor_scale", (1,), "float32"), c.count(rows_dev, "rows_dev"),
                                 c.ptr(codes, "codes", (rows, cols // 2), "uint8"),
                                 c.ptr(scales, "scales", (rows, _stride(cols, fmt)), "uint8"), c.stream(stream)))


def mxfp_dequantize(codes, scales, out, fmt, tensor_scale=None, rows_dev=None, stream=None):
    """moe_mxfp_dequantize: the values of codes and scales into out [rows, cols]."""
    c, f = _Call(), _format(fmt)
    rows, cols = _shape2(out, "out")
    _check("moe_mxfp_dequantize",
           LIB.moe_mxfp_dequantize(c.ptr(codes, "codes", (rows, cols // 2), "uint8"),
                                   c.ptr(scales, "scales", (rows, _stride(cols, fmt)), "uint8"), rows, cols, f,
                                   c.opt(tensor_scale, "tensor_scale", (1,), "float32"),
                                   c.count(rows_dev, "rows_dev"), c.ptr(out, "out"), _dtype(out, "out"),
                                   c.stream(stream)))


def mxfp_matmul(a_codes, a_scales, b_codes, b_scales, out, fmt, ws, offsets=None, a_tensor_scale=None,
                b_tensor_scale=None, stream=None):
    """moe_mxfp_matmul: rows a [R, K] times their expert's b [E, N, K] into out
    [R, N]; offsets [E+1] as moe_dispatch writes them (None: E = 1)."""
    c, f = _Call(), _format(fmt)
    R, N = _shape2(out, "out")
    if b_codes.dim() != 3:
        raise ValueError(f"b_codes: shape {tuple(b_codes.shape)}, expected [E, N, K/2]")
    E, _, half = b_codes.shape
    S = _stride(2 * half, fmt)
    w, n = c.ws(ws)
    _check("moe_mxfp_matmul",
           LIB.moe_mxfp_matmul(c.ptr(a_codes, "a_codes", (R, half), "uint8"),
                               c.ptr(a_scales, "a_scales", (R, S), "uint8"),
                               c.opt(a_tensor_scale, "a_tensor_scale", (1,), "float32"), R, 2 * half,
                               c.ptr(b_codes, "b_codes", (E, N, half), "uint8"),
                               c.ptr(b_scales, "b_scales", (E, N, S), "uint8"),
                               c.opt(b_tensor_scale, "b_tensor_scale", (E,), "float32"), E, N,
                               c.opt(offsets, "offsets", (E + 1,), "int32"), f, c.ptr(out, "out"),
                               _dtype(out, "out"), w, n, c.stream(stream)))
