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
_REAL = LIB     # the library the fast path is bound to (tests put others in LIB's place)
_native = None  # the fast path, bound on first use: it needs torch's libraries


def launch_count() -> int:
    """Kernels this library has launched in this process (host-side count)."""
    return int(LIB.moe_launch_count())


def set_wait_cycles(cycles: int) -> int:
    """Budget of every bounded wait of later fused decode launches and fp4
    products (testing the failure path); negative restores the default. Returns the previous."""
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
_torch = None  # the torch module and what the calls below need of it, on first use
_codes = {}    # torch.dtype -> MOE_DT_*
_raw_stream = None


def _fast():
    """The module of csrc/binding.cpp, which makes a call whose arguments are
    plainly right without the checks below; there is no running without it."""
    global _native
    if _native is None:
        _rt()
        if not os.path.exists(_build.NATIVE):
            raise ImportError(f"{_build.NATIVE} is missing: build it with `python -m bit_quantized_moe_gemv_b200.build`")
        from . import _native as m
        m.bind(LIB._name)
        _native = m
    return _native


def _rt():
    """Set up on the first call: importing torch here keeps the module's import
    light, and a call's checks cost less than its launch."""
    global _torch, _raw_stream
    import torch
    _torch = torch
    _codes.update({torch.bfloat16: 1, torch.float16: 2, torch.float32: 3, torch.uint8: 4})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch


def new_status_workspace(device="cuda"):
    """The smallest workspace: the status word of the calls below, cleared."""
    return (_torch or _rt()).zeros(MOE_STATUS_BYTES, dtype=_torch.uint8, device=device)


def _device():
    """The device whose stream a call runs on, and on which its tensors must
    be: the current one (-1, the CPU, in tests without a device)."""
    t = _torch or _rt()
    return t.cuda.current_device() if REQUIRE_CUDA else -1


def _on(stream, dev):
    """Address of the stream a call runs on: the current one, or `stream`."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(dev)
        return _torch.cuda.current_stream().cuda_stream
    d = getattr(stream, "device", None)
    if REQUIRE_CUDA and d is not None and d.index is not None and d.index != dev:
        raise ValueError(f"stream: on device {d.index}, the tensors are on {dev}")
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _p(t, name, dev, dtype, shape):
    """Address of a tensor argument: on the current device, contiguous, of the
    given torch dtype and exactly the given shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        raise ValueError(f"{name}: required (the call takes no NULL here)")
    if t.get_device() != dev:
        raise ValueError(f"{name}: must be a CUDA tensor on the current device {dev}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype} where the call takes {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _opt(t, name, dev, dtype, shape):
    return None if t is None else _p(t, name, dev, dtype, shape)


def _count(t, name, dev):
    """A device int32 scalar (or one-element slice), or None."""
    return None if t is None else _p(t.reshape(-1), name, dev, _torch.int32, (1,))


def _rows_of(t, name, bytes_ok=False):
    """(rows, columns, torch dtype, MOE_DT_* code) of the matrix a call goes by."""
    if t is None:
        raise ValueError(f"{name}: required (the call takes no NULL here)")
    n, m = _shape2(t, name)
    d = t.dtype
    c = _codes.get(d, 0)
    if c == 0 or (c == 4 and not bytes_ok):
        raise TypeError(f"{name}: dtype {d} where the call takes bf16, fp16 or fp32{' or uint8' if bytes_ok else ''}")
    return n, m, d, c


def _pairs(inv_perm, T, dev):
    """(address, k) of an inv_perm [T*k] (or [T, k])."""
    if inv_perm is None:
        raise ValueError("inv_perm: required (the call takes no NULL here)")
    n = inv_perm.numel()
    if n % T or n == 0:
        raise ValueError(f"inv_perm: {n} pairs for {T} tokens")
    return _p(inv_perm, "inv_perm", dev, _torch.int32, inv_perm.shape), n // T


def _status_ws(ws, dev):
    return _p(ws, "ws", dev, _torch.uint8, None if ws is None else ws.shape)


def permute(x, inv_perm, x_perm, ws, stream=None):
    """moe_permute: x [T, H] to the rows x_perm [T*k, H] sorted by expert."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).permute(x, inv_perm, x_perm, ws)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_permute", st)
    dev = _device()
    T, H, d, code = _rows_of(x, "x", True)
    if T == 0:
        return
    inv, k = _pairs(inv_perm, T, dev)
    st = LIB.moe_permute(_p(x, "x", dev, d, (T, H)), code, T, H, k, inv, _p(x_perm, "x_perm", dev, d, (T * k, H)),
                         _status_ws(ws, dev), ws.numel(), _on(stream, dev))
    if st:
        raise MoeError("moe_permute", st)


def permute_grad(dx_perm, inv_perm, dx, ws, stream=None):
    """moe_permute_grad: dx [T, H], the sum of each token's rows of dx_perm."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).permute_grad(dx_perm, inv_perm, dx, ws)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_permute_grad", st)
    dev = _device()
    T, H, d, code = _rows_of(dx, "dx")
    if T == 0:
        return
    inv, k = _pairs(inv_perm, T, dev)
    st = LIB.moe_permute_grad(_p(dx_perm, "dx_perm", dev, d, (T * k, H)), code, T, H, k, inv,
                              _p(dx, "dx", dev, d, (T, H)), _status_ws(ws, dev), ws.numel(), _on(stream, dev))
    if st:
        raise MoeError("moe_permute_grad", st)


def unpermute(y_perm, inv_perm, topk_w, out, ws, stream=None):
    """moe_unpermute: out [T, H], each token's rows weighted by topk_w [T, k]."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).unpermute(y_perm, inv_perm, topk_w, out, ws)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_unpermute", st)
    dev = _device()
    T, H, d, code = _rows_of(out, "out")
    if T == 0:
        return
    inv, k = _pairs(inv_perm, T, dev)
    st = LIB.moe_unpermute(_p(y_perm, "y_perm", dev, d, (T * k, H)), code, T, H, k, inv,
                           _p(topk_w, "topk_w", dev, _torch.float32, (T, k)), _p(out, "out", dev, d, (T, H)),
                           _status_ws(ws, dev), ws.numel(), _on(stream, dev))
    if st:
        raise MoeError("moe_unpermute", st)


def unpermute_grad(dout, y_perm, inv_perm, topk_w, dy_perm, dtopk_w, ws, stream=None):
    """moe_unpermute_grad: the gradients of y_perm and topk_w from dout [T, H]."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).unpermute_grad(dout, y_perm, inv_perm, topk_w, dy_perm, dtopk_w, ws)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_unpermute_grad", st)
    dev = _device()
    T, H, d, code = _rows_of(dout, "dout")
    if T == 0:
        return
    inv, k = _pairs(inv_perm, T, dev)
    f = _torch.float32
    st = LIB.moe_unpermute_grad(_p(dout, "dout", dev, d, (T, H)), _p(y_perm, "y_perm", dev, d, (T * k, H)), code, T, H,
                                k, inv, _p(topk_w, "topk_w", dev, f, (T, k)),
                                _p(dy_perm, "dy_perm", dev, d, (T * k, H)), _p(dtopk_w, "dtopk_w", dev, f, (T, k)),
                                _status_ws(ws, dev), ws.numel(), _on(stream, dev))
    if st:
        raise MoeError("moe_unpermute_grad", st)


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
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).quantize(x, codes, scales, fmt, tensor_scale, swiglu, rows_dev)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_mxfp_quantize", st)
    dev, f = _device(), _format(fmt)
    rows, wide, d, code = _rows_of(x, "x")
    cols = wide
    if swiglu:
        if wide % 2:
            raise ValueError(f"x: {wide} columns are no gate and up halves")
        cols = wide // 2
    u8 = _torch.uint8
    st = LIB.moe_mxfp_quantize(_p(x, "x", dev, d, (rows, wide)), code, rows, cols, f, MOE_FP_SWIGLU if swiglu else 0,
                               _opt(tensor_scale, "tensor_scale", dev, _torch.float32, (1,)),
                               _count(rows_dev, "rows_dev", dev), _p(codes, "codes", dev, u8, (rows, cols // 2)),
                               _p(scales, "scales", dev, u8, (rows, _stride(cols, fmt))), _on(stream, dev))
    if st:
        raise MoeError("moe_mxfp_quantize", st)


def mxfp_dequantize(codes, scales, out, fmt, tensor_scale=None, rows_dev=None, stream=None):
    """moe_mxfp_dequantize: the values of codes and scales into out [rows, cols]."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).dequantize(codes, scales, out, fmt, tensor_scale, rows_dev)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_mxfp_dequantize", st)
    dev, f = _device(), _format(fmt)
    rows, cols, d, code = _rows_of(out, "out")
    u8 = _torch.uint8
    st = LIB.moe_mxfp_dequantize(_p(codes, "codes", dev, u8, (rows, cols // 2)),
                                 _p(scales, "scales", dev, u8, (rows, _stride(cols, fmt))), rows, cols, f,
                                 _opt(tensor_scale, "tensor_scale", dev, _torch.float32, (1,)),
                                 _count(rows_dev, "rows_dev", dev), _p(out, "out", dev, d, (rows, cols)), code,
                                 _on(stream, dev))
    if st:
        raise MoeError("moe_mxfp_dequantize", st)


def mxfp_matmul(a_codes, a_scales, b_codes, b_scales, out, fmt, ws, offsets=None, a_tensor_scale=None,
                b_tensor_scale=None, stream=None):
    """moe_mxfp_matmul: rows a [R, K] times their expert's b [E, N, K] into out
    [R, N]; offsets [E+1] as moe_dispatch writes them (None: E = 1)."""
    if stream is None and LIB is _REAL:
        st = (_native or _fast()).matmul(a_codes, a_scales, b_codes, b_scales, out, fmt, ws, offsets, a_tensor_scale,
                                     b_tensor_scale)
        if st == 0:
            return
        if st > 0:
            raise MoeError("moe_mxfp_matmul", st)
    dev, f = _device(), _format(fmt)
    R, N, d, code = _rows_of(out, "out")
    if b_codes is None or b_codes.dim() != 3:
        raise ValueError("b_codes: expected [E, N, K/2]")
    E, _, half = b_codes.shape
    S, u8, f32 = _stride(2 * half, fmt), _torch.uint8, _torch.float32
    st = LIB.moe_mxfp_matmul(_p(a_codes, "a_codes", dev, u8, (R, half)), _p(a_scales, "a_scales", dev, u8, (R, S)),
                             _opt(a_tensor_scale, "a_tensor_scale", dev, f32, (1,)), R, 2 * half,
                             _p(b_codes, "b_codes", dev, u8, (E, N, half)), _p(b_scales, "b_scales", dev, u8, (E, N, S)),
                             _opt(b_tensor_scale, "b_tensor_scale", dev, f32, (E,)), E, N,
                             _opt(offsets, "offsets", dev, _torch.int32, (E + 1,)), f, _p(out, "out", dev, d, (R, N)),
                             code, _status_ws(ws, dev), ws.numel(), _on(stream, dev))
    if st:
        raise MoeError("moe_mxfp_matmul", st)
