"""Refusals of the row and fp4 operators, on CPU: the C entry points before any
CUDA call, the binding before any call; and the fp64 reference itself."""
import ctypes

import pytest
import torch

from bit_quantized_moe_gemv_b200 import build

from tests import mxfp_reference as ref
from tests.test_binding_checks import _Recorder

P, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)  # never read: the checks come first
WS = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def L():
    build.build()
    from bit_quantized_moe_gemv_b200 import _lib
    return _lib


def test_row_calls_check_their_arguments(L):
    f = L.LIB.moe_permute
    good = [P, 1, 4, 64, 2, P, P, WS, 8704, None]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_2=0) == 0  # no tokens: nothing to do
    for bad in (dict(_0=None), dict(_5=None), dict(_6=None), dict(_7=None), dict(_2=-1), dict(_3=0), dict(_3=1 << 25),
                dict(_4=0), dict(_4=65), dict(_2=1 << 30), dict(_2=1 << 14, _3=1 << 23), dict(_0=ODD), dict(_6=ODD), dict(_5=ODD), dict(_7=ODD)):
        assert call(**bad) == 1, bad
    assert call(_1=0) == 2 and call(_1=5) == 2
    assert call(_8=8703) == 3
    # sums and gradients have no byte form
    assert L.LIB.moe_permute_grad(P, 4, 4, 64, 2, P, P, WS, 8704, None) == 2
    assert L.LIB.moe_unpermute(P, 4, 4, 64, 2, P, P, P, WS, 8704, None) == 2
    assert L.LIB.moe_unpermute(P, 1, 4, 64, 2, P, None, P, WS, 8704, None) == 1
    assert L.LIB.moe_unpermute(P, 1, 4, 64, 2, P, ODD, P, WS, 8704, None) == 1
    for i in (1, 7, 8, 9):
        a = [P, P, 1, 4, 64, 2, P, P, P, P, WS, 8704, None]
        a[i] = None
        assert L.LIB.moe_unpermute_grad(*a) == 1, i
    assert L.LIB.moe_unpermute_grad(P, P, 1, 4, 64, 2, P, P, P, P, WS, 256, None) == 3


def test_fp_calls_check_their_arguments(L):
    assert L.LIB.moe_mxfp_scale_stride(2048, 1) == 64 and L.LIB.moe_mxfp_scale_stride(2080, 1) == 80
    assert L.LIB.moe_mxfp_scale_stride(32, 2) == 16 and L.LIB.moe_mxfp_scale_stride(768, 2) == 48
    for bad in ((0, 1), (48, 1), (16, 2), (64, 3), ((1 << 24) + 32, 1), (-32, 1)):
        assert L.LIB.moe_mxfp_scale_stride(*bad) == 0
    for cols in range(32, 4096, 32):
        for fmt in ("mx", "nv"):
            assert L.mxfp_scale_stride(cols, fmt) == L._stride(cols, fmt) == ref.stride(cols, fmt)

    q = [P, 1, 4, 64, 1, 0, None, None, P, P, None]
    qd = {"fn": L.LIB.moe_mxfp_quantize, "good": q}
    mm = [P, P, None, 4, 64, P, P, None, 3, 16, P, 1, P, 1, WS, 8704, None]
    md = {"fn": L.LIB.moe_mxfp_matmul, "good": mm}
    dq = [P, P, 4, 64, 1, None, None, P, 1, None]
    dd = {"fn": L.LIB.moe_mxfp_dequantize, "good": dq}

    def call(d, *changes):
        a = list(d["good"])
        for i, v in changes:
            a[i] = v
        return d["fn"](*a)

    assert call(qd, (2, 0)) == 0 and call(md, (3, 0)) == 0 and call(dd, (2, 0)) == 0
    for c in ((0, None), (0, ODD), (8, None), (8, ODD), (9, None), (2, -1), (3, 48), (3, 0), (3, (1 << 24) + 32), (5, 2),
              (6, P), (7, ODD), (2, 1 << 50)):
        assert call(qd, c) == 1, c
    assert call(qd, (4, 2), (6, ODD)) == 1
    assert call(qd, (4, 3)) == 2 and call(qd, (1, 4)) == 2 and call(qd, (1, 0)) == 2
    for c in ((0, None), (1, ODD), (7, None), (7, ODD), (2, -1), (3, 40), (5, P)):
        assert call(dd, c) == 1, c
    assert call(dd, (8, 4)) == 2
    for c in ((0, None), (1, None), (5, None), (6, None), (12, None), (0, ODD), (1, ODD), (5, ODD), (6, ODD), (12, ODD),
              (10, ODD), (3, -1), (3, (1 << 30) + 1), (4, 0), (4, 40), (8, 0), (8, 1025), (9, 0), (9, (1 << 24) + 1),
              (2, P), (7, P), (14, None), (14, ODD), (10, None)):
        assert call(md, c) == 1, c
    assert call(md, (9, 1 << 24), (4, 1 << 17)) == 1  # N K: more than a tensor map strides over
    assert call(md, (3, 1 << 30), (9, 1025)) == 1  # R N: more tiles than are counted
    assert call(qd, (2, (1 << 32) + 1)) == 1 and call(dd, (2, (1 << 32) + 1)) == 1  # rows * cols
    assert call(md, (11, 0)) == 2 and call(md, (13, 4)) == 2
    assert call(md, (15, 8000)) == 3


@pytest.fixture
def rec(monkeypatch, L):
    r = _Recorder()
    monkeypatch.setattr(L, "LIB", r)
    monkeypatch.setattr(L, "REQUIRE_CUDA", False)
    return r


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_the_binding_passes_good_calls(L, rec):
    inv, ws, w = _i32(12), _u8(8704), torch.zeros(4, 3)
    L.permute(_bf(4, 64), inv, _bf(12, 64), ws, stream=0)
    L.permute(_u8(4, 64), inv, _u8(12, 64), ws, stream=0)
    L.permute_grad(_bf(12, 64), inv, _bf(4, 64), ws, stream=0)
    L.unpermute(_bf(12, 64), inv, w, _bf(4, 64), ws, stream=0)
    L.unpermute_grad(_bf(4, 64), _bf(12, 64), inv, w, _bf(12, 64), torch.zeros(4, 3), ws, stream=0)
    L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 16), "mx", stream=0)
    L.mxfp_quantize(_bf(4, 128), _u8(4, 32), _u8(4, 16), "nv", torch.ones(1), True, _i32(5)[4:], stream=0)
    L.mxfp_dequantize(_u8(4, 32), _u8(4, 16), _bf(4, 64), "mx", stream=0)
    L.mxfp_matmul(_u8(4, 32), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 16), "nv", ws, _i32(4), torch.ones(1),
                  torch.ones(3), stream=0)
    assert rec.calls == ["moe_permute"] * 2 + ["moe_permute_grad", "moe_unpermute", "moe_unpermute_grad"] + \
        ["moe_mxfp_quantize"] * 2 + ["moe_mxfp_dequantize", "moe_mxfp_matmul"]


def test_the_binding_refuses_bad_ones(L, rec):
    inv, ws, w = _i32(12), _u8(8704), torch.zeros(4, 3)
    bad = [
        lambda: L.permute(_bf(4, 64), inv, _bf(11, 64), ws, stream=0),
        lambda: L.permute(_bf(4, 64), inv, torch.zeros(12, 64), ws, stream=0),
        lambda: L.permute(_bf(64, 4).t(), inv, _bf(12, 64), ws, stream=0),
        lambda: L.permute(_bf(5, 64), inv, _bf(12, 64), ws, stream=0),
        lambda: L.permute(_bf(4, 64), inv.long(), _bf(12, 64), ws, stream=0),
        lambda: L.permute(_bf(4, 64), inv, None, ws, stream=0),
        lambda: L.permute_grad(_u8(12, 64), inv, _u8(4, 64), ws, stream=0),
        lambda: L.unpermute(_bf(12, 64), inv, w[:, :2], _bf(4, 64), ws, stream=0),
        lambda: L.unpermute(_bf(12, 64), inv, w.double(), _bf(4, 64), ws, stream=0),
        lambda: L.unpermute_grad(_bf(4, 64), _bf(12, 64), inv, w, _bf(12, 64), torch.zeros(4, 2), ws, stream=0),
        lambda: L.mxfp_quantize(_bf(4, 64), _u8(4, 31), _u8(4, 16), "mx", stream=0),
        lambda: L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 2), "mx", stream=0),
        lambda: L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 16), "fp8", stream=0),
        lambda: L.mxfp_quantize(_u8(4, 64), _u8(4, 32), _u8(4, 16), "mx", stream=0),
        lambda: L.mxfp_quantize(_bf(4, 65), _u8(4, 16), _u8(4, 16), "mx", swiglu=True, stream=0),
        lambda: L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 16), "nv", torch.ones(2), stream=0),
        lambda: L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 16), "nv", rows_dev=_i32(2), stream=0),
        lambda: L.mxfp_dequantize(_u8(4, 32), _u8(3, 16), _bf(4, 64), "mx", stream=0),
        lambda: L.mxfp_matmul(_u8(4, 32), _u8(4, 16), _u8(16, 32), _u8(16, 16), _bf(4, 16), "mx", ws, stream=0),
        lambda: L.mxfp_matmul(_u8(4, 32), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 15), "mx", ws, _i32(4),
                              stream=0),
        lambda: L.mxfp_matmul(_u8(4, 32), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 16), "mx", ws, _i32(3),
                              stream=0),
        lambda: L.mxfp_matmul(_u8(4, 48), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 16), "mx", ws, _i32(4),
                              stream=0),
        lambda: L.mxfp_matmul(_u8(4, 32), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 16), "nv", ws, _i32(4),
                              b_tensor_scale=torch.ones(1), stream=0),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
        assert rec.calls == [], i


def test_host_tensors_are_refused(L, monkeypatch):
    monkeypatch.setattr(L, "LIB", _Recorder())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        L.mxfp_quantize(_bf(4, 64), _u8(4, 32), _u8(4, 16), "mx", stream=0)


def test_the_reference_rounds_by_hand():
    """Worked blocks: ties to the even code, the scale of a maximum, saturation."""
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :10] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.2501, -7.9])
    code, byte = ref.quantise(x, "mx")
    assert byte.tolist() == [[127]]  # floor(log2 7.9) - 2 = 0
    assert code[0, :10].tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 9, 15]
    code, byte = ref.quantise(2.0 ** -9 * x, "mx")
    assert byte.tolist() == [[118]] and code[0, :10].tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 9, 15]
    y = torch.zeros(1, 32, dtype=torch.float64)
    y[0, 0], y[0, 1], y[0, 16] = 12.0, -5.0, 6.0 * 2.0 ** -10  # scales 2 and, on a tie, 0
    code, byte = ref.quantise(y, "nv")
    assert byte.tolist() == [[0x40, 0]] and code[0, :2].tolist() == [7, 12] and code[0, 16] == 0
    v = ref.values(ref.pack(code), ref.pad_scales(byte, 32, "nv"), "nv", 0.5)
    assert v[0, :2].tolist() == [6.0, -2.0]
    assert ref.e4m3_table("cpu")[[1, 7, 8, 56, 126]].tolist() == [2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 448.0]


def test_the_fast_path_leaves_everything_doubtful_to_the_checks(L):
    """The native half of the binding answers -1, without a call, to anything
    that is not plainly right: here to host tensors, other objects, wrong counts."""
    f = L._fast()
    inv, ws, w = _i32(12), _u8(8704), torch.zeros(4, 3)
    good = {
        "permute": [_bf(4, 64), inv, _bf(12, 64), ws],
        "permute_grad": [_bf(12, 64), inv, _bf(4, 64), ws],
        "unpermute": [_bf(12, 64), inv, w, _bf(4, 64), ws],
        "unpermute_grad": [_bf(4, 64), _bf(12, 64), inv, w, _bf(12, 64), w.clone(), ws],
        "quantize": [_bf(4, 64), _u8(4, 32), _u8(4, 16), "mx", None, False, None],
        "dequantize": [_u8(4, 32), _u8(4, 16), _bf(4, 64), "mx", None, None],
        "matmul": [_u8(4, 32), _u8(4, 16), _u8(3, 16, 32), _u8(3, 16, 16), _bf(4, 16), "mx", ws, _i32(4), None, None],
    }
    for name, args in good.items():
        call = getattr(f, name)
        assert call(*args) == -1  # tensors of the host
        assert call(*args[:-1]) == -1 and call(*args, None) == -1 and call() == -1
        for i in range(len(args)):
            for other in (None, 3, "x", object()):
                assert call(*args[:i], other, *args[i + 1:]) == -1
    with pytest.raises(ImportError):
        f.bind("/nowhere/libmoe_b200.so")
    f.bind(L._build.LIB)


def test_a_missing_inv_perm_is_named(L, rec):
    ws, w = _u8(8704), torch.zeros(4, 3)
    for f in (lambda: L.permute(_bf(4, 64), None, _bf(12, 64), ws, stream=0),
              lambda: L.permute_grad(_bf(12, 64), None, _bf(4, 64), ws, stream=0),
              lambda: L.unpermute(_bf(12, 64), None, w, _bf(4, 64), ws, stream=0),
              lambda: L.unpermute_grad(_bf(4, 64), _bf(12, 64), None, w, _bf(12, 64), torch.zeros(4, 3), ws, stream=0)):
        with pytest.raises(ValueError, match="inv_perm: required"):
            f()
    assert rec.calls == []
