"""A call of the operators around the step that fails on the host does not fail
the next one."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_the_error_of_a_refused_launch_stays_with_its_call():
    """A launch into a stream whose capture was broken off is refused by the
    runtime. The call says so; a good call on another stream then succeeds."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, k, E, H = 4, 2, 8, 64
    x, xp = torch.ones(T, H, device="cuda"), torch.zeros(T * k, H, device="cuda")
    idx = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    inv, ws, dws = torch.arange(T * k, dtype=torch.int32, device="cuda"), L.new_status_workspace(), L.new_workspace(T, 64, 64, E, k)
    b = torch.zeros(1, 8, 32, dtype=torch.uint8, device="cuda")
    sc, out = torch.zeros(8, 16, dtype=torch.uint8, device="cuda"), torch.zeros(8, 8, device="cuda")
    calls = {
        "permute": lambda: L.permute(x, inv, xp, ws),
        "quantize": lambda: L.mxfp_quantize(xp, b[0], sc, "mx"),
        "matmul": lambda: L.mxfp_matmul(b[0], sc, b, sc[None], out, "mx", ws),
    }
    L.dispatch(idx, E, i32(E), i32(E + 1), i32(T * k), i32(T * k), dws)
    rt = ctypes.CDLL("libcudart.so.12")  # torch's: a graph of torch's own would not survive this
    for name, call in calls.items():
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), ctypes.c_void_p()
        raw = ctypes.c_void_p(s.cuda_stream)
        with torch.cuda.stream(s):
            assert rt.cudaStreamBeginCapture(raw, 1) == 0  # thread local
            assert rt.cudaStreamSynchronize(raw) != 0  # not allowed in a capture, and breaks it off
            with pytest.raises(L.MoeError) as e:
                call()
            assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0 and not graph.value
            rt.cudaGetLastError()
        assert e.value.status == 4, name  # MOE_ERR_CUDA
        L.dispatch(idx, E, i32(E), i32(E + 1), i32(T * k), i32(T * k), dws)  # on the default stream
        call()
        torch.cuda.synchronize()
        assert L.get_status(dws) == 0 and L.get_status(ws) == 0
