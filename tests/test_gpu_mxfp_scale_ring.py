"""Block scales on their way through the product: slots that are used again and
again, every byte of them another one, in calls that have to agree bit for bit."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes", [[1, 0, 20, 3], [300, 0, 40]], ids=["narrow", "wide"])
def test_slots_used_many_times(sizes, fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(6)
    E, R, N, K = len(sizes), sum(sizes), 1000, 16_416
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, generator=g).cuda()  # noqa: E731
    lo, hi = (117, 133) if fmt == "mx" else (1, 0x7F)
    S = ref.stride(K, fmt)
    a, a_s, b, b_s = u8(0, 256, R, K // 2), u8(lo, hi, R, S), u8(0, 256, E, N, K // 2), u8(lo, hi, E, N, S)
    off = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).int().cuda()
    ws, outs = L.new_status_workspace(), [torch.zeros(R, N, device="cuda") for _ in range(20)]
    for o in outs:
        L.mxfp_matmul(a, a_s, b, b_s, o, fmt, ws, offsets=off)
    y, s = ref.grouped(ref.values(a, a_s, fmt), ref.values(b, b_s, fmt), off.tolist())
    # K fp32 additions, rounded or cut, and one rounding of the result
    assert ((outs[0].double() - y).abs() <= K * 2.0 ** -23 * s + 2.0 ** -24 * y.abs()).all()
    assert all(torch.equal(o, outs[0]) for o in outs) and L.get_status(ws) == 0
