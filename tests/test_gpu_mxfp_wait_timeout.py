"""Bounded waits of the fp4 product that run out: the launch ends by itself,
reports MOE_ERR_TIMEOUT, leaves nothing in flight, and the next call is right.
The failure is made by the waits' budget alone."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu

MOE_ERR_TIMEOUT = 6


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes,N", [([3, 0, 20], 2000), ([400, 0, 161], 1000), ([2000], 8200)],
                         ids=["narrow", "wide", "many_tiles"])
def test_expired_waits_are_reported_and_the_next_call_is_right(sizes, N, fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(7)
    E, R, K = len(sizes), sum(sizes), 4128
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, generator=g).cuda()  # noqa: E731
    lo, hi = (120, 130) if fmt == "mx" else (24, 72)
    S = ref.stride(K, fmt)
    a, a_s, b, b_s = u8(0, 256, R, K // 2), u8(lo, hi, R, S), u8(0, 256, E, N, K // 2), u8(lo, hi, E, N, S)
    off = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).int().cuda()
    ws = L.new_status_workspace()

    def call(out):
        L.mxfp_matmul(a, a_s, b, b_s, out, fmt, ws, offsets=off)

    want = torch.zeros(R, N, device="cuda")
    call(want)
    assert L.get_status(ws) == 0
    y, s = ref.grouped(ref.values(a, a_s, fmt), ref.values(b, b_s, fmt), off.tolist())
    assert ((want.double() - y).abs() <= K * 2.0 ** -23 * s + 2.0 ** -24 * y.abs()).all()
    default = L.set_wait_cycles(-1)
    try:
        # from the first wait on, and wherever else in the pipeline a budget ends
        for cycles in [0] * 3 + [500 * i for i in range(1, 41)]:
            out, good = torch.empty_like(want), torch.zeros_like(want)
            assert L.set_wait_cycles(cycles) >= 0
            call(out)  # the host call itself succeeds
            L.set_wait_cycles(-1)
            call(good)  # follows at once, on the same SMs
            status = L.get_status(ws)
            assert status in (0, MOE_ERR_TIMEOUT) and (cycles or status == MOE_ERR_TIMEOUT), cycles
            assert torch.equal(good, want), cycles
            if status == 0:
                assert torch.equal(out, want), cycles
            L.reset_status(ws)
    finally:
        L.set_wait_cycles(-1)
    assert L.set_wait_cycles(-1) == default
