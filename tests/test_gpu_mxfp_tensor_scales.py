"""The grouped fp4 product under tensor scales of their whole range, 2^-90 to
2^90, against fp64. Tolerance: K 2^-23 sum|a b| for the fp32 sums, 2^-23 of the
value for ga gb[e] and its product, eps/2 of the value for the output type, and
half the smallest subnormal of either type where the value lies that low."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu

PAIRS = [(64, 64), (90, 90), (70, 40), (-70, -70), (-90, -90), (-75, -74), (-63, -64), (63, 64), (90, -90), (-90, 89), (0, -90), (2, 90)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [3, 200], ids=["narrow", "wide"])
def test_the_product_of_both_scales_may_leave_the_range(rows, dtype):
    from bit_quantized_moe_gemv_b200 import _lib as L
    r = torch.Generator().manual_seed(rows)
    E, N, K = len(PAIRS), 72, 288
    R = rows * E
    codes = [torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, generator=r) for n in (R, E * N)]
    scales = [torch.zeros(n, ref.stride(K, "nv"), dtype=torch.uint8) for n in (R, E * N)]
    for s in scales:  # rows of different size: sums of 2^-18 up to 2^23
        s[:, :K // 16] = torch.randint(0, 5, (s.shape[0], 1), generator=r).mul(25).to(torch.uint8) + \
            torch.randint(1, 20, (s.shape[0], K // 16), generator=r).to(torch.uint8)
    codes[0][1::rows] = 0  # rows of zeros, and of negative ones
    codes[0][2::rows] = 0x88
    a, b, a_s, b_s = (t.cuda() for t in codes + scales)
    out, ws = torch.empty(R, N, dtype=dtype, device="cuda"), L.new_status_workspace()
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * rows
    m = torch.rand(2, E, generator=r) * 0.9 + 1
    av, bv = ref.values(a, a_s, "nv"), ref.values(b, b_s, "nv").view(E, N, K)
    f = torch.finfo(dtype)
    for i, (p, _) in enumerate(PAIRS):
        ga = torch.tensor([2.0 ** p]).mul(m[0, i] if abs(p) < 90 else 1.0).cuda()
        gb = torch.tensor([2.0 ** q for _, q in PAIRS]).mul(torch.where(torch.tensor([abs(q) < 90 for _, q in PAIRS]), m[1], 1.0)).cuda()
        out.fill_(7)
        L.mxfp_matmul(a, a_s, b.view(E, N, -1), b_s.view(E, N, -1), out, "nv", ws, offsets=off, a_tensor_scale=ga,
                      b_tensor_scale=gb)
        y, s = ref.grouped(av, bv, off.tolist(), float(ga), gb)
        acc = K * 2.0 ** -23 * s + 2.0 ** -23 * y.abs() + 2.0 ** -149
        tol = acc + f.eps / 2 * (y.abs() + acc) + f.smallest_normal * f.eps / 2
        got = out.double()
        fits, over = y.abs() + tol < f.max, y.abs() - tol > 2.0 * f.max
        assert ((got - y).abs() <= tol)[fits].all(), (p, ((got - y).abs() - tol)[fits].max())
        assert (torch.isinf(got) & (got.sign() == y.sign()))[over].all(), p
        assert not torch.isnan(got).any(), p
    assert L.get_status(ws) == 0


def test_a_scale_of_zero_gives_zeros():
    """Not asked for, but what a matrix of zeros is scaled by: no NaN comes of it."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()  # noqa: E731
    out = torch.full((2, 8), 7.0, device="cuda")
    one, zero = torch.full((1,), 2.0 ** 80, device="cuda"), torch.zeros(1, device="cuda")
    sc = torch.full((8, 16), 56, dtype=torch.uint8, device="cuda")
    for ga, gb in ((one, zero), (zero, one), (zero, zero)):
        L.mxfp_matmul(u8(2, 32), sc[:2].contiguous(), u8(1, 8, 32), sc[None], out, "nv", L.new_status_workspace(), a_tensor_scale=ga, b_tensor_scale=gb)
        assert (out == 0).all()
