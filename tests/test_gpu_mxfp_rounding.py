"""NV values are code * scale * tensor scale, rounded once to the output type."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu


def _once(v, bits, lowest):
    """fp64 v rounded to `bits` significant bits, steps of at least 2^lowest, ties to even."""
    e = torch.frexp(v)[1]
    step = torch.clamp(e - bits, min=lowest)
    return torch.ldexp(torch.round(torch.ldexp(v, -step)), step)


@pytest.mark.parametrize("dtype,bits,lowest", [(torch.bfloat16, 8, -133), (torch.float16, 11, -24), (torch.float32, 24, -149)])
def test_dequantised_values_are_rounded_once(dtype, bits, lowest):
    """Every code with every scale, under tensor scales of full mantissas: among
    them products that fp32 would round onto a tie of 16 bits."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    r = torch.Generator().manual_seed(4)
    cols = 127 * 16 + 16
    codes = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * (cols // 16)], dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, L.mxfp_scale_stride(cols, "nv"), dtype=torch.uint8, device="cuda")
    scales[0, :127] = torch.arange(127, dtype=torch.uint8)
    g = torch.rand(600, generator=r) + 0.5
    g[0] = float.fromhex("0x1.5eaaaap-1")  # 0.5 x 1.5 x g is next to a tie of bf16
    # odd multiples of half a step of 16 bits, over a code times a scale, to either side
    for i in range(1, 300):
        n = int(torch.randint(1 << (bits % 24), 2 << (bits % 24), (1,), generator=r))
        near = torch.tensor((2 * n + 1) / float(torch.randint(3, 46, (1,), generator=r)))
        near = torch.nextafter(near, torch.tensor(0.0 if i % 2 else 1e30))
        g[i] = near / 2.0 ** int(torch.frexp(near)[1])
    g[-1], g[-2], g[-3] = 2.0 ** -90, 2.0 ** 90, 1.75 * 2.0 ** -20
    vals = ref.values(codes, scales, "nv")
    out, twice = torch.empty(1, cols, dtype=dtype, device="cuda"), 0
    for t in g.cuda():
        L.mxfp_dequantize(codes, scales, out, "nv", tensor_scale=t[None].contiguous())
        exact = vals * t.double()
        want = _once(exact, bits, lowest)
        want = torch.where(want.abs() > torch.finfo(dtype).max, torch.copysign(torch.full_like(want, float("inf")), want), want)
        assert torch.equal(out.double(), want), (float(t), (out.double() != want).sum())
        twice += int((exact.float().to(dtype).double() != want).sum())
    # the inputs do tell one rounding from two
    assert twice > 0 or dtype == torch.float32
