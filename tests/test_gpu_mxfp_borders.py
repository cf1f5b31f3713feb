"""SwiGLU quantisation at the ends of the fp32 range, byte for byte against
fp64: where a scale's border or an intermediate product lies next to or below
the smallest normal number, and where the values end."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu

FMAX = 2.0 ** 128 - 2.0 ** 104  # the largest fp32 number


def _check(gate, up, fmt, g=None):
    """gate, up [rows, cols] of one type."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    rows, cols = gate.shape
    x = torch.cat((gate, up), 1).contiguous().cuda()
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, L.mxfp_scale_stride(cols, fmt), dtype=torch.uint8, device="cuda")
    L.mxfp_quantize(x, codes, scales, fmt, None if g is None else torch.tensor([g], device="cuda"), swiglu=True)
    v = ref.swiglu(x)
    v = torch.where(v.abs() > FMAX, float("inf"), v)  # not held in fp32: the block becomes NaN
    code, byte = ref.quantise(v, fmt, 1.0 if g is None else float(torch.tensor(g)))
    torch.testing.assert_close(scales, ref.pad_scales(byte, cols, fmt), rtol=0, atol=0)
    torch.testing.assert_close(codes, ref.pack(code), rtol=0, atol=0)
    return code, byte


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_block_maxima_beside_the_smallest_scales(dtype):
    """silu(gate) up about 2^-124, where the MX byte changes from 0 to 1, and
    about its neighbours."""
    g = torch.Generator().manual_seed(1)
    gates, ups = [], []
    for e in (-127, -126, -125, -124, -123, -122):
        for k in (3, 4, 5, 6):  # gates of 8 to 64: silu is the gate less a part in 3,000 to 2^92
            gates.append(torch.full((32,), 2.0 ** k))
            ups.append(torch.full((32,), 2.0 ** (e - k)))
        for _ in range(40):
            gate = 40 * torch.rand(32, generator=g) + 0.5
            want = 2.0 ** e * (1 + (torch.rand(32, generator=g) - 0.5) * 2.0 ** -20)
            silu = gate.double() / (1 + torch.exp(-gate.double()))
            gates.append(gate)
            ups.append((want.double() / silu).float())
    code, byte = _check(torch.stack(gates).to(dtype), torch.stack(ups).to(dtype), "mx")
    assert {0, 1, 2} <= set(byte.reshape(-1).tolist())
    # silu(32) is 32 less a part in 2^46: 2^-124 is not reached
    code, byte = _check(torch.full((1, 32), 32.0).to(dtype), torch.full((1, 32), 2.0 ** -129).to(dtype), "mx")
    assert byte.item() == 0 and (code == 7).all()


@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 2.0 ** -88), ("nv", 2.0 ** -30)])
def test_gates_below_the_normal_range(fmt, g):
    """sigma(gate) gate has only the bits a subnormal number has, the values all of them."""
    r = torch.Generator().manual_seed(2)
    gate = torch.zeros(300, 64)
    gate[0, :2] = torch.tensor([2.0 ** -149, 2.0 ** -147])
    for i in range(1, 300):
        n = torch.randint(1, 1 << int(torch.randint(1, 25, (1,), generator=r)), (64,), generator=r)
        gate[i] = n.double().mul(2.0 ** -149).float() * (1 - 2 * torch.randint(0, 2, (64,), generator=r))
    up = torch.exp2(torch.randint(20, 127, (300, 1), generator=r).float()).expand(-1, 64) * (torch.rand(300, 64, generator=r) + 0.5)
    up[0] = 2.0 ** 100
    assert (gate != 0).any(1).all()
    code, byte = _check(gate, up, fmt, g)
    if fmt == "mx":
        assert code[0, :2].tolist() == [2, 6]


@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 2.0 ** 88)])
def test_values_beside_the_end_of_the_range(fmt, g):
    """Just below the largest fp32 number and just above: a block is NaN from there on."""
    r = torch.Generator().manual_seed(3)
    gate = 60 * torch.rand(400, 32, generator=r) + 1
    silu = gate.double() / (1 + torch.exp(-gate.double()))
    step = torch.randint(-3, 4, (400, 1), generator=r).double()
    up = (FMAX / silu * (1 + step * 2.0 ** -24)).float()
    few = torch.rand(400, 32, generator=r) < 0.9  # the rest of a block well inside
    up = torch.where(few, up / 8, up)
    nan = 255 if fmt == "mx" else 0x7F
    code, byte = _check(gate, up, fmt, g)
    assert (byte == nan).any() and (byte != nan).any()
    # infinities and NaN next to values at the end, in either half
    for half, v in ((0, float("inf")), (1, float("nan")), (1, float("-inf"))):
        halves = [gate.clone(), up.clone()]
        halves[half][::3, 5] = v
        _check(*halves, fmt, g)
