"""Quantisation to microscaled fp4 and back, byte for byte against fp64: the
rounding of scales and codes is decided on exact quotients, so every byte is
determined."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _quantise(x, fmt, g=None, swiglu=False, rows_dev=None, fill=0xAB):
    from bit_quantized_moe_gemv_b200 import _lib as L
    rows, cols = x.shape[0], x.shape[1] // (2 if swiglu else 1)
    codes = torch.full((rows, cols // 2), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, L.mxfp_scale_stride(cols, fmt)), fill, dtype=torch.uint8, device="cuda")
    L.mxfp_quantize(x, codes, scales, fmt, tensor_scale=g, swiglu=swiglu, rows_dev=rows_dev)
    return codes, scales


def _check(x, fmt, g=None, swiglu=False):
    codes, scales = _quantise(x, fmt, g, swiglu)
    v = ref.swiglu(x) if swiglu else x.double()
    want_c, want_s = ref.quantise(v, fmt, float(g) if g is not None else 1.0)
    cols = v.shape[1]
    torch.testing.assert_close(scales, ref.pad_scales(want_s, cols, fmt), rtol=0, atol=0)
    torch.testing.assert_close(codes, ref.pack(want_c), rtol=0, atol=0)
    return codes, scales


def _tscale(fmt, v):
    return torch.tensor([v], device="cuda") if fmt == "nv" else None


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (10, 768), (3, 96), (33, 2080), (7, 1056), (1031, 544)])
def test_codes_and_scales(rows, cols, dtype, fmt):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x = x.to(dtype).cuda()
    for ts in ((None,) if fmt == "mx" else (None, 7.3e-3, 0.25, 3.0)):
        codes, scales = _check(x, fmt, None if ts is None else _tscale(fmt, ts))
    from bit_quantized_moe_gemv_b200 import _lib as L
    for out_dtype in DTYPES:
        out = torch.empty(rows, cols, dtype=out_dtype, device="cuda")
        L.mxfp_dequantize(codes, scales, out, fmt, tensor_scale=_tscale(fmt, 3.0))
        want = ref.values(codes, scales, fmt, 3.0 if fmt == "nv" else 1.0)
        # fp32 first (one rounding for the tensor scale), then the output type
        assert torch.equal(out, want.float().to(out_dtype))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_large_inputs_take_the_unrolled_kernel(dtype, fmt):
    x = torch.randn(6000, 2080, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    _check(x, fmt, _tscale(fmt, 0.01))
    _check(x, fmt, _tscale(fmt, 0.01), swiglu=True) if x.shape[1] % 64 == 0 else _check(x[:, :2048].contiguous(), fmt,
                                                                                      _tscale(fmt, 0.01), True)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (10, 768), (129, 800)])
def test_swiglu_input(rows, cols, dtype, fmt):
    g = torch.Generator().manual_seed(rows)
    x = (2 * torch.randn(rows, 2 * cols, generator=g)).to(dtype).cuda()
    _check(x, fmt, _tscale(fmt, 0.02), swiglu=True)
    # gates far out: silu is about gate, about 0, or exactly so
    x[:, :cols] *= 30
    _check(x.clamp(-6e4, 6e4), fmt, _tscale(fmt, 0.02), swiglu=True)


@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 0.5), ("nv", 7.3e-3), ("nv", 1.7)])
def test_values_on_and_beside_rounding_borders(fmt, g):
    """Every border of E2M1 times every kind of scale, exactly and one fp32
    step to either side; block maxima beside the borders of the scale."""
    n = ref.BLOCK[fmt]
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    gg = g if g is not None else 1.0
    gf = float(torch.tensor(gg, dtype=torch.float32))
    rows = []
    scales = [2.0 ** e for e in (-20, -3, 0, 7)] if fmt == "mx" else [2.0 ** -9, 2.0 ** -6, 0.375, 1.0, 1.625, 13.0, 448.0]
    for s in scales:
        top = 6.0 * s * gf
        b = (borders * s * gf).float()
        for v in (b, torch.nextafter(b, torch.full_like(b, 1e30)), torch.nextafter(b, torch.zeros_like(b))):
            row = torch.zeros(32)
            row[0] = row[16] = top
            row[1:8], row[17:24] = v, -v
            rows.append(row)
    if fmt == "nv":  # block maxima about the borders between E4M3 values
        t = ref.e4m3_table("cpu")
        mid = ((t[:-1] + t[1:]) / 2 * 6.0 * gf).float()
        for v in (mid, torch.nextafter(mid, torch.full_like(mid, 1e30)), torch.nextafter(mid, torch.zeros_like(mid))):
            for m in v:
                row = torch.full((32,), float(m) / 3)
                row[0] = row[20] = m
                rows.append(row)
    else:
        for e in range(-40, 40):
            for m in (2.0 ** e, 2.0 ** e * (1 - 2.0 ** -24), 2.0 ** e * (1 + 2.0 ** -23)):
                row = torch.full((32,), m * 0.6)
                row[n - 1] = -m
                rows.append(row)
    _check(torch.stack(rows).float().cuda(), fmt, None if g is None else torch.tensor([g], device="cuda"))


def test_swiglu_beside_rounding_borders():
    """up chosen so that silu(gate) * up lands on borders as nearly as fp32
    inputs can: the fp32 product alone would take the wrong side for some."""
    g = torch.Generator().manual_seed(3)
    for fmt in ("mx", "nv"):
        gate = (torch.randn(512, 64, generator=g).abs() + 0.1)
        silu = gate.double() / (1 + torch.exp(-gate.double()))
        want = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)[
            torch.randint(0, 7, gate.shape, generator=g)]
        want[:, ::16] = torch.where(torch.rand(512, 4, generator=g) < 0.5, 4.0, 6.0).double()
        up = (want / silu).float()
        _check(torch.cat((gate, up), 1).cuda(), fmt, None, swiglu=True)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_values(dtype, fmt):
    f = torch.finfo(dtype)
    x = torch.zeros(12, 64)
    x[1] = f.max
    x[2, :40] = f.smallest_normal
    x[3] = f.smallest_normal * f.eps  # the smallest subnormal
    x[4, 5], x[4, 40] = float("inf"), 1.0
    x[5, 33], x[5, 3] = float("nan"), -2.0
    x[6, 0], x[6, 32] = float("-inf"), float("nan")
    x[7] = -0.0
    x[8, ::2], x[8, 1::2] = f.max, f.smallest_normal
    x[9, 31], x[9, 32] = 1e-30, -1e30
    x[10] = 1e-7
    x[11] = -f.max
    x = x.to(dtype).cuda()
    codes, scales = _check(x, fmt)
    from bit_quantized_moe_gemv_b200 import _lib as L
    out = torch.empty(12, 64, device="cuda")
    L.mxfp_dequantize(codes, scales, out, fmt)
    want = ref.values(codes, scales, fmt).float()
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(out[4:7]).any(1).all()
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("used", [-3, 0, 1, 5, 9, 100])
def test_only_the_rows_in_use_are_touched(used, fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    x = torch.randn(9, 96, generator=torch.Generator().manual_seed(1)).cuda()
    n = torch.tensor([used], dtype=torch.int32, device="cuda")
    codes, scales = _quantise(x, fmt, rows_dev=n)
    full_c, full_s = _quantise(x, fmt)
    m = min(9, max(0, used))
    assert torch.equal(codes[:m], full_c[:m]) and torch.equal(scales[:m], full_s[:m])
    assert (codes[m:] == 0xAB).all() and (scales[m:] == 0xAB).all()
    out = torch.full((9, 96), 7.0, device="cuda")
    L.mxfp_dequantize(full_c, full_s, out, fmt, rows_dev=n)
    assert torch.equal(out[:m], ref.values(full_c, full_s, fmt)[:m].float()) and (out[m:] == 7).all()


def test_empty_and_captured():
    from bit_quantized_moe_gemv_b200 import _lib as L
    _quantise(torch.empty(0, 64, device="cuda"), "mx")
    x = torch.randn(40, 512, generator=torch.Generator().manual_seed(1)).cuda()
    codes, scales = torch.empty(40, 256, dtype=torch.uint8, device="cuda"), torch.empty(40, 16, dtype=torch.uint8, device="cuda")
    out = torch.empty(40, 512, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.mxfp_quantize(x, codes, scales, "mx")
        L.mxfp_dequantize(codes, scales, out, "mx")
    x.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    want_c, want_s = ref.quantise(x, "mx")
    assert torch.equal(codes, ref.pack(want_c)) and torch.equal(scales, ref.pad_scales(want_s, 512, "mx"))
    assert torch.equal(out, ref.values(codes, scales, "mx").float())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("cols", [32, 96, 256, 320, 480, 768, 1312])
@pytest.mark.parametrize("swiglu", [False, True])
def test_large_inputs_of_every_row_split(cols, swiglu, fmt):
    """Rows that 4, 8, 16 and 32 lanes share, in ones to fours; the used rows end
    inside a warp's."""
    dtype = torch.bfloat16 if cols % 64 else torch.float32
    rows = 5_000_000 // cols + 3
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols * (2 if swiglu else 1), generator=g).to(dtype).cuda()
    codes, scales = _check(x, fmt, _tscale(fmt, 0.01), swiglu)
    n = torch.tensor([rows - 1234], dtype=torch.int32, device="cuda")
    c, s = _quantise(x, fmt, _tscale(fmt, 0.01), swiglu, n)
    assert torch.equal(c[:n], codes[:n]) and torch.equal(s[:n], scales[:n])
    assert (c[n:] == 0xAB).all() and (s[n:] == 0xAB).all()
