"""The row and fp4 operators where element offsets pass 32 bits: the first and
the last rows (and columns) against the same fp64 references."""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu

BIG = 2 ** 31


def _ends(n):
    return torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantise_and_back(fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    rows, cols = 134_000, 16_416
    assert rows * cols > BIG
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, L.mxfp_scale_stride(cols, fmt), dtype=torch.uint8, device="cuda")
    L.mxfp_quantize(x, codes, scales, fmt)
    at = _ends(rows)
    c, s = ref.quantise(x[at], fmt)
    assert torch.equal(codes[at], ref.pack(c)) and torch.equal(scales[at], ref.pad_scales(s, cols, fmt))
    L.mxfp_dequantize(codes, scales, x, fmt)
    assert torch.equal(x[at], ref.values(codes[at], scales[at], fmt).bfloat16())


def test_rows_and_back():
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, k, H = 66_000, 4, 8_192
    assert T * k * H > BIG
    g = torch.Generator("cuda").manual_seed(2)
    inv = torch.randperm(T * k, generator=g, device="cuda").int()
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(T, k, generator=g, device="cuda")
    ws, xp = L.new_status_workspace(), torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    L.permute(x, inv, xp, ws)
    at = _ends(T)
    rows = inv.view(T, k)[at].long()
    assert torch.equal(xp[rows], x[at][:, None].expand(-1, k, -1))
    assert torch.equal(xp[-1], x[torch.nonzero(inv == T * k - 1)[0, 0] // k])
    out, u = torch.empty_like(x), 2.0 ** -24
    eps = torch.finfo(torch.bfloat16).eps / 2 * (1 + 2.0 ** -10)
    for weights in (None, w):
        if weights is None:
            L.permute_grad(xp, inv, out, ws)
        else:
            L.unpermute(xp, inv, w, out, ws)
        want = x[at].double() * (k if weights is None else w[at].double().sum(1, keepdim=True))
        assert ((out[at].double() - want).abs() <= (eps + (k + 1) * u) * want.abs()).all()
    dw, want = torch.empty_like(w), x[at].double().square().sum(1, keepdim=True).expand(-1, k)
    dy = torch.empty_like(xp)
    L.unpermute_grad(x, xp, inv, w, dy, dw, ws)
    assert ((dw[at].double() - want).abs() <= H * u * want).all()
    ref_dy = w[at].double()[..., None] * x[at].double()[:, None]
    assert ((dy[rows].double() - ref_dy).abs() <= (eps + u) * ref_dy.abs()).all()
    assert L.get_status(ws) == 0


def test_the_most_tokens():
    from bit_quantized_moe_gemv_b200 import _lib as L
    T = BIG - 1
    x = torch.randint(0, 256, (T, 1), dtype=torch.uint8, device="cuda")
    inv = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    ws, xp = L.new_status_workspace(), torch.empty_like(x)
    L.permute(x, inv, xp, ws)
    assert torch.equal(xp, x.flip(0)) and L.get_status(ws) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_product(fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    R, N, K, E = 66_000, 33_000, 64, 2
    assert R * N > BIG
    g = torch.Generator("cuda").manual_seed(3)
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    a, b = u8(R, K // 2), u8(E, N, K // 2)
    a_s, b_s = (torch.randint(100, 110, (n, 16), dtype=torch.uint8, device="cuda", generator=g) for n in (R, E * N))
    b_s = b_s.view(E, N, 16)
    if fmt == "nv":
        a_s &= 0x7F - 64
    out, ws = torch.empty(R, N, dtype=torch.bfloat16, device="cuda"), L.new_status_workspace()
    off = torch.tensor([0, 1_000, R], dtype=torch.int32, device="cuda")
    L.mxfp_matmul(a, a_s, b, b_s, out, fmt, ws, offsets=off)
    at, cols = _ends(R), torch.cat((_ends(N), torch.tensor([N - 9, 127, 128], device="cuda")))
    av = ref.values(a[at], a_s[at], fmt)
    e = (at >= 1_000).long()
    bv = ref.values(b[:, cols], b_s[:, cols], fmt)[e]
    y, mag = (av[:, None] * bv).sum(2), (av[:, None] * bv).abs().sum(2)
    acc = K * 2.0 ** -23 * mag
    assert ((out[at][:, cols].double() - y).abs() <= acc + torch.finfo(torch.bfloat16).eps / 2 * (y.abs() + acc)).all()
    assert L.get_status(ws) == 0
