"""Microscaled fp4 in 64 bits, from the formats' definitions: the plain
implementation the fp4 operators are tested against. Works on any device and
shares nothing with the kernels.
"""
import torch

BLOCK = {"mx": 32, "nv": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def stride(cols, fmt):
    return -(-(cols // BLOCK[fmt]) // 16) * 16


def pow2(e):
    """2^e of whole e in [-200, 200], exactly: pow on CUDA is not exact, and a
    scale off by one bit hides the ties."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)[e.long() + 200]


def e4m3_table(device):
    b = torch.arange(0, 127, device=device)
    e, m = b // 8, (b % 8).double()
    return torch.where(e > 0, (1 + m / 8) * pow2(e - 7), m * 2.0 ** -9)


def nearest(values, x):
    """Index of the value of an ascending table nearest to x >= 0; ties to the
    even index; beyond the last value the last."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    d = (x - values[lo]) - (values[hi] - x)
    up = (d > 0) | ((d == 0) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def swiglu(x):
    gate, up = x.double().chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def quantise(x, fmt, g=1.0):
    """(codes [rows, cols] 0..15, scale bytes [rows, blocks]) of fp64 x."""
    b = x.double().reshape(x.shape[0], -1, BLOCK[fmt])
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    safe = torch.where(bad, torch.ones_like(amax), amax)
    if fmt == "mx":
        e = torch.frexp(safe)[1] - 1  # floor(log2)
        byte = torch.where(safe > 0, (e - 2 + 127).clamp(min=0), torch.zeros_like(e))
        scale = pow2(byte - 127)
        byte = torch.where(bad, 255, byte)
    else:
        table = e4m3_table(x.device)
        # a tensor divisor: on CUDA, division by a number multiplies by its rounded inverse and misses ties
        byte = nearest(table, safe / torch.full_like(safe, 6.0 * g))
        scale = table[byte] * g
        byte = torch.where(bad, 0x7F, byte)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    zero = bad | (scale == 0)
    v = b.abs() / torch.where(zero, torch.ones_like(scale), scale)[..., None]
    code = nearest(grid, torch.nan_to_num(v, nan=0.0, posinf=0.0).clamp(max=6.0)) + 8 * torch.signbit(b).long()
    code = torch.where(zero[..., None], 0, code)
    return code.reshape(x.shape[0], -1), byte


def pack(code):
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)


def pad_scales(byte, cols, fmt):
    out = torch.zeros(byte.shape[0], stride(cols, fmt), dtype=torch.uint8, device=byte.device)
    out[:, :byte.shape[1]] = byte.to(torch.uint8)
    return out


def scale_values(scales, cols, fmt):
    b = scales[..., :cols // BLOCK[fmt]].long()
    if fmt == "mx":
        return torch.where(b == 255, float("nan"), pow2(b - 127))
    table = torch.cat((e4m3_table(b.device), torch.full((1,), float("nan"), device=b.device, dtype=torch.float64)))
    return table[b & 127] * (1.0 - 2.0 * (b >> 7))


def values(codes, scales, fmt, g=1.0):
    """fp64 values of packed codes [..., K/2] and scale bytes [..., S]."""
    K = 2 * codes.shape[-1]
    c = codes.long()
    nib = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=codes.device)[nib]
    return v * scale_values(scales, K, fmt).repeat_interleave(BLOCK[fmt], -1) * g


def grouped(a, b, offsets, ga=1.0, gb=None):
    """(y, s): fp64 product of sorted rows a [R, K] with b [E, N, K], and the
    same sum over magnitudes; zeros outside the groups."""
    y = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
    s = torch.zeros_like(y)
    for e in range(b.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            f = ga * (float(gb[e]) if gb is not None else 1.0)
            y[lo:hi] = a[lo:hi] @ b[e].T * f
            s[lo:hi] = a[lo:hi].abs() @ b[e].abs().T * f
    return y, s
