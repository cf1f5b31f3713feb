"""Rows sorted by expert and back, with their gradients, against plain fp64
indexing; inv_perm comes from moe_dispatch.

Tolerances: a sum of n fp32 terms in any order is off by at most n u sum|terms|
(u = 2^-24), the rounding to the output type by eps/2 of the value, and by half
the smallest subnormal below the normal range.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _half(dtype, v):
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps / 2


def _routing(T, k, E, seed, drop=0.0):
    """(idx [T, k] with -1 for dropped tokens, inv_perm of moe_dispatch, ws)."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].int()
    idx[torch.rand(T, generator=g) < drop] = -1
    idx = idx.cuda()
    counts, offsets = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm, inv = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    L.dispatch(idx, E, counts, offsets, perm, inv, L.new_workspace(T, 64, 64, E, k))
    return idx, inv, L.new_status_workspace()


def _rand(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


SHAPES = [(1, 2048, 10, 512, 0.0), (4, 2048, 10, 64, 0.3), (3, 1, 1, 2, 0.0), (5, 7, 3, 8, 0.4), (130, 1030, 6, 16, 0.2),
          (67, 333, 5, 9, 0.0), (300, 128, 40, 64, 0.1), (2, 20000, 2, 4, 0.0), (1500, 64, 2, 4, 1.0)]


@pytest.mark.parametrize("dtype", DTYPES + [torch.uint8])
@pytest.mark.parametrize("T,H,k,E,drop", SHAPES)
def test_permute_moves_rows_and_leaves_the_others(T, H, k, E, drop, dtype):
    from bit_quantized_moe_gemv_b200 import _lib as L
    idx, inv, ws = _routing(T, k, E, T + H, drop)
    x = (torch.randint(0, 256, (T, H), dtype=torch.uint8).cuda() if dtype == torch.uint8
         else _rand(T, H, dtype=dtype, seed=1))
    xp = torch.full((T * k, H), 7, dtype=dtype, device="cuda")
    want = xp.clone()
    L.permute(x, inv, xp, ws)
    p = torch.nonzero(inv >= 0).reshape(-1)
    want[inv[p].long()] = x[p // k]
    assert torch.equal(xp, want)
    # rows are in expert order, tokens ascending inside an expert
    e = idx.reshape(-1)[p]
    order = torch.argsort(e.long() * (T * k) + p)
    assert torch.equal(inv[p[order]].long(), torch.arange(p.numel(), device="cuda"))
    assert L.get_status(ws) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,k,E,drop", SHAPES)
def test_sums_back_to_tokens(T, H, k, E, drop, dtype):
    from bit_quantized_moe_gemv_b200 import _lib as L
    _, inv, ws = _routing(T, k, E, T + H, drop)
    y, w = _rand(T * k, H, dtype=dtype, seed=2), _rand(T, k, dtype=torch.float32, seed=3)
    # rows no pair points to hold NaN: they must not be read
    y[torch.isin(torch.arange(T * k, device="cuda"), inv, invert=True)] = float("nan")
    at = inv.view(T, k).long()
    rows = torch.where((at >= 0)[..., None], y.double()[at.clamp(min=0)], 0.0)
    for weights in (None, w):
        got = torch.full((T, H), 7, dtype=dtype, device="cuda")
        if weights is None:
            L.permute_grad(y, inv, got, ws)
            terms = rows
        else:
            L.unpermute(y, inv, w, got, ws)
            terms = rows * w.double()[..., None]
        ref, mag = terms.sum(1), terms.abs().sum(1)
        err = (got.double() - ref).abs()
        assert (err <= _half(dtype, ref) * (1 + 2.0 ** -10) + (k + 1) * U * mag).all(), (weights is None, err.max())
    assert L.get_status(ws) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,k,E,drop", SHAPES)
def test_unpermute_gradient(T, H, k, E, drop, dtype):
    from bit_quantized_moe_gemv_b200 import _lib as L
    _, inv, ws = _routing(T, k, E, T + H, drop)
    y, w, d = (_rand(T * k, H, dtype=dtype, seed=2), _rand(T, k, dtype=torch.float32, seed=3),
               _rand(T, H, dtype=dtype, seed=4))
    unused = torch.isin(torch.arange(T * k, device="cuda"), inv, invert=True)
    y[unused] = float("nan")
    dy, dw = torch.full((T * k, H), 7, dtype=dtype, device="cuda"), torch.full((T, k), 7.0, device="cuda")
    L.unpermute_grad(d, y, inv, w, dy, dw, ws)
    at = inv.view(T, k).long()
    has = at >= 0
    terms = torch.where(has[..., None], y.double()[at.clamp(min=0)], 0.0) * d.double()[:, None]
    assert ((dw.double() - terms.sum(2)).abs() <= H * U * terms.abs().sum(2)).all()
    assert (dw[~has] == 0).all()
    ref = (w.double()[..., None] * d.double()[:, None]).reshape(T * k, H)
    p = torch.nonzero(inv >= 0).reshape(-1)
    got = dy[inv[p].long()].double()
    assert ((got - ref[p]).abs() <= _half(dtype, ref[p]) * (1 + 2.0 ** -10) + U * ref[p].abs()).all()
    assert (dy[unused] == 7).all()
    assert L.get_status(ws) == 0


def test_gradients_agree_with_differences():
    """out is linear in y and in w, so a difference over any step is the
    directional derivative up to rounding; the same for permute and its sum."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, H, k, E = 37, 96, 5, 8
    _, inv, ws = _routing(T, k, E, 5, 0.2)
    f = torch.float32
    y, w, d = _rand(T * k, H, dtype=f, seed=2), _rand(T, k, dtype=f, seed=3), _rand(T, H, dtype=f, seed=4)
    dy, dw = torch.zeros(T * k, H, device="cuda"), torch.zeros(T, k, device="cuda")
    L.unpermute_grad(d, y, inv, w, dy, dw, ws)

    def loss(y, w):
        out = torch.empty(T, H, device="cuda")
        L.unpermute(y, inv, w, out, ws)
        return (out.double() * d.double()).sum()

    ey, ew = _rand(T * k, H, dtype=f, seed=6), _rand(T, k, dtype=f, seed=7)
    y2, w2 = y + ey, w + ew
    at = inv.view(T, k).long().clamp(min=0)
    # every loss sums T*k*H products, each off by (k + 1) u of its size; the gradients by H u
    big = sum((v.double().abs()[..., None] * z.double()[at].abs() * d.double()[:, None].abs()).sum()
              for z, v in ((y, w), (y2, w), (y, w2)))
    tol = (k + 1 + H) * U * big
    dyd = (dy.double() * (y2.double() - y.double()))[inv[inv >= 0].long()].sum()
    assert abs(loss(y2, w) - loss(y, w) - dyd) <= tol
    assert abs(loss(y, w2) - loss(y, w) - (dw.double() * (w2.double() - w.double())).sum()) <= tol
    # <permute(x), g> = <x, permute_grad(g)>
    x, g = _rand(T, H, dtype=f, seed=8), _rand(T * k, H, dtype=f, seed=9)
    xp, dx = torch.zeros(T * k, H, device="cuda"), torch.empty(T, H, device="cuda")
    L.permute(x, inv, xp, ws)
    L.permute_grad(g, inv, dx, ws)
    lhs, rhs = (xp.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(lhs - rhs) <= k * U * (xp.double() * g.double()).abs().sum()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_rows_at_odd_addresses(off):
    """Slices that start off a 16-byte boundary."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, H, k, E = 9, 40, 3, 8
    _, inv, ws = _routing(T, k, E, 1)

    def at(n, m, fill):
        flat = torch.full((n * m + off,), fill, dtype=torch.bfloat16, device="cuda")
        return flat, flat[off:].view(n, m)

    x, y, w = _rand(T, H, dtype=torch.bfloat16, seed=1), _rand(T * k, H, dtype=torch.bfloat16, seed=2), None
    w = _rand(T, k, dtype=torch.float32, seed=3)
    _, x1 = at(T, H, 0)
    x1.copy_(x)
    f, xp1 = at(T * k, H, 5)
    xp = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    L.permute(x, inv, xp, ws)
    L.permute(x1, inv, xp1, ws)
    assert torch.equal(xp, xp1) and (f[:off] == 5).all()
    o, (f, o1) = torch.empty_like(x), at(T, H, 5)
    L.unpermute(y, inv, w, o, ws)
    L.unpermute(y, inv, w, o1, ws)
    assert torch.equal(o, o1) and (f[:off] == 5).all()
    dy, (_, dy1) = torch.empty_like(y), at(T * k, H, 5)
    dw, dw1 = torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")
    L.unpermute_grad(x, y, inv, w, dy, dw, ws)
    L.unpermute_grad(x1, y, inv, w, dy1, dw1, ws)
    assert torch.equal(dy, dy1)
    # another vector width sums in another order
    assert ((dw - dw1).abs() <= 2 * H * U * (x.float()[:, None] * y.float()[inv.view(T, k).long()]).abs().sum(2)).all()


def test_rows_outside_the_range_are_reported_and_left_out():
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, H, k = 4, 64, 2
    inv = torch.tensor([0, 1, 2, 8, 4, -2, 6, 7], dtype=torch.int32, device="cuda")  # 8 rows: 0..7
    x, y = torch.ones(T, H, device="cuda"), torch.ones(T * k, H, device="cuda")
    w, out, dw = torch.ones(T, k, device="cuda"), torch.zeros(T, H, device="cuda"), torch.full((T, k), 9.0, device="cuda")
    for call in (lambda ws: L.permute(x, inv, torch.zeros_like(y), ws), lambda ws: L.permute_grad(y, inv, out, ws),
                 lambda ws: L.unpermute(y, inv, w, out, ws),
                 lambda ws: L.unpermute_grad(x, y, inv, w, torch.zeros_like(y), dw, ws)):
        ws = L.new_status_workspace()
        call(ws)
        assert L.get_status(ws) == 5  # MOE_ERR_DEVICE_FAULT
    assert out[:, 0].tolist() == [2, 1, 1, 2]
    assert dw.tolist() == [[H, H], [H, 0], [H, 0], [H, H]]


def test_overlapping_calls_and_captured_graphs_share_a_status_workspace():
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, H, k, E = 64, 512, 4, 16
    _, inv, ws = _routing(T, k, E, 3)
    x, w = _rand(T, H, dtype=torch.bfloat16, seed=1), _rand(T, k, dtype=torch.float32, seed=3)
    outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        xp = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
        o = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        dy, dw = torch.zeros_like(xp), torch.zeros(T, k, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            L.permute(x, inv, xp, ws)
            L.unpermute(xp, inv, w, o, ws)
            L.unpermute_grad(x, xp, inv, w, dy, dw, ws)
        outs.append((xp, o, dy, dw))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    ref = (x.double() * w.double().sum(1, keepdim=True))
    mag = x.double().abs() * w.double().abs().sum(1, keepdim=True)
    assert ((outs[0][1].double() - ref).abs() <= _half(torch.bfloat16, ref) * (1 + 2.0 ** -10) + (k + 1) * U * mag).all()
    assert L.get_status(ws) == 0


def test_pairs_that_share_a_row():
    """All of them read it; what lands in it is one of theirs."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, H, k = 6, 72, 3
    inv = torch.tensor([0, 0, 1, 2, 3, 3, 0, 4, 5, 6, 6, 6, 7, 8, 2, -1, 17, 17], dtype=torch.int32, device="cuda")
    f, ws = torch.float32, L.new_status_workspace()
    x, y, w = _rand(T, H, dtype=f, seed=1), _rand(T * k, H, dtype=f, seed=2), _rand(T, k, dtype=f, seed=3)
    at, has = inv.view(T, k).long().clamp(min=0), (inv.view(T, k) >= 0)[..., None]
    terms = torch.where(has, y.double()[at], 0.0)
    out, dy, dw, xp = torch.empty_like(x), torch.zeros_like(y), torch.empty_like(w), torch.zeros_like(y)
    L.permute_grad(y, inv, out, ws)
    assert ((out.double() - terms.sum(1)).abs() <= (k + 1) * U * terms.abs().sum(1)).all()
    L.unpermute(y, inv, w, out, ws)
    v = terms * w.double()[..., None]
    assert ((out.double() - v.sum(1)).abs() <= (k + 1) * U * v.abs().sum(1)).all()
    L.unpermute_grad(x, y, inv, w, dy, dw, ws)
    v = terms * x.double()[:, None]
    assert ((dw.double() - v.sum(2)).abs() <= H * U * v.abs().sum(2)).all()
    L.permute(x, inv, xp, ws)
    for r in range(T * k):
        p = torch.nonzero(inv == r).reshape(-1)
        if p.numel() == 0:
            assert (xp[r] == 0).all() and (dy[r] == 0).all()
        else:
            assert (xp[r] == x[p // k]).any(0).all() and (dy[r] == w.view(-1)[p][:, None] * x[p // k]).any(0).all()
    assert L.get_status(ws) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 31, 127, 128, 129, 192, 193, 256, 260, 516, 1032, 1544])
def test_rows_of_every_number_of_segments(H, dtype):
    """One to many segments of a warp, powers of two and not, at tokens that end inside a block."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, k, E = 203, 3, 16
    _, inv, ws = _routing(T, k, E, H, 0.2)
    x, y, w = _rand(T, H, dtype=dtype, seed=1), _rand(T * k, H, dtype=dtype, seed=2), _rand(T, k, dtype=torch.float32, seed=3)
    at, has = inv.view(T, k).long().clamp(min=0), (inv.view(T, k) >= 0)[..., None]
    xp = torch.full((T * k, H), 7, dtype=dtype, device="cuda")
    want = xp.clone()
    p = torch.nonzero(inv >= 0).reshape(-1)
    want[inv[p].long()] = x[p // k]
    L.permute(x, inv, xp, ws)
    assert torch.equal(xp, want)
    terms = torch.where(has, y.double()[at] * w.double()[..., None], 0.0)
    out = torch.full((T, H), 7, dtype=dtype, device="cuda")
    L.unpermute(y, inv, w, out, ws)
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert ((out.double() - ref).abs() <= _half(dtype, ref) * (1 + 2.0 ** -10) + (k + 1) * U * mag).all()
    assert L.get_status(ws) == 0


@pytest.mark.parametrize("dtype", DTYPES + [torch.uint8])
@pytest.mark.parametrize("H", [1028, 2056, 2568, 4104])
def test_permute_with_and_without_surplus_warps(H, dtype):
    """Numbers of segments that are rounded up to a power of two, and that are too far from one."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    T, k, E = 203, 3, 16
    _, inv, ws = _routing(T, k, E, H, 0.2)
    x = (torch.randint(0, 256, (T, H), dtype=torch.uint8).cuda() if dtype == torch.uint8
         else _rand(T, H, dtype=dtype, seed=1))
    xp = torch.full((T * k, H), 7, dtype=dtype, device="cuda")
    want, p = xp.clone(), torch.nonzero(inv >= 0).reshape(-1)
    want[inv[p].long()] = x[p // k]
    L.permute(x, inv, xp, ws)
    assert torch.equal(xp, want) and L.get_status(ws) == 0
