"""The grouped fp4 product against fp64, and the operators together.

Tolerance: products of fp4 values and block scales are exact; a sum of K fp32
additions, rounded or cut, is off by at most K 2^-23 sum|a b|; the tensor scales
take two fp32 roundings and the output type eps/2 of the value.
"""
import pytest
import torch

from tests import mxfp_reference as ref

pytestmark = pytest.mark.gpu


def _matrix(g, rows, K, fmt, lo=None, hi=None):
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, generator=g)
    if lo is None:
        lo, hi = (120, 130) if fmt == "mx" else (1, 0x7F)
    scales = torch.randint(lo, hi, (rows, ref.stride(K, fmt)), dtype=torch.uint8, generator=g)
    scales[:, K // ref.BLOCK[fmt]:] = 255  # behind K: NaN for both formats, to be ignored
    return codes.cuda(), scales.cuda()


def _tol(y, s, K, dtype):
    f = torch.finfo(dtype)
    acc = K * 2.0 ** -23 * s + 3 * 2.0 ** -24 * y.abs()
    return acc + f.eps / 2 * (y.abs() + acc) + f.smallest_normal * f.eps / 2


def _case(sizes, N, K, fmt, dtype, seed=0, lead=0, behind=0, tensor_scales=True):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(seed)
    E, R = len(sizes), lead + sum(sizes) + behind
    a, a_s = _matrix(g, R, K, fmt)
    b, b_s = _matrix(g, E * N, K, fmt)
    b, b_s = b.view(E, N, -1), b_s.view(E, N, -1)
    off = [lead]
    for n in sizes:
        off.append(off[-1] + n)
    ga = gb = None
    if fmt == "nv" and tensor_scales:
        ga, gb = torch.rand(1, generator=g).cuda() + 0.5, torch.rand(E, generator=g).cuda() / 64 + 1e-3
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    ws = L.new_status_workspace()
    L.mxfp_matmul(a, a_s, b, b_s, out, fmt, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                  a_tensor_scale=ga, b_tensor_scale=gb)
    assert L.get_status(ws) == 0
    y, s = ref.grouped(ref.values(a, a_s, fmt), ref.values(b, b_s, fmt), off, float(ga) if ga is not None else 1.0, gb)
    lo, hi = off[0], off[-1]
    err = (out.double() - y).abs()[lo:hi]
    tol = _tol(y, s, K, dtype)[lo:hi]
    big = torch.finfo(dtype).max
    fits = (y.abs() < big / 2)[lo:hi]
    assert (err <= tol)[fits].all(), ((err - tol)[fits].max(), err.max(), y.abs().max())
    assert (out[:lo] == 7).all() and (out[hi:] == 7).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("K", [32, 64, 96, 256, 288, 768, 2080])
def test_one_row(K, fmt):
    _case([1], 128, K, fmt, torch.float32, K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N", [1, 8, 127, 200, 257])
def test_widths_and_output_types(N, dtype, fmt):
    _case([5, 0, 17, 1], N, 320, fmt, dtype, N)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes", [
    [0, 0, 3], [16, 0, 32, 33], [0] * 100 + [1] + [0] * 100, [1] * 300, [31, 1, 64, 97, 2],  # narrow tiles
    [33], [128, 129], [191, 192, 193, 0, 1], [385, 2], [700, 0, 40], [1000],  # wide tiles
], ids=lambda s: f"{len(s)}g{sum(s)}r{max(s)}")
def test_group_sizes(sizes, fmt):
    _case(sizes, 192, 288, fmt, torch.bfloat16, sum(sizes))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("E,rows", [(1024, 1), (1023, 2), (1024, 33), (512, 33), (513, 1)])
def test_as_many_groups_as_there_may_be(E, rows, fmt):
    sizes = [rows] * E
    sizes[0], sizes[E - 1] = 5 * rows, 3 * rows  # the list's ends
    _case(sizes, 72, 96, fmt, torch.float32, E)
    _case([0] * (E - 1) + [40 * rows], 72, 96, fmt, torch.bfloat16, E)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_more_tiles_than_are_listed_at_once(fmt):
    """Over 256 tiles per CTA (128 of narrow ones): the list is written again,
    the rings go on where they were."""
    for rows in (32, 33):  # narrow, wide
        _case([rows], 128 * 38000 + 8, 32, fmt, torch.bfloat16, rows)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("K", [32, 256, 288, 768, 1056, 2080])
@pytest.mark.parametrize("N,dtype", [(2048, torch.bfloat16), (2184, torch.float16), (2307, torch.float32)])
def test_experts_with_none_one_and_many_tiles(N, dtype, K, fmt):
    _case([1, 0, 4700, 40, 0, 161, 320, 129], N, K, fmt, dtype, N + K, lead=3, behind=5)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_before_and_behind_the_groups_are_left(fmt):
    _case([3, 4], 136, 256, fmt, torch.float32, 1, lead=5, behind=70)
    _case([300, 4], 136, 256, fmt, torch.bfloat16, 2, lead=9, behind=33)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_more_tiles_than_processors(fmt):
    _case([900, 0, 1100, 7], 2050, 800, fmt, torch.bfloat16, 3)  # wide, unaligned rows
    _case([9] * 64, 1536, 2048, fmt, torch.bfloat16, 4)  # narrow: 768 tiles of 8 stages


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_dense_without_offsets(fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(8)
    for R in (1, 77, 500):
        a, a_s = _matrix(g, R, 544, fmt)
        b, b_s = _matrix(g, 264, 544, fmt)
        out = torch.empty(R, 264, device="cuda")
        ws = L.new_status_workspace()
        L.mxfp_matmul(a, a_s, b[None], b_s[None], out, fmt, ws)
        y, s = ref.grouped(ref.values(a, a_s, fmt), ref.values(b, b_s, fmt)[None], [0, R])
        assert ((out.double() - y).abs() <= _tol(y, s, 544, torch.float32)).all()
        assert L.get_status(ws) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_scales_over_their_whole_range(fmt):
    """Products from 2^-60 up to 2^60: each output against its own magnitude."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(9)
    K, N, R = 256, 64, 40
    lo, hi = (97, 157) if fmt == "mx" else (1, 0x7F)
    a, a_s = _matrix(g, R, K, fmt, lo, hi)
    b, b_s = _matrix(g, N, K, fmt, lo, hi)
    out = torch.empty(R, N, device="cuda")
    L.mxfp_matmul(a, a_s, b[None], b_s[None], out, fmt, L.new_status_workspace())
    y, s = ref.grouped(ref.values(a, a_s, fmt), ref.values(b, b_s, fmt)[None], [0, R])
    assert ((out.double() - y).abs() <= _tol(y, s, K, torch.float32)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_nan_scale_stays_in_its_row_and_column(fmt):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(10)
    K, N, R = 512, 160, 50
    nan = 255 if fmt == "mx" else 0x7F
    a, a_s = _matrix(g, R, K, fmt)
    b, b_s = _matrix(g, N, K, fmt)
    a_s[3, K // ref.BLOCK[fmt] - 1] = nan
    b_s[131, 2] = nan
    out = torch.empty(R, N, device="cuda")
    L.mxfp_matmul(a, a_s, b[None], b_s[None], out, fmt, L.new_status_workspace())
    want = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    want[3], want[:, 131] = True, True
    assert torch.equal(torch.isnan(out), want)


def test_zero_rows_write_nothing():
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(1)
    a, a_s = _matrix(g, 4, 64, "mx")
    b, b_s = _matrix(g, 3 * 16, 64, "mx")
    b, b_s = b.view(3, 16, 32), b_s.view(3, 16, 16)
    out = torch.full((4, 16), 7.0, device="cuda")
    ws = L.new_status_workspace()
    L.mxfp_matmul(a, a_s, b, b_s, out, "mx", ws, offsets=torch.tensor([2, 2, 2, 2], dtype=torch.int32, device="cuda"))
    L.mxfp_matmul(a[:0], a_s[:0], b, b_s, out[:0], "mx", ws, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (out == 7).all() and L.get_status(ws) == 0


@pytest.mark.parametrize("off", [[0, 3, 2, 4], [-1, 0, 1, 2], [0, 1, 2, 5], [4, 3, 2, 1]])
def test_bad_offsets_are_reported_and_nothing_is_written(off):
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(1)
    a, a_s = _matrix(g, 4, 64, "nv")
    b, b_s = _matrix(g, 3 * 16, 64, "nv")
    out = torch.full((4, 16), 7.0, device="cuda")
    ws = L.new_status_workspace()
    L.mxfp_matmul(a, a_s, b.view(3, 16, 32), b_s.view(3, 16, 16), out, "nv", ws,
                  offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    assert L.get_status(ws) == 5 and (out == 7).all()
    L.reset_status(ws)
    L.mxfp_matmul(a, a_s, b.view(3, 16, 32), b_s.view(3, 16, 16), out, "nv", ws,
                  offsets=torch.tensor([0, 1, 2, 4], dtype=torch.int32, device="cuda"))
    assert L.get_status(ws) == 0 and not (out == 7).all()


def test_graphs_on_two_streams_share_a_workspace():
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(2)
    a, a_s = _matrix(g, 300, 512, "mx", 120, 125)
    b, b_s = _matrix(g, 4 * 256, 512, "mx", 120, 125)
    b, b_s = b.view(4, 256, -1), b_s.view(4, 256, -1)
    off = torch.tensor([0, 7, 7, 250, 300], dtype=torch.int32, device="cuda")
    ws = L.new_status_workspace()
    outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        out, gr = torch.zeros(300, 256, device="cuda"), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr, stream=s):
            L.mxfp_matmul(a, a_s, b, b_s, out, "mx", ws, offsets=off)
        outs.append(out)
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    y, s = ref.grouped(ref.values(a, a_s, "mx"), ref.values(b, b_s, "mx"), off.tolist())
    for out in outs:
        assert ((out.double() - y).abs() <= _tol(y, s, 512, torch.float32)).all()
    assert L.get_status(ws) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 4, 150])
def test_a_layer_of_fp4_experts(T, fmt):
    """route, dispatch, quantise x, permute its codes and scales, gate|up
    product, SwiGLU and quantise, down product, unpermute: each step against
    fp64 on the step's own inputs, and the whole near the unrounded layer."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    H, I, E, k = 256, 192, 16, 4
    g = torch.Generator().manual_seed(T)
    dev = "cuda"
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev)
    ws = L.new_workspace(T, H, I, E, k)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    tsc = (lambda n: torch.full((n,), 0.004, device=dev)) if fmt == "nv" else (lambda n: None)
    gv = 0.004 if fmt == "nv" else 1.0

    def weights(n, kk):
        w = (torch.randn(E * n, kk, generator=g) / kk ** 0.5).to(dev)
        c, s = u8(E * n, kk // 2), u8(E * n, L.mxfp_scale_stride(kk, fmt))
        L.mxfp_quantize(w, c, s, fmt, tensor_scale=tsc(1))
        return w.view(E, n, kk), c.view(E, n, -1), s.view(E, n, -1)

    w1, c1, s1 = weights(2 * I, H)
    w2, c2, s2 = weights(H, I)
    idx, gates = i32(T, k), torch.empty(T, k, device=dev)
    w_r = torch.randn(E, H, generator=g).to(dev)
    L.route(x, w_r, None, 0, k, idx, gates, ws)
    counts, off, perm, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    L.dispatch(idx, E, counts, off, perm, inv, ws)
    xc, xs = u8(T, H // 2), u8(T, L.mxfp_scale_stride(H, fmt))
    L.mxfp_quantize(x, xc, xs, fmt, tensor_scale=tsc(1))
    pc, ps = u8(T * k, H // 2), u8(T * k, xs.shape[1])
    L.permute(xc, inv, pc, ws)
    L.permute(xs, inv, ps, ws)
    gu = torch.empty(T * k, 2 * I, dtype=torch.bfloat16, device=dev)
    L.mxfp_matmul(pc, ps, c1, s1, gu, fmt, ws, offsets=off, a_tensor_scale=tsc(1), b_tensor_scale=tsc(E))
    hc, hs = u8(T * k, I // 2), u8(T * k, L.mxfp_scale_stride(I, fmt))
    L.mxfp_quantize(gu, hc, hs, fmt, tensor_scale=tsc(1), swiglu=True, rows_dev=off[E:])
    y = torch.empty(T * k, H, dtype=torch.bfloat16, device=dev)
    L.mxfp_matmul(hc, hs, c2, s2, y, fmt, ws, offsets=off, a_tensor_scale=tsc(1), b_tensor_scale=tsc(E))
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    L.unpermute(y, inv, gates, out, ws)
    torch.cuda.synchronize()
    assert L.get_status(ws) == 0

    o = off.tolist()
    assert o[-1] == T * k
    rows = perm.long() // k
    assert torch.equal(pc, xc[rows]) and torch.equal(ps, xs[rows])
    gb = [gv] * E
    v1 = ref.values(c1, s1, fmt)
    r, s = ref.grouped(ref.values(pc, ps, fmt), v1, o, float(torch.tensor(gv)), [float(torch.tensor(gv))] * E)
    assert ((gu.double() - r).abs() <= _tol(r, s, H, torch.bfloat16)).all()
    want_c, want_s = ref.quantise(ref.swiglu(gu), fmt, float(torch.tensor(gv)))
    assert torch.equal(hc, ref.pack(want_c)) and torch.equal(hs, ref.pad_scales(want_s, I, fmt))
    r, s = ref.grouped(ref.values(hc, hs, fmt), ref.values(c2, s2, fmt), o, float(torch.tensor(gv)),
                       [float(torch.tensor(gv))] * E)
    assert ((y.double() - r).abs() <= _tol(r, s, I, torch.bfloat16)).all()
    terms = gates.double()[..., None] * y.double()[inv.view(T, k).long()]
    tol = torch.finfo(torch.bfloat16).eps / 2 * (1 + 2.0 ** -10) * terms.sum(1).abs() + (k + 1) * 2.0 ** -24 * terms.abs().sum(1)
    assert ((out.double() - terms.sum(1)).abs() <= tol).all()

    # the whole layer without fp4: four 4-bit roundings (x, w1, h, w2), each at
    # most half a step of 1/3 of the value (5 -> 6), 1/6 relative, plus small
    # values lost in their block; that it is the same layer, not how exact, is asked
    ex = torch.zeros(T, H, dtype=torch.float64, device=dev)
    for j in range(k):
        e = idx[:, j].long()
        h = ref.swiglu(torch.einsum("th,tnh->tn", x.double(), w1[e].double()))
        ex += gates[:, j, None].double() * torch.einsum("ti,thi->th", h, w2[e].double())
    cos = (ex * out.double()).sum() / ex.norm() / out.double().norm()
    assert cos > 0.9
