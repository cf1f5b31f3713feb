"""The row and fp4 operators one after another on a stream, where a call's
kernel is launched while its predecessor still runs: every call sees what came
before it, whoever wrote it, and nobody reads what it has yet to write."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 64), (40, 64), (600, 96), (2000, 1030)])
def test_two_buffers_written_in_turn(T, H, dtype):
    """x -> xp -> x -> ..., each step another permutation of all rows."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(T)
    there, back = (torch.randperm(T, generator=g).int().cuda() for _ in range(2))
    ones, ws = torch.ones(T, 1, device="cuda"), L.new_status_workspace()
    x = torch.randn(T, H, generator=g).to(dtype).cuda()
    xp, want, step = torch.empty_like(x), x.clone(), torch.empty(T, dtype=torch.long, device="cuda")
    step[there.long()] = torch.arange(T, device="cuda")  # xp[r] = x[step[r]], then x[t] = xp[back[t]]
    step = step[back.long()]
    at = torch.arange(T, device="cuda")
    torch.cuda.synchronize()
    for i in range(300):
        L.permute(x, there, xp, ws)
        if i % 2:
            L.permute_grad(xp, back, x, ws)
        else:
            L.unpermute(xp, back, ones, x, ws)
        at = at if i % 60 else at.clone()  # another library's kernel in between, now and then
    for _ in range(300):
        want = want[step]
    assert torch.equal(x, want) and L.get_status(ws) == 0


def _layer(fmt, T, k=4, E=8, H=256, D=128):
    """Buffers of one layer of fp4 experts and a function that runs it on them."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(7)
    z = lambda *s, d=torch.uint8: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    S = lambda n: L.mxfp_scale_stride(n, fmt)  # noqa: E731
    w = {}
    for n, rows, cols in (("up", 2 * D, H), ("down", H, D)):
        w[n] = z(E, rows, cols // 2), z(E, rows, S(cols))
        L.mxfp_quantize((torch.randn(E * rows, cols, generator=g) / cols ** 0.5).cuda(), w[n][0].view(E * rows, -1),
                        w[n][1].view(E * rows, -1), fmt)
    R, bf = T * k, torch.bfloat16
    o = {"x": z(T, H, d=bf), "w": z(T, k, d=torch.float32), "idx": z(T, k, d=torch.int32), "out": z(T, H, d=bf),
         "c": z(T, H // 2), "s": z(T, S(H)), "pc": z(R, H // 2), "ps": z(R, S(H)), "gu": z(R, 2 * D, d=bf),
         "hc": z(R, D // 2), "hs": z(R, S(D)), "y": z(R, H, d=bf), "dy": z(R, H, d=bf), "dw": z(T, k, d=torch.float32),
         "counts": z(E, d=torch.int32), "off": z(E + 1, d=torch.int32), "perm": z(R, d=torch.int32),
         "inv": z(R, d=torch.int32), "v": z(R, D, d=bf)}
    dws, ws = L.new_workspace(T, 64, 64, E, k), L.new_status_workspace()

    def run(after=lambda: None, status=ws):
        steps = (
            lambda: L.reset_status(status),
            lambda: L.dispatch(o["idx"], E, o["counts"], o["off"], o["perm"], o["inv"], dws),
            lambda: L.mxfp_quantize(o["x"], o["c"], o["s"], fmt),
            lambda: L.permute(o["c"], o["inv"], o["pc"], status),
            lambda: L.permute(o["s"], o["inv"], o["ps"], status),
            lambda: L.mxfp_matmul(o["pc"], o["ps"], *w["up"], o["gu"], fmt, status, offsets=o["off"]),
            lambda: L.mxfp_quantize(o["gu"], o["hc"], o["hs"], fmt, swiglu=True, rows_dev=o["off"][E:]),
            lambda: L.mxfp_matmul(o["hc"], o["hs"], *w["down"], o["y"], fmt, status, offsets=o["off"]),
            lambda: L.unpermute(o["y"], o["inv"], o["w"], o["out"], status),
            lambda: L.unpermute_grad(o["out"], o["y"], o["inv"], o["w"], o["dy"], o["dw"], status),
            lambda: L.mxfp_dequantize(o["hc"], o["hs"], o["v"], fmt, rows_dev=o["off"][E:]),
        )
        for f in steps:
            f()
            after()

    def fill(seed):
        h = torch.Generator("cuda").manual_seed(seed)
        o["x"].normal_(generator=h)
        o["w"].uniform_(generator=h)
        o["idx"].copy_(torch.rand(T, E, generator=h, device="cuda").argsort(1)[:, :k])

    return o, run, fill, ws, ("out", "dy", "dw", "v")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 30, 400])
def test_layer_after_layer_with_new_inputs(T, fmt):
    """Layers on the same buffers, filled by torch in between, against the same
    layers with every call waited for."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    o, run, fill, ws, outs = _layer(fmt, T)
    want, got = [], []
    for after, res in ((torch.cuda.synchronize, want), (lambda: None, got)):
        for seed in range(12):
            fill(seed)
            run(after)
            res.append([o[n].clone() for n in outs])
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert want[0][0].float().abs().sum() > 0 and L.get_status(ws) == 0


def test_captured_with_a_fork_and_a_memset():
    """A graph whose chained calls follow a memset, a copy, and a join of two streams."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    parts = [_layer("mx", 30), _layer("nv", 30)]
    both = torch.zeros(30, 256, dtype=torch.bfloat16, device="cuda")
    inv, ws = torch.randperm(30).int().cuda(), L.new_status_workspace()
    sums = [torch.zeros_like(both) for _ in range(2)]

    def step(fork):
        s = torch.cuda.current_stream()
        if fork:
            side = torch.cuda.Stream()
            side.wait_stream(s)
            with torch.cuda.stream(side):
                parts[0][1]()
            parts[1][1]()
            s.wait_stream(side)
        else:
            parts[0][1](torch.cuda.synchronize)
            parts[1][1](torch.cuda.synchronize)
        for p, t in zip(parts, sums):  # the first follows the join
            L.permute(p[0]["out"], inv, t, ws)
        both.copy_(sums[0])
        L.permute(both, inv, sums[1], ws)

    want = []
    for seed in range(4):
        for p in parts:
            p[2](seed)
        step(False)
        want.append([sums[0].clone(), sums[1].clone(), parts[0][0]["dw"].clone(), parts[1][0]["dw"].clone()])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(True)
    for seed in range(4):
        for p in parts:
            p[2](seed)
        g.replay()
        got = [sums[0], sums[1], parts[0][0]["dw"], parts[1][0]["dw"]]
        assert all(torch.equal(a, b) for a, b in zip(want[seed], got))
    assert all(L.get_status(p[3]) == 0 for p in parts) and L.get_status(ws) == 0


def test_calls_on_two_streams_at_once():
    """Narrow and wide products, sums and conversions on two streams that share
    a status workspace, call after call: the same results as one after another."""
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator("cuda").manual_seed(4)
    E, N, K, T, k = 24, 512, 512, 60, 4
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    b, b_s = u8(E, N, K // 2), torch.full((E, N, 16), 120, dtype=torch.uint8, device="cuda")
    inv = torch.randperm(T * k, generator=g, device="cuda").int()
    w, ws = torch.rand(T, k, generator=g, device="cuda"), L.new_status_workspace()
    kinds = ("narrow", "wide")  # 240 rows of 24 experts, of one
    offs = torch.arange(E + 1, dtype=torch.int32, device="cuda") * (T * k // E)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()

    def chain(kind, o):
        L.mxfp_quantize(x, o["c"], o["s"], "mx")
        L.permute(o["c"], inv, o["pc"], ws)
        L.permute(o["s"], inv, o["ps"], ws)
        if kind == "narrow":
            L.mxfp_matmul(o["pc"], o["ps"], b, b_s, o["y"], "mx", ws, offsets=offs)
        else:
            L.mxfp_matmul(o["pc"], o["ps"], b[:1], b_s[:1], o["y"], "mx", ws)
        L.unpermute(o["y"], inv, w, o["out"], ws)

    def buffers():
        z = lambda *s, d=torch.uint8: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        return {"c": z(T, K // 2), "s": z(T, 16), "pc": z(T * k, K // 2), "ps": z(T * k, 16),
                "y": z(T * k, N, d=torch.bfloat16), "out": z(T, N, d=torch.bfloat16)}

    want = {}
    for kind in kinds:
        o = buffers()
        chain(kind, o)
        torch.cuda.synchronize()
        want[kind] = o["out"]
    streams = {kind: torch.cuda.Stream() for kind in kinds}
    got = {kind: [buffers() for _ in range(4)] for kind in kinds}
    torch.cuda.synchronize()
    for i in range(40):
        for kind, s in streams.items():
            with torch.cuda.stream(s):
                chain(kind, got[kind][i % 4])
    torch.cuda.synchronize()
    for kind in kinds:
        for o in got[kind]:
            assert torch.equal(o["out"], want[kind]) and want[kind].float().abs().sum() > 0
    assert L.get_status(ws) == 0
