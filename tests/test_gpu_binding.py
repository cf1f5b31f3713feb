"""The binding of the row and fp4 operators on a device: what is refused, and
that a call on a given stream (checked step by step) and one on the current
stream (the native path) do the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _tensors():
    from bit_quantized_moe_gemv_b200 import _lib as L
    g = torch.Generator().manual_seed(0)
    T, k, H, E, N = 6, 2, 64, 3, 32
    inv = torch.randperm(T * k, generator=g).int().cuda()
    t = {
        "x": torch.randn(T, H, generator=g).bfloat16().cuda(), "inv": inv, "w": torch.rand(T, k, generator=g).cuda(),
        "y": torch.randn(T * k, H, generator=g).bfloat16().cuda(), "ws": L.new_status_workspace(),
        "codes": torch.randint(0, 256, (T, H // 2), dtype=torch.uint8, generator=g).cuda(),
        "scales": torch.full((T, 16), 120, dtype=torch.uint8).cuda(),
        "b": torch.randint(0, 256, (E, N, H // 2), dtype=torch.uint8, generator=g).cuda(),
        "bs": torch.full((E, N, 16), 120, dtype=torch.uint8).cuda(),
        "off": torch.tensor([0, 1, 4, T], dtype=torch.int32).cuda(),
    }
    return L, t, (T, k, H, E, N)


def _calls(L, t, dims, o, **kw):
    T, k, H, E, N = dims
    return {
        "permute": lambda: L.permute(t["x"], t["inv"], o["rows"], t["ws"], **kw),
        "permute_grad": lambda: L.permute_grad(t["y"], t["inv"], o["tokens"], t["ws"], **kw),
        "unpermute": lambda: L.unpermute(t["y"], t["inv"], t["w"], o["tokens2"], t["ws"], **kw),
        "unpermute_grad": lambda: L.unpermute_grad(t["x"], t["y"], t["inv"], t["w"], o["rows2"], o["dw"], t["ws"], **kw),
        "quantize": lambda: L.mxfp_quantize(t["x"], o["codes"], o["scales"], "nv", **kw),
        "dequantize": lambda: L.mxfp_dequantize(t["codes"], t["scales"], o["values"], "mx", **kw),
        "matmul": lambda: L.mxfp_matmul(t["codes"], t["scales"], t["b"], t["bs"], o["out"], "mx", t["ws"], t["off"], **kw),
    }


def _outs(dims):
    T, k, H, E, N = dims
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    return {"rows": z(T * k, H), "tokens": z(T, H), "tokens2": z(T, H), "rows2": z(T * k, H), "dw": z(T, k, d=torch.float32),
            "codes": z(T, H // 2, d=torch.uint8), "scales": z(T, 16, d=torch.uint8), "values": z(T, H), "out": z(T, N)}


def test_a_given_stream_and_the_current_one_do_the_same():
    L, t, dims = _tensors()
    a, b, s = _outs(dims), _outs(dims), torch.cuda.Stream()
    torch.cuda.synchronize()
    before = L.launch_count()
    for f in _calls(L, t, dims, a).values():
        f()
    assert L.launch_count() == before + 7
    for f in _calls(L, t, dims, b, stream=s).values():
        f()
    with torch.cuda.stream(s):
        for f in _calls(L, t, dims, b).values():  # the native path takes the current stream
            f()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]) and a[n].float().abs().sum() > 0, n
    assert L.get_status(t["ws"]) == 0


@pytest.mark.parametrize("broken", ["x", "inv", "w", "y", "ws", "codes", "scales", "b", "bs", "off"])
@pytest.mark.parametrize("how", ["host", "strided", "dtype", "none"])
def test_wrong_tensors_raise_and_launch_nothing(broken, how):
    L, t, dims = _tensors()
    v = t[broken]
    if how == "host":
        t[broken] = v.cpu()
    elif how == "strided":
        t[broken] = torch.stack((v, v), -1)[..., 0]
    elif how == "dtype":
        t[broken] = v.double()
    elif broken == "off":
        return  # no offsets: one group, refused below for E = 3 by the library itself
    else:
        t[broken] = None
    before, calls = L.launch_count(), 0
    used = {"permute": "x inv ws", "permute_grad": "y inv ws", "unpermute": "y inv w ws", "unpermute_grad": "x y inv w ws",
            "quantize": "x", "dequantize": "codes scales", "matmul": "codes scales b bs ws off"}
    for name, f in _calls(L, t, dims, _outs(dims)).items():
        if broken in used[name].split():
            with pytest.raises((ValueError, TypeError, AttributeError)):
                f()
            calls += 1
    assert calls and L.launch_count() == before


def test_the_library_refuses_what_the_shapes_allow():
    L, t, dims = _tensors()
    T, k, H, E, N = dims
    o = _outs(dims)
    with pytest.raises(L.MoeError):  # three groups need offsets
        L.mxfp_matmul(t["codes"], t["scales"], t["b"], t["bs"], o["out"], "mx", t["ws"])
    with pytest.raises(L.MoeError):  # MX has no tensor scale
        L.mxfp_quantize(t["x"], o["codes"], o["scales"], "mx", tensor_scale=torch.ones(1, device="cuda"))
    with pytest.raises(L.MoeError):  # a workspace without room for the status
        L.permute(t["x"], t["inv"], o["rows"], t["ws"][:256])
    with pytest.raises(L.MoeError):  # 48 columns are no whole blocks
        L.mxfp_quantize(torch.zeros(2, 48, device="cuda"), torch.zeros(2, 24, dtype=torch.uint8, device="cuda"),
                        torch.zeros(2, 16, dtype=torch.uint8, device="cuda"), "nv")
