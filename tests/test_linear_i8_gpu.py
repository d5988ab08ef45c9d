"""The channel products in 8-bit integers and their 8-bit form against the formulas in fp64.

Tolerances are sums of the roundings that each result passes (u the unit roundoff of the output's type, v = 2^-24 fp32's):
the form's scale one, the product four of fp32 (the sum's conversion, two scales, the bias) and the output's; the gradients
one of the data type a term (the 8-bit operand times its scale), fp32's of the sum (n v of the terms' sizes) and the output's.
An activation function is evaluated within ACT of its argument's size: the normal tail by its rational form is off by
0.75e-7, its exponential, reciprocal and the products by 6 v of at most 1/2, and two products follow; a slope is a sum of
two such terms, v phi(v) <= 1/4 among them."""
import pytest
import torch

import sparse_gather_contraction_amd as sgc

pytestmark = pytest.mark.gpu

V = 2.0 ** -24
ACT = 0.75e-7 + 6 * V / 2 + 2 * V
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}  # half a step of the type's subnormals (others: far below the data)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def u_of(name):
    return torch.finfo(DT[name]).eps / 2


def shape_of(points, channels):
    return (points[0], channels) + tuple(points[1:])


def normal(points, channels, dt, seed, std=1.0):
    return (torch.randn(shape_of(points, channels), generator=gen(seed), device="cuda") * std).to(DT[dt])


def rows(t):
    return t.double().movedim(1, -1).reshape(-1, t.shape[1])


def act64(x, act):
    return x if act is None else x * torch.special.ndtr(x) if act == "gelu" else x * torch.sigmoid(x)


def slope64(x, act):
    if act == "gelu":
        return torch.special.ndtr(x) + x * torch.exp(-x * x / 2) / (2 * torch.pi) ** 0.5
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def form(points, channels, seed, std=1.0):
    """A form made here, apart from the library: (q, scale, values as rows in fp64)."""
    n = 1
    for p in points:
        n *= p
    x = torch.randn((n, channels), generator=gen(seed), device="cuda") * std
    scale = (x.abs().amax(1) / 127).clamp(min=2.0 ** -126)
    q = torch.zeros((n, -(-channels // 16) * 16), dtype=torch.int8, device="cuda")
    q[:, :channels] = torch.round(x / scale[:, None])
    return q.reshape(tuple(points) + (-1,)), scale.reshape(points), q[:, :channels].double() * scale.double()[:, None]


POINTS = [(1,), (17,), (64,), (300,), (1, 5, 7), (3, 9, 13), (2, 1, 1), (5, 1, 3), (1, 16, 64), (2, 91, 181)]
CHANNELS = [1, 16, 33, 80, 256, 600]


def check_form(q, scale, x, v, err, act, exact32=None):
    """q, scale: the form of v (rows, fp64), of values that may be off by err."""
    P, C = v.shape
    assert q.dtype == torch.int8 and q.shape[-1] == -(-C // 16) * 16 and q.shape[:-1] == scale.shape
    codes, s = q.reshape(P, -1).double(), scale.reshape(P).double()
    assert bool((codes[:, C:] == 0).all()) and float(codes.abs().max()) <= 127
    want = (v.abs().amax(1) / 127).clamp(min=2.0 ** -126)
    assert bool(((s - want).abs() <= err.amax(1) / 127 + V * want * 1.01).all())
    # a quotient is off by 127 v and is rounded to the nearest whole number
    assert bool(((codes[:, :C] * s[:, None] - v).abs() <= s[:, None] * (0.5 + 128 * V) + err).all())
    if exact32 is not None:
        s32 = (exact32.abs().amax(1) / 127).clamp(min=2.0 ** -126)
        assert torch.equal(scale.reshape(P).cpu(), s32)
        assert torch.equal(codes[:, :C].cpu(), torch.round(exact32 / s32[:, None]).double())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("points", POINTS, ids=str)
def test_quantize(points, dt):
    for C in CHANNELS:
        x = normal(points, C, dt, C, 3.0)
        q, s = sgc.disco_quantize_i8(x)
        v = rows(x)
        check_form(q, s, x, v, torch.zeros_like(v), None, v.float().cpu())
        for act in ("gelu", "silu"):
            q, s, k, ks = sgc.disco_quantize_i8(x, act=act, keep=True)
            check_form(q, s, x, act64(v, act), v.abs() * (ACT if act == "gelu" else 6 * V), act)
            check_form(k, ks, x, v, torch.zeros_like(v), None, v.float().cpu())
            q2, s2 = sgc.disco_quantize_i8(x, act=act)
            assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("points", POINTS, ids=str)
def test_dequantize(points, dt):
    for C in CHANNELS:
        q, s, v = form(points, C, C + 1)
        out = sgc.disco_dequantize_i8(q, s, channels=C, dtype=DT[dt])
        assert out.shape == shape_of(points, C) and out.dtype == DT[dt]
        want = (q.float() * s.unsqueeze(-1)).reshape(-1, q.shape[-1])[:, :C].to(DT[dt])  # one rounding to fp32, one to dt
        assert torch.equal(rows(out), want.double())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(3, 2100, 4, 70), (2, 5000, 3, 5), (4, 40000), (1, 1 << 20)], ids=str)
def test_long_axes(shape, dt):
    # channels beyond what a workgroup's registers or its LDS hold
    x = (torch.randn(shape, generator=gen(5), device="cuda") * 2).to(DT[dt])
    v = rows(x)
    q, s = sgc.disco_quantize_i8(x)
    check_form(q, s, x, v, torch.zeros_like(v), None, v.float().cpu())
    q, s, k, ks = sgc.disco_quantize_i8(x, act="silu", keep=True)
    check_form(q, s, x, act64(v, "silu"), v.abs() * 6 * V, "silu")
    check_form(k, ks, x, v, torch.zeros_like(v), None, v.float().cpu())
    out = sgc.disco_dequantize_i8(k, ks, channels=shape[1], dtype=DT[dt])
    assert torch.equal(rows(out), (k.float() * ks.unsqueeze(-1)).reshape(-1, k.shape[-1])[:, :shape[1]].to(DT[dt]).double())


def test_axes_and_dimensions():
    x = torch.randn((3, 4, 5, 6, 7), generator=gen(1), device="cuda")
    for axis in range(-5, 5):
        q, s = sgc.disco_quantize_i8(x, axis=axis)
        lead = [n for i, n in enumerate(x.shape) if i != axis % 5]
        assert list(s.shape) == lead and list(q.shape) == lead + [16]
        back = sgc.disco_dequantize_i8(q, s, channels=x.shape[axis], dtype=torch.float32, axis=axis)
        assert back.shape == x.shape and bool(((back - x).abs() <= 0.51 * s.unsqueeze(axis)).all())
    q, s = sgc.disco_quantize_i8(x[0, 0, 0, 0], axis=0)
    assert q.shape == (16,) and s.shape == ()


def test_rows_of_nothing_extremes_and_what_is_not_finite():
    x = torch.randn((40, 200), generator=gen(2), device="cuda")
    x[0] = 0
    x[1] = 1e-42                       # subnormal
    x[2, 3], x[3, 199], x[4, 0] = float("nan"), float("inf"), float("-inf")
    x[5] = 3.4e38
    x[6] = torch.finfo(torch.float32).tiny
    x[7] = torch.nan_to_num(x[7], nan=0.0)
    bits = torch.full((200,), 0x7fc000ab, dtype=torch.int32, device="cuda").view(torch.float32)
    x[8] = bits                        # NaNs whose low bits are set
    for y in (x, x.t().contiguous().view(1, 200, 40, 1).movedim(2, 0).contiguous().view(40, 200, 1, 1), x.t().reshape(1, 200, 5, 8).contiguous()):
        q, s = sgc.disco_quantize_i8(y)
        q, s = q.reshape(40, -1), s.reshape(40)
        bad = torch.tensor([i in (2, 3, 4, 8) for i in range(40)], device="cuda")
        assert torch.equal(torch.isnan(s), bad) and bool((q[bad] == 0).all())
        assert float(s[0]) == 2.0 ** -126 and bool((q[0] == 0).all()) and float(s[1]) == 2.0 ** -126 and bool((q[1] == 0).all())
        assert bool((q[5, :200] == 127).all()) and float(s[5]) == float(torch.tensor(3.4e38) / 127)
        # the smallest scale is 2^-126: values of it are the code 1
        assert float(s[6]) == 2.0 ** -126 and bool((q[6, :200] == 1).all())
        ok = ~bad
        ok[:9] = False
        assert bool(((q[ok][:, :200].float() * s[ok][:, None] - x[ok]).abs() <= 0.501 * s[ok][:, None]).all())
    for act in ("gelu", "silu"):
        q, s, k, ks = sgc.disco_quantize_i8(x, act=act, keep=True)
        assert torch.equal(torch.isnan(s), bad) and torch.equal(torch.isnan(ks), bad)
        assert bool((q[5, :200] == 127).all())


# ---------------------------------------------------------------- the product

PRODUCTS = [((1,), 1, 1), ((1,), 512, 2048), ((5,), 16, 3), ((16,), 1000, 70), ((17,), 33, 65), ((33,), 2064, 31), ((64,), 64, 256), ((65,), 80, 73),
            ((129,), 128, 257), ((300,), 272, 130), ((1000,), 48, 300), ((16500,), 64, 1100), ((4100,), 200, 4200),
            ((1, 5, 7), 33, 20), ((3, 9, 13), 80, 73), ((2, 1, 1), 16, 8), ((5, 1, 3), 100, 40), ((7, 6, 2), 64, 130), ((1, 16, 64), 256, 256),
            ((2, 91, 181), 73, 41), ((2, 181, 360), 48, 200)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("points,C,Co", PRODUCTS, ids=str)
def test_linear(points, C, Co, dt):
    q, s, _ = form(points, C, 10)
    w, ws, _ = form((Co,), C, 11, C ** -0.5)
    bias = torch.randn(Co, generator=gen(12), device="cuda")
    # the sum of whole numbers is exact in fp64 (of scaled values it is not: sums that are 0 come out as 1e-17)
    t = (q.reshape(-1, q.shape[-1]).double() @ w.double().t()) * s.reshape(-1, 1).double() * ws.double()
    for b in (None, bias):
        y = sgc.disco_linear_i8(q, s, w, ws, bias=b, dtype=DT[dt])
        assert y.shape == shape_of(points, Co) and y.dtype == DT[dt]
        want = t if b is None else t + b.double()
        tol = 1.01 * (3 * V * t.abs() + V * want.abs() + u_of(dt) * want.abs()) + SMALLEST[dt] + 2.0 ** -120
        assert bool(((rows(y) - want).abs() <= tol).all())


def test_linear_of_all_codes_and_the_most_channels():
    # 131056 channels of -128 x -128 (no writer gives -128, a caller's own codes may): the sum is 2^31 - 2^18
    C = 131056
    q = torch.full((70, C), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, C), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    w[2, ::2] = 127
    w[3] = 0
    one = torch.ones(70, device="cuda")
    for n in (3, 70):
        y = sgc.disco_linear_i8(q[:n], one[:n], w, one[:5], dtype=torch.float32)
        want = q[:n].double() @ w.double().t()
        assert torch.equal(y.double(), want.float().double())
    with pytest.raises(sgc.DiscoError):
        sgc.disco_linear_i8(torch.zeros((2, C + 16), dtype=torch.int8, device="cuda"), one[:2],
                            torch.zeros((2, C + 16), dtype=torch.int8, device="cuda"), one[:2])


@pytest.mark.parametrize("points", [(5,), (200,), (3, 9, 13)], ids=str)
def test_linear_nan_point_and_channel(points):
    q, s, _ = form(points, 80, 1)
    w, ws, _ = form((70,), 80, 2)
    clean = sgc.disco_linear_i8(q, s, w, ws)
    s.view(-1)[3] = float("nan")
    ws[7] = float("inf")
    y = rows(sgc.disco_linear_i8(q, s, w, ws))
    want = rows(clean)
    assert bool(torch.isnan(y[3]).all())
    keep = [i for i in range(y.shape[0]) if i != 3]
    assert not bool(torch.isfinite(y[keep][:, 7]).any())
    cols = [i for i in range(70) if i != 7]
    assert torch.equal(y[keep][:, cols], want[keep][:, cols])


# ---------------------------------------------------------------- the gradients

GRADS = [((1,), 1, 1), ((1,), 256, 256), ((5,), 16, 3), ((17,), 33, 65), ((64,), 64, 256), ((65,), 80, 73), ((129,), 128, 257), ((300,), 272, 130),
         ((1000,), 48, 300), ((33000,), 300, 40), ((1, 5, 7), 33, 20), ((3, 9, 13), 80, 73), ((2, 1, 1), 16, 8), ((5, 1, 3), 100, 40),
         ((7, 6, 2), 64, 130), ((1, 16, 64), 256, 256), ((2, 91, 181), 73, 41), ((2, 181, 360), 200, 48)]


def reach(points, n):
    """gy of these points as a view whose surroundings are NaN: what a call reads beside it shows."""
    whole = 1
    for v in shape_of(points, n):
        whole *= v
    return whole


def surrounded(t, before=3):
    buf = torch.full((t.numel() + 64 + before,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[before:before + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co", GRADS, ids=str)
def test_bwd_input(points, C, Co, dt):
    gy = surrounded(normal(points, Co, dt, 20, 0.5))
    w, ws, W = form((Co,), C, 21, Co ** -0.5)
    k, ks, kv = form(points, C, 22, 1.5)
    g = rows(gy)
    t, size = g @ W, g.abs() @ W.abs()
    for act in (None, "gelu", "silu"):
        gx = sgc.disco_linear_i8_bwd_input(gy, w, ws, channels=C, act=act, kept=None if act is None else k, kept_scale=None if act is None else ks)
        assert gx.shape == shape_of(points, C) and gx.dtype == DT[dt]
        f = torch.ones_like(t) if act is None else slope64(kv, act)
        want = t * f
        terms = size * (u_of(dt) + (Co + 2) * V) + g.abs().sum(1, keepdim=True) * SMALLEST[dt]
        # the slope: its own error, and the argument kept kept_scale rounded once (|act''| <= 1, times |x| v)
        slope = 0 if act is None else t.abs() * (2 * ACT + kv.abs() * V + 4 * V)
        tol = 1.02 * (terms * f.abs() + slope + u_of(dt) * want.abs()) + SMALLEST[dt] + 2.0 ** -120
        assert bool(((rows(gx) - want).abs() <= tol).all()), act


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co", GRADS + [((70000,), 140, 130), ((1,), 300, 700), ((2, 300, 333), 256, 256)], ids=str)
def test_bwd_weight(points, C, Co, dt):
    gy = surrounded(normal(points, Co, dt, 30, 0.5))
    q, s, x = form(points, C, 31)
    g = rows(gy)
    P = g.shape[0]
    want, size = g.t() @ x, g.abs().t() @ x.abs()
    tol = 1.02 * (size * (u_of(dt) + (P + 2) * V) + g.abs().sum(0)[:, None] * SMALLEST[dt] + u_of(dt) * want.abs()) + SMALLEST[dt] + 2.0 ** -120
    dw = sgc.disco_linear_i8_bwd_weight(gy, q, s, channels=C)
    assert dw.shape == (Co, C) and dw.dtype == DT[dt]
    assert bool(((dw.double() - want).abs() <= tol).all())
    dw2, db = sgc.disco_linear_i8_bwd_weight(gy, q, s, channels=C, bias=True)
    assert torch.equal(dw, dw2) and db.shape == (Co,) and db.dtype == DT[dt]
    wb, sb = g.sum(0), g.abs().sum(0)
    assert bool(((db.double() - wb).abs() <= 1.01 * (sb * (P + 2) * V + u_of(dt) * wb.abs()) + SMALLEST[dt]).all())
