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
@pytest.mark.parametrize("shape", [(1, 1024, 3, 70), (1, 1030, 9, 80), (3, 2048, 4, 70), (2, 1500, 3, 5), (3, 2100, 4, 70), (2, 5000, 3, 5), (4, 40000), (1, 1 << 20)], ids=str)
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
            ((2, 91, 181), 73, 41), ((2, 181, 360), 48, 200),
            # the weights in registers: rows and fields, whole and ragged planes, outputs stored past the caches and not
            ((33000,), 500, 300), ((33001,), 100, 513), ((40000,), 17, 70), ((33000,), 512, 256), ((1, 181, 360), 300, 70), ((3, 91, 181), 400, 130),
            ((9, 60, 61), 272, 300), ((1, 512, 1024), 80, 160), ((2, 512, 520), 33, 130), ((1, 512, 1024), 256, 128)]


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
         ((7, 6, 2), 64, 130), ((1, 16, 64), 256, 256), ((2, 91, 181), 73, 41), ((2, 181, 360), 200, 48),
         # 32 input channels at most: tiles of their own
         ((3000,), 8, 307), ((2001,), 32, 600), ((3, 61, 67), 8, 307), ((2, 40, 64), 30, 512), ((1, 128, 64), 1, 33)]


def surrounded(t, before=3):
    """t as a view whose surroundings are NaN: what a call reads beside it shows."""
    buf = torch.full((t.numel() + 64 + before,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[before:before + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# rows with the weights in registers: every bucket of output channels, ragged channels and points
STAYS = [((33001,), 301, 8), ((33001,), 300, 64), ((33001,), 257, 72), ((20000,), 600, 128), ((16500,), 600, 200), ((16401,), 520, 256),
         ((9000,), 1030, 264), ((9001,), 1100, 512), ((70000,), 40, 512), ((40000,), 512, 136)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co,before", [g + (3,) for g in GRADS] + [g + (8,) for g in STAYS] + [STAYS[0] + (4,), STAYS[7] + (4,)], ids=str)
def test_bwd_input(points, C, Co, before, dt):
    # (the rows of gy start at 16 bytes' alignment with 8 elements before them, at none with 3 and 4)
    gy = surrounded(normal(points, Co, dt, 20, 0.5), before)
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


# ---------------------------------------------------------------- how they are called


CALLS = {
    "quantize": lambda s: sgc.disco_quantize_i8(s["x"], act="gelu", keep=True),
    "dequantize": lambda s: sgc.disco_dequantize_i8(s["q"], s["s"], channels=s["C"]),
    "linear": lambda s: sgc.disco_linear_i8(s["q"], s["s"], s["w"], s["ws"], bias=s["b"]),
    "bwd_input": lambda s: sgc.disco_linear_i8_bwd_input(s["gy"], s["w"], s["ws"], channels=s["C"], act="gelu", kept=s["q"], kept_scale=s["s"]),
    "bwd_weight": lambda s: sgc.disco_linear_i8_bwd_weight(s["gy"], s["q"], s["s"], channels=s["C"], bias=True),
}
SIZES = [((1,), 40, 50), ((100,), 256, 64), ((900,), 80, 200), ((40000,), 64, 300), ((40000,), 300, 304), ((33000,), 200, 40), ((9000,), 1030, 512),
         ((2, 91, 181), 73, 41), ((1, 360, 128), 256, 256), ((1, 181, 360), 300, 70)]


def state(points, C, Co, seed=0):
    q, s, _ = form(points, C, seed + 1)
    w, ws, _ = form((Co,), C, seed + 2, C ** -0.5)
    return {"C": C, "x": normal(points, C, "bf16", seed + 3, 2.0), "q": q, "s": s, "w": w, "ws": ws,
            "b": torch.randn(Co, generator=gen(seed + 4), device="cuda"), "gy": normal(points, Co, "bf16", seed + 5, 0.5)}


def flat(r):
    return list(r) if isinstance(r, tuple) else [r]


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("points,C,Co", SIZES, ids=str)
def test_replays_streams_and_repeats(points, C, Co, call):
    s, f = state(points, C, Co), CALLS[call]
    first = flat(f(s))
    assert all(torch.equal(a, b) for a, b in zip(first, flat(f(s))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = flat(f(s))
        here_too = flat(f(s))
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, there, here_too))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = flat(f(s))
    for k in range(3):
        t = state(points, C, Co, 100 * (k + 1))
        for n in s:
            if n != "C":
                s[n].copy_(t[n])
        eager = flat(f(t))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), k


@pytest.mark.parametrize("points,C,Co", SIZES, ids=str)
def test_two_streams_at_once(points, C, Co):
    one, two = state(points, C, Co, 7), state(points, C, Co, 9)
    want = [[flat(f(s)) for f in CALLS.values()] for s in (one, two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for f in CALLS.values():
        for k, s in enumerate((one, two)):
            with torch.cuda.stream(streams[k]):
                got[k].append(flat(f(s)))
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(want[k], got[k]):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("points,C,Co", [((7,), 33, 9), ((500,), 73, 65), ((40000,), 100, 257), ((40001,), 100, 264), ((3, 9, 13), 80, 73), ((2, 91, 181), 48, 41), ((1, 360, 128), 300, 130)], ids=str)
@pytest.mark.parametrize("dt", list(DT))
def test_given_outputs_at_any_element_are_filled_and_nothing_beside_them(points, C, Co, dt):
    s = state(points, C, Co)

    def inside(t, skip):
        buf = torch.full((t.numel() + 40,), 77, dtype=t.dtype, device="cuda")
        v = buf[skip:skip + t.numel()].view(t.shape)
        return buf, v, skip

    def check(holder, want):
        buf, v, skip = holder
        assert torch.equal(v, want)
        assert bool((buf[:skip] == 77).all()) and bool((buf[skip + want.numel():] == 77).all())

    x = s["x"].to(DT[dt])
    xs = inside(x, 5)
    xs[1].copy_(x)
    want = sgc.disco_quantize_i8(x, act="silu", keep=True)
    outs = [inside(w, 16 if w.dtype == torch.int8 else 3) for w in want]
    got = sgc.disco_quantize_i8(xs[1], act="silu", keep=True, q=outs[0][1], scale=outs[1][1], kept=outs[2][1], kept_scale=outs[3][1])
    assert all(a is b[1] for a, b in zip(got, outs))
    for o, w in zip(outs, want):
        check(o, w)
    want = sgc.disco_dequantize_i8(s["q"], s["s"], channels=C, dtype=DT[dt])
    o = inside(want, 1)
    sgc.disco_dequantize_i8(s["q"], s["s"], out=o[1], dtype=DT[dt])
    check(o, want)
    want = sgc.disco_linear_i8(s["q"], s["s"], s["w"], s["ws"], bias=s["b"], dtype=DT[dt])
    o = inside(want, 1)
    sgc.disco_linear_i8(s["q"], s["s"], s["w"], s["ws"], bias=s["b"], out=o[1], dtype=DT[dt])
    check(o, want)
    if dt == "f32":
        return
    gy = s["gy"].to(DT[dt])
    g = inside(gy, 3)
    g[1].copy_(gy)
    for act in (None, "gelu"):
        k = {} if act is None else {"act": act, "kept": s["q"], "kept_scale": s["s"]}
        want = sgc.disco_linear_i8_bwd_input(gy, s["w"], s["ws"], channels=C, **k)
        o = inside(want, 1)
        sgc.disco_linear_i8_bwd_input(g[1], s["w"], s["ws"], gx=o[1], **k)
        check(o, want)
    want = sgc.disco_linear_i8_bwd_weight(gy, s["q"], s["s"], channels=C, bias=True)
    outs = [inside(w, 1) for w in want]
    need = sgc.disco_linear_i8_bwd_weight_workspace(gy, C, bias=True)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    sgc.disco_linear_i8_bwd_weight(g[1], s["q"], s["s"], dw=outs[0][1], db=outs[1][1], workspace=ws[:need] if need else None)
    for o, w in zip(outs, want):
        check(o, w)
    assert bool((ws[need:] == 255).all())


def test_refusals_on_the_device():
    s = state((64,), 64, 64)
    big = torch.zeros(64 * 64 + 16, dtype=torch.int8, device="cuda")
    off = big[1:1 + 64 * 64].view(64, 64)
    gy = normal((40000,), 64, "bf16", 1)
    q, sc, _ = form((40000,), 64, 2)
    small = torch.zeros(64, dtype=torch.uint8, device="cuda")
    for call in (lambda: sgc.disco_linear_i8(off, s["s"], s["w"], s["ws"]), lambda: sgc.disco_linear_i8(s["q"], s["s"], off, s["ws"]),
                 lambda: sgc.disco_quantize_i8(s["x"], q=off), lambda: sgc.disco_dequantize_i8(off, s["s"]),
                 lambda: sgc.disco_linear_i8_bwd_input(s["gy"], off, s["ws"]), lambda: sgc.disco_linear_i8_bwd_weight(s["gy"], off, s["s"]),
                 lambda: sgc.disco_linear_i8_bwd_weight(gy, q, sc, workspace=small), lambda: sgc.disco_linear_i8(s["q"], s["s"].cpu(), s["w"], s["ws"]),
                 lambda: sgc.disco_linear_i8_bwd_input(s["gy"], s["w"], s["ws"], gx=s["gy"]),
                 lambda: sgc.disco_linear_i8_bwd_weight(s["gy"], s["q"], s["s"], dw=s["gy"]),
                 lambda: sgc.disco_dequantize_i8(s["q"], s["s"], out=s["q"].view(torch.bfloat16).view(64, 32)[:, :16].contiguous().t().contiguous().t())):
        with pytest.raises((sgc.DiscoError, ValueError)):
            call()
    with pytest.raises(sgc.DiscoError) as e:  # the whole of x would be overwritten as it is read
        sgc.disco_quantize_i8(s["x"], q=s["x"].view(torch.int8)[:, :64].contiguous().view(64, 64), scale=s["x"].view(-1)[:128].view(torch.float32))
    assert e.value.status_name == "DISCO_ERR_INVALID_ARGUMENT"


def test_no_points():
    q, s = torch.zeros((0, 48), dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    w, ws, _ = form((5,), 40, 1)
    gy = torch.zeros((0, 5), dtype=torch.bfloat16, device="cuda")
    assert sgc.disco_linear_i8(q, s, w, ws).shape == (0, 5)
    assert sgc.disco_linear_i8_bwd_input(gy, w, ws, channels=40).shape == (0, 40)
    assert sgc.disco_quantize_i8(torch.zeros((0, 40), device="cuda"))[0].shape == (0, 48)
    assert sgc.disco_dequantize_i8(q, s, channels=40).shape == (0, 40)
    dw = torch.full((5, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    db = torch.full((5,), float("nan"), dtype=torch.bfloat16, device="cuda")
    sgc.disco_linear_i8_bwd_weight(gy, q, s, dw=dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_a_nan_point_stays_its_own_in_the_input_gradient():
    for points in ((300,), (3, 9, 13), (40000,), (1, 91, 181)):  # the third: weights in registers
        gy = normal(points, 80, "bf16", 1)
        w, ws, _ = form((80,), 260, 2)
        k, ks, _ = form(points, 260, 3)
        clean = rows(sgc.disco_linear_i8_bwd_input(gy, w, ws, channels=260, act="gelu", kept=k, kept_scale=ks))
        rows_of = gy.movedim(1, -1).reshape(-1, 80)
        bad = rows_of.clone()
        bad[7, 3], bad[11, 79] = float("nan"), float("inf")
        g = bad.reshape(gy.movedim(1, -1).shape).movedim(-1, 1).contiguous()
        ks.view(-1)[20] = float("nan")   # a checkpoint that held a NaN
        got = rows(sgc.disco_linear_i8_bwd_input(g, w, ws, channels=260, act="gelu", kept=k, kept_scale=ks))
        hit = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
        hit[[7, 11, 20]] = True
        assert torch.equal(got[~hit], clean[~hit]) and bool(torch.isnan(got[7]).all()) and bool(torch.isnan(got[20]).all())
        assert not bool(torch.isfinite(got[11]).any())


def test_gradients_against_differences():
    # the product is linear in its operands' values: <gy, y(W + e D) - y(W)> / e = <dw, D>, and the same for the input
    points, C, Co = (500,), 64, 48
    q, s, x = form(points, C, 1)
    w, ws, W = form((Co,), C, 2)
    gy = normal(points, Co, "f16", 3)
    g = rows(gy)
    dw = sgc.disco_linear_i8_bwd_weight(gy, q, s).double()
    gx = rows(sgc.disco_linear_i8_bwd_input(gy, w, ws))
    y = lambda qq, ss, ww, wws: rows(sgc.disco_linear_i8(qq, ss, ww, wws, dtype=torch.float32))
    base = y(q, s, w, ws)
    for o, c in ((0, 0), (17, 33), (47, 63)):
        step = 1 if int(w[o, c]) < 127 else -1
        w2 = w.clone()
        w2[o, c] += step
        diff = float((g * (y(q, s, w2, ws) - base)).sum()) / (step * float(ws[o]))
        size = float((g[:, o].abs() * x[:, c].abs()).sum())
        # fp32 outputs: their roundings, as large as the outputs themselves; dw: fp16 operands and result
        slack = 8 * V * float((g[:, o].abs() * base[:, o].abs()).sum()) / float(ws[o]) + 2.0 ** -11 * (size + abs(diff)) * 1.1
        assert abs(diff - float(dw[o, c])) <= slack, (o, c)
    for p, c in ((0, 0), (123, 45), (499, 63)):
        step = 1 if int(q[p, c]) < 127 else -1
        q2 = q.clone()
        q2[p, c] += step
        diff = float((g * (y(q2, s, w, ws) - base)).sum()) / (step * float(s[p]))
        size = float((g[p].abs() * W[:, c].abs()).sum())
        slack = 8 * V * float((g[p].abs() * base[p].abs()).sum()) / float(s[p]) + 2.0 ** -11 * (size + abs(diff)) * 1.1
        assert abs(diff - float(gx[p, c])) <= slack, (p, c)


@pytest.mark.parametrize("rows_or_field", ["rows", "field"])
def test_elements_beyond_32_bits(rows_or_field):
    # 2^21 + 3 points of 2064 channels: 4.3e9 codes, and as many values read and written
    n, C, Co = (1 << 21) + 3, 2064, 32
    shape = (n, C) if rows_or_field == "rows" else (1, C, 1, n)
    points = (n,) if rows_or_field == "rows" else (1, 1, n)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(1))
    q, s = sgc.disco_quantize_i8(x)
    pick = torch.tensor([0, 1, 1 << 20, (1 << 21) - 1, n - 2, n - 1], device="cuda")
    xr = (x[pick] if rows_or_field == "rows" else x[0, :, 0, pick].t()).float()
    qr, sr = q.reshape(n, C)[pick], s.reshape(n)[pick]
    want = (xr.abs().amax(1).cpu() / 127)
    assert torch.equal(sr.cpu(), want) and torch.equal(qr.float().cpu(), torch.round(xr.cpu() / want[:, None]))
    back = sgc.disco_dequantize_i8(q, s)
    br = back[pick] if rows_or_field == "rows" else back[0, :, 0, pick].t()
    assert torch.equal(br, (qr.float() * sr[:, None]).bfloat16())
    del back, x
    w, ws, W = form((Co,), C, 2, C ** -0.5)
    y = sgc.disco_linear_i8(q, s, w, ws, dtype=torch.float32)
    yr = (y[pick] if rows_or_field == "rows" else y[0, :, 0, pick].t()).double()
    t = (qr.double() @ w.double().t()) * sr.double()[:, None] * ws.double()
    assert bool(((yr - t).abs() <= 4.1 * V * t.abs()).all())
    del y
    gy = torch.zeros(points[:1] + (Co,) + points[1:], dtype=torch.bfloat16, device="cuda")
    if rows_or_field == "rows":
        gy[pick] = torch.randn((6, Co), generator=gen(3), device="cuda").bfloat16()
        g = gy[pick].double()
    else:
        gy[0, :, 0, pick] = torch.randn((Co, 6), generator=gen(3), device="cuda").bfloat16()
        g = gy[0, :, 0, pick].t().double()
    xv = qr.double() * sr.double()[:, None]
    dw = sgc.disco_linear_i8_bwd_weight(gy, q, s).double()
    want, size = g.t() @ xv, g.abs().t() @ xv.abs()
    assert bool(((dw - want).abs() <= 1.02 * (size * (2.0 ** -8 + 16 * V) + 2.0 ** -8 * want.abs())).all())
    gx = sgc.disco_linear_i8_bwd_input(gy, w, ws)
    gr = (gx[pick] if rows_or_field == "rows" else gx[0, :, 0, pick].t()).double()
    want, size = g @ W, g.abs() @ W.abs()
    assert bool(((gr - want).abs() <= 1.02 * (size * (2.0 ** -8 + 40 * V) + 2.0 ** -8 * want.abs())).all())
    del gx, gy, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("C", [1 << 24, (1 << 25) + 16, 1 << 26])
def test_bwd_input_checkpoint_rows_beyond_32_bits(C):
    # 64 points' checkpoints of 2^30 to 2^32 bytes: past 31 bits they fit no tile's offsets
    n, Co = 64, 8
    kept = torch.randint(-127, 128, (n, C), generator=gen(1), device="cuda", dtype=torch.int8)
    ks = torch.rand(n, generator=gen(2), device="cuda") * 0.03 + 0.001
    w = torch.randint(-127, 128, (Co, C), generator=gen(3), device="cuda", dtype=torch.int8)
    ws = torch.rand(Co, generator=gen(4), device="cuda") * 0.01 + 0.001
    gy = torch.randn((n, Co), generator=gen(5), device="cuda").bfloat16()
    gx = sgc.disco_linear_i8_bwd_input(gy, w, ws, act="gelu", kept=kept, kept_scale=ks)
    pick = torch.tensor([0, 1, 255, 256, C // 2 - 1, C // 2, C - 257, C - 1], device="cuda")
    a = kept[:, pick].double() * ks.double()[:, None]
    slope = 0.5 * (1 + torch.erf(a / 2 ** 0.5)) + a * torch.exp(-a * a / 2) / (2 * torch.pi) ** 0.5
    wv, g = w[:, pick].double() * ws.double()[:, None], gy.double()
    t, size = g @ wv, g.abs() @ wv.abs()
    want = slope * t
    # the weights' rounding to bf16 and the fp32 sum of 8 terms, the slope (5.1e-7 and its argument's rounding), the result
    bar = 1.02 * (slope.abs() * size * (2.0 ** -8 + 40 * V) + 8e-7 * size + 2.0 ** -8 * want.abs())
    assert bool(((gx[:, pick].double() - want).abs() <= bar).all())
    del kept, w, gx
    torch.cuda.empty_cache()
