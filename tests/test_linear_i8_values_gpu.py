"""The channel products' values where a bound of the terms' sizes says little: the lower tail of gelu, ties of the codes, the
gradients of many points, and the product over large fields, against the formulas in fp64 (V = 2^-24, fp32's unit roundoff)."""
import pytest
import torch

import sparse_gather_contraction_amd as sgc
from test_linear_i8_gpu import DT, V, gen, rows, shape_of, u_of

pytestmark = pytest.mark.gpu


def points_as(x, layout):
    """Rows (P, C) as rows or as a field (the first axis in two, planes of P / 2)."""
    if layout == "rows":
        return x
    return x.view(2, x.shape[0] // 2, 1, x.shape[1]).permute(0, 3, 2, 1).contiguous()


def tail_error(v):
    """How far gelu(v) may be off in relation to its size for v <= 0: the polynomial 9.1e-8 (1 + v^2 / 8); the exponent's argument,
    v^2 / 2 with the roundings of a square, a constant and a product; twelve for its exponential (one unit in the last place, two
    V), the polynomial's last steps and its argument, whose errors it passes on with a factor below one, and two products."""
    return 9.1e-8 * (1 + v * v / 8) + V * (1.5 * v * v + 12)


# rows in one wave, in several and past the registers; fields in registers and past them
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("layout,C", [("rows", 1), ("rows", 3), ("rows", 200), ("rows", 2064), ("rows", 33000), ("field", 1), ("field", 40), ("field", 2064)])
def test_gelu_of_points_in_the_lower_tail(layout, C, dt):
    # every value of a point lies within 1/4 of one place between -12 and -2: the point's scale and codes come from the tail alone
    P = 80 if C > 20000 else 1000
    top = -2 - 10 * torch.arange(P, device="cuda") / P
    x = (top[:, None] - torch.rand((P, C), generator=gen(1), device="cuda") / 4).to(DT[dt])
    q, s = sgc.disco_quantize_i8(points_as(x, layout), act="gelu")
    q, s, v = q.reshape(P, -1)[:, :C].double(), s.reshape(P).double(), x.double()
    g = v * torch.erfc(v * -0.5 ** 0.5) / 2
    err = g.abs() * tail_error(v)
    want = g.abs().amax(1) / 127
    assert bool(((s - want).abs() <= err.amax(1) / 127 + V * want * 1.01).all())
    assert bool(((q * s[:, None] - g).abs() <= s[:, None] * (0.5 + 128 * V) + err).all())


@pytest.mark.parametrize("layout", ["rows", "field", "rows_narrow", "field_narrow", "rows_stay"])
def test_gelu_slope_in_the_lower_tail(layout):
    # gy w = 1 in one term, so the gradient is the slope at the kept values: -12 .. -0.76 in every channel, and their negatives
    P, C = (40000, 257) if layout == "rows_stay" else (1000, 20 if "narrow" in layout else 129)
    Co = 8
    ks = (torch.arange(P, device="cuda") % 1000 + 64) * (12 / 1064 / 127)
    k = torch.randint(-127, -125, (P, -(-C // 16) * 16), generator=gen(1), device="cuda", dtype=torch.int8)
    k[P // 2:] *= -1
    w, ws = torch.zeros((Co, k.shape[1]), dtype=torch.int8, device="cuda"), torch.ones(Co, device="cuda")
    w[3] = 1
    gy = torch.zeros((P, Co), dtype=torch.bfloat16, device="cuda")
    gy[:, 3] = 1
    kept, kept_scale = (k, ks) if layout.startswith("rows") else (k.view(2, 1, P // 2, -1), ks.view(2, 1, P // 2))
    gx = rows(sgc.disco_linear_i8_bwd_input(points_as(gy, layout.split("_")[0]), w, ws, channels=C, act="gelu", kept=kept, kept_scale=kept_scale))
    v = (k[:, :C].float() * ks[:, None]).double()   # rounded to fp32 as the kernels do
    t = v.abs()
    R = torch.special.erfcx(t / 2 ** 0.5) / 2
    e, d = torch.exp(-t * t / 2), t / (2 * torch.pi) ** 0.5
    z = e * (R - d)                                  # the slope at -t; at t it is 1 - z
    want = torch.where(v < 0, z, 1 - z)
    # R - t / sqrt(2 pi): the polynomial, six of its last steps and of the difference; the exponential and two products
    err = e * (9.1e-8 * (1 + t * t / 8) * R + 8 * V * (R + d)) + z.abs() * V * (1.5 * t * t + 6) + V * want.abs() * (v > 0)
    assert bool(((gx - want).abs() <= (err + u_of("bf16") * want.abs()) * 1.01).all())


@pytest.mark.parametrize("layout,C", [("rows", 128), ("rows", 2064), ("rows", 33000), ("field", 128), ("field", 2064)])
@pytest.mark.parametrize("act", [None, "gelu", "silu"])
def test_codes_are_the_quotients_by_the_stored_scale(layout, C, act):
    # From 17 on both functions give their argument itself in fp32, so the codes are those of x.  A point's largest value is 127 times
    # a scale of its own, and its other values lie at (k + 1/2) scale and beside it: exact ties go to the even code.
    P = 64
    scale = torch.tensor([3.0, 7.0, 11.0, 1.0, 5.5, 9.0, 13.0, 1.3, 2.7, 6.1], device="cuda").repeat(7)[:P]
    k = torch.randint(17, 126, (P, C), generator=gen(1), device="cuda").float()
    x = ((k + 0.5) * scale[:, None]) * (1 + torch.randint(-1, 2, (P, C), generator=gen(2), device="cuda") * 2.0 ** -23)
    x[:, 5] = 127 * scale
    q, s = sgc.disco_quantize_i8(points_as(x, layout), act=act)
    s32 = x.cpu().abs().amax(1) / 127
    assert torch.equal(s.reshape(P).cpu(), s32)
    assert torch.equal(q.reshape(P, -1)[:, :C].cpu().float(), torch.round(x.cpu() / s32[:, None]))


# one step, several steps a split, many splits; tiles of 256 x 256, 128 x 128 and 32 x 256; shared sums of db; whole and ragged planes
WEIGHTS = [((64,), 256, 256), ((1000,), 48, 300), ((33000,), 300, 40), ((70000,), 140, 130), ((70001,), 512, 1030), ((200000,), 256, 256), ((130000,), 20, 600),
           ((3, 9, 13), 80, 73), ((2, 181, 360), 200, 48), ((2, 300, 333), 256, 256), ((2, 300, 334), 256, 512), ((3, 285, 291), 8, 307), ((1, 361, 720), 600, 260)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co", WEIGHTS, ids=str)
def test_bwd_weight_of_whole_numbers(points, C, Co, dt):
    # gy in eighths, codes and scales of 1/2, 1 and 2: every term is a whole number of at most 1016 sixteenths, so fp32 sums of up to
    # 16,000 points (no split here is longer) are exact in any order, the fp64 ones over the splits too, and the results are the true
    # sums rounded once.  A point that is left out or met twice shows.
    P = 1
    for n in points:
        P *= n
    g = torch.randint(-2, 3, (P, Co), generator=gen(1), device="cuda").double() / 8
    q = torch.zeros((P, -(-C // 16) * 16), dtype=torch.int8, device="cuda")
    q[:, :C] = torch.randint(-127, 128, (P, C), generator=gen(2), device="cuda")
    s = torch.tensor([0.5, 1.0, 2.0], device="cuda")[torch.randint(0, 3, (P,), generator=gen(3), device="cuda")]
    gy = g.to(DT[dt]).view(tuple(points) + (Co,)).movedim(-1, 1).contiguous()
    assert gy.shape == shape_of(points, Co)
    x = q[:, :C].double() * s.double()[:, None]
    want = g.t() @ x
    dw, db = sgc.disco_linear_i8_bwd_weight(gy, q.view(tuple(points) + (-1,)), s.view(points), channels=C, bias=True)
    assert torch.equal(dw, want.to(DT[dt])) and torch.equal(db, g.sum(0).to(DT[dt]))
    assert torch.equal(dw, sgc.disco_linear_i8_bwd_weight(gy, q.view(tuple(points) + (-1,)), s.view(points), channels=C))
    # the comparison sees one point in the middle
    less = want - g[P // 2][:, None] * x[P // 2][None, :]
    assert not torch.equal(less.to(DT[dt]), want.to(DT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co", [((70000,), 140, 130), ((200000,), 256, 256), ((2, 300, 333), 256, 256), ((2, 181, 360), 200, 160)], ids=str)
def test_bwd_weight_error_of_its_norm(points, C, Co, dt):
    # Rounding a value to 16 bits is off by 0.425 u of it in the root mean square (uniform within a step, over mantissas spread as
    # their logarithms).  Each term passes one such rounding and the result one, independent of each other and of the terms' signs, so
    # the error's norm is 0.425 sqrt(2) u = 0.6 u of the result's; 0.75 u leaves out no more than a point in 300,000 (bf16).
    # db: its rounding alone, at most u.  fp32 sums of up to n steps of 16 points: sqrt(n) V, 1e-5 here.
    P = 1
    for n in points:
        P *= n
    gy = (torch.randn(shape_of(points, Co), generator=gen(1), device="cuda") / 2).to(DT[dt])
    x = torch.randn((P, C), generator=gen(2), device="cuda")
    q, s = sgc.disco_quantize_i8(x)
    v, g = q[:, :C].double() * s.double()[:, None], rows(gy)
    dw, db = sgc.disco_linear_i8_bwd_weight(gy, q.view(tuple(points) + (-1,)), s.view(points), channels=C, bias=True)
    want, wb = g.t() @ v, g.sum(0)
    assert float((dw.double() - want).norm()) <= (0.75 * u_of(dt) + 1e-5) * float(want.norm())
    assert float((db.double() - wb).norm()) <= (u_of(dt) + 1e-5) * float(wb.norm())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("points,C,Co", [((2, 721, 1440), 256, 256), ((2, 721, 1440), 48, 70), ((2, 721, 1440), 100, 70), ((2, 721, 1440), 300, 65), ((1, 512, 1024), 256, 160),
                                         ((3, 361, 720), 130, 257)], ids=str)
def test_linear_over_large_fields(points, C, Co, dt):
    # more than 128 MiB of output: the weights stay in registers, for every bucket of channels; planes that end half way through
    # a tile of 64 points (721 x 1440 and 361 x 720), so a tile crosses from one plane to the next
    P = points[0] * points[1] * points[2]
    q = torch.zeros((P, -(-C // 16) * 16), dtype=torch.int8, device="cuda")
    q[:, :C] = torch.randint(-127, 128, (P, C), generator=gen(1), device="cuda", dtype=torch.int8)
    w = torch.zeros((Co, q.shape[1]), dtype=torch.int8, device="cuda")
    w[:, :C] = torch.randint(-127, 128, (Co, C), generator=gen(2), device="cuda", dtype=torch.int8)
    s = torch.rand(P, generator=gen(3), device="cuda") * 0.02 + 0.005
    ws = (torch.rand(Co, generator=gen(4), device="cuda") + 0.5) / (127 * C ** 0.5)
    bias = torch.randn(Co, generator=gen(5), device="cuda")
    y = sgc.disco_linear_i8(q.view(points + (-1,)), s.view(points), w, ws, bias=bias, dtype=DT[dt])
    assert y.shape == shape_of(points, Co) and y.numel() * 2 > 128 << 20
    M = points[1] * points[2]
    for b in range(points[0]):
        t = (q[b * M:(b + 1) * M].double() @ w.double().t()).mul_(s[b * M:(b + 1) * M].double()[:, None]).mul_(ws.double())
        want = t + bias.double()
        # the sum's conversion and two scales, the bias, the output's rounding (fp16's subnormals: half a step)
        tol = 1.01 * (3 * V * t.abs() + (V + u_of(dt)) * want.abs()) + 2.0 ** -25
        assert bool(((y[b].reshape(Co, M).t().double() - want).abs() <= tol).all()), b


@pytest.mark.parametrize("layout,C", [("rows", 1), ("rows", 200), ("field", 40)])
def test_silu_of_points_in_the_lower_tail(layout, C):
    # as for gelu, down to where e^x leaves fp32's range
    P = 1000
    top = -2 - 85 * torch.arange(P, device="cuda") / P
    x = top[:, None] - torch.rand((P, C), generator=gen(1), device="cuda") / 4
    q, s = sgc.disco_quantize_i8(points_as(x, layout), act="silu")
    q, s, v = q.reshape(P, -1)[:, :C].double(), s.reshape(P).double(), x.double()
    g = v / (1 + torch.exp(-v))
    # the exponent's argument (a constant's rounding and a product's), the exponential, the sum, the reciprocal and the product
    err = g.abs() * V * (2 * v.abs() + 8)
    want = (g.abs().amax(1) / 127).clamp(min=2.0 ** -126)
    assert bool(((s - want).abs() <= err.amax(1) / 127 + V * want * 1.01).all())
    assert bool(((q * s[:, None] - g).abs() <= s[:, None] * (0.5 + 128 * V) + err).all())


def test_functions_beyond_their_tails():
    # from where the exponential leaves fp32's range on both functions are 0, whatever the size of what they are taken of
    x = torch.tensor([-13.3, -14.5, -20.0, -1e4, -1e30, -3.4e38], device="cuda").view(-1, 1)
    for act, shift in (("gelu", 0.0), ("silu", -76.0)):
        q, s, k, ks = sgc.disco_quantize_i8(x + shift, act=act, keep=True)
        assert bool((s == 2.0 ** -126).all()) and bool((q == 0).all()) and bool((k[:, 0] == -127).all())
        w, ws = torch.ones((1, 16), dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda")
        gx = sgc.disco_linear_i8_bwd_input(torch.ones((6, 1), dtype=torch.bfloat16, device="cuda"), w, ws, channels=1, act=act, kept=k, kept_scale=ks)
        assert bool((gx.abs() <= 2.0 ** -115).all())
