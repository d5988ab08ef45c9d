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
