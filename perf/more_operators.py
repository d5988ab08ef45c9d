"""Workloads of the channel products in 8-bit integers that stand beside the spherical convolution.

A channel product mixes the channels of each grid point (of each row), y = x W^T + bias.  Its operands are held as
8-bit integers with a scale for each point and one for each output channel; the same 8-bit form is the checkpoint that
the backward pass reads.  Five operators: the form's writer, with an activation function before it and a checkpoint of
what the function was taken of, and its reader ("store"); the product ("linear"); the gradient of its input, through
the activation function by its checkpoint ("bwd_input"); the gradients of its weight and bias from the 8-bit input
("bwd_weight").

The form: a point's channels lie together, padded with zeros to a multiple of 16, whatever the order of the tensor it
was made from; q = x / scale to whole numbers (ties to even), scale = max(max |x| / 127, 2^-126).

Fields (B, C, H, W) have their channels at axis 1, rows (points, C) too.  With ``own`` false, ``run`` evaluates the
plain form in fp32 torch operations; with ``own`` true it calls ``sparse_gather_contraction_amd``.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = 2.0 ** -126
MAX_ELEMENTS = 2 * 256 * 721 * 1440
MAX_PRODUCT = 8192 ** 3
STEP = 1 << 27  # elements of a piece in 64 bits


def listed():
    return [
        # one grid point's 256 channels on their way into a product: the calls' latency is all that counts
        {"name": "store_one_point", "op": "store", "points": "1", "C": 256, "dtype": "bf16", "act": "none", "keep": False},
        # the residual stream of the 256-channel model at 721x1440, batch 2, into the 8-bit form and back
        {"name": "store_721x1440", "op": "store", "points": "2x721x1440", "C": 256, "dtype": "bf16", "act": "none", "keep": False},
        # hidden rows of the 512-channel model (360x720 points, four times as wide): the next product's operand and the checkpoint
        {"name": "store_rows_gelu_keep", "op": "store", "points": "259200", "C": 2048, "dtype": "bf16", "act": "gelu", "keep": True},
        # one point through the 512-channel model's first product
        {"name": "linear_one_point", "op": "linear", "points": "1", "C": 512, "Co": 2048, "dtype": "bf16", "bias": True},
        # a few rows against large weights: the weights are all there is to read
        {"name": "linear_16_rows_8192", "op": "linear", "points": "16", "C": 8192, "Co": 8192, "dtype": "f16", "bias": False},
        # 256 channels to 256 at 721x1440, batch 2, into a field
        {"name": "linear_721x1440", "op": "linear", "points": "2x721x1440", "C": 256, "Co": 256, "dtype": "bf16", "bias": True},
        # the 512-channel model's first product over its 360x720 points
        {"name": "linear_rows_512", "op": "linear", "points": "259200", "C": 512, "Co": 2048, "dtype": "bf16", "bias": True},
        # a large square product
        {"name": "linear_8192", "op": "linear", "points": "8192", "C": 8192, "Co": 8192, "dtype": "bf16", "bias": False},
        # gradient of the input at an odd regional grid with 80 channels in and 73 out: no row or plane is aligned
        {"name": "bwd_input_odd_91x181", "op": "bwd_input", "points": "3x91x181", "C": 80, "Co": 73, "dtype": "f16", "act": "silu"},
        # gradient of the hidden rows of the 512-channel model, through their activation function
        {"name": "bwd_input_rows_gelu", "op": "bwd_input", "points": "259200", "C": 2048, "Co": 512, "dtype": "bf16", "act": "gelu"},
        # gradients of weight and bias of the 256-channel product at 721x1440, batch 2
        {"name": "bwd_weight_721x1440", "op": "bwd_weight", "points": "2x721x1440", "C": 256, "Co": 256, "dtype": "bf16", "bias": True},
        # gradients of the first product's weight and bias in the 512-channel model
        {"name": "bwd_weight_rows_512", "op": "bwd_weight", "points": "259200", "C": 512, "Co": 2048, "dtype": "bf16", "bias": True},
    ]


def _size(rng, low, high):
    """A whole number whose logarithm is uniform in [low, high]; every second one is made odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    if rng.random() < 0.5 and v % 2 == 0 and v > low:
        v -= 1
    return v


def draw(rng):
    op = rng.choice(["store", "linear", "linear", "bwd_input", "bwd_weight"])
    while True:
        if rng.random() < 0.5:  # a field
            points = [rng.randint(1, 4), _size(rng, 1, 721), _size(rng, 1, 1440)]
            C, Co = _size(rng, 1, 512), _size(rng, 1, 512)
        else:
            points = [_size(rng, 1, 259200)]
            C, Co = _size(rng, 1, 8192), _size(rng, 1, 8192)
        n = math.prod(points)
        wide = C if op == "store" else max(C, Co)
        if n * wide <= MAX_ELEMENTS // 2 and (op == "store" or n * C * Co <= MAX_PRODUCT // 4):
            break
    case = {"op": op, "points": "x".join(map(str, points)), "C": C}
    if op != "store":
        case["Co"] = Co
    case["dtype"] = rng.choice(["bf16", "f16"] if op.startswith("bwd") else list(DTYPES))
    if op in ("store", "bwd_input"):
        case["act"] = rng.choice(["none", "gelu", "silu"])
    if op == "store":
        case["keep"] = case["act"] != "none" and rng.random() < 0.5
    if op in ("linear", "bwd_weight"):
        case["bias"] = rng.random() < 0.5
    return case


def _points(case):
    return tuple(int(v) for v in case["points"].split("x"))


def _shape(case, channels):
    """The tensor of these points: channels at axis 1."""
    p = _points(case)
    return (p[0], channels) + p[1:]


def _read_dtype(case):
    return DTYPES["bf16" if case["dtype"] == "f32" else case["dtype"]]


def _codes(x, axis):
    """x in whole numbers (in x's type), and the scales of what lies along the axis."""
    scale = (x.abs().amax(axis) / 127.0).clamp(min=TINY)
    return torch.round(x / scale.unsqueeze(axis)), scale


def _act(x, name):
    if name == "gelu":
        return x * (0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))))
    return x * torch.sigmoid(x) if name == "silu" else x


def _act_slope(x, name):
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "silu":
        s = torch.sigmoid(x)
        return s * (1.0 + x * (1.0 - s))
    return None


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op, C, dt = case["op"], case["C"], DTYPES[case["dtype"]]

    def normal(shape, dtype, std=1.0):
        t = torch.randn(shape, generator=gen, dtype=dtype, device=dev)
        return t.mul_(std) if std != 1.0 else t

    def form(n, channels, lead, std=1.0):
        """The 8-bit form of normal rows."""
        q, scale = _codes(normal((n, channels), torch.float32, std), 1)
        padded = torch.zeros((n, -(-channels // 16) * 16), dtype=torch.int8, device=dev)
        padded[:, :channels] = q
        return padded.reshape(lead + (padded.shape[1],)), scale.reshape(lead)

    s = {"case": case}
    points = _points(case)
    n = math.prod(points)
    if op == "store":
        spread = torch.empty((1, C) + (1,) * (len(points) - 1), device=dev).uniform_(0.25, 4.0, generator=gen)  # channels differ in size
        s["x"] = normal(_shape(case, C), dt).mul_(spread.to(dt))
        return s
    Co = case["Co"]
    if op in ("linear", "bwd_weight"):
        s["q"], s["scale"] = form(n, C, points)
    if op in ("linear", "bwd_input"):
        s["w"], s["wscale"] = form(Co, C, (Co,), 1.0 / math.sqrt(C if op == "linear" else Co))
    if op == "linear":
        s["bias"] = normal((Co,), torch.float32, 0.5) if case["bias"] else None
        return s
    s["gy"] = normal(_shape(case, Co), dt, 0.125)
    if op == "bwd_input" and case["act"] != "none":
        s["kept"], s["kept_scale"] = form(n, C, points, 1.5)
    return s


def _values(q, scale, case):
    """The 8-bit form's values as (first axis, points after it, channels)."""
    return (q.float() * scale.unsqueeze(-1)).reshape(q.shape[0], -1, q.shape[-1])[..., :case["C"]]


def _plain(s):
    case = s["case"]
    op, C, dt = case["op"], case["C"], DTYPES[case["dtype"]]
    points = _points(case)
    if op == "store":
        x = s["x"].float()
        q, scale = _codes(_act(x, case["act"]), 1)
        out = {"values": (q * scale.unsqueeze(1)).to(_read_dtype(case)), "scale": scale}
        if case["keep"]:
            q, scale = _codes(x, 1)
            out["kept"], out["kept_scale"] = (q * scale.unsqueeze(1)).to(_read_dtype(case)), scale
        return out
    field = len(points) > 1
    if op == "linear":
        q, w = s["q"].float(), s["w"].float()
        if field:
            y = w @ q.reshape(points[0], -1, q.shape[-1]).transpose(1, 2)  # (first axis, Co, points after it)
            y = y * s["scale"].reshape(points[0], 1, -1) * s["wscale"][:, None]
            y = y if s["bias"] is None else y + s["bias"][:, None]
        else:
            y = (q @ w.t()) * s["scale"][:, None] * s["wscale"]
            y = y if s["bias"] is None else y + s["bias"]
        return {"y": y.to(dt).reshape(_shape(case, case["Co"]))}
    gy = s["gy"].float()
    if op == "bwd_input":
        w = (s["w"].float() * s["wscale"][:, None])[:, :C]
        gx = w.t() @ gy.flatten(2) if field else gy @ w
        if case["act"] != "none":
            kept = _values(s["kept"], s["kept_scale"], case)
            gx = gx * _act_slope(kept.transpose(1, 2) if field else kept[:, 0], case["act"])
        return {"gx": gx.to(dt).reshape(_shape(case, C))}
    x = _values(s["q"], s["scale"], case)
    out = {"dw": ((gy.flatten(2) @ x).sum(0) if field else gy.t() @ x[:, 0]).to(dt)}
    if case["bias"]:
        out["db"] = (gy.sum((0, 2, 3)) if field else gy.sum(0)).to(dt)
    return out


def _own(s):
    import sparse_gather_contraction_amd as sgc

    case = s["case"]
    op, C, dt = case["op"], case["C"], DTYPES[case["dtype"]]
    if op == "store":
        act = None if case["act"] == "none" else case["act"]
        form = sgc.disco_quantize_i8(s["x"], act=act, keep=case["keep"], axis=1)
        out = {"values": sgc.disco_dequantize_i8(form[0], form[1], channels=C, dtype=_read_dtype(case), axis=1), "scale": form[1]}
        if case["keep"]:
            out["kept"], out["kept_scale"] = sgc.disco_dequantize_i8(form[2], form[3], channels=C, dtype=_read_dtype(case), axis=1), form[3]
        return out
    if op == "linear":
        return {"y": sgc.disco_linear_i8(s["q"], s["scale"], s["w"], s["wscale"], bias=s["bias"], dtype=dt, axis=1)}
    if op == "bwd_input":
        act = None if case["act"] == "none" else case["act"]
        return {"gx": sgc.disco_linear_i8_bwd_input(s["gy"], s["w"], s["wscale"], channels=C, act=act, kept=s.get("kept"),
                                                    kept_scale=s.get("kept_scale"), axis=1)}
    if not case["bias"]:
        return {"dw": sgc.disco_linear_i8_bwd_weight(s["gy"], s["q"], s["scale"], channels=C, axis=1)}
    dw, db = sgc.disco_linear_i8_bwd_weight(s["gy"], s["q"], s["scale"], channels=C, bias=True, axis=1)
    return {"dw": dw, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, n, C = case["op"], math.prod(_points(case)), case["C"]
    esz = 4 if case["dtype"] == "f32" else 2
    padded = -(-C // 16) * 16
    form = n * (padded + 4)
    if op == "store":
        k = 2 if case["keep"] else 1
        return {"bytes": n * C * esz + k * (2 * form + 2 * n * C), "flops": n * C * (4 * k + (12 if case["act"] != "none" else 0))}
    Co = case["Co"]
    weights = Co * (padded + 4)
    flops = 2 * n * C * Co
    if op == "linear":
        return {"bytes": form + weights + (4 * Co if case["bias"] else 0) + n * Co * esz, "flops": flops}
    if op == "bwd_input":
        return {"bytes": n * Co * esz + weights + n * C * esz + (form if case["act"] != "none" else 0), "flops": flops}
    return {"bytes": n * Co * esz + form + Co * C * esz + (Co * esz if case["bias"] else 0), "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    op, C, points = case["op"], case["C"], _points(case)
    n = math.prod(points)
    step = max(1, STEP // max(C, case.get("Co", 1)))

    def pieces(v):
        """Consecutive points of a tensor with its channels at axis 1 or a form's leading axes, as rows in 64 bits."""
        for a in range(0, n, step):
            yield v[a:a + step].to(torch.float64)

    def slope_or_value(x, slope):
        """The activation function's value, or its slope, in 64 bits."""
        if case["act"] == "silu":
            e = 1.0 / (1.0 + torch.exp(-x))
            return e + x * e * (1.0 - e) if slope else x * e
        if case["act"] == "gelu":
            phi = 0.5 * torch.special.erfc(x * -(0.5 ** 0.5))
            return torch.exp(x.square() * -0.5).mul_((2.0 * math.pi) ** -0.5).mul_(x).add_(phi) if slope else x * phi
        return torch.ones_like(x) if slope else x

    def rounded(x):
        """Rows after their way through the 8-bit form, and their scales."""
        largest = x.abs().max(1)[0]
        unit = torch.maximum(largest / 127.0, torch.full_like(largest, TINY))
        return torch.round(x / unit[:, None]) * unit[:, None], unit

    def whole(parts):
        v = torch.cat(parts)
        if v.dim() == 1:
            return v.view(points)
        if len(points) == 1:
            return v
        return v.view(points + (v.shape[1],)).permute((0, len(points)) + tuple(range(1, len(points)))).contiguous()

    def dense(q, scale):
        return pieces_of(q.reshape(n, -1)[:, :C], scale.reshape(n))

    def pieces_of(q, scale):
        for a, b in zip(pieces(q), pieces(scale)):
            yield a * b[:, None]

    def as_rows(v):
        return v if v.dim() == 2 else v.permute((0,) + tuple(range(2, v.dim())) + (1,)).reshape(n, v.shape[1])

    if op == "store":
        parts = [[], [], [], []]
        for x in pieces(as_rows(s["x"])):
            for k, v in enumerate([slope_or_value(x, False), x] if case["keep"] else [slope_or_value(x, False)]):
                y, unit = rounded(v)
                parts[2 * k].append(y)
                parts[2 * k + 1].append(unit)
        out = {"values": whole(parts[0]), "scale": whole(parts[1])}
        if case["keep"]:
            out["kept"], out["kept_scale"] = whole(parts[2]), whole(parts[3])
        return out
    if op in ("linear", "bwd_input"):
        w = s["w"][:, :C].to(torch.float64) * s["wscale"].to(torch.float64)[:, None]
    if op == "linear":
        b = 0.0 if s["bias"] is None else s["bias"].to(torch.float64)
        return {"y": whole([torch.mm(x, w.t()).add_(b) for x in dense(s["q"], s["scale"])])}
    if op == "bwd_input":
        parts = [torch.mm(g, w) for g in pieces(as_rows(s["gy"]))]
        if case["act"] != "none":
            parts = [p.mul_(slope_or_value(x, True)) for p, x in zip(parts, dense(s["kept"], s["kept_scale"]))]
        return {"gx": whole(parts)}
    dw = torch.zeros((case["Co"], C), dtype=torch.float64, device=s["gy"].device)
    db = torch.zeros(case["Co"], dtype=torch.float64, device=s["gy"].device)
    for g, x in zip(pieces(as_rows(s["gy"])), dense(s["q"], s["scale"])):
        dw.addmm_(g.t(), x)
        db += g.sum(0)
    return {"dw": dw, "db": db} if case["bias"] else {"dw": dw}
