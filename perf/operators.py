"""Workloads of the operators that surround the spherical convolution in a residual model's training step.

Five operators: the root-mean-square norm of x + residual ("norm"), the same with an 8-bit output and
scales ("norm8"), the norm's backward ("bwd"), the 8-bit form's reader ("dequant"), and the global norm of
many gradients with clipping ("clip").  A case of the first four is a dense tensor whose normalised axis is
axis 1: fields (B, C, H, W) are normalised over the channels of each grid point, rows (rows, C) over the row.

With ``own`` false, ``run`` evaluates the plain form in fp32 torch operations; with ``own`` true it calls
``sparse_gather_contraction_amd``.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
TINY = 2.0 ** -126  # smallest scale: the reciprocal of a smaller one leaves fp32's range
MAX_ELEMENTS = 2 * 256 * 721 * 1440
MAX_PARAMS = 1 << 28


def listed():
    return [
        # one grid point's 256 channels: the norm inside a point-wise head; the call's latency is all that counts
        {"name": "norm_one_row_bf16", "op": "norm", "shape": "1x256", "dtype": "bf16", "weight": "bf16", "residual": True},
        # fields of the fp32 training workload, 181x360 with 32 channels and batch 4
        {"name": "norm_181x360_f32", "op": "norm", "shape": "4x32x181x360", "dtype": "f32", "weight": "f32", "residual": True},
        # residual stream of the 256-channel model at 721x1440, batch 2
        {"name": "norm_721x1440_bf16", "op": "norm", "shape": "2x256x721x1440", "dtype": "bf16", "weight": "f32", "residual": True},
        # an 80-channel input field kept in 8 bits, one scale per grid point
        {"name": "norm8_721x1440_80", "op": "norm8", "shape": "1x80x721x1440", "dtype": "bf16", "weight": "f32", "residual": True,
         "f8": "e4m3", "group": 0},
        # channels-last rows of the 512-channel model (360x720 points), a scale for each 128 channels
        {"name": "norm8_rows_512", "op": "norm8", "shape": "259200x512", "dtype": "f16", "weight": "f16", "residual": False,
         "f8": "e4m3", "group": 128},
        # backward at an odd, ragged regional grid: no row of it is aligned to 16 bytes
        {"name": "bwd_odd_91x181", "op": "bwd", "shape": "3x73x91x181", "dtype": "bf16", "weight": "bf16", "residual": True},
        # backward of the fp32 training workload
        {"name": "bwd_181x360_f32", "op": "bwd", "shape": "4x32x181x360", "dtype": "f32", "weight": "f32", "residual": True},
        # backward of the 256-channel model at 721x1440, batch 2
        {"name": "bwd_721x1440_bf16", "op": "bwd", "shape": "2x256x721x1440", "dtype": "bf16", "weight": "f32", "residual": True},
        # the kept 8-bit field read back for the convolution's backward
        {"name": "dequant_721x1440_80", "op": "dequant", "shape": "1x80x721x1440", "dtype": "bf16", "f8": "e4m3", "group": 0},
        # channels-last rows read back, a scale for each 128 channels
        {"name": "dequant_rows_512", "op": "dequant", "shape": "259200x512", "dtype": "f16", "f8": "e4m3", "group": 128},
        # one step's gradients of a 12-block model with 256x256x16 convolution weights: they fit the last-level cache
        {"name": "clip_12_blocks", "op": "clip", "tensors": 25, "params": 12 * 256 * 256 * 16 + 13 * 257, "dtype": "bf16",
         "max_norm": 1.0, "write": True},
        # gradients of a large fp32 model in 400 tensors: far beyond every cache
        {"name": "clip_400_tensors_f32", "op": "clip", "tensors": 400, "params": MAX_PARAMS, "dtype": "f32", "max_norm": 1.0,
         "write": True},
    ]


def _size(rng, low, high):
    """A whole number whose logarithm is uniform in [low, high]; every second one is made odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    if rng.random() < 0.5 and v % 2 == 0 and v > low:
        v -= 1
    return v if v != 3 << 10 else v - 1


def draw(rng):
    op = rng.choice(["norm", "norm8", "bwd", "dequant", "clip"])
    if op == "clip":
        params = _size(rng, 256, MAX_PARAMS)
        return {"op": op, "tensors": min(_size(rng, 1, 400), params // 2), "params": params, "dtype": rng.choice(list(DTYPES)),
                "max_norm": rng.choice([1.0, 1.0, 1e30]), "write": rng.random() < 0.75}
    while True:
        if rng.random() < 0.6:
            dims = [rng.randint(1, 4), _size(rng, 1, 512), _size(rng, 1, 721), _size(rng, 1, 1440)]
        else:
            dims = [_size(rng, 1, 262144), _size(rng, 1, 8192)]
        if math.prod(dims) <= MAX_ELEMENTS // 2:
            break
    case = {"op": op, "shape": "x".join(map(str, dims)), "dtype": rng.choice(list(DTYPES))}
    if op != "dequant":
        case["weight"] = rng.choice(["f32", case["dtype"]])
        case["residual"] = rng.random() < 0.7
    if op in ("norm8", "dequant"):
        case["f8"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        case["group"] = rng.choice([0, 32, 64, 128])
    return case


def _shape(case):
    return tuple(int(v) for v in case["shape"].split("x"))


def _groups(case):
    D = _shape(case)[1]
    return 1 if not case["group"] else -(-D // case["group"])


def _sizes(case):
    """Elements of each gradient: weights in the even places, small vectors (norm weights, biases) in the odd ones."""
    n, total = case["tensors"], case["params"]
    big = (n + 1) // 2
    small = min(257, total // (2 * n))
    rest = total - (n - big) * small
    each = [rest // big + (1 if i < rest % big else 0) for i in range(big)]
    return [each[i // 2] if i % 2 == 0 else small for i in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(shape, dtype, std=1.0):
        t = torch.randn(shape, generator=gen, dtype=torch.float32 if dtype == "f32" else DTYPES[dtype], device=dev)
        return t.mul_(std) if std != 1.0 else t

    if case["op"] == "clip":
        # gradients are consecutive views of one flat buffer, as gradient buckets hold them
        sizes = _sizes(case)
        flat = normal((sum(sizes),), case["dtype"], 1.0 if case["dtype"] == "f16" else 0.02)  # fp16 ones carry a loss scale
        out = torch.empty_like(flat)
        return {"case": case, "flat": flat, "out": out, "grads": list(flat.split(sizes)), "outs": list(out.split(sizes))}
    shape, dt = _shape(case), case["dtype"]
    per_channel = (1, shape[1]) + (1,) * (len(shape) - 2)
    spread = torch.empty(per_channel, device=dev).uniform_(0.25, 4.0, generator=gen)  # channels differ in size
    s = {"case": case}
    if case["op"] == "dequant":
        s["q"] = normal(shape, "bf16", 64.0).clamp_(-448.0, 448.0).to(F8[case["f8"]][0])
        s["scale"] = torch.empty((shape[0], _groups(case)) + shape[2:], device=dev).uniform_(0.001, 0.02, generator=gen)
        return s
    s["w"] = torch.empty(shape[1], device=dev).uniform_(0.5, 1.5, generator=gen).to(DTYPES[case["weight"]])
    s["x"] = normal(shape, dt).mul_(spread.to(DTYPES[dt]))
    s["r"] = normal(shape, dt) if case["residual"] else None
    if case["op"] == "bwd":
        s["gy"] = normal(shape, dt, 0.125)
    return s


def _per_channel(w, x):
    return w.view((1, -1) + (1,) * (x.dim() - 2))


def _over_groups(v, case):
    """v (N, D, ...) as (N, G, group, ...), zeros past D."""
    g = case["group"] or v.shape[1]
    G = _groups(case)
    if G * g != v.shape[1]:
        v = torch.cat([v, v.new_zeros((v.shape[0], G * g - v.shape[1]) + tuple(v.shape[2:]))], 1)
    return v.reshape((v.shape[0], G, g) + tuple(v.shape[2:]))


def _from_groups(v, D):
    return v.flatten(1, 2)[:, :D].contiguous()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip":
        total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
        if case["write"]:
            coef = torch.clamp(case["max_norm"] / (total + EPS), max=1.0).float()
            [o.copy_(g.float() * coef) for o, g in zip(s["outs"], s["grads"])]
        return {"norm": total.float(), "out": s["out"] if case["write"] else None}
    if op == "dequant":
        v = _over_groups(s["q"].float(), case) * s["scale"].unsqueeze(2)
        return {"out": _from_groups(v, s["q"].shape[1]).to(DTYPES[case["dtype"]])}
    x, w, dt = s["x"], _per_channel(s["w"].float(), s["x"]), DTYPES[case["dtype"]]
    if op == "bwd":  # x is the sum that the forward stored, r the gradient that reaches that sum by the residual path
        h, gy = x.float(), s["gy"].float()
        rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        g = gy * w
        gx = rstd * g - h * (rstd.pow(3) * (g * h).mean(1, keepdim=True))
        if s["r"] is not None:
            gx = gx + s["r"].float()
        dw = (gy * h * rstd).sum([0] + list(range(2, h.dim())), dtype=torch.float64)
        return {"gx": gx.to(dt), "dw": dw.to(s["w"].dtype)}
    h = x.float() if s["r"] is None else x.float() + s["r"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
    stored = None if s["r"] is None else h.to(dt)
    if op == "norm":
        return {"y": y.to(dt), "h": stored}
    f8, qmax = F8[case["f8"]]
    v = _over_groups(y, case)
    scale = (v.abs().amax(2) / qmax).clamp(min=TINY)
    return {"q": _from_groups(v / scale.unsqueeze(2), y.shape[1]).to(f8), "scale": scale, "h": stored}


def _own(s):
    import sparse_gather_contraction_amd as sgc

    case = s["case"]
    op = case["op"]
    if op == "clip":
        if not case["write"]:
            return {"norm": sgc.disco_grad_norm(s["grads"]), "out": None}
        return {"norm": sgc.disco_clip_grads(s["grads"], case["max_norm"], out=s["outs"]), "out": s["out"]}
    if op == "dequant":
        return {"out": sgc.disco_dequantize(s["q"], s["scale"], dtype=DTYPES[case["dtype"]], axis=1, group=case["group"])}
    if op == "bwd":
        gx, dw = sgc.disco_rms_norm_bwd(s["x"], s["w"], s["gy"], gh=s["r"], axis=1, eps=EPS)
        return {"gx": gx, "dw": dw}
    if op == "norm":
        y = sgc.disco_rms_norm(s["x"], s["w"], residual=s["r"], axis=1, eps=EPS)
        return {"y": y, "h": None} if s["r"] is None else {"y": y[0], "h": y[1]}
    q = sgc.disco_rms_norm_f8(s["x"], s["w"], residual=s["r"], axis=1, eps=EPS, group=case["group"], dtype=F8[case["f8"]][0])
    return {"q": q[0], "scale": q[1], "h": None if s["r"] is None else q[2]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    esz = 4 if case["dtype"] == "f32" else 2
    if op == "clip":
        n = case["params"]
        return {"bytes": n * esz * (2 if case["write"] else 1) + 4, "flops": n * (3 if case["write"] else 2)}
    shape = _shape(case)
    n = math.prod(shape)
    if op == "dequant":
        return {"bytes": n * (1 + esz) + 4 * n // shape[1] * _groups(case), "flops": n}
    w = shape[1] * (4 if case["weight"] == "f32" else esz)
    r = 1 if case["residual"] else 0
    if op == "norm":
        return {"bytes": n * esz * (2 + 2 * r) + w, "flops": n * (4 + r)}
    if op == "norm8":
        return {"bytes": n * (esz * (1 + 2 * r) + 1) + 4 * n // shape[1] * _groups(case) + w, "flops": n * (6 + r)}
    return {"bytes": n * esz * (3 + r) + 2 * w, "flops": n * (11 + r)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        g = s["flat"].to(torch.float64)
        norm = torch.sqrt(torch.dot(g, g))
        if not case["write"]:
            return {"norm": norm, "out": None}
        factor = min(1.0, case["max_norm"] / (norm.item() + EPS))
        return {"norm": norm, "out": g.mul_(factor)}
    D = _shape(case)[1]
    if op == "dequant":
        v = s["q"].to(torch.float64)
        for k in range(_groups(case)):
            a, b = (0, D) if not case["group"] else (k * case["group"], min(D, (k + 1) * case["group"]))
            v[:, a:b].mul_(s["scale"][:, k:k + 1].to(torch.float64))
        return {"out": v}
    parts = [[] for _ in range(4)]
    dw = torch.zeros(D, dtype=torch.float64, device=s["x"].device)
    w = s["w"].to(torch.float64)
    step = max(1, (1 << 27) // max(1, math.prod(_shape(case)[1:])))
    for n0 in range(0, _shape(case)[0], step):  # the first axis in pieces: the 64-bit intermediates are large
        x = s["x"][n0:n0 + step].to(torch.float64).flatten(2) if len(_shape(case)) > 2 else s["x"][n0:n0 + step].to(torch.float64).unsqueeze(2)
        r = None if s["r"] is None else s["r"][n0:n0 + step].to(torch.float64).reshape(x.shape)
        if op != "bwd" and r is not None:
            x += r
        inv = (x * x).sum(1).div_(D).add_(EPS).pow_(-0.5)
        u = x * inv[:, None]  # the normalised rows
        if op == "bwd":
            gy = s["gy"][n0:n0 + step].to(torch.float64).reshape(x.shape)
            dw += (gy * u).sum((0, 2))
            gy *= w[None, :, None]
            proj = (gy * u).sum(1).div_(D)
            gy -= u.mul_(proj[:, None])
            gy *= inv[:, None]
            parts[0].append(gy if r is None else gy.add_(r))
            continue
        if r is not None:
            parts[3].append(x)
        u *= w[None, :, None]
        if op == "norm":
            parts[0].append(u)
            continue
        f8, qmax = F8[case["f8"]]
        scales = []
        for k in range(_groups(case)):
            a, b = (0, D) if not case["group"] else (k * case["group"], min(D, (k + 1) * case["group"]))
            sc = u[:, a:b].abs().max(1)[0].div_(qmax).clamp_(min=TINY)
            u[:, a:b] /= sc[:, None]
            scales.append(sc)
        parts[0].append(u.to(f8).to(torch.float64))
        parts[1].append(torch.stack(scales, 1))

    def whole(p, like):
        return torch.cat(p).reshape(like) if p else None

    shape = _shape(case)
    if op == "bwd":
        return {"gx": whole(parts[0], shape), "dw": dw}
    if op == "norm":
        return {"y": whole(parts[0], shape), "h": whole(parts[3], shape)}
    return {"q": whole(parts[0], shape), "scale": whole(parts[1], (shape[0], _groups(case)) + shape[2:]), "h": whole(parts[3], shape)}
