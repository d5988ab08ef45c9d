"""The operators around the convolution in a training step (norm, 8-bit norm and its reader, norm backward, gradient
norm and clipping) against their formulas in fp64.

Bounds.  u = 2^-24 is half a step of fp32, half(t) half a step of the output's type, both relative.  A sum of fp32 terms
along a chain of n additions is off by at most n u times the sum of the terms' sizes; the kernels' chains (a thread's
terms, the lanes, the workgroup's parts) are shorter than 80 for every size used here.  So the mean of squares is
off by 80 u, its inverse root by 40 u and 2 u of its own, y by 45 u and the rounding of the output; the other bounds
count the same way beside each check.  fp16 results below its normal range are off by up to 2^-25 beside that."""
import math

import pytest
import torch

import sparse_gather_contraction_amd as sgc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10), "e5m2": (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}
U = 2.0 ** -24
EPS = 1e-6


def half(dt):
    return torch.finfo(dt).eps / 2


def floor_of(dt):
    return 2.0 ** -25 if dt == torch.float16 else 1e-40


def randn(shape, dt, seed, std=1.0, shift=0):
    """A tensor that starts `shift` elements into its storage."""
    g = torch.Generator().manual_seed(seed)
    n = math.prod(shape)
    flat = (torch.randn(n + shift, generator=g) * std).to(dt).to(DEV)
    return flat[shift:].view(shape)


def per(w, x, axis):
    s = [1] * x.dim()
    s[axis] = -1
    return w.view(s)


def close(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape
    assert bool(torch.isfinite(got).all()), what + ": non-finite"
    worst = float(((got - ref).abs() / bound).max()) if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst} times its bound"


SHAPES = [  # (shape, axis): fields with aligned, odd and tiny grids, rows of every kind, middle axes
    ((1, 1), -1), ((3, 5), -1), ((1, 256), -1), ((67, 8), -1), ((5, 9), -1), ((33, 260), -1), ((129, 512), -1), ((17, 1000), -1),
    ((9, 1025), -1), ((5, 2048), -1), ((3, 4100), -1), ((3, 8191), -1), ((2, 16385), -1), ((2, 70001), -1), ((1029, 7), -1),
    ((2, 1, 8, 16), 1), ((2, 3, 5, 7), 1), ((1, 8, 1, 1), 1), ((3, 73, 9, 11), 1), ((2, 32, 18, 36), 1), ((1, 80, 13, 41), 1),
    ((2, 256, 8, 17), 1), ((1, 257, 3, 43), 1), ((1, 512, 9, 16), 1), ((1, 1000, 8, 9), 1), ((1, 2048, 8, 8), 1), ((1, 2500, 5, 13), 1),
    ((300, 4, 3), 1), ((64, 33, 2), 1), ((4, 6, 50), 0), ((2, 3, 40, 5), 2), ((70,), 0), ((2, 16, 4, 5, 6), 1), ((1, 32, 400, 333), 1),
]


def ids(v):
    return "x".join(map(str, v[0])) + f"@{v[1]}"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", SHAPES, ids=ids)
def test_norm(case, dtype):
    shape, axis = case
    dt = T[dtype]
    for shift, residual, wdt in ((0, True, torch.float32), (1, False, dt)):
        print(f"[norm] {shape} axis {axis} {dtype} shift {shift} residual {residual}", flush=True)
        x, r = randn(shape, dt, 1, 2.0, shift), randn(shape, dt, 2, 1.0, shift) if residual else None
        w = randn((shape[axis],), wdt, 3, 1.0, shift)
        got = sgc.disco_rms_norm(x, w, residual=r, axis=axis, eps=EPS)
        y, h = got if residual else (got, None)
        H = x.double() + (r.double() if residual else 0)
        ref = H * (H.square().mean(axis, keepdim=True) + EPS).rsqrt() * per(w.double(), x, axis)
        close(y, ref, ref.abs() * (half(dt) + 46 * U) * 1.001 + floor_of(dt), "y")
        if residual:
            close(h, H, H.abs() * (half(dt) + U) * 1.001 + floor_of(dt), "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", SHAPES, ids=ids)
def test_norm_f8_and_reader(case, dtype):
    shape, axis = case
    dt = T[dtype]
    D = shape[axis]
    for shift, residual, f8, group in ((0, True, "e4m3", 0), (1, False, "e4m3", 128), (0, False, "e5m2", 32), (1, True, "e4m3", 96)):
        print(f"[f8] {shape} axis {axis} {dtype} shift {shift} residual {residual} {f8} group {group}", flush=True)
        qt, qmax, qhalf, qfloor = F8[f8]
        x, r = randn(shape, dt, 11, 2.0, shift), randn(shape, dt, 12, 1.0, shift) if residual else None
        w = randn((D,), torch.float32, 13, 1.0, shift)
        got = sgc.disco_rms_norm_f8(x, w, residual=r, axis=axis, eps=EPS, group=group, dtype=qt)
        q, scale = got[0], got[1]
        H = x.double() + (r.double() if residual else 0)
        if residual:
            close(got[2], H, H.abs() * (half(dt) + U) * 1.001 + floor_of(dt), "h")
        Y = H * (H.square().mean(axis, keepdim=True) + EPS).rsqrt() * per(w.double(), x, axis)
        g = group or D
        for k, (ys, qs) in enumerate(zip(Y.split(g, axis), q.float().split(g, axis))):
            ref = (ys.abs().amax(axis, keepdim=True) / qmax).clamp(min=2.0 ** -126)
            mine = scale.narrow(axis, k, 1)
            close(mine, ref, ref * 48 * U, "scale")  # y's 46 u, the quotient's rounding
            v = ys / ref
            close(qs, v, v.abs() * (qhalf + 100 * U) + qfloor, "q")  # y and scale perturb v by 96 u
            for out in (torch.float32, torch.bfloat16, torch.float16):
                back = sgc.disco_dequantize(q, scale, dtype=out, axis=axis, group=group).narrow(axis, k * g, ys.shape[axis])
                ref2 = qs.double() * mine.double()
                close(back, ref2, ref2.abs() * half(out) * 1.001 + floor_of(out), "reader")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", SHAPES, ids=ids)
def test_norm_bwd(case, dtype):
    shape, axis = case
    dt = T[dtype]
    for shift, with_gh, wdt in ((0, True, dt), (1, False, torch.float32)):
        print(f"[bwd] {shape} axis {axis} {dtype} shift {shift} gh {with_gh}", flush=True)
        h, gy = randn(shape, dt, 21, 2.0, shift), randn(shape, dt, 22, 1.0, shift)
        gh = randn(shape, dt, 23, 1.0, shift) if with_gh else None
        w = randn((shape[axis],), wdt, 24, 1.0, shift)
        gx, dw = sgc.disco_rms_norm_bwd(h, w, gy, gh=gh, axis=axis, eps=EPS)
        H, G = h.double(), gy.double() * per(w.double(), h, axis)
        rstd = (H.square().mean(axis, keepdim=True) + EPS).rsqrt()
        mean, size = (G * H).mean(axis, keepdim=True), (G * H).abs().mean(axis, keepdim=True)
        a, b, c = rstd * G, H * rstd ** 3 * mean, gh.double() if with_gh else torch.zeros_like(H)
        ref = a - b + c
        # rstd 42 u and two products; rstd^3 126 u and four products, the mean's own 82 u of its terms' sizes; two sums
        bound = U * (46 * a.abs() + 134 * b.abs() + 84 * H.abs() * rstd ** 3 * size + 3 * (a.abs() + b.abs() + c.abs()))
        close(gx, ref, ref.abs() * half(dt) * 1.001 + bound + floor_of(dt), "gx")
        terms = gy.double() * H * rstd
        dims = [i for i in range(h.dim()) if i != axis % h.dim()]
        rdw, sdw = (terms.sum(dims), terms.abs().sum(dims)) if dims else (terms, terms.abs())
        # each term 44 u; chains of at most 200 additions in fp32, then fp64
        close(dw, rdw, rdw.abs() * half(wdt) * 1.001 + 244 * U * sdw + floor_of(wdt), "dw")


def bwd_reference(h, w, gy, gh, axis):
    """gx, the bound of its fp32 steps, dw and the sum of its terms' sizes, by the formula in fp64."""
    H, G = h.double(), gy.double() * per(w.double(), h, axis)
    rstd = (H.square().mean(axis, keepdim=True) + EPS).rsqrt()
    mean, size = (G * H).mean(axis, keepdim=True), (G * H).abs().mean(axis, keepdim=True)
    a, b, c = rstd * G, H * rstd ** 3 * mean, gh.double() if gh is not None else torch.zeros_like(H)
    bound = U * (46 * a.abs() + 134 * b.abs() + 84 * H.abs() * rstd ** 3 * size + 3 * (a.abs() + b.abs() + c.abs()))
    terms = gy.double() * H * rstd
    dims = [i for i in range(h.dim()) if i != axis % h.dim()]
    return a - b + c, bound, terms.sum(dims), terms.abs().sum(dims)


@pytest.mark.parametrize("scale", [2.0 ** 50, 2.0 ** -50])
@pytest.mark.parametrize("case", [((40, 256), -1), ((2, 32, 16, 16), 1), ((9, 24, 3), 1), ((3, 20000), -1)], ids=ids)
def test_norm_bwd_of_large_and_small_values(case, scale):
    # rstd^3 leaves fp32's range at 2^50 where h^2 does not; at 2^-50 eps alone is left of the mean
    shape, axis = case
    print(f"[bwd] {shape} axis {axis} scale {scale}", flush=True)
    for dt in (torch.float32, torch.bfloat16):
        h, gy, gh = randn(shape, dt, 111, 2.0) * scale, randn(shape, dt, 112), randn(shape, dt, 113) / scale
        w = randn((shape[axis],), torch.float32, 114)
        gx, dw = sgc.disco_rms_norm_bwd(h, w, gy, gh=gh, axis=axis, eps=EPS)
        ref, bound, rdw, sdw = bwd_reference(h, w, gy, gh, axis)
        close(gx, ref, ref.abs() * half(dt) * 1.001 + bound + 1e-40, "gx")
        close(dw, rdw, rdw.abs() * U * 1.001 + 244 * U * sdw + 1e-40, "dw")


# Outputs beyond the sizes from which stores go past the L2: whole sectors, runs that end inside a sector, an
# unaligned base, rows.
LARGE = [((1, 256, 512, 520), 1, 0), ((1, 72, 721, 1441), 1, 0), ((1, 256, 512, 520), 1, 3), ((40000, 512), -1, 0), ((40000, 511), -1, 0), ((70001, 264), -1, 1)]


@pytest.mark.parametrize("case", LARGE, ids=lambda v: ids(v) + f"+{v[2]}")
def test_large_outputs(case):
    shape, axis, shift = case
    print(f"[large] {shape} axis {axis} shift {shift}", flush=True)
    dt = torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(121)
    n = math.prod(shape)
    x, r, gy = (torch.randn(n + shift, generator=gen, dtype=dt, device=DEV)[shift:].view(shape) for _ in range(3))
    w = randn((shape[axis],), torch.float32, 122)
    y, h = (torch.empty(n + shift, dtype=dt, device=DEV)[shift:].view(shape) for _ in range(2))
    sgc.disco_rms_norm(x, w, residual=r, axis=axis, eps=EPS, y=y, h=h)
    q, scale, h8 = sgc.disco_rms_norm_f8(x, w, residual=r, axis=axis, eps=EPS)
    back = sgc.disco_dequantize(q, scale, axis=axis)
    gx, dw = sgc.disco_rms_norm_bwd(h, w, gy, gh=r, axis=axis, eps=EPS, gx=torch.empty_like(h) if shift == 0 else y.clone())
    assert torch.equal(h8, h)
    total = torch.zeros(shape[axis], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(total)
    cut = 0 if axis == -1 else 2  # in pieces: the fp64 intermediates are large
    for lo in range(0, shape[cut], -(-shape[cut] // 8)):
        k = min(-(-shape[cut] // 8), shape[cut] - lo)
        X, R, GY, Y, H, B, GX = (t.narrow(cut, lo, k) for t in (x, r, gy, y, h, back, gx))
        S = X.double() + R.double()
        close(H, S, S.abs() * (half(dt) + U) * 1.001 + 1e-40, "h")
        ref = S * (S.square().mean(axis, keepdim=True) + EPS).rsqrt() * per(w.double(), S, axis)
        close(Y, ref, ref.abs() * (half(dt) + 46 * U) * 1.001 + 1e-40, "y")
        top = ref.abs().amax(axis, keepdim=True)
        close(B, ref, ref.abs() * (2 ** -4 + 2 ** -8) * 1.01 + top / 448 * 2.0 ** -10 * 1.01, "back")
        gref, bound, rdw, sdw = bwd_reference(H, w, GY, R, axis)
        close(GX, gref, gref.abs() * half(dt) * 1.001 + bound + 1e-40, "gx")
        total += rdw
        size += sdw
    close(dw, total, total.abs() * U * 1.001 + 244 * U * size + 1e-40, "dw")


def test_norm_bwd_against_differences():
    # the directional derivative of <gy, y> + <gh, h> in x and in w, by central differences in fp64 of the formula
    shape = (2, 24, 9, 15)
    h, gy, gh = (randn(shape, torch.float32, s) for s in (31, 32, 33))
    w = randn((24,), torch.float32, 34)
    gx, dw = sgc.disco_rms_norm_bwd(h, w, gy, gh=gh, axis=1, eps=EPS)

    def loss(h, w):
        y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * per(w, h, 1)
        return float((gy.double() * y).sum() + (gh.double() * h).sum())

    dx, dv = randn(shape, torch.float32, 35).double(), randn((24,), torch.float32, 36).double()
    s = 2.0 ** -12  # the difference's own error is of the order s^2, 6e-8 of the third derivative
    fx = (loss(h.double() + s * dx, w.double()) - loss(h.double() - s * dx, w.double())) / (2 * s)
    fw = (loss(h.double(), w.double() + s * dv) - loss(h.double(), w.double() - s * dv)) / (2 * s)
    assert abs(float((gx.double() * dx).sum()) - fx) <= 1e-5 * float((gx.double() * dx).abs().sum())
    assert abs(float((dw.double() * dv).sum()) - fw) <= 1e-5 * float((dw.double() * dv).abs().sum())


@pytest.mark.parametrize("case", [((40, 256), -1), ((40, 1000), -1), ((2, 32, 16, 16), 1), ((3, 20000), -1), ((1, 5000, 4, 16), 1), ((9, 24, 3), 1)], ids=ids)
def test_norm_special_values(case):
    shape, axis = case
    dt = torch.bfloat16
    x = randn(shape, dt, 41)
    view = x.movedim(axis, -1)  # (..., D): the points in front
    pts = [tuple(i) for i in torch.cartesian_prod(*[torch.arange(s) for s in view.shape[:-1]]).view(-1, view.dim() - 1).tolist()][:3]
    view[pts[0]][:] = 0.0
    view[pts[1]][1] = float("nan")
    view[pts[2]][2] = float("inf")
    w = randn((shape[axis],), torch.float32, 42)
    X = x.double()
    ref = (X * (X.square().mean(axis, keepdim=True) + EPS).rsqrt() * per(w.double(), x, axis)).movedim(axis, -1)
    y = sgc.disco_rms_norm(x, w, axis=axis, eps=EPS).movedim(axis, -1)
    assert bool((y[pts[0]] == 0).all())
    assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.isinf(), ref.isinf())
    q, scale = sgc.disco_rms_norm_f8(x, w, axis=axis, eps=EPS)
    qv, sv = q.float().movedim(axis, -1), scale.movedim(axis, -1)
    assert bool((qv[pts[0]] == 0).all()) and float(sv[pts[0]][0]) == 2.0 ** -126
    for p in pts[1:]:
        assert bool(qv[p].isnan().all()) and bool(sv[p].isnan().all())
    assert int(sv.isnan().sum()) == 2
    gy = randn(shape, dt, 43)
    gx, dw = sgc.disco_rms_norm_bwd(x, w, gy, axis=axis, eps=EPS)
    bad = gx.movedim(axis, -1).isnan().any(-1)
    assert int(bad.sum()) == 2 and bool(bad[pts[1]]) and bool(bad[pts[2]])
    assert bool(dw.isnan().any())


def test_f8_of_huge_weights():
    # y beyond fp32's range: infinite scales, as amax / qmax gives them, and quotients of 0 and NaN
    x = torch.ones((2, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    x[0, 5] = 2.0
    w[5] = 3.0e38
    q, scale = sgc.disco_rms_norm_f8(x, w, axis=-1, group=32)
    y = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w).view(2, 2, 32)
    ref_s = (y.abs().amax(2) / 448.0).clamp(min=2.0 ** -126)
    assert torch.equal(scale.isinf(), ref_s.isinf()) and torch.equal(scale.isnan(), ref_s.isnan())
    ref_q = (y / ref_s.unsqueeze(2)).view(2, 64)
    assert torch.equal(q.float().isnan(), ref_q.isnan())
    fine = ~ref_q.isnan()
    assert torch.equal((q.float() == 0)[fine], (ref_q.to(torch.float8_e4m3fn).float() == 0)[fine])


def test_every_f8_code_is_read():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    for qt in (torch.float8_e4m3fn, torch.float8_e5m2):
        ref = codes.view(qt).float()
        for shape in ((1, 256), (1, 2, 128)):
            q = codes.view(shape).to(DEV).view(qt)
            s = torch.full((1, 1) if len(shape) == 2 else (1, 1, 128), 2.0, device=DEV)
            out = sgc.disco_dequantize(q, s, dtype=torch.float32, axis=1).cpu().flatten()
            assert torch.equal(out.isnan(), ref.isnan())
            assert torch.equal(out[~ref.isnan()], (2 * ref)[~ref.isnan()])


def test_norm_empty_and_strided():
    w = torch.ones(4, device=DEV)
    x = torch.empty((0, 4, 3), device=DEV)
    assert sgc.disco_rms_norm(x, w).shape == x.shape
    gx, dw = sgc.disco_rms_norm_bwd(x, w, x)
    assert gx.shape == x.shape and bool((dw == 0).all())
    with pytest.raises(ValueError):
        sgc.disco_rms_norm(torch.ones((3, 2, 4), device=DEV).movedim(1, 2), w)


def test_outputs_may_not_overlap():
    x = torch.ones((8, 32), device=DEV)
    w = torch.ones(32, device=DEV)
    for call in (lambda: sgc.disco_rms_norm(x, w, axis=-1, y=x),
                 lambda: sgc.disco_rms_norm(x, w, residual=x, axis=-1, h=x),
                 lambda: sgc.disco_rms_norm_bwd(x, w, x, axis=-1, gx=x),
                 lambda: sgc.disco_rms_norm_bwd(x, w, x, axis=-1, dw=w),
                 lambda: sgc.disco_clip_grads([x, w], 1.0, out=[torch.empty_like(x), x.view(-1)[:32]]),
                 lambda: sgc.disco_clip_grads([x, x], 1.0)):
        with pytest.raises(sgc.DiscoError) as e:
            call()
        assert e.value.status_name == "DISCO_ERR_INVALID_ARGUMENT" and "overlap" in str(e.value)
    torch.cuda.synchronize()
    assert bool((x == 1).all()) and bool((w == 1).all())


LISTS = [[1], [0], [5, 0, 7], [257] * 9, [1 << 20, 3, 70001, 12], [2048, 2049, 4095, 4097], [17] * 130, [3] * 400, [5000] * 260, [9_000_001]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda v: f"{len(v)}x{v[0]}")
def test_grad_norm_and_clip(sizes, dtype):
    print(f"[clip] {len(sizes)} tensors of {sizes[0]}.. {dtype}", flush=True)
    flat = {d: randn((sum(sizes) + 1,), T[d], 51, 0.5) for d in T}
    grads, at = [], 1  # views into flat buffers: no start is aligned
    for i, n in enumerate(sizes):
        grads.append(flat[dtype if dtype != "mixed" else ("f32", "bf16", "f16")[i % 3]][at:at + n])
        at += n
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm = sgc.disco_grad_norm(grads)
    assert norm.shape == () and abs(float(norm) - ref) <= 2 * U * ref  # fp64 sums, one rounding
    for max_norm in (ref / 3 + 1e-3, 1e30):
        factor = min(1.0, max_norm / (ref + EPS))
        outs = [torch.full_like(g, float("nan")) for g in grads]
        n2 = sgc.disco_clip_grads(grads, max_norm, out=outs)
        assert float(n2) == float(norm)
        for g, o in zip(grads, outs):
            r = g.double() * factor
            close(o, r, r.abs() * (half(g.dtype) + 4 * U) * 1.001 + floor_of(g.dtype), "out")  # the factor 3 u, the product 1
        mine = [g.clone() for g in grads]
        sgc.disco_clip_grads(mine, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gap", [0, 5])
def test_gradients_in_one_buffer(dtype, gap):
    # tensors that follow each other are walked as one run; the result may not depend on the outputs' places
    sizes = [3, 257, 0, 70001, 8192, 5, 44_000_000 if gap == 0 else 100_001, 9001]
    print(f"[clip] one buffer {dtype} gap {gap}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(131)
    flat = torch.randn(sum(sizes) + gap * len(sizes), generator=gen, device=DEV).to(T[dtype])
    at = [sum(sizes[:i]) + gap * i for i in range(len(sizes))]
    grads = [flat[a:a + n] for a, n in zip(at, sizes)]
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm = sgc.disco_grad_norm(grads)
    assert abs(float(norm) - ref) <= 2 * U * ref
    factor = min(1.0, 0.25 / (ref + EPS))
    into = torch.full_like(flat, 7.0)
    apart = [torch.empty_like(g) for g in grads]
    n1 = sgc.disco_clip_grads(grads, 0.25, out=[into[a:a + n] for a, n in zip(at, sizes)])
    n2 = sgc.disco_clip_grads(grads, 0.25, out=apart)
    assert float(n1) == float(norm) == float(n2)
    for g, a, n, o in zip(grads, at, sizes, apart):
        r = g.double() * factor
        close(o, r, r.abs() * (half(g.dtype) + 4 * U) * 1.001 + floor_of(g.dtype), "out")
        assert torch.equal(into[a:a + n], o) and bool((into[a + n:a + n + gap] == 7).all())
    n3 = sgc.disco_clip_grads(grads, 0.25)
    assert float(n3) == float(norm) and all(torch.equal(g, o) for g, o in zip(grads, apart))


def test_grad_norm_of_none_and_of_extremes():
    assert float(sgc.disco_grad_norm([])) == 0.0
    assert float(sgc.disco_clip_grads([], 1.0)) == 0.0
    big = torch.full((3,), 1e30, device=DEV)  # squares beyond fp32's range
    assert abs(float(sgc.disco_grad_norm([big])) / (1e30 * math.sqrt(3)) - 1) <= 2 ** -22
    small = torch.full((4,), 1e-40, device=DEV)  # and below it
    assert abs(float(sgc.disco_grad_norm([small])) / 2e-40 - 1) <= 2 ** -5  # a subnormal norm has few bits
    for bad in (float("nan"), float("inf")):
        g = torch.ones(70000, device=DEV)
        g[6] = bad
        n = sgc.disco_clip_grads([g], 1.0)
        ref = torch.tensor(bad)
        assert torch.equal(n.cpu().isnan(), ref.isnan()) and torch.equal(n.cpu().isinf(), ref.isinf())
        assert bool(g.isnan().all()) if bad != bad else (bool(g[6].isnan()) and bool((g[7:] == 0).all()))


def test_results_repeat_and_streams():
    x, gy = randn((2, 96, 40, 51), torch.bfloat16, 61), randn((2, 96, 40, 51), torch.bfloat16, 62)
    w = randn((96,), torch.float32, 63)
    first = [*sgc.disco_rms_norm(x, w, residual=gy), *sgc.disco_rms_norm_bwd(x, w, gy, gh=gy),
             sgc.disco_grad_norm([x, gy])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in streams:
        with torch.cuda.stream(s):
            runs.append([*sgc.disco_rms_norm(x, w, residual=gy), *sgc.disco_rms_norm_bwd(x, w, gy, gh=gy),
                         sgc.disco_grad_norm([x, gy])])
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_graph_replays():
    x, r = randn((2, 80, 20, 33), torch.bfloat16, 71), randn((2, 80, 20, 33), torch.bfloat16, 72)
    w = randn((80,), torch.float32, 73)

    def step():
        y, h = sgc.disco_rms_norm(x, w, residual=r)
        q, s, h2 = sgc.disco_rms_norm_f8(x, w, residual=r, group=32)
        back = sgc.disco_dequantize(q, s, group=32)
        gx, dw = sgc.disco_rms_norm_bwd(h, w, y, gh=back)
        outs = [torch.empty_like(gx), torch.empty_like(dw)]
        n = sgc.disco_clip_grads([gx, dw], 0.5, out=outs)
        return [y, h, q.view(torch.uint8), s, back, gx, dw, n, *outs]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(randn(x.shape, torch.bfloat16, 80 + k))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), f"replay {k}"


def test_graph_replays_of_small_calls():
    # the forms of one launch: a backward of one tile, gradients that one workgroup sums and scales
    x, gy = randn((4, 617), torch.bfloat16, 141), randn((4, 617), torch.bfloat16, 142)
    w = randn((617,), torch.float32, 143)

    def step():
        gx, dw = sgc.disco_rms_norm_bwd(x, w, gy, axis=-1)
        outs = [torch.empty_like(gx), torch.empty_like(dw)]
        return [gx, dw, sgc.disco_grad_norm([gx, dw]), sgc.disco_clip_grads([gx, dw], 0.5, out=outs), *outs]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(randn(x.shape, torch.bfloat16, 150 + k))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), f"replay {k}"


@pytest.mark.parametrize("sizes", [[16384], [16385], [8192, 8192], [8193, 8191], [2000] * 8, [2000] * 9, [1] * 8, [1] * 9], ids=str)
def test_clip_at_the_border_of_one_workgroup(sizes):
    print(f"[clip] {sizes}", flush=True)
    grads = [randn((n,), torch.float32, 160 + i, 0.5) for i, n in enumerate(sizes)]  # apart from each other
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    factor = min(1.0, 0.125 / (ref + EPS))
    whole = torch.empty(sum(sizes), device=DEV)
    for outs in (list(whole.split(sizes)), [torch.empty_like(g) for g in grads]):
        n = sgc.disco_clip_grads(grads, 0.125, out=outs)
        assert float(n) == float(sgc.disco_grad_norm(grads)) and abs(float(n) - ref) <= 2 * U * ref
        for g, o in zip(grads, outs):
            r = g.double() * factor
            close(o, r, r.abs() * (half(g.dtype) + 4 * U) * 1.001 + 1e-40, "out")


def test_offsets_beyond_32_bits():
    # 3 x (2^30 + 72) points of bf16: byte offsets pass 2^32 and element offsets 2^31
    M = (1 << 30) + 72
    x = torch.empty((1, 3, M), dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(5))
    w = randn((3,), torch.float32, 91)
    y = sgc.disco_rms_norm(x, w)
    q, s = sgc.disco_rms_norm_f8(x, w)
    back = sgc.disco_dequantize(q, s)
    gx, dw = sgc.disco_rms_norm_bwd(x, w, x)
    torch.cuda.synchronize()
    for lo in (0, M // 2, M - 4096):
        c = slice(lo, lo + 4096)
        H = x[..., c].double()
        rstd = (H.square().mean(1, keepdim=True) + EPS).rsqrt()
        W = w.double().view(1, 3, 1)
        ref = H * rstd * W
        close(y[..., c], ref, ref.abs() * (half(torch.bfloat16) + 46 * U) * 1.001 + 1e-40, "y")
        top = ref.abs().amax(1, keepdim=True)
        close(back[..., c], ref, ref.abs() * (2 ** -4 + 2 ** -8) * 1.01 + top / 448 * 2.0 ** -10 * 1.01, "back")
        a, b = rstd * H * W, H * rstd ** 3 * (H * H * W).mean(1, keepdim=True)
        size = (H * H * W).abs().mean(1, keepdim=True)
        bound = U * (49 * a.abs() + 137 * b.abs() + 84 * H.abs() * rstd ** 3 * size)
        close(gx[..., c], a - b, (a - b).abs() * half(torch.bfloat16) * 1.001 + bound + 1e-40, "gx")
    del y, q, s, back, gx
    n = float(sgc.disco_grad_norm([x]))
    ref = math.sqrt(sum(float(x[0, i, j:j + (1 << 28)].double().square().sum()) for i in range(3) for j in range(0, M, 1 << 28)))
    assert abs(n - ref) <= 2 * U * ref


# Rows in registers with one group, groups joined over lanes and through LDS, several vectors a thread, single
# elements; columns, flat tiles; the looping kernels.
QUOTIENTS = [((300, 512), -1, 128), ((300, 512), -1, 0), ((99, 1000), -1, 96), ((40, 4100), -1, 64), ((1029, 7), -1, 0), ((3, 70001), -1, 128),
             ((2, 80, 13, 41), 1, 0), ((1, 257, 9, 43), 1, 32), ((64, 66, 3), 1, 32), ((1, 2500, 5, 13), 1, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", QUOTIENTS, ids=lambda v: ids(v) + f"g{v[2]}")
def test_f8_codes_are_the_quotients_by_the_stored_scale(case, dtype):
    # Whole numbers up to 8 (e4m3) and 14 (e5m2) with weights of 1: the sums of squares are exact in any order, so the
    # fp32 norm of the same numbers gives the y that the 8-bit form rounds, and multiples of 448 / 8 and 57344 / 14 are
    # often half way between two codes, where the last bit of y / scale decides.  The quotient is rounded once to fp32
    # and that once to 8 bits.
    shape, axis, group = case
    for f8, top in (("e4m3", 8), ("e5m2", 14)):
        print(f"[quotients] {shape} axis {axis} group {group} {dtype} {f8}", flush=True)
        qt, qmax = F8[f8][0], F8[f8][1]
        gen = torch.Generator().manual_seed(171)
        x = torch.randint(-top, top + 1, shape, generator=gen).to(T[dtype]).to(DEV)
        w = torch.ones(shape[axis], device=DEV)
        y = sgc.disco_rms_norm(x.float(), w, axis=axis, eps=EPS).cpu()
        q, scale = (t.cpu() for t in sgc.disco_rms_norm_f8(x, w, axis=axis, eps=EPS, group=group, dtype=qt))
        g = group or shape[axis]
        for k, ys in enumerate(y.split(g, axis)):
            s = (ys.abs().amax(axis, keepdim=True) / qmax).clamp(min=2.0 ** -126)
            assert torch.equal(scale.narrow(axis, k, 1), s)
            assert torch.equal(q.narrow(axis, k * g, ys.shape[axis]).float(), (ys / s).to(qt).float())


# dw over many rows of long axes: rows in registers with four vectors a thread (fp32 and 16 bits), the looping kernel
# with more tiles than workgroups and a last round that is not full, over rows and over columns.
LONG = [((2500, 16390), -1), ((9, 20000), -1), ((3000, 20011), -1), ((700, 8201), -1), ((600, 32776), -1), ((1, 1040, 96, 97), 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LONG, ids=ids)
def test_dw_of_long_axes(case, dtype):
    # Against the formula, and in a workspace of NaN and one of large values: nothing of it may be taken over.
    shape, axis = case
    print(f"[long dw] {shape} axis {axis} {dtype}", flush=True)
    dt = T[dtype]
    gen = torch.Generator(device=DEV).manual_seed(181)
    h, gy, gh = (torch.randn(shape, generator=gen, device=DEV).to(dt) for _ in range(3))
    w = randn((shape[axis],), torch.float32, 182)
    need = sgc.disco_rms_norm_bwd_workspace(h, axis=axis)
    first = None
    for fill in (255, 0x7e):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        got = sgc.disco_rms_norm_bwd(h, w, gy, gh=gh, axis=axis, eps=EPS, workspace=ws)
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    gx, dw = first
    total = torch.zeros(shape[axis], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(total)
    cut = 0 if axis == -1 else 2  # in pieces: the fp64 intermediates are large
    for lo in range(0, shape[cut], -(-shape[cut] // 8)):
        k = min(-(-shape[cut] // 8), shape[cut] - lo)
        H, GY, GH, GX = (t.narrow(cut, lo, k) for t in (h, gy, gh, gx))
        ref, bound, rdw, sdw = bwd_reference(H, w, GY, GH, axis)
        close(GX, ref, ref.abs() * half(dt) * 1.001 + bound + 1e-40, "gx")
        total += rdw
        size += sdw
    # each term 44 u, summed in fp64
    close(dw, total, total.abs() * U * 1.001 + 50 * U * size + 1e-40, "dw")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", [((15616, 16390), -1), ((15616, 9000), -1), ((15616, 20000), -1), ((1, 1040, 704, 710), 1)], ids=ids)
def test_dw_of_long_axes_keeps_small_terms(case, dtype):
    # |h| = 1, so rstd is one number r just below 1 and every term is r gy.  A large term in the first tile of each of
    # 256 workgroups, then 60 small ones, each 3/8 of a step of the large one: an fp32 sum over the tiles drops them all
    # (22 u), fp64 keeps them.  r is off by 3 u (mean 1 u, root 2 u), a term by 1 u more, the sum of a vector's or a
    # wave's equal terms by nothing (powers of two of them), the result is rounded once: 5 u.
    shape, axis = case
    print(f"[small terms] {shape} axis {axis} {dtype}", flush=True)
    dt = T[dtype]
    D = shape[axis]
    points, many, big, small = math.prod(shape) // D, 8192 if axis == 1 else 256, 2.0 ** 12, 1.5 * 2.0 ** -14
    h = torch.ones(shape, dtype=dt, device=DEV)
    gy = torch.full(shape, small, dtype=dt, device=DEV)
    (gy.view(D, -1)[:, :many] if axis == 1 else gy[:many])[:] = big
    _, dw = sgc.disco_rms_norm_bwd(h, torch.ones(D, device=DEV), gy, axis=axis, eps=EPS)
    ref = (many * big + (points - many) * small) / math.sqrt(1 + EPS)
    worst = float((dw.double() / ref - 1).abs().max())
    assert worst <= 5 * U, worst / U


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", [((1, 64, 361, 720), 1), ((3, 73, 91, 181), 1), ((1, 300, 128, 129), 1), ((6000, 24, 3), 1), ((40960, 512), -1), ((4096, 1), -1),
                                  ((4, 617), -1), ((512, 9000), -1), ((256, 40000), -1), ((1, 2050, 64, 128), 1), ((1, 2050, 64, 128), 1, 2)],
                         ids=lambda v: ids(v) + "+" * (len(v) - 2))
def test_dw_of_sums_that_cancel(case, dtype):
    # |h| = 1, so every term is r gy with one number r: 2^12 and -2^12 in the first and third quarters of the points,
    # 1.5 2^-14 in the others.  The large terms cancel, so dw is the small ones' sum if every sum on the way keeps them;
    # rounded to fp32 anywhere (in a vector, over lanes, in a workgroup, between launches) it is off by the large ones'
    # half steps.  With a stride of 2 every second point is small in the large quarters too (the looping kernel).  r is off
    # by 3 u, a term by 1 u more, the result is rounded once.
    shape, axis, step = case if len(case) == 3 else (*case, 1)
    print(f"[cancel] {shape} axis {axis} {dtype}", flush=True)
    dt = T[dtype]
    D = shape[axis]
    points = math.prod(shape) // D
    quarter = points // 4 // 64 * 64 if points >= 256 else points // 4
    small = 1.5 * 2.0 ** -14
    gy = torch.full((points,), small, dtype=dt, device=DEV)
    gy[:quarter:step] = 2.0 ** 12
    gy[2 * quarter:3 * quarter:step] = -2.0 ** 12
    many = int((gy == small).sum()) if dt == torch.float32 else points - 2 * len(range(0, quarter, step))
    gy = gy.view([s for i, s in enumerate(shape) if i != axis % len(shape)]).unsqueeze(axis).expand(shape).contiguous()
    _, dw = sgc.disco_rms_norm_bwd(torch.ones_like(gy), torch.ones(D, device=DEV), gy, axis=axis, eps=EPS)
    ref = many * small / math.sqrt(1 + EPS)
    worst = float((dw.double() / ref - 1).abs().max())
    assert worst <= 5 * U, worst / U


def test_dw_of_very_long_axes():
    # 2^26 columns and more: 16 a workgroup of 1024 threads are more threads than a launch has
    D = (1 << 26) + 3
    e, w = torch.empty((0, D), dtype=torch.bfloat16, device=DEV), torch.ones(D, device=DEV)
    dw = torch.full((D,), float("nan"), device=DEV)
    sgc.disco_rms_norm_bwd(e, w, e, axis=1, dw=dw)
    assert bool((dw == 0).all())
    shape = (1, (1 << 20) + 77, 2)  # more columns than that launch's workgroups take at once
    h, gy = randn(shape, torch.bfloat16, 191), randn(shape, torch.bfloat16, 192)
    w = randn((shape[1],), torch.float32, 193)
    gx, dw = sgc.disco_rms_norm_bwd(h, w, gy, axis=1, eps=EPS)
    # chains of 2^20 / 32 terms and a tree of 32 in the sums over the axis: 32773 u of their terms' sizes; the root half
    # of that, and the bounds of test_norm_bwd follow with 16387 and 32775 in the place of 40 and 82
    H, G = h.double(), gy.double() * per(w.double(), h, 1)
    rstd = (H.square().mean(1, keepdim=True) + EPS).rsqrt()
    mean, size = (G * H).mean(1, keepdim=True), (G * H).abs().mean(1, keepdim=True)
    a, b = rstd * G, H * rstd ** 3 * mean
    bound = U * (16396 * a.abs() + 49170 * b.abs() + 32780 * H.abs() * rstd ** 3 * size)
    close(gx, a - b, (a - b).abs() * half(torch.bfloat16) * 1.001 + bound + 1e-40, "gx")
    terms = gy.double() * H * rstd
    close(dw, terms.sum((0, 2)), U * (1 + 16396) * terms.abs().sum((0, 2)) + 1e-40, "dw")


@pytest.mark.parametrize("n", [5, 70000])
def test_clip_factor_at_its_limits(n):
    print(f"[clip] limits of {n}", flush=True)
    inf, nan = float("inf"), float("nan")

    def clip(values, max_norm, eps=EPS):
        g = torch.ones(n, device=DEV) * values[0]
        g[3] = values[-1]
        out = torch.full_like(g, 7.0)
        norm = float(sgc.disco_clip_grads([g], max_norm, out=[out], eps=eps))
        mine = g.clone()
        sgc.disco_clip_grads([mine], max_norm, eps=eps)
        assert torch.equal(mine.isnan(), out.isnan()) and torch.equal(mine[~mine.isnan()], out[~out.isnan()])
        return norm, out

    norm, out = clip([0.0], 0.0, eps=0.0)  # 0 / 0: there is nothing to clip
    assert norm == 0 and bool((out == 0).all())
    norm, out = clip([2.0], 0.0, eps=0.0)
    assert bool((out == 0).all())
    for max_norm in (1.0, inf, 1e300):  # an infinite norm makes finite elements 0, also where no limit is set
        norm, out = clip([2.0, -inf], max_norm)
        assert norm == inf and bool(out[3].isnan()) and bool((out[4:] == 0).all()) and bool((out[:3] == 0).all())
    norm, out = clip([2.0], inf)
    assert bool((out == 2).all())
    for max_norm in (0.0, 1.0, inf):
        norm, out = clip([2.0, nan], max_norm)
        assert norm != norm and bool(out.isnan().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [6, 70001])
def test_clip_by_a_factor_below_the_normal_range(n, dtype):
    # gradients of 1e37 by factors of 1e-40 and less: the products are ordinary numbers (but the last, which is below the
    # normal range: half a subnormal step, 2^-150 in fp32 and 2^-134 in bf16).  The factor 3 u, the product 1.
    print(f"[clip] tiny factors {n} {dtype}", flush=True)
    g = (randn((n,), torch.float32, 201) * 1e37).to(T[dtype])
    g[-1] = 1.5
    total = float(g.double().square().sum().sqrt())
    for max_norm in (1e-3, 1e-6, 1e-12):
        ref = g.double() * (max_norm / (total + EPS))
        for src, out in ((g, torch.empty_like(g)), 2 * (g.clone(),)):
            sgc.disco_clip_grads([src], max_norm, out=[out])
            close(out, ref, ref.abs() * (half(T[dtype]) + 4 * U) * 1.001 + (2.0 ** -150 if dtype == "f32" else 2.0 ** -134), "out")


def test_written_tensors_count_as_changed_in_place():
    x, w = randn((40, 64), torch.bfloat16, 211), randn((64,), torch.float32, 212)
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)
    y, h, gx, dw = e(40, 64), e(40, 64), e(40, 64), e(64, dt=torch.float32)
    q, scale, out = e(40, 64, dt=torch.float8_e4m3fn), e(40, 1, dt=torch.float32), e(40, 64)
    versions = [t._version for t in (x, w, y, h, gx, dw, q, scale, out)]
    sgc.disco_rms_norm(x, w, residual=x, axis=-1, y=y, h=h)
    sgc.disco_rms_norm_f8(x, w, axis=-1, q=q, scale=scale)
    sgc.disco_dequantize(q, scale, axis=-1, out=out)
    sgc.disco_rms_norm_bwd(h, w, y, axis=-1, gx=gx, dw=dw)
    assert [t._version for t in (x, w, y, h, gx, dw, q, scale, out)] == [v + (i >= 2) for i, v in enumerate(versions)]
    sgc.disco_grad_norm([gx, dw])
    outs = [torch.empty_like(gx), torch.empty_like(dw)]
    before = [t._version for t in (gx, dw, *outs)]
    sgc.disco_clip_grads([gx, dw], 1e-3, out=outs)
    sgc.disco_clip_grads([gx], 1e-3)
    assert [t._version for t in (gx, dw, *outs)] == [before[0] + 1, before[1], before[2] + 1, before[3] + 1]
    leaf = torch.ones(64, device=DEV, requires_grad=True)
    saved = torch.full((64,), 3.0, device=DEV)
    loss = (leaf * saved).sum()
    sgc.disco_clip_grads([saved], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # tensors without a count
        t = torch.full((64,), 3.0, device=DEV)
    sgc.disco_clip_grads([t], 1e-3)
    assert float(t[0]) < 1


BWD_PATHS = [((259, 512), -1), ((40, 9000), -1), ((40, 20000), -1), ((20, 40000), -1), ((2, 80, 20, 33), 1), ((900, 24, 3), 1), ((1, 1040, 96, 97), 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", BWD_PATHS, ids=ids)
def test_bwd_workspace_at_fp32_alignment(case, dtype):
    # four bytes past an allocation's start is alignment enough, and nothing outside of the workspace is written
    shape, axis = case
    print(f"[workspace] {shape} axis {axis} {dtype}", flush=True)
    h, gy = randn(shape, T[dtype], 221), randn(shape, T[dtype], 222)
    w = randn((shape[axis],), torch.float32, 223)
    want = sgc.disco_rms_norm_bwd(h, w, gy, axis=axis, eps=EPS)
    need = sgc.disco_rms_norm_bwd_workspace(h, axis=axis)
    ws = torch.full((need + 68,), 0x5a, dtype=torch.uint8, device=DEV)
    got = sgc.disco_rms_norm_bwd(h, w, gy, axis=axis, eps=EPS, workspace=ws[4:4 + need])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((ws[:4] == 0x5a).all()) and bool((ws[4 + need:] == 0x5a).all())
    with pytest.raises(sgc.DiscoError):
        sgc.disco_rms_norm_bwd(h, w, gy, axis=axis, eps=EPS, workspace=ws[:need - 1])


@pytest.mark.parametrize("case", BWD_PATHS, ids=ids)
def test_graph_replays_of_the_backward(case):
    shape, axis = case
    print(f"[graph] {shape} axis {axis}", flush=True)
    h, gy = randn(shape, torch.bfloat16, 231), randn(shape, torch.bfloat16, 232)
    w = randn((shape[axis],), torch.float32, 233)
    sgc.disco_rms_norm_bwd(h, w, gy, gh=gy, axis=axis)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = sgc.disco_rms_norm_bwd(h, w, gy, gh=gy, axis=axis)
    for k in range(4):
        h.copy_(randn(shape, torch.bfloat16, 240 + k))
        graph.replay()
        torch.cuda.synchronize()
        eager = sgc.disco_rms_norm_bwd(h, w, gy, gh=gy, axis=axis)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), f"replay {k}"
