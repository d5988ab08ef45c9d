"""Refusals of the training-step operators, and the replay of their index arithmetic, without a GPU.

Every argument is checked on the host before the device is looked at, so a refusal here never reaches one; calls whose
arguments are in order end at the device check (or, with no elements, succeed)."""
import ctypes
import os
import subprocess

import pytest
import torch

import sparse_gather_contraction_amd as sgc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_gather_contraction_amd", "csrc")


def desc(shape, dtype=sgc.DISCO_BF16, ndim=None, data=0x1000):
    return sgc.TensorDesc(data, dtype, len(shape) if ndim is None else ndim, tuple(shape)[:5])


def status(name, *args):
    lib = sgc.load_library()
    st = getattr(lib, name)(*args)
    return sgc.STATUS_NAMES[st], lib.disco_last_error().decode()


X, W, S = (2, 64, 3, 5), (64,), (2, 1, 3, 5)
F8 = sgc.DISCO_F8_E4M3


def norm(x=desc(X), r=None, w=desc(W), axis=1, eps=1e-6, y=desc(X), h=None):
    return status("disco_rms_norm", x, r, w, axis, eps, y, h, None)


def norm8(x=desc(X), r=None, w=desc(W), axis=1, eps=1e-6, group=0, q=desc(X, F8), scale=desc(S, sgc.DISCO_F32), h=None):
    return status("disco_rms_norm_f8", x, r, w, axis, eps, group, q, scale, h, None)


def dequant(q=desc(X, F8), scale=desc(S, sgc.DISCO_F32), axis=1, group=0, out=desc(X)):
    return status("disco_dequantize", q, scale, axis, group, out, None)


def bwd(h=desc(X), w=desc(W), gy=desc(X), gh=None, axis=1, eps=1e-6, gx=desc(X), dw=desc(W)):
    return status("disco_rms_norm_bwd", h, w, gy, gh, axis, eps, gx, dw, 0x1000, 1 << 20, None)


BAD = [
    (lambda: norm(x=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: norm(w=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: norm(y=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: norm(r=desc(X)), "INVALID_ARGUMENT", "together"),
    (lambda: norm(h=desc(X)), "INVALID_ARGUMENT", "together"),
    (lambda: norm(x=desc(X, 99)), "DTYPE", "x"),
    (lambda: norm(x=desc(X, F8), y=desc(X, F8)), "DTYPE", "x"),
    (lambda: norm(y=desc(X, sgc.DISCO_F16)), "DTYPE", "y"),
    (lambda: norm(w=desc(W, sgc.DISCO_F16)), "DTYPE", "w"),
    (lambda: norm(r=desc(X, sgc.DISCO_F32), h=desc(X)), "DTYPE", "residual"),
    (lambda: norm(w=desc((63,))), "SHAPE", "w"),
    (lambda: norm(w=desc((64, 1))), "SHAPE", "w"),
    (lambda: norm(y=desc((2, 64, 3, 6))), "SHAPE", "y dimension 3 is 6, expected 5"),
    (lambda: norm(y=desc((2, 64, 15))), "SHAPE", "number of dimensions"),
    (lambda: norm(r=desc((2, 64, 4, 5)), h=desc(X)), "SHAPE", "residual"),
    (lambda: norm(axis=4), "SHAPE", "axis"),
    (lambda: norm(axis=-5), "SHAPE", "axis"),
    (lambda: norm(x=desc(X, ndim=6)), "SHAPE", "dimensions"),
    (lambda: norm(x=desc((), ndim=0)), "SHAPE", "dimensions"),
    (lambda: norm(x=desc((2, -64, 3, 5))), "SHAPE", "negative"),
    (lambda: norm(x=desc((1 << 40, 64, 1 << 20, 5))), "SHAPE", "too many"),
    (lambda: norm(x=desc((2, 0, 3, 5)), w=desc((0,)), y=desc((2, 0, 3, 5))), "SHAPE", "along the axis"),
    (lambda: norm(x=desc((1 << 34, 1)), w=desc((1,)), y=desc((1 << 34, 1))), "SHAPE", "workgroups"),
    (lambda: norm(eps=-1e-6), "INVALID_ARGUMENT", "eps"),
    (lambda: norm(eps=float("nan")), "INVALID_ARGUMENT", "eps"),
    (lambda: norm(eps=float("inf")), "INVALID_ARGUMENT", "eps"),
    (lambda: norm8(q=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: norm8(scale=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: norm8(q=desc(X)), "DTYPE", "q"),
    (lambda: norm8(scale=desc(S)), "DTYPE", "scale"),
    (lambda: norm8(group=16), "SHAPE", "group"),
    (lambda: norm8(group=-32), "SHAPE", "group"),
    (lambda: norm8(group=32), "SHAPE", "scale dimension 1 is 1, expected 2"),
    (lambda: norm8(scale=desc((2, 2, 3, 5), sgc.DISCO_F32)), "SHAPE", "scale"),
    (lambda: dequant(q=desc(X)), "DTYPE", "q"),
    (lambda: dequant(scale=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: dequant(scale=desc(S)), "DTYPE", "scale"),
    (lambda: dequant(out=desc(X, F8)), "DTYPE", "out"),
    (lambda: dequant(group=33), "SHAPE", "group"),
    (lambda: dequant(group=32), "SHAPE", "scale"),
    (lambda: dequant(out=desc((2, 64, 5, 3))), "SHAPE", "out"),
    (lambda: bwd(gy=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: bwd(gx=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: bwd(gy=desc(X, sgc.DISCO_F32)), "DTYPE", "gy"),
    (lambda: bwd(dw=desc(W, sgc.DISCO_F32)), "DTYPE", "dw"),
    (lambda: bwd(gh=desc((2, 64, 3, 4))), "SHAPE", "gh"),
    (lambda: bwd(dw=desc((65,))), "SHAPE", "dw"),
    (lambda: bwd(eps=-1.0), "INVALID_ARGUMENT", "eps"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    call, want, word = BAD[i]
    st, msg = call()
    assert st == "DISCO_ERR_" + want and word in msg, (st, msg)


def test_a_tensor_without_points_is_accepted():
    e = (0, 64, 3, 5)
    assert norm(x=desc(e, data=None), y=desc(e, data=None))[0] == "DISCO_OK"
    assert norm8(x=desc(e), q=desc(e, F8), scale=desc((0, 1, 3, 5), sgc.DISCO_F32))[0] == "DISCO_OK"
    assert dequant(q=desc(e, F8), scale=desc((0, 1, 3, 5), sgc.DISCO_F32), out=desc(e))[0] == "DISCO_OK"


def grads(*descs):
    return (sgc.TensorDesc * max(len(descs), 1))(*descs)


def clip(g, o=None, n=None, max_norm=1.0, eps=1e-6, norm=desc((1,), sgc.DISCO_F32)):
    a = grads(*g)
    b = a if o is None else grads(*o)
    return status("disco_clip_grads", len(g) if n is None else n, a, max_norm, eps, b, norm, 0x1000, 1 << 20, None)


G = desc((4, 4))
BAD_GRADS = [
    (lambda: clip([G], n=-1), "INVALID_ARGUMENT", "number"),
    (lambda: status("disco_grad_norm", 1, None, desc((1,), 0), 0x1000, 64, None), "INVALID_ARGUMENT", "NULL"),
    (lambda: status("disco_clip_grads", 1, grads(G), 1.0, 0.0, None, desc((1,), 0), 0x1000, 64, None), "INVALID_ARGUMENT", "outs"),
    (lambda: clip([G], norm=None), "INVALID_ARGUMENT", "norm"),
    (lambda: clip([G], norm=desc((1,))), "DTYPE", "norm"),
    (lambda: clip([G], norm=desc((2,), sgc.DISCO_F32)), "SHAPE", "norm"),
    (lambda: clip([G, desc((4,), F8)]), "DTYPE", "grads[1]"),
    (lambda: clip([G], o=[desc((4, 4), sgc.DISCO_F32)]), "DTYPE", "grads[0]"),
    (lambda: clip([G], o=[desc((4, 5))]), "SHAPE", "outs"),
    (lambda: clip([desc((4, -4))]), "SHAPE", "grads[0]"),
    (lambda: clip([desc((4, 4), ndim=6)]), "SHAPE", "grads[0]"),
    (lambda: clip([G], max_norm=-1.0), "INVALID_ARGUMENT", "max_norm"),
    (lambda: clip([G], max_norm=float("nan")), "INVALID_ARGUMENT", "max_norm"),
    (lambda: clip([G], eps=float("inf")), "INVALID_ARGUMENT", "eps"),
]


@pytest.mark.parametrize("i", range(len(BAD_GRADS)))
def test_refusals_of_gradients(i):
    call, want, word = BAD_GRADS[i]
    st, msg = call()
    assert st == "DISCO_ERR_" + want and word in msg, (st, msg)


def test_workspaces():
    lib, n = sgc.load_library(), ctypes.c_size_t()
    assert lib.disco_rms_norm_bwd_workspace(desc((2, 256, 721, 1440)), 1, n) == 0
    assert 0 < n.value <= 4096 * 256 * 4 and n.value % (256 * 4) == 0  # rows of D floats, one for each workgroup
    assert lib.disco_rms_norm_bwd_workspace(desc((0, 256)), 1, n) == 0 and n.value == 0
    assert sgc.STATUS_NAMES[lib.disco_rms_norm_bwd_workspace(desc((2, 256)), 2, n)] == "DISCO_ERR_SHAPE"
    assert lib.disco_grad_norm_workspace(0, None, n) == 0 and n.value == 8
    many = grads(*[desc((1 << 28,))] * 500)
    assert lib.disco_grad_norm_workspace(500, many, n) == 0 and 8 <= n.value <= 500 * 1024 * 8
    assert sgc.STATUS_NAMES[lib.disco_grad_norm_workspace(2, None, n)] == "DISCO_ERR_INVALID_ARGUMENT"


def test_binding_refuses_strided_tensors_and_a_short_output_list():
    a, w = torch.zeros((4, 6)), torch.ones(4)
    for call in (lambda: sgc.disco_rms_norm(a.t(), w), lambda: sgc.disco_rms_norm(a, w, residual=a.t()),
                 lambda: sgc.disco_rms_norm_f8(a.t(), w), lambda: sgc.disco_rms_norm_bwd(a, w, a.t()),
                 lambda: sgc.disco_rms_norm_bwd_workspace(a.t()), lambda: sgc.disco_clip_grads([a, a.t()], 1.0),
                 lambda: sgc.disco_grad_norm([a.t()]), lambda: sgc.disco_clip_grads([a], 1.0, out=[a.t()]),
                 lambda: sgc.disco_clip_grads([a, a], 1.0, out=[a])):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_what_is_no_tensor_and_passes_refusals_on():
    a, w = torch.zeros((4, 6)), torch.ones(6)
    for call in (lambda: sgc.disco_rms_norm(None, w), lambda: sgc.disco_rms_norm([1.0], w), lambda: sgc.disco_rms_norm(a, w, axis="1"),
                 lambda: sgc.disco_clip_grads([a, 3], 1.0), lambda: sgc.disco_grad_norm(3), lambda: sgc.disco_clip_grads([a], "x")):
        with pytest.raises(TypeError):
            call()
    for call, want in ((lambda: sgc.disco_rms_norm(a.long(), w), "DTYPE"), (lambda: sgc.disco_rms_norm(a, w, axis=5), "SHAPE"),
                       (lambda: sgc.disco_rms_norm(a, w, axis=1 << 40), "SHAPE"), (lambda: sgc.disco_rms_norm(a, torch.ones(5), axis=1), "SHAPE"),
                       (lambda: sgc.disco_rms_norm(a, w, axis=1, h=a), "INVALID_ARGUMENT"), (lambda: sgc.disco_rms_norm_f8(a, w, axis=-3), "SHAPE"),
                       (lambda: sgc.disco_rms_norm_f8(a, w, dtype=torch.int8), "DTYPE"), (lambda: sgc.disco_rms_norm_f8(a, w, group=-32), "SHAPE"),
                       (lambda: sgc.disco_rms_norm_f8(a, w, q=a), "DTYPE"), (lambda: sgc.disco_dequantize(a, a), "DTYPE"),
                       (lambda: sgc.disco_dequantize(a, a, dtype=torch.int8), "DTYPE"), (lambda: sgc.disco_rms_norm_bwd(a, w, a.half()), "DTYPE"),
                       (lambda: sgc.disco_rms_norm_bwd(a, w, a, axis=2), "SHAPE"), (lambda: sgc.disco_grad_norm([a, a.int()]), "DTYPE"),
                       (lambda: sgc.disco_clip_grads([a], -1.0), "INVALID_ARGUMENT"), (lambda: sgc.disco_clip_grads([a], 1.0, out=[a.half()]), "DTYPE")):
        with pytest.raises(sgc.DiscoError) as e:
            call()
        assert e.value.status_name == "DISCO_ERR_" + want and str(e.value), e.value


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("norm_check") / "norm_check")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    os.path.join(CSRC, "norm_check.cpp"), "-o", exe], check=True)
    return exe


def test_every_access_of_the_norm_kernels_lies_inside(checker):
    r = subprocess.run([checker], capture_output=True, text=True)
    assert r.returncode == 0 and "geometries checked" in r.stdout, r.stdout + r.stderr


def test_the_workspace_of_long_rows_stays_small():
    lib, n = sgc.load_library(), ctypes.c_size_t()
    for rows, D in ((100000, 1 << 20), (5000, 40000), (40000, 20000), (33, 1 << 26)):
        assert lib.disco_rms_norm_bwd_workspace(desc((rows, D)), 1, n) == 0
        # fp64 sums of dw for the chunks of rows that fill the GPU (2048 x 256 threads of 8 columns, or one row), rstd
        assert D * 8 <= n.value <= max(2048 * 256 * 8, D) * 8 + rows * 4, (rows, D, n.value)


@pytest.mark.parametrize("shape", [(6, 4), (24,), (4, 6, 1), (1, 4, 6)], ids=str)
def test_binding_refuses_outputs_of_another_shape(shape):
    # as many elements, laid out otherwise: a gradient's transpose among them
    a = torch.zeros((4, 6))
    for grads, out in (([a], [torch.zeros(shape)]), ([a, a.clone()], [torch.zeros((4, 6)), torch.zeros(shape)])):
        with pytest.raises(sgc.DiscoError) as e:
            sgc.disco_clip_grads(grads, 1.0, out=out)
        assert e.value.status_name == "DISCO_ERR_SHAPE" and f"out[{len(out) - 1}]" in str(e.value)


def test_binding_holds_the_tensors_of_its_lists():
    # `out` is walked after the gradients: what its walk does to the list of gradients must not free them
    from torch.multiprocessing.reductions import StorageWeakRef

    grads = [torch.zeros(1000 + i) for i in range(3)]
    kept = [StorageWeakRef(g.untyped_storage()) for g in grads]
    seen = []

    class Out:
        def __iter__(self):
            grads.clear()
            seen.extend(k.expired() for k in kept)
            return iter([torch.zeros(1000 + i) for i in range(3)])

    with pytest.raises(sgc.DiscoError):  # host memory
        sgc.disco_clip_grads(grads, 1.0, out=Out())
    assert seen == [False] * 3 and all(k.expired() for k in kept)


def test_a_given_output_of_another_dtype_than_asked_for_is_refused():
    a, w, s = torch.zeros((4, 6)), torch.ones(6), torch.ones((4, 1))
    q = a.to(torch.float8_e4m3fn)
    for call in (lambda: sgc.disco_rms_norm_f8(a, w, axis=1, dtype=torch.float8_e5m2, q=q),
                 lambda: sgc.disco_dequantize(q, s, dtype=torch.float32, out=a.half()),
                 lambda: sgc.disco_dequantize(q, s, dtype=torch.int8, out=a.to(torch.int8))):
        with pytest.raises(sgc.DiscoError) as e:
            call()
        assert e.value.status_name == "DISCO_ERR_DTYPE", e.value
