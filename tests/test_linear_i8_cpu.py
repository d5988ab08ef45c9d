"""Refusals of the channel products in 8-bit integers, and the replay of their index arithmetic, without a GPU.

Every argument is checked on the host before the device is looked at, so a refusal here never reaches one; calls whose
arguments are in order end at the device check (or, with no points, succeed)."""
import ctypes
import os
import subprocess

import pytest
import torch

import sparse_gather_contraction_amd as sgc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_gather_contraction_amd", "csrc")
F32, BF16, F16, I8 = sgc.DISCO_F32, sgc.DISCO_BF16, sgc.DISCO_F16, sgc.DISCO_I8


def desc(shape, dtype=BF16, ndim=None, data=0x1000):
    return sgc.TensorDesc(data, dtype, len(shape) if ndim is None else ndim, tuple(shape)[:5])


def status(name, *args):
    lib = sgc.load_library()
    st = getattr(lib, name)(*args)
    return sgc.STATUS_NAMES[st], lib.disco_last_error().decode()


X, Q, S = (2, 70, 3, 5), (2, 3, 5, 80), (2, 3, 5)
Y, W, WS = (2, 40, 3, 5), (40, 80), (40,)


def quant(x=desc(X), act=0, axis=1, q=desc(Q, I8), scale=desc(S, F32), k=None, ks=None):
    return status("disco_quantize_i8", x, act, axis, q, scale, k, ks, None)


def dequant(q=desc(Q, I8), scale=desc(S, F32), axis=1, out=desc(X)):
    return status("disco_dequantize_i8", q, scale, axis, out, None)


def linear(q=desc(Q, I8), scale=desc(S, F32), w=desc(W, I8), ws=desc(WS, F32), bias=None, axis=1, y=desc(Y)):
    return status("disco_linear_i8", q, scale, w, ws, bias, axis, y, None)


def grad_x(gy=desc(Y), w=desc(W, I8), ws=desc(WS, F32), act=0, k=None, ks=None, axis=1, gx=desc(X)):
    return status("disco_linear_i8_bwd_input", gy, w, ws, act, k, ks, axis, gx, None)


def grad_w(gy=desc(Y), q=desc(Q, I8), scale=desc(S, F32), axis=1, dw=desc((40, 70)), db=None):
    return status("disco_linear_i8_bwd_weight", gy, q, scale, axis, dw, db, 0x1000, 1 << 20, None)


K, KS = desc(Q, I8), desc(S, F32)
BAD = [
    (lambda: quant(x=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: quant(q=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: quant(scale=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: quant(act=1, k=K), "INVALID_ARGUMENT", "together"),
    (lambda: quant(act=1, ks=KS), "INVALID_ARGUMENT", "together"),
    (lambda: quant(k=K, ks=KS), "INVALID_ARGUMENT", "checkpoint"),
    (lambda: quant(act=3), "INVALID_ARGUMENT", "act"),
    (lambda: quant(act=-1), "INVALID_ARGUMENT", "act"),
    (lambda: quant(x=desc(X, I8)), "DTYPE", "x"),
    (lambda: quant(q=desc(Q, BF16)), "DTYPE", "q"),
    (lambda: quant(scale=desc(S, F16)), "DTYPE", "scale"),
    (lambda: quant(act=2, k=desc(Q, F32), ks=KS), "DTYPE", "kept"),
    (lambda: quant(q=desc((2, 3, 5, 70), I8)), "SHAPE", "expected 80"),
    (lambda: quant(q=desc((2, 3, 5, 96), I8)), "SHAPE", "expected 80"),
    (lambda: quant(q=desc((2, 5, 3, 80), I8)), "SHAPE", "q dimension 1"),
    (lambda: quant(scale=desc((2, 3, 4), F32)), "SHAPE", "scale dimension 2"),
    (lambda: quant(scale=desc((2, 3, 5, 1), F32)), "SHAPE", "number of dimensions"),
    (lambda: quant(q=desc((30, 80), I8)), "SHAPE", "number of dimensions"),
    (lambda: quant(axis=4), "SHAPE", "axis"),
    (lambda: quant(x=desc((2, 0, 3, 5))), "SHAPE", "along the axis"),
    (lambda: quant(x=desc((2, -70, 3, 5))), "SHAPE", "negative"),
    (lambda: quant(x=desc((1 << 20, 16, 1 << 11)), q=desc((1 << 20, 1 << 11, 16), I8), scale=desc((1 << 20, 1 << 11), F32)), "SHAPE", "points"),
    (lambda: dequant(out=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: dequant(out=desc(X, I8)), "DTYPE", "out"),
    (lambda: dequant(q=desc(Q, sgc.DISCO_F8_E4M3)), "DTYPE", "q"),
    (lambda: dequant(scale=desc(S, BF16)), "DTYPE", "scale"),
    (lambda: dequant(out=desc((2, 60, 3, 5))), "SHAPE", "expected 64"),
    (lambda: dequant(out=desc((2, 70, 5, 3))), "SHAPE", "dimension"),
    (lambda: linear(w=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: linear(y=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: linear(y=desc(Y, I8)), "DTYPE", "y"),
    (lambda: linear(q=desc(Q, F32)), "DTYPE", "q"),
    (lambda: linear(w=desc(W, BF16)), "DTYPE", "w"),
    (lambda: linear(ws=desc(WS, BF16)), "DTYPE", "wscale"),
    (lambda: linear(bias=desc(WS, BF16)), "DTYPE", "bias"),
    (lambda: linear(bias=desc((41,), F32)), "SHAPE", "bias"),
    (lambda: linear(w=desc((40, 64), I8)), "SHAPE", "w must be (40, 80)"),
    (lambda: linear(w=desc((39, 80), I8)), "SHAPE", "w must be (40, 80)"),
    (lambda: linear(ws=desc((39,), F32)), "SHAPE", "wscale"),
    (lambda: linear(q=desc((2, 3, 5, 72), I8), w=desc((40, 72), I8)), "SHAPE", "multiple of 16"),
    (lambda: linear(q=desc((2, 3, 5, 0), I8), w=desc((40, 0), I8)), "SHAPE", "at least 16"),
    (lambda: linear(q=desc((2, 3, 5, 131072), I8), w=desc((40, 131072), I8)), "SHAPE", "131056"),
    (lambda: linear(q=desc((30, 80), I8)), "SHAPE", "number of dimensions"),
    (lambda: linear(y=desc((2, 40, 3, 6))), "SHAPE", "points"),
    (lambda: linear(axis=-1), "SHAPE", "points"),
    (lambda: linear(q=desc((1 << 30, 16), I8), scale=desc((1 << 30,), F32), w=desc((1 << 28, 16), I8), ws=desc((1 << 28,), F32),
                    y=desc((1 << 30, 1 << 28))), "SHAPE", "workgroups"),
    (lambda: linear(q=desc((1, 16), I8), scale=desc((1,), F32), w=desc((1 << 28, 16), I8), ws=desc((1 << 28,), F32), y=desc((1, 1 << 28))),
     "SHAPE", "workgroups"),
    (lambda: grad_x(gx=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: grad_x(act=1), "INVALID_ARGUMENT", "checkpoint"),
    (lambda: grad_x(k=K, ks=KS), "INVALID_ARGUMENT", "checkpoint"),
    (lambda: grad_x(act=1, k=K), "INVALID_ARGUMENT", "together"),
    (lambda: grad_x(act=7, k=K, ks=KS), "INVALID_ARGUMENT", "act"),
    (lambda: grad_x(gy=desc(Y, F32)), "DTYPE", "gy"),
    (lambda: grad_x(gx=desc(X, F16)), "DTYPE", "dtypes differ"),
    (lambda: grad_x(w=desc(W, F32)), "DTYPE", "w"),
    (lambda: grad_x(act=2, k=desc(Q, BF16), ks=KS), "DTYPE", "kept"),
    (lambda: grad_x(w=desc((41, 80), I8)), "SHAPE", "w must be (40, 80)"),
    (lambda: grad_x(gx=desc((2, 81, 3, 5))), "SHAPE", "w must be (40, 96)"),
    (lambda: grad_x(gx=desc((2, 70, 3, 4))), "SHAPE", "gy dimension 3"),
    (lambda: grad_x(gy=desc((2, 40, 15))), "SHAPE", "number of dimensions"),
    (lambda: grad_x(gy=desc((2, 0, 3, 5))), "SHAPE", "along the axis"),
    (lambda: grad_x(act=1, k=desc((2, 3, 5, 96), I8), ks=KS), "SHAPE", "kept"),
    (lambda: grad_w(dw=None), "INVALID_ARGUMENT", "NULL"),
    (lambda: grad_w(gy=desc(Y, F32), dw=desc((40, 70), F32)), "DTYPE", "gy"),
    (lambda: grad_w(dw=desc((40, 70), F32)), "DTYPE", "dtypes differ"),
    (lambda: grad_w(db=desc((40,), F32)), "DTYPE", "dtypes differ"),
    (lambda: grad_w(q=desc(Q, BF16)), "DTYPE", "q"),
    (lambda: grad_w(dw=desc((41, 70))), "SHAPE", "dw"),
    (lambda: grad_w(dw=desc((40, 70, 1))), "SHAPE", "dw"),
    (lambda: grad_w(dw=desc((40, 60))), "SHAPE", "expected 64"),
    (lambda: grad_w(dw=desc((40, 0))), "SHAPE", "channels"),
    (lambda: grad_w(db=desc((39,))), "SHAPE", "db"),
    (lambda: grad_w(scale=desc((2, 3, 6), F32)), "SHAPE", "scale"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    call, want, word = BAD[i]
    st, msg = call()
    assert st == "DISCO_ERR_" + want and word in msg, (st, msg)


def test_a_tensor_without_points_is_accepted():
    x, q, s, y = desc((0, 70, 3, 5), data=None), desc((0, 3, 5, 80), I8, data=None), desc((0, 3, 5), F32, data=None), desc((0, 40, 3, 5), data=None)
    assert quant(x=x, q=q, scale=s)[0] == "DISCO_OK"
    assert dequant(q=q, scale=s, out=x)[0] == "DISCO_OK"
    assert linear(q=q, scale=s, y=y)[0] == "DISCO_OK"
    assert grad_x(gy=y, gx=x)[0] == "DISCO_OK"


def test_workspaces():
    lib, n = sgc.load_library(), ctypes.c_size_t()
    call = lib.disco_linear_i8_bwd_weight_workspace
    assert call(desc((2, 256, 721, 1440)), 1, 256, 1, n) == 0 and n.value == 256 * (256 * 256 + 256) * 4  # a split a CU
    assert call(desc((64, 256)), 1, 256, 1, n) == 0 and n.value == 0      # one step of points: no partial sums
    assert call(desc((0, 256)), 1, 256, 1, n) == 0 and n.value == 0
    assert call(desc((1 << 30, 8192)), 1, 8192, 0, n) == 0 and n.value == 0  # 1024 tiles fill the GPU
    assert sgc.STATUS_NAMES[call(desc((64, 256), F32), 1, 256, 1, n)] == "DISCO_ERR_DTYPE"
    assert sgc.STATUS_NAMES[call(desc((64, 256)), 2, 256, 1, n)] == "DISCO_ERR_SHAPE"
    assert sgc.STATUS_NAMES[call(desc((64, 256)), 1, 0, 1, n)] == "DISCO_ERR_SHAPE"
    assert sgc.STATUS_NAMES[call(None, 1, 16, 1, n)] == "DISCO_ERR_INVALID_ARGUMENT"


def test_binding_refuses_what_is_wrong():
    x = torch.zeros((6, 32))
    q, s = torch.zeros((6, 32), dtype=torch.int8), torch.ones(6)
    w, ws = torch.zeros((4, 32), dtype=torch.int8), torch.ones(4)
    gy = torch.zeros((6, 4), dtype=torch.bfloat16)
    for call in (lambda: sgc.disco_quantize_i8(x.t()), lambda: sgc.disco_dequantize_i8(q.t(), s), lambda: sgc.disco_linear_i8(q, s, w.t(), ws),
                 lambda: sgc.disco_linear_i8(q, s, w, ws, bias=torch.ones(8)[::2]), lambda: sgc.disco_linear_i8_bwd_input(gy.t(), w, ws),
                 lambda: sgc.disco_linear_i8_bwd_weight(gy, q.t(), s)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sgc.disco_quantize_i8(None), lambda: sgc.disco_quantize_i8(x, axis="1"), lambda: sgc.disco_dequantize_i8(q, 1.0),
                 lambda: sgc.disco_linear_i8(q, s, w, None), lambda: sgc.disco_linear_i8_bwd_input(gy, [w], ws),
                 lambda: sgc.disco_linear_i8_bwd_weight(gy, q, s, workspace=3)):
        with pytest.raises(TypeError):
            call()
    for call, want in ((lambda: sgc.disco_quantize_i8(x, act="relu"), "INVALID_ARGUMENT"), (lambda: sgc.disco_quantize_i8(x, act=["gelu"]), "INVALID_ARGUMENT"),
                       (lambda: sgc.disco_quantize_i8(x, keep=True), "INVALID_ARGUMENT"), (lambda: sgc.disco_quantize_i8(x.int()), "DTYPE"),
                       (lambda: sgc.disco_quantize_i8(x, axis=2), "SHAPE"), (lambda: sgc.disco_quantize_i8(x, axis=1 << 40), "SHAPE"),
                       (lambda: sgc.disco_quantize_i8(torch.tensor(1.0)), "SHAPE"), (lambda: sgc.disco_quantize_i8(x, q=x), "DTYPE"),
                       (lambda: sgc.disco_dequantize_i8(q, s, dtype=torch.int8), "DTYPE"), (lambda: sgc.disco_dequantize_i8(q, s, channels=40), "SHAPE"),
                       (lambda: sgc.disco_dequantize_i8(q, s, channels=-3), "SHAPE"), (lambda: sgc.disco_dequantize_i8(q, s, channels=0), "SHAPE"),
                       (lambda: sgc.disco_dequantize_i8(q, s, dtype=torch.float32, out=x.half()), "DTYPE"), (lambda: sgc.disco_linear_i8(q, s, w[:, :16].contiguous(), ws), "SHAPE"),
                       (lambda: sgc.disco_linear_i8(q, s, w, ws, axis=5), "SHAPE"), (lambda: sgc.disco_linear_i8(q, s, w, ws, dtype=torch.int32), "DTYPE"),
                       (lambda: sgc.disco_linear_i8(q, s, torch.tensor(1, dtype=torch.int8), ws), "SHAPE"),
                       (lambda: sgc.disco_linear_i8_bwd_input(gy, w, ws, act="gelu"), "INVALID_ARGUMENT"), (lambda: sgc.disco_linear_i8_bwd_input(gy.float(), w, ws), "DTYPE"),
                       (lambda: sgc.disco_linear_i8_bwd_input(gy, w, ws, channels=10), "SHAPE"), (lambda: sgc.disco_linear_i8_bwd_weight(gy, q, s, channels=50), "SHAPE"),
                       (lambda: sgc.disco_linear_i8_bwd_weight(gy, q, s[:5]), "SHAPE"), (lambda: sgc.disco_linear_i8_bwd_weight(gy, q, s, axis=3), "SHAPE"),
                       (lambda: sgc.disco_linear_i8_bwd_weight_workspace(gy.float(), 32), "DTYPE")):
        with pytest.raises(sgc.DiscoError) as e:
            call()
        assert e.value.status_name == "DISCO_ERR_" + want and str(e.value), e.value


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("linear_check") / "linear_check")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    os.path.join(CSRC, "linear_check.cpp"), "-o", exe], check=True)
    return exe


def test_every_access_of_the_kernels_lies_inside(checker):
    r = subprocess.run([checker], capture_output=True, text=True)
    assert r.returncode == 0 and "geometries checked" in r.stdout, r.stdout + r.stderr
