"""Python binding of libdisco.so — argument marshalling only.

Every step of the DISCO contraction runs in the library's HIP kernels; this
module turns torch tensors into ``disco_tensor`` views (device pointer, dtype,
shape), passes torch's current HIP stream, and raises on a non-OK status.
The names mirror the C ABI in ``include/disco.h``:

    psi = disco_psi_create(csr, device)      # csr: K, Ho, Wo, Hi, Wi, row_ptr, col_hi, col_wi, val
    out = disco_fwd(psi, x)                  # (B,C,Hi,Wi) -> (B,C,K,Ho,Wo)
    gx  = disco_bwd(psi, gout)               # (B,C,K,Ho,Wo) -> (B,C,Hi,Wi)
    y   = disco_fused_conv(psi, x, W)        # (B,C,Hi,Wi), (Co,C,K) -> (B,Co,Ho,Wo)

The operators around the convolution (disco_rms_norm and below) are marshalled by a
compiled module, ``_disco_bind.so`` (csrc/bind.cpp), in the same way.

There is no fallback: if a library is not built, loading raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdisco.so")

DISCO_OK = 0
STATUS_NAMES = {
    0: "DISCO_OK",
    1: "DISCO_ERR_INVALID_ARGUMENT",
    2: "DISCO_ERR_SHAPE",
    3: "DISCO_ERR_DTYPE",
    4: "DISCO_ERR_PSI",
    5: "DISCO_ERR_UNSUPPORTED_DEVICE",
    6: "DISCO_ERR_OOM",
    7: "DISCO_ERR_HIP",
}
DISCO_F32 = 0
DISCO_BF16 = 1
DISCO_F16 = 2
DISCO_F8_E4M3 = 3
DISCO_F8_E5M2 = 4
DISCO_I8 = 5
ACTS = {None: 0, "gelu": 1, "silu": 2}  # disco_act: activation functions of the channel products
EXPORTED = ("disco_psi_create", "disco_psi_destroy", "disco_fwd", "disco_bwd", "disco_fused_conv",
            "disco_fused_conv_save", "disco_einsum", "disco_fused_conv_bwd_workspace", "disco_fused_conv_bwd",
            "disco_fused_conv_bwd_saved", "disco_fused_conv_bwd_noalloc", "disco_rms_norm", "disco_rms_norm_f8",
            "disco_dequantize", "disco_rms_norm_bwd_workspace", "disco_rms_norm_bwd", "disco_grad_norm_workspace",
            "disco_grad_norm", "disco_clip_grads", "disco_quantize_i8", "disco_dequantize_i8", "disco_linear_i8",
            "disco_linear_i8_bwd_input", "disco_linear_i8_bwd_weight_workspace", "disco_linear_i8_bwd_weight", "disco_last_error")


class DiscoError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{self.status_name}: {message}")


class CSRDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("Ho", ctypes.c_int32), ("Wo", ctypes.c_int32), ("Hi", ctypes.c_int32),
                ("Wi", ctypes.c_int32), ("nnz", ctypes.c_int64), ("row_ptr", ctypes.c_void_p),
                ("col_hi", ctypes.c_void_p), ("col_wi", ctypes.c_void_p), ("val", ctypes.c_void_p)]


class TensorDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 5)]


_lib = None


def load_library():
    """Load libdisco.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m sparse_gather_contraction_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        lib.disco_psi_create.argtypes = [ctypes.POINTER(CSRDesc), ctypes.c_int, ctypes.POINTER(P)]
        lib.disco_psi_destroy.argtypes = [P]
        lib.disco_fwd.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), P]
        lib.disco_bwd.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), P]
        lib.disco_fused_conv.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc),
                                         ctypes.POINTER(TensorDesc), P]
        lib.disco_einsum.argtypes = [ctypes.POINTER(TensorDesc)] * 3 + [P]
        lib.disco_fused_conv_save.argtypes = [P] + [ctypes.POINTER(TensorDesc)] * 4 + [P]
        lib.disco_fused_conv_bwd_saved.argtypes = [P] + [ctypes.POINTER(TensorDesc)] * 5 + [P, ctypes.c_size_t, P]
        lib.disco_fused_conv_bwd_workspace.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                       ctypes.POINTER(ctypes.c_size_t)]
        lib.disco_fused_conv_bwd.argtypes = [P] + [ctypes.POINTER(TensorDesc)] * 5 + [P, ctypes.c_size_t, P]
        lib.disco_fused_conv_bwd_noalloc.argtypes = [P] + [ctypes.POINTER(TensorDesc)] * 5 + [P]
        T, I64, F, SZ = ctypes.POINTER(TensorDesc), ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.disco_rms_norm.argtypes = [T, T, T, ctypes.c_int, F, T, T, P]
        lib.disco_rms_norm_f8.argtypes = [T, T, T, ctypes.c_int, F, I64, T, T, T, P]
        lib.disco_dequantize.argtypes = [T, T, ctypes.c_int, I64, T, P]
        lib.disco_rms_norm_bwd_workspace.argtypes = [T, ctypes.c_int, ctypes.POINTER(SZ)]
        lib.disco_rms_norm_bwd.argtypes = [T, T, T, T, ctypes.c_int, F, T, T, P, SZ, P]
        lib.disco_grad_norm_workspace.argtypes = [I64, P, ctypes.POINTER(SZ)]
        lib.disco_grad_norm.argtypes = [I64, P, T, P, SZ, P]
        lib.disco_clip_grads.argtypes = [I64, P, F, F, P, T, P, SZ, P]
        lib.disco_quantize_i8.argtypes = [T, ctypes.c_int, ctypes.c_int, T, T, T, T, P]
        lib.disco_dequantize_i8.argtypes = [T, T, ctypes.c_int, T, P]
        lib.disco_linear_i8.argtypes = [T, T, T, T, T, ctypes.c_int, T, P]
        lib.disco_linear_i8_bwd_input.argtypes = [T, T, T, ctypes.c_int, T, T, ctypes.c_int, T, P]
        lib.disco_linear_i8_bwd_weight_workspace.argtypes = [T, ctypes.c_int, I64, ctypes.c_int, ctypes.POINTER(SZ)]
        lib.disco_linear_i8_bwd_weight.argtypes = [T, T, T, ctypes.c_int, T, T, P, SZ, P]
        lib.disco_last_error.restype = ctypes.c_char_p
        for f in ("disco_psi_create", "disco_psi_destroy", "disco_fwd", "disco_bwd", "disco_fused_conv",
                  "disco_fused_conv_save", "disco_einsum", "disco_fused_conv_bwd_workspace", "disco_fused_conv_bwd",
                  "disco_fused_conv_bwd_saved", "disco_fused_conv_bwd_noalloc", "disco_rms_norm", "disco_rms_norm_f8",
                  "disco_dequantize", "disco_rms_norm_bwd_workspace", "disco_rms_norm_bwd",
                  "disco_grad_norm_workspace", "disco_grad_norm", "disco_clip_grads", "disco_quantize_i8", "disco_dequantize_i8",
                  "disco_linear_i8", "disco_linear_i8_bwd_input", "disco_linear_i8_bwd_weight_workspace",
                  "disco_linear_i8_bwd_weight"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(status: int):
    if status != DISCO_OK:
        raise DiscoError(status, load_library().disco_last_error().decode())


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return DISCO_F32
    if t.dtype == torch.bfloat16:
        return DISCO_BF16
    if t.dtype == torch.float16:
        return DISCO_F16
    return 99  # rejected by the library with DISCO_ERR_DTYPE


def tensor_desc(t) -> TensorDesc:
    """View of a contiguous torch tensor for the C ABI."""
    if not t.is_contiguous():
        raise ValueError("disco tensors must be contiguous")
    d = TensorDesc()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _dtype_code(t)
    d.ndim = t.dim()
    for i, s in enumerate(t.shape[:5]):
        d.shape[i] = int(s)
    return d


def _stream(device) -> int:
    import torch

    return torch.cuda.current_stream(device).cuda_stream


def csr_desc(csr):
    """CSRDesc over host numpy arrays; returns (desc, arrays kept alive)."""
    rp = np.ascontiguousarray(csr.row_ptr, dtype=np.int64)
    ch = np.ascontiguousarray(csr.col_hi, dtype=np.int32)
    cw = np.ascontiguousarray(csr.col_wi, dtype=np.int32)
    v = np.ascontiguousarray(csr.val, dtype=np.float32)
    d = CSRDesc(int(csr.K), int(csr.Ho), int(csr.Wo), int(csr.Hi), int(csr.Wi), int(rp[-1]) if rp.size else 0,
                rp.ctypes.data, ch.ctypes.data, cw.ctypes.data, v.ctypes.data)
    return d, (rp, ch, cw, v)


class Psi:
    """Owner of a disco_psi handle (device plans of one CSR filter)."""

    def __init__(self, handle: int, csr, device: int):
        self.handle = ctypes.c_void_p(handle)
        self.K, self.Ho, self.Wo, self.Hi, self.Wi = (int(csr.K), int(csr.Ho), int(csr.Wo), int(csr.Hi), int(csr.Wi))
        self.nnz = int(np.asarray(csr.row_ptr)[-1])
        self.device = device

    def close(self):
        if self.handle:
            load_library().disco_psi_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def disco_psi_create(csr, device=None) -> Psi:
    import torch

    lib = load_library()
    if device is None:
        device = torch.cuda.current_device()
    desc, keep = csr_desc(csr)
    h = ctypes.c_void_p()
    _check(lib.disco_psi_create(ctypes.byref(desc), int(device), ctypes.byref(h)))
    return Psi(h.value, csr, int(device))


def disco_fwd(psi: Psi, x, out=None):
    import torch

    if out is None:
        out = torch.empty((x.shape[0], x.shape[1], psi.K, psi.Ho, psi.Wo), dtype=x.dtype, device=x.device)
    xd, od = tensor_desc(x), tensor_desc(out)
    _check(load_library().disco_fwd(psi.handle, ctypes.byref(xd), ctypes.byref(od), _stream(x.device)))
    return out


def disco_bwd(psi: Psi, gout, gx=None):
    import torch

    if gx is None:
        gx = torch.empty((gout.shape[0], gout.shape[1], psi.Hi, psi.Wi), dtype=gout.dtype, device=gout.device)
    gd, xd = tensor_desc(gout), tensor_desc(gx)
    _check(load_library().disco_bwd(psi.handle, ctypes.byref(gd), ctypes.byref(xd), _stream(gout.device)))
    return gx


def disco_fused_conv(psi: Psi, x, W, y=None):
    import torch

    if y is None:
        y = torch.empty((x.shape[0], W.shape[0], psi.Ho, psi.Wo), dtype=x.dtype, device=x.device)
    xd, wd, yd = tensor_desc(x), tensor_desc(W), tensor_desc(y)
    _check(load_library().disco_fused_conv(psi.handle, ctypes.byref(xd), ctypes.byref(wd), ctypes.byref(yd),
                                           _stream(x.device)))
    return y




def disco_fused_conv_save(psi: Psi, x, W, y=None, out=None):
    """(y, out): the fused convolution and the contraction F x it multiplied (kept for the backward)."""
    import torch

    if y is None:
        y = torch.empty((x.shape[0], W.shape[0], psi.Ho, psi.Wo), dtype=x.dtype, device=x.device)
    if out is None:
        out = torch.empty((x.shape[0], x.shape[1], psi.K, psi.Ho, psi.Wo), dtype=x.dtype, device=x.device)
    xd, wd, yd, od = tensor_desc(x), tensor_desc(W), tensor_desc(y), tensor_desc(out)
    _check(load_library().disco_fused_conv_save(psi.handle, ctypes.byref(xd), ctypes.byref(wd), ctypes.byref(yd),
                                                ctypes.byref(od), _stream(x.device)))
    return y, out

def disco_einsum(W, t, y=None):
    """y[b, o, ho, wo] = sum_{c,k} W[o, c, k] t[b, c, k, ho, wo] on the current device (no psi)."""
    import torch

    if y is None:
        y = torch.empty((t.shape[0], W.shape[0], t.shape[3], t.shape[4]), dtype=t.dtype, device=t.device)
    wd, td, yd = tensor_desc(W), tensor_desc(t), tensor_desc(y)
    _check(load_library().disco_einsum(ctypes.byref(wd), ctypes.byref(td), ctypes.byref(yd), _stream(t.device)))
    return y

def disco_fused_conv_bwd_workspace(psi: Psi, B: int, C: int, Co: int) -> int:
    """Workspace bytes disco_fused_conv_bwd needs for these sizes."""
    n = ctypes.c_size_t()
    _check(load_library().disco_fused_conv_bwd_workspace(psi.handle, int(B), int(C), int(Co), ctypes.byref(n)))
    return int(n.value)


def disco_fused_conv_bwd(psi: Psi, x, W, gy, gx=None, dW=None, workspace=None):
    """(gx, dW): gradients of <gy, disco_fused_conv(x, W)>.  The workspace (a uint8 device tensor)
    is allocated here when not given."""
    import torch

    if gx is None:
        gx = torch.empty_like(x)
    if dW is None:
        dW = torch.empty_like(W)
    need = disco_fused_conv_bwd_workspace(psi, x.shape[0], x.shape[1], W.shape[0])
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    descs = [tensor_desc(t) for t in (x, W, gy, gx, dW)]
    _check(load_library().disco_fused_conv_bwd(psi.handle, *[ctypes.byref(d) for d in descs],
                                               ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                               _stream(x.device)))
    return gx, dW


def disco_fused_conv_bwd_noalloc(psi: Psi, x, W, gy, gx=None, dW=None):
    """(gx, dW) as disco_fused_conv_bwd, with the library's per-device scratch array as workspace
    (no device allocation inside the call; gx and dW are allocated here when not given)."""
    import torch

    if gx is None:
        gx = torch.empty_like(x)
    if dW is None:
        dW = torch.empty_like(W)
    descs = [tensor_desc(t) for t in (x, W, gy, gx, dW)]
    _check(load_library().disco_fused_conv_bwd_noalloc(psi.handle, *[ctypes.byref(d) for d in descs],
                                                       _stream(x.device)))
    return gx, dW


def disco_fused_conv_bwd_saved(psi: Psi, out, W, gy, gx=None, dW=None, workspace=None):
    """(gx, dW) as disco_fused_conv_bwd, with the contraction `out` from disco_fused_conv_save in place of x."""
    import torch

    B, C = out.shape[0], out.shape[1]
    if gx is None:
        gx = torch.empty((B, C, psi.Hi, psi.Wi), dtype=out.dtype, device=out.device)
    if dW is None:
        dW = torch.empty_like(W)
    need = disco_fused_conv_bwd_workspace(psi, B, C, W.shape[0])
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=out.device)
    descs = [tensor_desc(t) for t in (out, W, gy, gx, dW)]
    _check(load_library().disco_fused_conv_bwd_saved(psi.handle, *[ctypes.byref(d) for d in descs],
                                                     ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                                     _stream(out.device)))
    return gx, dW


# ---- the operators around the convolution in a residual model's training step

BIND_PATH = os.path.join(_PKG, "_disco_bind.so")
_bind = None


def _binding():
    """The compiled marshalling of these operators (csrc/bind.cpp); raise if it has not been built."""
    global _bind
    if _bind is None:
        import torch

        load_library()
        if not os.path.exists(BIND_PATH):
            raise RuntimeError(f"{BIND_PATH} is not built; run `python -m sparse_gather_contraction_amd.build`")
        from . import _disco_bind as bind

        bind.setup(DiscoError, torch._C._cuda_getCurrentRawStream)
        _bind = bind
    return _bind


def disco_rms_norm(x, w, residual=None, axis=1, eps=1e-6, y=None, h=None):
    """y = h w / sqrt(mean(h^2) + eps) over `axis`, h = x + residual.

    Returns y, or (y, h) with a residual.  axis 1 normalises fields (B, C, H, W) over their channels, -1 rows
    (points, C); w (D,) is fp32 or of x's type."""
    return (_bind or _binding()).rms_norm(x, w, residual, axis, eps, y, h)


def disco_rms_norm_f8(x, w, residual=None, axis=1, eps=1e-6, group=0, dtype=None, q=None, scale=None, h=None):
    """disco_rms_norm with its output in 8 bits: (q, scale), or (q, scale, h) with a residual.

    q is of `dtype` (torch.float8_e4m3fn, the default, or torch.float8_e5m2), which a given q must have too; scale (fp32)
    has x's shape with the axis replaced by the number of runs of `group` entries (0: one run, the whole axis; else a
    multiple of 32)."""
    code = 0 if dtype is None else _f8_code(dtype, q)
    return (_bind or _binding()).rms_norm_f8(x, w, residual, axis, eps, group, code, q, scale, h)


def _given_of(dtype, given, name):
    if given is not None and getattr(given, "dtype", dtype) != dtype:
        raise DiscoError(3, f"{name} is given and not of the dtype asked for")


def _f8_code(dtype, q):
    import torch

    _given_of(dtype, q, "q")
    if dtype == torch.float8_e4m3fn:
        return 0
    if dtype == torch.float8_e5m2:
        return 1
    raise DiscoError(3, "q must be e4m3 or e5m2")


def disco_dequantize(q, scale, dtype=None, axis=1, group=0, out=None):
    """out = q * scale in `dtype` (default bf16, or the given out's): the reader of disco_rms_norm_f8's form."""
    code = DISCO_BF16 if dtype is None else _data_code(dtype, out)
    return (_bind or _binding()).dequantize(q, scale, code, axis, group, out)


def _data_code(dtype, out):
    import torch

    _given_of(dtype, out, "out")
    code = {torch.float32: DISCO_F32, torch.bfloat16: DISCO_BF16, torch.float16: DISCO_F16}.get(dtype)
    if code is None:
        raise DiscoError(3, "out has an unsupported dtype")
    return code


def disco_rms_norm_bwd_workspace(h, axis=1) -> int:
    """Workspace bytes disco_rms_norm_bwd needs for this h."""
    n = ctypes.c_size_t()
    _check(load_library().disco_rms_norm_bwd_workspace(ctypes.byref(tensor_desc(h)), axis, ctypes.byref(n)))
    return int(n.value)


def disco_rms_norm_bwd(h, w, gy, gh=None, axis=1, eps=1e-6, gx=None, dw=None, workspace=None):
    """(gx, dw): gradients of disco_rms_norm at h (the stored sum, or x without a residual).

    gh is the gradient that reaches h past the norm; gx is the gradient of x and of the residual alike.  The
    workspace (a uint8 device tensor) is allocated here when not given."""
    return (_bind or _binding()).rms_norm_bwd(h, w, gy, gh, axis, eps, gx, dw, workspace)


def _result_on(grads, device):
    """A tensor for the norm where the list alone does not say its device."""
    if device is None and len(grads):
        return None
    import torch

    return torch.empty((), dtype=torch.float32, device="cuda" if device is None else device)


def disco_grad_norm(grads, device=None):
    """The norm over all elements of all tensors of the list `grads`, as a 0-dimensional fp32 tensor on their device.

    The tensors may differ in shape and type (fp32, bf16, fp16); squares are summed in fp64."""
    grads = grads if type(grads) is list else list(grads)
    return (_bind or _binding()).grad_norm(grads, _result_on(grads, device))


def disco_clip_grads(grads, max_norm, out=None, eps=1e-6, device=None):
    """Scale all gradients by min(1, max_norm / (norm + eps)), norm = disco_grad_norm(grads); returns that norm.

    In place, or into the tensors of the list `out`.  The factor never leaves the device."""
    grads = grads if type(grads) is list else list(grads)
    return (_bind or _binding()).clip_grads(grads, max_norm, eps, out, _result_on(grads, device))


# ---- channel products in 8-bit integers, and 8-bit activation checkpoints


def _act_code(act) -> int:
    try:
        return ACTS[act]
    except (KeyError, TypeError):
        raise DiscoError(1, "act must be None, 'gelu' or 'silu'") from None


def _channels(channels, given, axis, name) -> int:
    """`channels` (-1: not asked for), which a given output has to have at `axis`."""
    if channels is None:
        return -1
    if channels < 0:
        raise DiscoError(2, "the number of channels is out of range")
    shape = getattr(given, "shape", ())
    if -len(shape) <= axis < len(shape) and shape[axis] != channels:  # (an axis out of range is the library's to refuse)
        raise DiscoError(2, f"{name} has {shape[axis]} channels, {channels} were asked for")
    return channels


def disco_quantize_i8(x, act=None, keep=False, axis=1, q=None, scale=None, kept=None, kept_scale=None):
    """The 8-bit form of act(x) over its channel axis: (q, scale), or with `keep` (q, scale, kept, kept_scale).

    q (int8) holds a point's channels together, in x's shape with `axis` moved last and padded with zeros to a multiple of
    16; scale (fp32) has x's shape without `axis`.  act is None, "gelu" or "silu".  kept and kept_scale are the form of x
    itself, the checkpoint that disco_linear_i8_bwd_input takes act's slope from.  A weight (Co, C) takes axis=1."""
    return (_bind or _binding()).quantize_i8(x, _act_code(act), keep or kept is not None or kept_scale is not None, axis, q, scale,
                                             kept, kept_scale)


def disco_dequantize_i8(q, scale, channels=None, dtype=None, axis=1, out=None):
    """out = q * scale in `dtype` (default bf16, or the given out's), `channels` of them (default: all of q's) at `axis`."""
    code = DISCO_BF16 if dtype is None else _data_code(dtype, out)
    return (_bind or _binding()).dequantize_i8(q, scale, _channels(channels, out, axis, "out"), code, axis, out)


def disco_linear_i8(q, scale, w, wscale, bias=None, dtype=None, axis=1, out=None):
    """y = (q scale) (w wscale)^T + bias over the channels of each point, from the 8-bit forms of both.

    q (points..., Cp), scale (points...): disco_quantize_i8 of the input; w (Co, Cp), wscale (Co): of the weight; bias (Co)
    fp32.  y has the Co channels at `axis`, in `dtype` (default bf16, or the given out's)."""
    code = DISCO_BF16 if dtype is None else _data_code(dtype, out)
    return (_bind or _binding()).linear_i8(q, scale, w, wscale, bias, code, axis, out)


def disco_linear_i8_bwd_input(gy, w, wscale, channels=None, act=None, kept=None, kept_scale=None, axis=1, gx=None):
    """The gradient of disco_linear_i8's input (before it was put into 8 bits): gy w, channels at `axis` of both.

    With act, kept and kept_scale the gradient of what act was taken of before the product: times act'(kept kept_scale).
    `channels` is the input's number of channels (default: all of w's)."""
    return (_bind or _binding()).linear_i8_bwd_input(gy, w, wscale, _channels(channels, gx, axis, "gx"), _act_code(act), kept, kept_scale,
                                                       axis, gx)


def disco_linear_i8_bwd_weight_workspace(gy, channels, bias=False, axis=1) -> int:
    """Workspace bytes disco_linear_i8_bwd_weight needs for this gy."""
    return _binding().linear_i8_bwd_weight_workspace(gy, channels, bias, axis)


def disco_linear_i8_bwd_weight(gy, q, scale, channels=None, bias=False, axis=1, dw=None, db=None, workspace=None):
    """dw, or (dw, db) with `bias`: the gradients of disco_linear_i8's weight (Co, channels) and bias (Co).

    q, scale: the 8-bit input that the forward took; gy has its Co channels at `axis`.  The workspace (a uint8 device
    tensor) is allocated here when not given."""
    return (_bind or _binding()).linear_i8_bwd_weight(gy, q, scale, _channels(channels, dw, -1, "dw"), bias or db is not None, axis, dw, db,
                                                        workspace)
