// linear_api.hip — C ABI of the channel products in 8-bit integers and of their 8-bit form: validation and launches.
#include <cstdint>
#include <string>

#include "api_common.hpp"
#include "disco.h"
#include "linear.hpp"
#include "tensor_checks.hpp"

using namespace disco;

namespace {

bool is_16bit(int dtype) { return dtype == DISCO_BF16 || dtype == DISCO_F16; }

disco_status check_act(int act)
{
    if (act != DISCO_ACT_NONE && act != DISCO_ACT_GELU && act != DISCO_ACT_SILU)
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "act is no activation function");
    return DISCO_OK;
}

// The dense tensor x around its channel axis, with point numbers of 32 bits.
disco_status points_of(const disco_tensor *x, const char *name, int axis, View *v)
{
    const disco_status st = view_of(x, name, axis, v);
    if (st != DISCO_OK) return st;
    if (v->N > 0 && v->M > kMaxPoints / v->N) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has too many points");
    if (v->D > kMaxPoints) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has too many channels");
    return DISCO_OK;
}

// q and scale are the form of the dense tensor x (dimensions before and after the axis, then the padded channels).
disco_status check_form(const disco_tensor *q, const disco_tensor *scale, const char *qname, const char *sname,
                        const disco_tensor *x, int axis, int64_t Cp)
{
    if (q->dtype != DISCO_I8) return api_fail(DISCO_ERR_DTYPE, std::string(qname) + " must be int8");
    if (scale->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, std::string(sname) + " must be fp32");
    if (q->ndim != x->ndim) return api_fail(DISCO_ERR_SHAPE, std::string(qname) + " has the wrong number of dimensions");
    if (scale->ndim != x->ndim - 1) return api_fail(DISCO_ERR_SHAPE, std::string(sname) + " has the wrong number of dimensions");
    for (int i = 0, k = 0; i < x->ndim; ++i) {
        if (i == axis) continue;
        if (q->shape[k] != x->shape[i] || scale->shape[k] != x->shape[i])
            return api_fail(DISCO_ERR_SHAPE, std::string(q->shape[k] != x->shape[i] ? qname : sname) + " dimension " + std::to_string(k) +
                                             " is not that of the points (" + std::to_string(x->shape[i]) + ")");
        ++k;
    }
    if (q->shape[x->ndim - 1] != Cp)
        return api_fail(DISCO_ERR_SHAPE, std::string(qname) + " has " + std::to_string(q->shape[x->ndim - 1]) +
                                         " channels, expected " + std::to_string(Cp) + " (padded to a multiple of 16)");
    return DISCO_OK;
}

disco_status check_form_pointers(const disco_tensor *q, const disco_tensor *scale, const char *qname, const char *sname, int dev)
{
    disco_status st;
    if ((st = check_pointer(q->data, qname, dev)) != DISCO_OK) return st;
    if ((uintptr_t)q->data & 15) return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(qname) + " is not 16-byte aligned");
    return check_pointer(scale->data, sname, dev);
}

// w (Co, Cp) with wscale (Co)
disco_status check_w(const disco_tensor *w, const disco_tensor *wscale, int64_t Co, int64_t Cp)
{
    if (w->dtype != DISCO_I8) return api_fail(DISCO_ERR_DTYPE, "w must be int8");
    if (wscale->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, "wscale must be fp32");
    if (w->ndim != 2 || w->shape[0] != Co || w->shape[1] != Cp)
        return api_fail(DISCO_ERR_SHAPE, "w must be (" + std::to_string(Co) + ", " + std::to_string(Cp) + ")");
    if (wscale->ndim != 1 || wscale->shape[0] != Co) return api_fail(DISCO_ERR_SHAPE, "wscale must be (Co,)");
    return DISCO_OK;
}

disco_status check_channels(int64_t Cp)
{
    if (Cp > kMaxChannels) return api_fail(DISCO_ERR_SHAPE, "a product has at most " + std::to_string(kMaxChannels) + " channels");
    return DISCO_OK;
}

disco_status check_tiles(int64_t a, int64_t b, int64_t threads)
{
    // products of tile counts stay far below 63 bits: both come from 32-bit sizes
    return check_grid(a * b, threads);
}

disco_status quantize_impl(const disco_tensor *x, int act, int axis, disco_tensor *q, disco_tensor *scale, disco_tensor *kept,
                           disco_tensor *kept_scale, void *stream)
{
    if (!x || !q || !scale) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "x, q or scale is NULL");
    if ((kept == nullptr) != (kept_scale == nullptr))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "kept and kept_scale come together");
    disco_status st;
    if ((st = check_act(act)) != DISCO_OK) return st;
    if (kept && act == DISCO_ACT_NONE)
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "kept is the checkpoint of an activation function: without one it is q");
    if (!is_data(x->dtype)) return api_fail(DISCO_ERR_DTYPE, "x has an unsupported dtype");
    View v;
    if ((st = points_of(x, "x", axis, &v)) != DISCO_OK) return st;
    const int64_t Cp = padded_channels(v.D);
    if ((st = check_form(q, scale, "q", "scale", x, v.axis, Cp)) != DISCO_OK) return st;
    if (kept && (st = check_form(kept, kept_scale, "kept", "kept_scale", x, v.axis, Cp)) != DISCO_OK) return st;
    if (v.N == 0 || v.M == 0) return DISCO_OK;
    const FormGeom g = form_geom(v.N, v.D, v.M, (int)elem_size(x->dtype));
    if ((st = check_grid(g.tiles, g.threads)) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_pointer(x->data, "x", dev)) != DISCO_OK) return st;
    if ((st = check_form_pointers(q, scale, "q", "scale", dev)) != DISCO_OK) return st;
    if (kept && (st = check_form_pointers(kept, kept_scale, "kept", "kept_scale", dev)) != DISCO_OK) return st;
    const Range ins[1] = {range_of(x, "x")};
    Range outs[4] = {range_of(q, "q"), range_of(scale, "scale")};
    int no = 2;
    if (kept) {
        outs[no++] = range_of(kept, "kept");
        outs[no++] = range_of(kept_scale, "kept_scale");
    }
    if ((st = check_ranges(outs, no, ins, 1)) != DISCO_OK) return st;
    FormLaunch l;
    l.x = x->data; l.q = (int8_t *)q->data; l.scale = (float *)scale->data;
    l.kq = kept ? (int8_t *)kept->data : nullptr; l.kscale = kept ? (float *)kept_scale->data : nullptr;
    l.dtype = x->dtype; l.act = act; l.N = v.N; l.D = v.D; l.M = v.M;
    return launched(launch_quantize_i8(l, (hipStream_t)stream), "quantize");
}

disco_status dequantize_impl(const disco_tensor *q, const disco_tensor *scale, int axis, disco_tensor *out, void *stream)
{
    if (!q || !scale || !out) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "q, scale or out is NULL");
    if (!is_data(out->dtype)) return api_fail(DISCO_ERR_DTYPE, "out has an unsupported dtype");
    View v;
    disco_status st;
    if ((st = points_of(out, "out", axis, &v)) != DISCO_OK) return st;
    if ((st = check_form(q, scale, "q", "scale", out, v.axis, padded_channels(v.D))) != DISCO_OK) return st;
    if (v.N == 0 || v.M == 0) return DISCO_OK;
    const FormGeom g = form_geom(v.N, v.D, v.M, (int)elem_size(out->dtype));
    if ((st = check_grid(g.tiles, g.threads)) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_form_pointers(q, scale, "q", "scale", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(out->data, "out", dev)) != DISCO_OK) return st;
    const Range ins[2] = {range_of(q, "q"), range_of(scale, "scale")}, outs[1] = {range_of(out, "out")};
    if ((st = check_ranges(outs, 1, ins, 2)) != DISCO_OK) return st;
    FormLaunch l;
    l.q = (int8_t *)q->data; l.scale = (float *)scale->data; l.out = out->data;
    l.dtype = out->dtype; l.N = v.N; l.D = v.D; l.M = v.M;
    return launched(launch_dequantize_i8(l, (hipStream_t)stream), "dequantize");
}

disco_status linear_impl(const disco_tensor *q, const disco_tensor *scale, const disco_tensor *w, const disco_tensor *wscale,
                         const disco_tensor *bias, int axis, disco_tensor *y, void *stream)
{
    if (!q || !scale || !w || !wscale || !y) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "q, scale, w, wscale or y is NULL");
    if (!is_data(y->dtype)) return api_fail(DISCO_ERR_DTYPE, "y has an unsupported dtype");
    if (bias && bias->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, "bias must be fp32");
    View v;
    disco_status st;
    if ((st = points_of(y, "y", axis, &v)) != DISCO_OK) return st;
    if (q->ndim != y->ndim) return api_fail(DISCO_ERR_SHAPE, "q has the wrong number of dimensions");
    const int64_t Cp = q->shape[q->ndim - 1];
    if (Cp < 16 || Cp % 16) return api_fail(DISCO_ERR_SHAPE, "q's last dimension must be a multiple of 16, at least 16");
    if ((st = check_channels(Cp)) != DISCO_OK) return st;
    if ((st = check_form(q, scale, "q", "scale", y, v.axis, Cp)) != DISCO_OK) return st;
    if ((st = check_w(w, wscale, v.D, Cp)) != DISCO_OK) return st;
    if (bias && (bias->ndim != 1 || bias->shape[0] != v.D)) return api_fail(DISCO_ERR_SHAPE, "bias must be (Co,)");
    if (v.N == 0 || v.M == 0) return DISCO_OK;
    const int64_t P = v.N * v.M;
    if ((st = check_grid(lin_blocks(P, v.D), lin_threads(P))) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_form_pointers(q, scale, "q", "scale", dev)) != DISCO_OK) return st;
    if ((st = check_form_pointers(w, wscale, "w", "wscale", dev)) != DISCO_OK) return st;
    if (bias && (st = check_pointer(bias->data, "bias", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(y->data, "y", dev)) != DISCO_OK) return st;
    Range ins[5] = {range_of(q, "q"), range_of(scale, "scale"), range_of(w, "w"), range_of(wscale, "wscale")};
    const Range outs[1] = {range_of(y, "y")};
    int ni = 4;
    if (bias) ins[ni++] = range_of(bias, "bias");
    if ((st = check_ranges(outs, 1, ins, ni)) != DISCO_OK) return st;
    LinearLaunch l;
    l.q = (const int8_t *)q->data; l.scale = (const float *)scale->data;
    l.w = (const int8_t *)w->data; l.wscale = (const float *)wscale->data;
    l.bias = bias ? (const float *)bias->data : nullptr; l.y = y->data; l.dtype = y->dtype;
    l.P = P; l.M = v.M; l.Cp = Cp; l.Co = v.D;
    return launched(launch_linear_i8(l, (hipStream_t)stream), "linear");
}

disco_status bwd_input_impl(const disco_tensor *gy, const disco_tensor *w, const disco_tensor *wscale, int act,
                            const disco_tensor *kept, const disco_tensor *kept_scale, int axis, disco_tensor *gx, void *stream)
{
    if (!gy || !w || !wscale || !gx) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "gy, w, wscale or gx is NULL");
    if ((kept == nullptr) != (kept_scale == nullptr))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "kept and kept_scale come together");
    disco_status st;
    if ((st = check_act(act)) != DISCO_OK) return st;
    if ((act != DISCO_ACT_NONE) != (kept != nullptr))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "an activation function and its checkpoint (kept) come together");
    if (!is_16bit(gy->dtype)) return api_fail(DISCO_ERR_DTYPE, "gy must be bf16 or fp16");
    if (gx->dtype != gy->dtype) return api_fail(DISCO_ERR_DTYPE, "gy and gx dtypes differ");
    View v, u;
    if ((st = points_of(gx, "gx", axis, &v)) != DISCO_OK) return st;
    if (gy->ndim != gx->ndim) return api_fail(DISCO_ERR_SHAPE, "gy has the wrong number of dimensions");
    if ((st = points_of(gy, "gy", axis, &u)) != DISCO_OK) return st;
    if ((st = same_shape(gy, "gy", gx, v.axis, u.D)) != DISCO_OK) return st;
    const int64_t Cp = padded_channels(v.D);
    if ((st = check_w(w, wscale, u.D, Cp)) != DISCO_OK) return st;
    if (kept && (st = check_form(kept, kept_scale, "kept", "kept_scale", gx, v.axis, Cp)) != DISCO_OK) return st;
    if (v.N == 0 || v.M == 0) return DISCO_OK;
    const int64_t P = v.N * v.M;
    if ((st = check_tiles(ceil_div64(P, 128), ceil_div64(v.D, 128), 256)) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_pointer(gy->data, "gy", dev)) != DISCO_OK) return st;
    if ((st = check_form_pointers(w, wscale, "w", "wscale", dev)) != DISCO_OK) return st;
    if (kept && (st = check_form_pointers(kept, kept_scale, "kept", "kept_scale", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(gx->data, "gx", dev)) != DISCO_OK) return st;
    Range ins[5] = {range_of(gy, "gy"), range_of(w, "w"), range_of(wscale, "wscale")};
    const Range outs[1] = {range_of(gx, "gx")};
    int ni = 3;
    if (kept) {
        ins[ni++] = range_of(kept, "kept");
        ins[ni++] = range_of(kept_scale, "kept_scale");
    }
    if ((st = check_ranges(outs, 1, ins, ni)) != DISCO_OK) return st;
    LinearBwdLaunch l;
    l.gy = gy->data; l.q = (const int8_t *)w->data; l.scale = (const float *)wscale->data;
    l.kept = kept ? (const int8_t *)kept->data : nullptr; l.kept_scale = kept ? (const float *)kept_scale->data : nullptr;
    l.out = gx->data; l.dtype = gy->dtype; l.act = act;
    l.P = P; l.M = v.M; l.C = v.D; l.Cp = Cp; l.Co = u.D;
    return launched(launch_linear_bwd_input(l, (hipStream_t)stream), "linear backward");
}

// The checks that the weight's gradient and its workspace share.
disco_status weight_view(const disco_tensor *gy, int axis, int64_t C, View *v)
{
    if (!is_16bit(gy->dtype)) return api_fail(DISCO_ERR_DTYPE, "gy must be bf16 or fp16");
    disco_status st;
    if ((st = points_of(gy, "gy", axis, v)) != DISCO_OK) return st;
    if (C < 1 || C > kMaxPoints) return api_fail(DISCO_ERR_SHAPE, "the number of channels is out of range");
    return check_tiles(ceil_div64(C, 128), ceil_div64(v->D, 128), 256);
}

disco_status bwd_weight_impl(const disco_tensor *gy, const disco_tensor *q, const disco_tensor *scale, int axis, disco_tensor *dw,
                             disco_tensor *db, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!gy || !q || !scale || !dw) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "gy, q, scale or dw is NULL");
    if (dw->dtype != gy->dtype || (db && db->dtype != gy->dtype)) return api_fail(DISCO_ERR_DTYPE, "gy, dw and db dtypes differ");
    if (dw->ndim != 2) return api_fail(DISCO_ERR_SHAPE, "dw must be (Co, C)");
    View v;
    disco_status st;
    const int64_t C = dw->shape[1];
    if ((st = weight_view(gy, axis, C, &v)) != DISCO_OK) return st;
    if (dw->shape[0] != v.D) return api_fail(DISCO_ERR_SHAPE, "dw must be (Co, C)");
    if (db && (db->ndim != 1 || db->shape[0] != v.D)) return api_fail(DISCO_ERR_SHAPE, "db must be (Co,)");
    const int64_t Cp = padded_channels(C), P = v.N * v.M;
    if ((st = check_form(q, scale, "q", "scale", gy, v.axis, Cp)) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_pointer(dw->data, "dw", dev)) != DISCO_OK) return st;
    if (db && (st = check_pointer(db->data, "db", dev)) != DISCO_OK) return st;
    Range ins[3] = {range_of(gy, "gy"), range_of(q, "q"), range_of(scale, "scale")}, outs[3] = {range_of(dw, "dw")};
    int no = 1;
    if (db) outs[no++] = range_of(db, "db");
    LinearBwdLaunch l;
    l.out = dw->data; l.db = db ? db->data : nullptr; l.dtype = gy->dtype; l.P = P; l.M = v.M; l.C = C; l.Cp = Cp; l.Co = v.D;
    if (P > 0) {
        if ((st = check_pointer(gy->data, "gy", dev)) != DISCO_OK) return st;
        if ((st = check_form_pointers(q, scale, "q", "scale", dev)) != DISCO_OK) return st;
        const WeightPlan p = weight_plan(P, C, v.D);
        const size_t need = weight_bytes(p, C, v.D, db != nullptr);
        if (need > 0) {
            if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15))
                return api_fail(DISCO_ERR_INVALID_ARGUMENT, "workspace is NULL, not 16-byte aligned or too small");
            if ((st = check_pointer(workspace, "workspace", dev)) != DISCO_OK) return st;
            outs[no++] = {(uintptr_t)workspace, (uintptr_t)workspace + need, "workspace"};
        }
        l.gy = gy->data; l.q = (const int8_t *)q->data; l.scale = (const float *)scale->data;
        l.workspace = (float *)workspace;
        l.splits = p.splits;
    }
    if ((st = check_ranges(outs, no, ins, P > 0 ? 3 : 0)) != DISCO_OK) return st;
    return launched(launch_linear_bwd_weight(l, (hipStream_t)stream), "linear backward");
}

// No C++ exception leaves a C entry: what the host allocates (messages) may not be had.
template <typename F>
disco_status guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return api_fail_oom();
    }
}

}  // namespace

extern "C" {

disco_status disco_quantize_i8(const disco_tensor *x, disco_act act, int axis, disco_tensor *q, disco_tensor *scale,
                               disco_tensor *kept, disco_tensor *kept_scale, void *stream)
{
    return guarded([&] { return quantize_impl(x, (int)act, axis, q, scale, kept, kept_scale, stream); });
}

disco_status disco_dequantize_i8(const disco_tensor *q, const disco_tensor *scale, int axis, disco_tensor *out, void *stream)
{
    return guarded([&] { return dequantize_impl(q, scale, axis, out, stream); });
}

disco_status disco_linear_i8(const disco_tensor *q, const disco_tensor *scale, const disco_tensor *w, const disco_tensor *wscale,
                             const disco_tensor *bias, int axis, disco_tensor *y, void *stream)
{
    return guarded([&] { return linear_impl(q, scale, w, wscale, bias, axis, y, stream); });
}

disco_status disco_linear_i8_bwd_input(const disco_tensor *gy, const disco_tensor *w, const disco_tensor *wscale, disco_act act,
                                       const disco_tensor *kept, const disco_tensor *kept_scale, int axis, disco_tensor *gx,
                                       void *stream)
{
    return guarded([&] { return bwd_input_impl(gy, w, wscale, (int)act, kept, kept_scale, axis, gx, stream); });
}

disco_status disco_linear_i8_bwd_weight_workspace(const disco_tensor *gy, int axis, int64_t C, int db, size_t *bytes)
{
    return guarded([&]() -> disco_status {
        if (!gy || !bytes) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "gy or bytes is NULL");
        View v;
        const disco_status st = weight_view(gy, axis, C, &v);
        if (st != DISCO_OK) return st;
        const int64_t P = v.N * v.M;
        *bytes = P == 0 ? 0 : weight_bytes(weight_plan(P, C, v.D), C, v.D, db != 0);
        return DISCO_OK;
    });
}

disco_status disco_linear_i8_bwd_weight(const disco_tensor *gy, const disco_tensor *q, const disco_tensor *scale, int axis,
                                        disco_tensor *dw, disco_tensor *db, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] { return bwd_weight_impl(gy, q, scale, axis, dw, db, workspace, workspace_bytes, stream); });
}

}  // extern "C"
