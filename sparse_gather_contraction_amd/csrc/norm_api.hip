// norm_api.hip — C ABI of the training-step operators beside the convolution: validation and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>
#include <string>
#include <vector>

#include "api_common.hpp"
#include "disco.h"
#include "norm.hpp"
#include "tensor_checks.hpp"

using namespace disco;

namespace {

disco_status check_weight(const disco_tensor *w, const char *name, const disco_tensor *x, int64_t D)
{
    if (w->dtype != DISCO_F32 && w->dtype != x->dtype)
        return api_fail(DISCO_ERR_DTYPE, std::string(name) + " must be fp32 or of the data's type");
    if (w->ndim != 1 || w->shape[0] != D) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " must be (D,)");
    return DISCO_OK;
}

disco_status norm_impl(const disco_tensor *x, const disco_tensor *residual, const disco_tensor *w, int axis, float eps,
                       int64_t group, disco_tensor *y, disco_tensor *scale, disco_tensor *h, bool f8, void *stream)
{
    if (!x || !w || !y || (f8 && !scale))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, f8 ? "x, w, q or scale is NULL" : "x, w or y is NULL");
    if ((residual == nullptr) != (h == nullptr))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "residual and h come together: the sum is stored where there is one");
    const char *yname = f8 ? "q" : "y";
    if (!is_data(x->dtype)) return api_fail(DISCO_ERR_DTYPE, "x has an unsupported dtype");
    if (f8 ? !is_f8(y->dtype) : y->dtype != x->dtype)
        return api_fail(DISCO_ERR_DTYPE, f8 ? "q must be e4m3 or e5m2" : "x and y dtypes differ");
    if (residual && (residual->dtype != x->dtype || h->dtype != x->dtype))
        return api_fail(DISCO_ERR_DTYPE, "x, residual and h dtypes differ");
    if (f8 && scale->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, "scale must be fp32");
    View v;
    disco_status st;
    if ((st = view_of(x, "x", axis, &v)) != DISCO_OK) return st;
    if ((st = check_weight(w, "w", x, v.D)) != DISCO_OK) return st;
    if ((st = same_shape(y, yname, x, v.axis, v.D)) != DISCO_OK) return st;
    if (residual && (st = same_shape(residual, "residual", x, v.axis, v.D)) != DISCO_OK) return st;
    if (h && (st = same_shape(h, "h", x, v.axis, v.D)) != DISCO_OK) return st;
    int64_t ngroups = 1;
    if (f8) {
        if (group < 0 || group % 32 != 0)
            return api_fail(DISCO_ERR_SHAPE, "group must be 0 (the whole axis) or a multiple of 32");
        if (group == 0 || group > v.D) group = v.D;
        ngroups = disco::ceil_div64(v.D, group);
        if ((st = same_shape(scale, "scale", x, v.axis, ngroups)) != DISCO_OK) return st;
    }
    if (!(eps >= 0.0f) || std::isinf(eps)) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    if (v.N == 0 || v.M == 0) return DISCO_OK;
    const disco::NormGeom g = disco::norm_geom(v.N, v.D, v.M, (int)elem_size(x->dtype), false);
    if ((st = check_grid(g.tiles, g.threads)) != DISCO_OK) return st;
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    if ((st = check_pointer(x->data, "x", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(w->data, "w", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(y->data, yname, dev)) != DISCO_OK) return st;
    if (residual && (st = check_pointer(residual->data, "residual", dev)) != DISCO_OK) return st;
    if (h && (st = check_pointer(h->data, "h", dev)) != DISCO_OK) return st;
    if (f8 && (st = check_pointer(scale->data, "scale", dev)) != DISCO_OK) return st;
    Range ins[3] = {range_of(x, "x"), range_of(w, "w")}, outs[3] = {range_of(y, yname)};
    int ni = 2, no = 1;
    if (residual) ins[ni++] = range_of(residual, "residual");
    if (h) outs[no++] = range_of(h, "h");
    if (f8) outs[no++] = range_of(scale, "scale");
    if ((st = check_ranges(outs, no, ins, ni)) != DISCO_OK) return st;
    disco::NormLaunch a;
    a.x = x->data; a.r = residual ? residual->data : nullptr; a.w = w->data;
    a.y = y->data; a.h = h ? h->data : nullptr; a.scale = f8 ? (float *)scale->data : nullptr;
    a.dtype = x->dtype; a.wf32 = w->dtype == DISCO_F32;
    a.N = v.N; a.D = v.D; a.M = v.M; a.eps = eps;
    a.f8 = f8 ? (y->dtype == DISCO_F8_E5M2 ? 1 : 0) : -1;
    a.group = (int32_t)group; a.ngroups = (int32_t)ngroups;
    return launched(disco::launch_norm(a, (hipStream_t)stream), "norm");
}

// ---- gradients

constexpr int64_t kGradElements = (int64_t)1 << 40;  // of all tensors: chunk numbers stay below 2^30

disco_status check_grads(int64_t n, const disco_tensor *g)
{
    if (n < 0 || n > (1 << 24)) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "the number of tensors is out of range");
    if (n > 0 && !g) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "grads is NULL");
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (!is_data(g[i].dtype)) return api_fail(DISCO_ERR_DTYPE, "grads[" + std::to_string(i) + "] has an unsupported dtype");
        if (g[i].ndim < 0 || g[i].ndim > 5)
            return api_fail(DISCO_ERR_SHAPE, "grads[" + std::to_string(i) + "] must have at most 5 dimensions");
        int64_t all = 8;
        for (int k = 0; k < g[i].ndim; ++k) {
            const int64_t s = g[i].shape[k];
            if (s < 0 || (s > 0 && all > INT64_MAX / s))
                return api_fail(DISCO_ERR_SHAPE, "grads[" + std::to_string(i) + "] has a bad dimension");
            if (s > 0) all *= s;
        }
        const int64_t len = numel(&g[i]);
        if (len > kGradElements - total) return api_fail(DISCO_ERR_SHAPE, "grads have too many elements");
        total += len;
    }
    return DISCO_OK;
}

// Elements of a chunk: up to 8192, a workgroup's loads of 16-bit elements in one go, as long as half the
// workgroups of a launch have one.  (4 times that for 2^28 fp32 elements: the scaling pass 384 against 374 us.)
int64_t chunk_of(int64_t total)
{
    int64_t c = 2048;
    while (c < 8192 && total / c > disco::kGradBlocks / 2) c *= 2;
    return c;
}

// Tensors that follow each other in memory are walked as one.
struct Run {
    const char *p;
    char *o;
    int64_t n;
    int dtype;
};

// The runs of the gradients, and with `o` of their outputs too (both must follow each other).
void runs_of(int64_t n, const disco_tensor *g, const disco_tensor *o, std::vector<Run> *runs)
{
    runs->clear();
    for (int64_t i = 0; i < n; ++i) {
        const int64_t len = numel(&g[i]), esz = elem_size(g[i].dtype);
        if (len == 0) continue;
        const char *p = (const char *)g[i].data;
        char *q = o ? (char *)o[i].data : nullptr;
        if (!runs->empty()) {
            Run &b = runs->back();
            if (b.dtype == g[i].dtype && p == b.p + b.n * esz && (!o || q == b.o + b.n * esz)) {
                b.n += len;
                continue;
            }
        }
        runs->push_back({p, q, len, g[i].dtype});
    }
}

// How the runs fall into launches.
struct GradPlan {
    std::vector<disco::GradBatch> batches;
    int64_t slots = 0;                 // workgroups of all batches: the partial sums that they leave
};

int32_t blocks_of(const disco::GradBatch &b) { return std::min<int32_t>(b.chunks, disco::kGradBlocks); }

void plan_grads(const std::vector<Run> &runs, int64_t total, GradPlan *p)
{
    const int64_t chunk = chunk_of(total);
    int64_t bytes = 0;
    for (const Run &r : runs) bytes += r.n * elem_size(r.dtype);
    p->batches.reserve((runs.size() + disco::kGradBatch - 1) / disco::kGradBatch);
    for (const Run &r : runs) {
        if (p->batches.empty() || p->batches.back().count == disco::kGradBatch) {
            p->batches.emplace_back();
            disco::GradBatch &nb = p->batches.back();
            nb.count = nb.chunks = 0;
            nb.chunk = (int32_t)chunk;
            nb.stream = bytes > disco::kStreamBytes;
        }
        disco::GradBatch &b = p->batches.back();
        b.t[b.count++] = {r.p, r.o, r.n, b.chunks, r.dtype};
        b.chunks += (int32_t)disco::ceil_div64(r.n, chunk);
    }
    for (const disco::GradBatch &b : p->batches) p->slots += blocks_of(b);
}

// The runs in chunks for one workgroup, if they are few; false otherwise.
bool small_of(const std::vector<Run> &runs, int64_t total, disco::GradSmall *s)
{
    s->count = 0;
    if (total > disco::kSmallElements) return false;
    for (const Run &r : runs)
        for (int64_t off = 0; off < r.n; off += disco::kSmallChunk) {
            if (s->count == disco::kSmallChunks) return false;
            const int64_t esz = elem_size(r.dtype);
            s->t[s->count++] = {r.p + off * esz, r.o ? r.o + off * esz : nullptr, std::min(r.n - off, disco::kSmallChunk), 0, r.dtype};
        }
    return true;
}

// Partial sums that tensors of these sizes leave at most, however they lie in memory: runs of several tensors
// have no more chunks and launches than the tensors have.
int64_t slots_of(int64_t n, const disco_tensor *g)
{
    int64_t total = 0, tensors = 0, chunks = 0;
    for (int64_t i = 0; i < n; ++i) total += numel(&g[i]);
    const int64_t chunk = chunk_of(total);
    for (int64_t i = 0; i < n; ++i) {
        const int64_t len = numel(&g[i]);
        tensors += len > 0;
        chunks += disco::ceil_div64(len, chunk);
    }
    return std::min<int64_t>(chunks, disco::ceil_div64(tensors, disco::kGradBatch) * disco::kGradBlocks);
}

// Checks that pointers are device memory, asking the runtime once for each allocation that a call meets in a row.
struct PointerCheck {
    int device;
    uintptr_t lo = 0, hi = 0;
    disco_status operator()(const void *p, int64_t bytes, const char *name)
    {
        const uintptr_t a = (uintptr_t)p;
        if (a >= lo && a < hi && (uintptr_t)bytes <= hi - a) return DISCO_OK;
        const disco_status st = check_pointer(p, name, device);
        if (st != DISCO_OK) return st;
        hipDeviceptr_t base = nullptr;
        size_t size = 0;
        if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)p) == hipSuccess) {
            lo = (uintptr_t)base;
            hi = lo + size;
        } else {
            (void)hipGetLastError();
        }
        return DISCO_OK;
    }
};

disco_status grads_impl(int64_t n, const disco_tensor *grads, bool clip, float max_norm, float eps, disco_tensor *outs,
                        disco_tensor *norm, void *workspace, size_t workspace_bytes, void *stream)
{
    disco_status st;
    if ((st = check_grads(n, grads)) != DISCO_OK) return st;
    if (!norm) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "norm is NULL");
    if (norm->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, "norm must be fp32");
    if (norm->ndim < 0 || norm->ndim > 5 || numel(norm) != 1) return api_fail(DISCO_ERR_SHAPE, "norm must have one element");
    if (clip) {
        if (n > 0 && !outs) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "outs is NULL");
        for (int64_t i = 0; i < n; ++i) {
            if (outs[i].dtype != grads[i].dtype)
                return api_fail(DISCO_ERR_DTYPE, "grads[" + std::to_string(i) + "] and its output's dtypes differ");
            if ((st = same_shape(&outs[i], "outs", &grads[i], -1, 0)) != DISCO_OK) return st;
        }
        if (!(max_norm >= 0.0f)) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "max_norm must not be negative");
        if (!(eps >= 0.0f) || std::isinf(eps)) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    }
    int dev = -1;
    if ((st = current_device(&dev)) != DISCO_OK) return st;
    const size_t need = (size_t)std::max<int64_t>(slots_of(n, grads), 1) * sizeof(double);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 7))
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, "workspace is NULL, not 8-byte aligned or too small");
    if ((st = check_pointer(workspace, "workspace", dev)) != DISCO_OK) return st;
    if ((st = check_pointer(norm->data, "norm", dev)) != DISCO_OK) return st;
    // outputs: disjoint from each other and from the gradients, but for an output that is its own gradient
    struct Span {
        uintptr_t lo, hi;
        bool out;
    };
    std::vector<Span> spans;
    spans.reserve((size_t)n * 2 + 2);
    auto add = [&](const void *p, int64_t bytes, bool out) {
        if (bytes > 0) spans.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, out});
    };
    PointerCheck in{dev}, into{dev};
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t len = numel(&grads[i]), bytes = len * elem_size(grads[i].dtype);
        if (bytes == 0) continue;
        total += len;
        if ((st = in(grads[i].data, bytes, "grads")) != DISCO_OK) return st;
        if (clip && outs[i].data != grads[i].data) {
            if ((st = into(outs[i].data, bytes, "outs")) != DISCO_OK) return st;
            add(outs[i].data, bytes, true);
            add(grads[i].data, bytes, false);
        } else {
            add(grads[i].data, bytes, clip);
        }
    }
    add(norm->data, 4, true);
    add(workspace, (int64_t)need, true);
    auto before = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
    uintptr_t any = 0, out = 0;  // the furthest end of the spans so far, and of the outputs among them
    for (const Span &s : spans) {
        if (s.lo < out || (s.out && s.lo < any))
            return api_fail(DISCO_ERR_INVALID_ARGUMENT, "an output, norm or the workspace overlaps another tensor");
        any = std::max(any, s.hi);
        if (s.out) out = std::max(out, s.hi);
    }
    // The sum's runs go by the gradients alone, so its order and result are one and the same whatever the outputs.
    std::vector<Run> runs;
    runs_of(n, grads, nullptr, &runs);
    double *partial = (double *)workspace;
    hipStream_t sm = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    float *nd = (float *)norm->data;
    int32_t slots = 1;  // partial sums that the scaling pass finds
    disco::GradSmall few, scaled;
    bool done = false;
    if (small_of(runs, total, &few)) {
        scaled.count = 0;
        if (clip) {
            runs_of(n, grads, outs, &runs);
            done = small_of(runs, total, &scaled);
            if (!done) scaled.count = 0;
        }
        e = disco::launch_grad_small(few, scaled, partial, nd, max_norm, eps, sm);
        nd = nullptr;
    } else {
        GradPlan p;
        plan_grads(runs, total, &p);
        int64_t at = 0;
        for (const disco::GradBatch &b : p.batches) {
            if (e == hipSuccess) e = disco::launch_grad_partials(b, blocks_of(b), partial + at, sm);
            at += blocks_of(b);
        }
        slots = (int32_t)p.slots;
        if (e == hipSuccess && (!clip || slots > disco::kGradDirect)) {
            e = disco::launch_grad_total(partial, slots, nd, sm);
            slots = 1;
            nd = nullptr;
        }
        if (clip) runs_of(n, grads, outs, &runs);
    }
    if (clip && !done) {
        GradPlan q;
        plan_grads(runs, total, &q);
        for (size_t i = 0; i < q.batches.size() && e == hipSuccess; ++i) {
            const disco::GradBatch &b = q.batches[q.batches.size() - 1 - i];
            e = disco::launch_grad_scale(b, blocks_of(b), partial, slots, i == 0 ? nd : nullptr, max_norm, eps, sm);
        }
    }
    return launched(e, "gradient norm");
}

// No C++ exception leaves a C entry: what the host allocates (messages, launch tables) may not be had.
template <typename F>
disco_status guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return disco::api_fail_oom();
    }
}

}  // namespace

extern "C" {

disco_status disco_rms_norm(const disco_tensor *x, const disco_tensor *residual, const disco_tensor *w, int axis,
                            float eps, disco_tensor *y, disco_tensor *h, void *stream)
{
    return guarded([&] { return norm_impl(x, residual, w, axis, eps, 0, y, nullptr, h, false, stream); });
}

disco_status disco_rms_norm_f8(const disco_tensor *x, const disco_tensor *residual, const disco_tensor *w, int axis,
                               float eps, int64_t group, disco_tensor *q, disco_tensor *scale, disco_tensor *h,
                               void *stream)
{
    return guarded([&] { return norm_impl(x, residual, w, axis, eps, group, q, scale, h, true, stream); });
}

disco_status disco_dequantize(const disco_tensor *q, const disco_tensor *scale, int axis, int64_t group,
                              disco_tensor *out, void *stream)
{
    return guarded([&]() -> disco_status {
        if (!q || !scale || !out) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "q, scale or out is NULL");
        if (!is_f8(q->dtype)) return api_fail(DISCO_ERR_DTYPE, "q must be e4m3 or e5m2");
        if (scale->dtype != DISCO_F32) return api_fail(DISCO_ERR_DTYPE, "scale must be fp32");
        if (!is_data(out->dtype)) return api_fail(DISCO_ERR_DTYPE, "out has an unsupported dtype");
        View v;
        disco_status st;
        if ((st = view_of(q, "q", axis, &v)) != DISCO_OK) return st;
        if (group < 0 || group % 32 != 0)
            return api_fail(DISCO_ERR_SHAPE, "group must be 0 (the whole axis) or a multiple of 32");
        if (group == 0 || group > v.D) group = v.D;
        const int64_t ngroups = disco::ceil_div64(v.D, group);
        if ((st = same_shape(scale, "scale", q, v.axis, ngroups)) != DISCO_OK) return st;
        if ((st = same_shape(out, "out", q, v.axis, v.D)) != DISCO_OK) return st;
        if (v.N == 0 || v.M == 0) return DISCO_OK;
        const int esz = (int)elem_size(out->dtype);
        if ((st = check_grid(disco::dequant_geom(v.N, v.D, v.M, esz).blocks, 256)) != DISCO_OK) return st;
        int dev = -1;
        if ((st = current_device(&dev)) != DISCO_OK) return st;
        if ((st = check_pointer(q->data, "q", dev)) != DISCO_OK) return st;
        if ((st = check_pointer(scale->data, "scale", dev)) != DISCO_OK) return st;
        if ((st = check_pointer(out->data, "out", dev)) != DISCO_OK) return st;
        const Range ins[2] = {range_of(q, "q"), range_of(scale, "scale")}, outs[1] = {range_of(out, "out")};
        if ((st = check_ranges(outs, 1, ins, 2)) != DISCO_OK) return st;
        disco::DequantLaunch a;
        a.q = (const uint8_t *)q->data; a.scale = (const float *)scale->data; a.out = out->data;
        a.dtype = out->dtype; a.f8 = q->dtype == DISCO_F8_E5M2 ? 1 : 0;
        a.N = v.N; a.D = v.D; a.M = v.M; a.group = (int32_t)group; a.ngroups = (int32_t)ngroups;
        return launched(disco::launch_dequant(a, (hipStream_t)stream), "dequantize");
    });
}

disco_status disco_rms_norm_bwd_workspace(const disco_tensor *h, int axis, size_t *bytes)
{
    return guarded([&]() -> disco_status {
        if (!h || !bytes) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "h or bytes is NULL");
        if (!is_data(h->dtype)) return api_fail(DISCO_ERR_DTYPE, "h has an unsupported dtype");
        View v;
        const disco_status st = view_of(h, "h", axis, &v);
        if (st != DISCO_OK) return st;
        *bytes = disco::norm_bwd_plan(v.N, v.D, v.M, (int)elem_size(h->dtype)).bytes(v.N, v.D);
        return DISCO_OK;
    });
}

disco_status disco_rms_norm_bwd(const disco_tensor *h, const disco_tensor *w, const disco_tensor *gy,
                                const disco_tensor *gh, int axis, float eps, disco_tensor *gx, disco_tensor *dw,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> disco_status {
        if (!h || !w || !gy || !gx || !dw) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "h, w, gy, gx or dw is NULL");
        if (!is_data(h->dtype)) return api_fail(DISCO_ERR_DTYPE, "h has an unsupported dtype");
        if (gy->dtype != h->dtype || gx->dtype != h->dtype || (gh && gh->dtype != h->dtype))
            return api_fail(DISCO_ERR_DTYPE, "h, gy, gh and gx dtypes differ");
        if (dw->dtype != w->dtype) return api_fail(DISCO_ERR_DTYPE, "w and dw dtypes differ");
        View v;
        disco_status st;
        if ((st = view_of(h, "h", axis, &v)) != DISCO_OK) return st;
        if ((st = check_weight(w, "w", h, v.D)) != DISCO_OK) return st;
        if ((st = check_weight(dw, "dw", h, v.D)) != DISCO_OK) return st;
        if ((st = same_shape(gy, "gy", h, v.axis, v.D)) != DISCO_OK) return st;
        if ((st = same_shape(gx, "gx", h, v.axis, v.D)) != DISCO_OK) return st;
        if (gh && (st = same_shape(gh, "gh", h, v.axis, v.D)) != DISCO_OK) return st;
        if (!(eps >= 0.0f) || std::isinf(eps))
            return api_fail(DISCO_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
        const disco::BwdPlan plan = disco::norm_bwd_plan(v.N, v.D, v.M, (int)elem_size(h->dtype));
        const size_t need = plan.bytes(v.N, v.D);
        int dev = -1;
        if ((st = current_device(&dev)) != DISCO_OK) return st;
        if ((st = check_pointer(dw->data, "dw", dev)) != DISCO_OK) return st;
        Range ins[4] = {range_of(h, "h"), range_of(w, "w"), range_of(gy, "gy")}, outs[3] = {range_of(gx, "gx"), range_of(dw, "dw")};
        int ni = 3;
        if (plan.blocks > 0) {  // without points only dw is written, as zeros
            if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3))
                return api_fail(DISCO_ERR_INVALID_ARGUMENT, "workspace is NULL, not 4-byte aligned or too small");
            if ((st = check_pointer(h->data, "h", dev)) != DISCO_OK) return st;
            if ((st = check_pointer(w->data, "w", dev)) != DISCO_OK) return st;
            if ((st = check_pointer(gy->data, "gy", dev)) != DISCO_OK) return st;
            if ((st = check_pointer(gx->data, "gx", dev)) != DISCO_OK) return st;
            if (gh && (st = check_pointer(gh->data, "gh", dev)) != DISCO_OK) return st;
            if ((st = check_pointer(workspace, "workspace", dev)) != DISCO_OK) return st;
            if (gh) ins[ni++] = range_of(gh, "gh");
            outs[2] = {(uintptr_t)workspace, (uintptr_t)workspace + need, "workspace"};
            if ((st = check_ranges(outs, 3, ins, ni)) != DISCO_OK) return st;
        }
        disco::NormLaunch a;
        a.x = h->data; a.r = gh ? gh->data : nullptr; a.gy = gy->data; a.w = w->data;
        a.y = gx->data; a.dw = dw->data; a.workspace = workspace;
        a.dtype = h->dtype; a.wf32 = w->dtype == DISCO_F32;
        a.N = v.N; a.D = v.D; a.M = v.M; a.eps = eps;
        return launched(disco::launch_norm_bwd(a, (hipStream_t)stream), "norm backward");
    });
}

disco_status disco_grad_norm_workspace(int64_t n, const disco_tensor *grads, size_t *bytes)
{
    return guarded([&]() -> disco_status {
        if (!bytes) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "bytes is NULL");
        const disco_status st = check_grads(n, grads);
        if (st != DISCO_OK) return st;
        *bytes = (size_t)std::max<int64_t>(slots_of(n, grads), 1) * sizeof(double);
        return DISCO_OK;
    });
}

disco_status disco_grad_norm(int64_t n, const disco_tensor *grads, disco_tensor *norm, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        return grads_impl(n, grads, false, 0.0f, 0.0f, nullptr, norm, workspace, workspace_bytes, stream);
    });
}

disco_status disco_clip_grads(int64_t n, const disco_tensor *grads, float max_norm, float eps, disco_tensor *outs,
                              disco_tensor *norm, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        return grads_impl(n, grads, true, max_norm, eps, outs, norm, workspace, workspace_bytes, stream);
    });
}

}  // extern "C"
