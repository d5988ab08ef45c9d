// tensor_checks.hpp — the argument checks that the operators without a psi share (host side).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "api_common.hpp"
#include "disco.h"

namespace disco {

inline int64_t elem_size(int dtype)
{
    return dtype == DISCO_F32 ? 4 : dtype == DISCO_BF16 || dtype == DISCO_F16 ? 2 : 1;
}

inline bool is_data(int dtype) { return dtype == DISCO_F32 || dtype == DISCO_BF16 || dtype == DISCO_F16; }
inline bool is_f8(int dtype) { return dtype == DISCO_F8_E4M3 || dtype == DISCO_F8_E5M2; }

inline int64_t numel(const disco_tensor *t)
{
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

// The launches' device: the current one, gfx950.
inline disco_status current_device(int *dev)
{
    if (hipGetDevice(dev) != hipSuccess) {
        (void)hipGetLastError();
        return api_fail(DISCO_ERR_HIP, "hipGetDevice failed");
    }
    if (*dev < 0 || *dev >= 64) return api_fail(DISCO_ERR_INVALID_ARGUMENT, "device ordinal out of range");
    static std::atomic<int> ok[64];  // the architecture of a device cannot change
    if (ok[*dev].load() != 1) {
        const disco_status st = api_check_device(*dev);
        if (st != DISCO_OK) return st;
        ok[*dev].store(1);
    }
    return DISCO_OK;
}

inline disco_status check_pointer(const void *p, const char *name, int device)
{
    if (!p) return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(name) + "->data is NULL");
    hipPointerAttribute_t attr;
    if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
        (void)hipGetLastError();
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(name) + "->data is not device memory");
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged)
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(name) + "->data is not device memory");
    if (attr.device != device)
        return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(name) + "->data lives on another device");
    return DISCO_OK;
}

struct View {  // a tensor around its normalised axis
    int64_t N = 1, D = 0, M = 1;
    int axis = 0;
};

// Dimensions of x around `axis` (negative: from the end); sizes whose products leave 63 bits are refused.
inline disco_status view_of(const disco_tensor *x, const char *name, int axis, View *v)
{
    if (x->ndim < 1 || x->ndim > 5) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " must have 1 to 5 dimensions");
    if (axis < 0) axis += x->ndim;
    if (axis < 0 || axis >= x->ndim) return api_fail(DISCO_ERR_SHAPE, "axis out of range");
    v->axis = axis;
    int64_t all = 8;
    for (int i = 0; i < x->ndim; ++i) {
        const int64_t s = x->shape[i];
        if (s < 0) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has a negative dimension");
        if (s > 0 && all > INT64_MAX / s) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has too many elements");
        if (s > 0) all *= s;
        if (i < axis) v->N *= s;
        else if (i > axis) v->M *= s;
        else v->D = s;
    }
    if (v->D < 1) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has no elements along the axis");
    if (v->D > (1 << 30)) return api_fail(DISCO_ERR_SHAPE, "the axis is longer than 2^30");
    return DISCO_OK;
}

inline disco_status same_shape(const disco_tensor *t, const char *name, const disco_tensor *x, int axis, int64_t along)
{
    if (t->ndim != x->ndim) return api_fail(DISCO_ERR_SHAPE, std::string(name) + " has the wrong number of dimensions");
    for (int i = 0; i < x->ndim; ++i) {
        const int64_t want = i == axis ? along : x->shape[i];
        if (t->shape[i] != want)
            return api_fail(DISCO_ERR_SHAPE, std::string(name) + " dimension " + std::to_string(i) + " is " +
                                             std::to_string(t->shape[i]) + ", expected " + std::to_string(want));
    }
    return DISCO_OK;
}

struct Range {
    uintptr_t lo, hi;
    const char *name;
};

inline Range range_of(const disco_tensor *t, const char *name)
{
    const uintptr_t lo = (uintptr_t)t->data;
    return {lo, lo + (uintptr_t)(numel(t) * elem_size(t->dtype)), name};
}

// Outputs may share no byte with each other or with an input.
inline disco_status check_ranges(const Range *outs, int no, const Range *ins, int ni)
{
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni + i; ++j) {
            const Range &b = j < ni ? ins[j] : outs[j - ni];
            if (outs[i].lo < b.hi && b.lo < outs[i].hi)
                return api_fail(DISCO_ERR_INVALID_ARGUMENT, std::string(outs[i].name) + " overlaps " + b.name);
        }
    }
    return DISCO_OK;
}

inline disco_status check_grid(int64_t blocks, int64_t threads)
{
    if (blocks > INT32_MAX || blocks * threads > (int64_t)UINT32_MAX)
        return api_fail(DISCO_ERR_SHAPE, "the tensor needs more workgroups than a launch has");
    return DISCO_OK;
}

inline disco_status launched(hipError_t e, const char *what)
{
    if (e == hipSuccess) return DISCO_OK;
    return api_fail(DISCO_ERR_HIP, std::string(what) + " launch failed: " + hipGetErrorString(e));
}

}  // namespace disco
