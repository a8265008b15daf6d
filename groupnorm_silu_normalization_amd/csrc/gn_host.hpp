// gn_host.hpp -- host-side pieces shared by the library's entry points: the
// dtype argument, the device and pointer checks, launch status.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gn_types.hpp"
#include "gnsilu.h"

namespace gnsilu {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// The dtype argument: a gn_dtype for x and y in the low bits, or-ed with at
// most one GN_AFFINE_* value for gamma and beta (none: fp32).
inline int x_dtype(int dtype) { return dtype & ~GN_AFFINE_MASK; }
inline bool valid_dtype(int dtype) {
    const int xd = x_dtype(dtype), ad = dtype & GN_AFFINE_MASK;
    return (xd == GN_DTYPE_BF16 || xd == GN_DTYPE_F16 || xd == GN_DTYPE_F32) &&
           (ad == 0 || ad == GN_AFFINE_F32 || ad == GN_AFFINE_BF16 || ad == GN_AFFINE_F16);
}
inline int affine_type(int dtype) {
    switch (dtype & GN_AFFINE_MASK) {
        case GN_AFFINE_BF16: return Affine::kBf16;
        case GN_AFFINE_F16: return Affine::kF16;
        default: return Affine::kF32;
    }
}
inline int64_t elem_bytes(int dtype) { return x_dtype(dtype) == GN_DTYPE_F32 ? 4 : 2; }

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    gn_status enter(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) return GN_DEVICE_ERROR;
        if (prev != dev) {
            if (hipSetDevice(dev) != hipSuccess) return GN_DEVICE_ERROR;
            changed = true;
        }
        return GN_OK;
    }
    ~DeviceGuard() {
        if (changed) (void)hipSetDevice(prev);
    }
};

inline gn_status stream_device(hipStream_t s, int *dev) {
    if (s == nullptr) return hipGetDevice(dev) == hipSuccess ? GN_OK : GN_DEVICE_ERROR;
    hipDevice_t d;
    if (hipStreamGetDevice(s, &d) != hipSuccess) {
        (void)hipGetLastError();
        return GN_INVALID_ARGUMENT;
    }
    *dev = static_cast<int>(d);
    return GN_OK;
}

// A pointer the kernels may dereference: device (or managed) memory on `dev`.
inline bool on_device(const void *ptr, int dev) {
    if (ptr == nullptr) return true;  // optional argument absent
    hipPointerAttribute_t a;
    if (hipPointerGetAttributes(&a, ptr) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    if (a.type != hipMemoryTypeDevice && a.type != hipMemoryTypeManaged) return false;
    return a.device == dev;
}

// Everything a compute entry point needs after its argument checks.
struct Call {
    hipStream_t stream;
    int dev;
    DeviceGuard guard;
};

inline gn_status begin_call(void *stream, std::initializer_list<const void *> ptrs, Call *c) {
    c->stream = static_cast<hipStream_t>(stream);
    gn_status st = stream_device(c->stream, &c->dev);
    if (st != GN_OK) return st;
    st = c->guard.enter(c->dev);
    if (st != GN_OK) return st;
    for (const void *q : ptrs)
        if (!on_device(q, c->dev)) return GN_UNSUPPORTED;
    return GN_OK;
}

// gamma and beta aligned to their element type.
inline gn_status check_affine(const void *gamma, const void *beta, int dtype) {
    const uintptr_t m = affine_type(dtype) == Affine::kF32 ? 3u : 1u;
    for (const void *q : {gamma, beta})
        if (q != nullptr && (reinterpret_cast<uintptr_t>(q) & m) != 0) return GN_UNSUPPORTED;
    return GN_OK;
}

inline gn_status finish_launch() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GN_OK : GN_DEVICE_ERROR;
}

}  // namespace gnsilu
