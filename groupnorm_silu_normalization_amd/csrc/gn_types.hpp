// gn_types.hpp -- element types, SiLU and the 16-byte accesses shared by the
// library's kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gnsilu {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ---- element types ---------------------------------------------------------
// storage: the in-memory type; to_f32 widens exactly; pack2 rounds two fp32
// values to the type (round to nearest even: v_cvt_pk_bf16_f32 /
// v_cvt_pk_f16_f32 on gfx950) and packs them, lower address first.
struct Bf16 {
    using storage = uint16_t;
    __device__ __forceinline__ static float to_f32(uint16_t b) {
        return __uint_as_float(static_cast<uint32_t>(b) << 16);
    }
    __device__ __forceinline__ static float lo(uint32_t w) { return __uint_as_float(w << 16); }
    __device__ __forceinline__ static float hi(uint32_t w) {
        return __uint_as_float(w & 0xffff0000u);
    }
    __device__ __forceinline__ static uint32_t pack2(float a, float b) {
        f32x2 v = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    __device__ __forceinline__ static uint16_t from_f32(float f) {
        return static_cast<uint16_t>(pack2(f, 0.0f) & 0xffffu);
    }
};

struct Fp16 {
    using storage = uint16_t;
    __device__ __forceinline__ static float to_f32(uint16_t b) {
        return static_cast<float>(__builtin_bit_cast(_Float16, b));
    }
    __device__ __forceinline__ static float lo(uint32_t w) {
        return to_f32(static_cast<uint16_t>(w & 0xffffu));
    }
    __device__ __forceinline__ static float hi(uint32_t w) {
        return to_f32(static_cast<uint16_t>(w >> 16));
    }
    __device__ __forceinline__ static uint32_t pack2(float a, float b) {
        f32x2 v = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
    __device__ __forceinline__ static uint16_t from_f32(float f) {
        return static_cast<uint16_t>(pack2(f, 0.0f) & 0xffffu);
    }
};

struct F32 {
    using storage = float;
    __device__ __forceinline__ static float to_f32(float v) { return v; }
    __device__ __forceinline__ static float from_f32(float f) { return f; }
};

// SiLU(t) = t * sigmoid(t) = t / (1 + e^-t), with e^-t = 2^(-t*log2 e):
// one v_exp_f32 and one v_rcp_f32.  t << 0 gives 2^(+big) = inf, 1/inf = 0,
// t*0 = -0, the limit; t >> 0 gives t.
__device__ __forceinline__ float silu_f32(float t) {
    const float e = __builtin_amdgcn_exp2f(t * -1.4426950408889634f);
    return t * __builtin_amdgcn_rcpf(1.0f + e);
}

// NT: the access carries the nontemporal hint (streaming cache policy), for
// data the pass touches once.
template <bool NT, class T>
__device__ __forceinline__ T ld(const T *p) {
    if constexpr (NT)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}
template <bool NT, class T>
__device__ __forceinline__ void st(T *p, T v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

// ---- one access of W consecutive elements -----------------------------------
template <class D, int W> struct Vec;

template <class D> struct Vec16x8 {  // 8 16-bit values, one 16-byte access
    u32x4 w;
    __device__ __forceinline__ float get(int j) const {
        const uint32_t word = w[j >> 1];
        return (j & 1) ? D::hi(word) : D::lo(word);
    }
    template <bool NT>
    __device__ __forceinline__ void load(const uint16_t *p) {
        w = ld<NT>(reinterpret_cast<const u32x4 *>(p));
    }
    template <bool NT>
    __device__ __forceinline__ static void store(uint16_t *p, const float *o) {
        u32x4 v;
        v[0] = D::pack2(o[0], o[1]);
        v[1] = D::pack2(o[2], o[3]);
        v[2] = D::pack2(o[4], o[5]);
        v[3] = D::pack2(o[6], o[7]);
        st<NT>(reinterpret_cast<u32x4 *>(p), v);
    }
};
template <> struct Vec<Bf16, 8> : Vec16x8<Bf16> {};
template <> struct Vec<Fp16, 8> : Vec16x8<Fp16> {};

template <> struct Vec<F32, 4> {  // 4 fp32 values, one 16-byte access
    u32x4 w;
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(w[j]); }
    template <bool NT>
    __device__ __forceinline__ void load(const float *p) {
        w = ld<NT>(reinterpret_cast<const u32x4 *>(p));
    }
    template <bool NT>
    __device__ __forceinline__ static void store(float *p, const float *o) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(o[j]);
        st<NT>(reinterpret_cast<u32x4 *>(p), v);
    }
};

template <class D> struct Vec<D, 1> {  // one value
    typename D::storage b;
    __device__ __forceinline__ float get(int) const { return D::to_f32(b); }
    template <bool NT>
    __device__ __forceinline__ void load(const typename D::storage *p) { b = ld<NT>(p); }
    template <bool NT>
    __device__ __forceinline__ static void store(typename D::storage *p, const float *o) {
        st<NT>(p, D::from_f32(o[0]));
    }
};

// gamma and beta: C values each, or null (1 and 0), of element type kF32,
// kBf16 or kF16; widened exactly to fp32 before the fold.
struct Affine {
    enum : int { kF32 = 0, kBf16 = 1, kF16 = 2 };
    const void *gamma;
    const void *beta;
    int type;
};

}  // namespace gnsilu
