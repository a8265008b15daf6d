// gn_rows8.hpp -- rows in 8 bits with one scale each: the device side of the
// format, shared by the kernels that write it.
//
// Of a row t of fp32 values with the largest magnitude `top` the code of t[c] is
//     q = rint(127 * t[c] / top)      (half to even, of the exact quotient)
// and stands for q * top / 127.  One factor common to the whole row (the
// root-mean-square norm's rstd) does not change q, so codes never depend on the
// order of a sum.  A row that holds an infinity or a NaN has the scale NaN and
// codes 0; a row of zeros has codes 0.
//
// The quotient is taken as t * (127 * (1 / top)) with v_rcp_f32 (one unit in the
// last place), one rounding and a fused product: off by less than 127 * 1.5 * 2^-23,
// which is less than 2^-15, so only a value that close to a border between two codes
// may get the wrong one.  Those (one value in 2^14) are settled in fp64, where
// 127 * t - q * top and top / 2 are exact: 31 bits of products.
#pragma once

#include "gn_rows.hpp"

namespace gnsilu {

// What a row's values are multiplied by: 127 / top, with values and `top` brought
// nearer to one first where 1 / top would not be a normal number (v_rcp_f32 gives 0
// for top > 2^126) or 127 / top would leave fp32's range.  By powers of two: only
// values below 2^-26 of a row above 2^100 round, far below half a code.
struct Rows8Scale {
    float top, inv, up;
    uint32_t keep;  // mask of the codes' bytes: 0 for a row without values
    // top_bits: the largest |t| as bits (a NaN's are above infinity's)
    __device__ __forceinline__ explicit Rows8Scale(uint32_t top_bits) {
        const bool none = top_bits == 0u || top_bits >= 0x7f800000u;
        top = none ? 1.0f : __uint_as_float(top_bits);
        up = top < 0x1p-100f ? 0x1p100f : top > 0x1p100f ? 0x1p-100f : 1.0f;
        inv = 127.0f * __builtin_amdgcn_rcpf(top * up);
        keep = none ? 0u : ~0u;
    }
    // top / 127; NaN, 0 or the quotient
    __device__ __forceinline__ static float step(uint32_t top_bits) {
        const float s = __uint_as_float(top_bits) / 127.0f;
        return top_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s;
    }
    // top / 127 * rstd, where top / 127 alone may be subnormal
    __device__ __forceinline__ static float step(uint32_t top_bits, float rstd) {
        const bool small = top_bits < 0x0d800000u;  // 2^-100
        const float s = step(__float_as_uint(__uint_as_float(top_bits) * (small ? 0x1p100f : 1.0f)));
        return s * rstd * (small ? 0x1p-100f : 1.0f);
    }
};

// A value next to a border between two codes: its code among q and q's neighbours.
__device__ __forceinline__ float rows8_settle(float t, float top, float q) {
    const double half = 0.5 * static_cast<double>(top);
    const double off = static_cast<double>(t) * 127.0 - static_cast<double>(q) * static_cast<double>(top);
    const float to = off < 0.0 ? -1.0f : 1.0f;
    const double a = off < 0.0 ? -off : off;
    const bool odd = (static_cast<int>(q) & 1) != 0;
    return a > half || (a == half && odd) ? q + to : q;
}

// W codes of t.  rint by adding 1.5 * 2^23: the sum's low byte is the code in
// two's complement (as in block8_encode).
template <int W>
__device__ __forceinline__ Codes<W> rows8_encode(const float (&t)[W], const Rows8Scale &s) {
    uint32_t b[W];
    float far = 0.0f, v[W];
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = t[j];
    if (s.up != 1.0f) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] *= s.up;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const float r = fmaf(v[j], s.inv, 12582912.0f);
        b[j] = __float_as_uint(r);
        far = fmaxf(far, fabsf(fmaf(v[j], s.inv, 12582912.0f - r)));
    }
    if (far > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float q = __uint_as_float(b[j]) - 12582912.0f;
            b[j] = __float_as_uint(rows8_settle(t[j], s.top, q) + 12582912.0f);
        }
    }
    Codes<W> q;
    if constexpr (W == 1) {
        q.w = b[0] & s.keep & 0xffu;
    } else {
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
            q.set4(k, (__builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0c0c0400u) |
                       __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000c0cu)) &
                          s.keep);
    }
    return q;
}

}  // namespace gnsilu
