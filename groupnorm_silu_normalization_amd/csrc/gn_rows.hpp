// gn_rows.hpp -- device pieces shared by the row kernels (layer norm, the
// backward passes, the 8-bit checkpoints): accesses of W consecutive channels
// at any element alignment, lane-group sums and the 8-bit block format.
//
// A row of C channels is P = ceil(C / W) pieces of W channels, W = 16 bytes'
// worth of the element type (1 when C is smaller than that).  Piece p covers
// channels p*W .. p*W+W-1; when W does not divide C the last piece would run
// past the row, so it is read at channel C-W instead and its first `lo`
// channels, which the piece before it covers, are left out of every sum.
// Every lane thus makes the same full-width accesses whatever C is.  Rows of
// such a C start at any multiple of the element size: the accesses are
// declared with that alignment, which gfx950 serves with the same wide
// instructions (unaligned access mode, on for every HSA queue).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gn_types.hpp"

namespace gnsilu {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// ---- one piece -----------------------------------------------------------------
// NT: nontemporal, for data that no later pass reads from a cache.
template <class D, int W> struct Piece;

template <class D> struct Piece16x8 {
    u32x4 w;
    __device__ __forceinline__ float get(int j) const {
        return (j & 1) ? D::hi(w[j >> 1]) : D::lo(w[j >> 1]);
    }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
    template <bool NT>
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (NT)
            w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2 *>(p));
        else
            w = *reinterpret_cast<const u32x4_a2 *>(p);
    }
    template <bool NT>
    __device__ __forceinline__ static void store(uint16_t *p, const float (&o)[8]) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = D::pack2(o[2 * j], o[2 * j + 1]);
        if constexpr (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2 *>(p));
        else
            *reinterpret_cast<u32x4_a2 *>(p) = v;
    }
};
template <> struct Piece<Bf16, 8> : Piece16x8<Bf16> {};
template <> struct Piece<Fp16, 8> : Piece16x8<Fp16> {};

template <> struct Piece<F32, 4> {
    u32x4 w;
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(w[j]); }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
    template <bool NT>
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (NT)
            w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4 *>(p));
        else
            w = *reinterpret_cast<const u32x4_a4 *>(p);
    }
    template <bool NT>
    __device__ __forceinline__ static void store(float *p, const float (&o)[4]) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(o[j]);
        if constexpr (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4 *>(p));
        else
            *reinterpret_cast<u32x4_a4 *>(p) = v;
    }
};

template <class D> struct Piece<D, 1> {
    typename D::storage b;
    __device__ __forceinline__ float get(int) const { return D::to_f32(b); }
    __device__ __forceinline__ void opaque() {}
    template <bool NT>
    __device__ __forceinline__ void load(const typename D::storage *p) { b = ld<NT>(p); }
    template <bool NT>
    __device__ __forceinline__ static void store(typename D::storage *p, const float (&o)[1]) {
        st<NT>(p, D::from_f32(o[0]));
    }
};

// Stores the channels j >= lo of a piece one by one (the last piece of a row
// whose other channels another lane owns).
template <class D, int W>
__device__ __forceinline__ void store_from(typename D::storage *p, const float (&o)[W], int lo) {
#pragma unroll
    for (int j = 0; j < W; ++j)
        if (j >= lo) p[j] = D::from_f32(o[j]);
}

// W consecutive values of gamma or beta, widened exactly; `absent` where the
// pointer is null.  Aligned to their element type only.
template <int W>
__device__ __forceinline__ void load_affine(const void *p, int type, int64_t c, float absent,
                                            float (&o)[W]) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = absent;
        return;
    }
    if (type == Affine::kF32) {
        const float *f = static_cast<const float *>(p) + c;
        if constexpr (W == 1) {
            o[0] = f[0];
        } else {
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const u32x4 v = *reinterpret_cast<const u32x4_a4 *>(f + j);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[j + k] = __uint_as_float(v[k]);
            }
        }
        return;
    }
    const uint16_t *h = static_cast<const uint16_t *>(p) + c;
    uint32_t w[(W + 1) / 2];
    if constexpr (W == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4_a2 *>(h);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j];
    } else if constexpr (W == 4) {
        const u32x2 v = *reinterpret_cast<const u32x2_a2 *>(h);
        w[0] = v[0];
        w[1] = v[1];
    } else {
        w[0] = h[0];
    }
    if (type == Affine::kBf16) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = (j & 1) ? Bf16::hi(w[j >> 1]) : Bf16::lo(w[j >> 1]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = (j & 1) ? Fp16::hi(w[j >> 1]) : Fp16::lo(w[j >> 1]);
    }
}

// A gradient of gamma or beta, rounded once to their element type.
__device__ __forceinline__ void store_affine(void *p, int type, int64_t c, float v) {
    if (type == Affine::kF32)
        static_cast<float *>(p)[c] = v;
    else if (type == Affine::kBf16)
        static_cast<uint16_t *>(p)[c] = Bf16::from_f32(v);
    else
        static_cast<uint16_t *>(p)[c] = Fp16::from_f32(v);
}

// ---- sums over aligned groups of N lanes (N a power of two up to 64) -------------
// The butterfly's five first steps move data within a row of 16 lanes (DPP) or
// swap rows (v_permlane16_swap / v_permlane32_swap): no LDS round trips.  Both
// operands of every step's sum are the same two values in every lane of the
// pair, so all N lanes end with the same bits.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false));
}
constexpr int kDppXor1 = 0xB1;        // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2,3,0,1]
constexpr int kDppHalfMirror = 0x141; // lane i of a half row <-> 7 - i
constexpr int kDppMirror = 0x140;     // lane i of a row <-> 15 - i
constexpr int kDppRor4 = 0x124;       // rotations within a row of 16 lanes
constexpr int kDppRor8 = 0x128;

template <int N, class F>
__device__ __forceinline__ uint32_t lane_fold(uint32_t v, F op) {
    if constexpr (N >= 2) v = op(v, dpp<kDppXor1>(v));
    if constexpr (N >= 4) v = op(v, dpp<kDppXor2>(v));
    // the lanes of a quad are equal now, so a mirror pairs the quads
    if constexpr (N >= 8) v = op(v, dpp<kDppHalfMirror>(v));
    if constexpr (N >= 16) v = op(v, dpp<kDppMirror>(v));
    if constexpr (N >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if constexpr (N >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
    return __uint_as_float(lane_fold<N>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int N>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
    return lane_fold<N>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// ---- the 8-bit block format --------------------------------------------------------
// Blocks of kBlock8 consecutive channels of a row (the last one of a row may be
// shorter) share a scale byte E, the exponent field (biased by 127) of the
// block's largest magnitude as an fp32 number; a value x is kept as
//     code = clamp(rint(x * 2^(133 - E)), -127, 127)
// and stands for code * 2^(E - 133): the element and scale formats of OCP MX
// "MXINT8".  Powers of two scale exactly, so the only rounding is rint's and
// the code is the same in any precision.  A block holding an infinity or a NaN
// has E = 255 and stands for NaN throughout.
constexpr int kBlock8 = 32;

// 2^(E - 133); NaN for E = 255, by bits: a select of the NaN would be moved
// behind every product with the step.
__device__ __forceinline__ float block8_step(uint32_t E) {
    const float s = __builtin_ldexpf(1.0f, static_cast<int>(E) - 133);
    return __uint_as_float(__float_as_uint(s) | (E == 255u ? 0x7fc00000u : 0u));
}

template <int W> struct Codes;  // a piece's W codes, one byte each
template <> struct Codes<8> {
    u32x2 w;
    __device__ __forceinline__ void load(const int8_t *p) {
        w = *reinterpret_cast<const u32x2_a1 *>(p);
    }
    template <bool NT> __device__ __forceinline__ void store(int8_t *p) const {
        if constexpr (NT)
            __builtin_nontemporal_store(w, reinterpret_cast<u32x2_a1 *>(p));
        else
            *reinterpret_cast<u32x2_a1 *>(p) = w;
    }
    __device__ __forceinline__ int get(int j) const {
        return static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
    }
    __device__ __forceinline__ void set4(int q, uint32_t v) { w[q] = v; }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
};
template <> struct Codes<4> {
    uint32_t w;
    __device__ __forceinline__ void load(const int8_t *p) {
        w = *reinterpret_cast<const u32_a1 *>(p);
    }
    template <bool NT> __device__ __forceinline__ void store(int8_t *p) const {
        if constexpr (NT)
            __builtin_nontemporal_store(w, reinterpret_cast<u32_a1 *>(p));
        else
            *reinterpret_cast<u32_a1 *>(p) = w;
    }
    __device__ __forceinline__ int get(int j) const { return static_cast<int8_t>(w >> (8 * j)); }
    __device__ __forceinline__ void set4(int, uint32_t v) { w = v; }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
};
template <> struct Codes<1> {
    uint32_t w;
    __device__ __forceinline__ void load(const int8_t *p) { w = static_cast<uint8_t>(*p); }
    template <bool NT> __device__ __forceinline__ void store(int8_t *p) const {
        *p = static_cast<int8_t>(w);
    }
    __device__ __forceinline__ int get(int) const { return static_cast<int8_t>(w); }
    __device__ __forceinline__ void opaque() {}
};

// A piece of saved values: its codes and the scale bytes of its first and last
// channel (different only for a last piece read at C-W).
template <int W, bool TAIL> struct Piece8At {  // where a row's piece at channel c lies
    const int8_t *q;
    const uint8_t *e0, *e1;
    __device__ __forceinline__ Piece8At(const int8_t *codes, const uint8_t *scales, int64_t row,
                                        int C, int c)
        : q(codes + row * C + c),
          e0(scales + row * ((C + kBlock8 - 1) / kBlock8) + c / kBlock8),
          e1(scales + row * ((C + kBlock8 - 1) / kBlock8) + (c + W - 1) / kBlock8) {}
};
template <int W, bool TAIL> struct Piece8 {
    Codes<W> q;
    uint32_t e0, e1;
    // `dq` codes and `de` scales further on
    __device__ __forceinline__ void load(const Piece8At<W, TAIL> &at, int64_t dq, int64_t de) {
        q.load(at.q + dq);
        e0 = at.e0[de];
        if constexpr (TAIL) e1 = at.e1[de];
    }
    // The values less mu, in one fma each.  edge: whether a lane of the wave
    // holds a last piece read at C-W (wave_has_edge); only that one can lie in
    // two blocks.
    __device__ __forceinline__ void widen_less(int c, const float (&mu)[W], bool edge,
                                               float (&o)[W]) const {
        const float s0 = block8_step(e0);
        if (TAIL && edge) {
            const float s1 = block8_step(e1);
            const int split = kBlock8 - c % kBlock8;
#pragma unroll
            for (int j = 0; j < W; ++j)
                o[j] = fmaf(static_cast<float>(q.get(j)), j < split ? s0 : s1, -mu[j]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = fmaf(static_cast<float>(q.get(j)), s0, -mu[j]);
        }
    }
    __device__ __forceinline__ void widen(int c, bool edge, float (&o)[W]) const {
        const float s0 = block8_step(e0);
        if (TAIL && edge) {
            const float s1 = block8_step(e1);
            const int split = kBlock8 - c % kBlock8;
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = static_cast<float>(q.get(j)) * (j < split ? s0 : s1);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = static_cast<float>(q.get(j)) * s0;
        }
    }
    __device__ __forceinline__ void opaque() { q.opaque(); }
};

// Whether a lane of the wave holds a last piece whose first channels are
// another piece's (0 < lo < W): the work such a piece needs is left out of the
// waves that have none.
template <int W, bool TAIL> __device__ __forceinline__ bool wave_has_edge(int lo) {
    return TAIL && __builtin_amdgcn_ballot_w64(lo > 0 && lo < W) != 0;
}

// Which bits of a raw piece count for its block's maximum: the magnitudes of
// the channels j >= lo.  Cleared words cost nothing, as the signs have to be
// masked off anyway.
template <class D, int W> struct Magnitudes {
    static constexpr bool k16 = sizeof(typename D::storage) == 2;
    static constexpr int kWords = W == 8 ? 4 : W;
    uint32_t m[kWords];
    __device__ __forceinline__ explicit Magnitudes(int lo) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (k16 && W == 8)
                m[k] = (2 * k >= lo ? 0x7fffu : 0u) | (2 * k + 1 >= lo ? 0x7fff0000u : 0u);
            else if constexpr (k16)
                m[k] = k >= lo ? 0x7fffu : 0u;
            else
                m[k] = k >= lo ? 0x7fffffffu : 0u;
        }
    }
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max2_u16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                        __builtin_bit_cast(u16x2, b)));
}

// The scale byte of the block that the calling lane's piece belongs to; the
// block's pieces are held by GROUP consecutive, aligned lanes -- or, where rows
// are that short, by `group` of them, a smaller power of two, the same for all
// lanes -- all of which call this.  Magnitudes of every type order like their bits, so the maxima
// are taken on the raw words, two 16-bit values at a time.
template <class D, int W, int GROUP>
__device__ __forceinline__ uint32_t block8_exponent(const Piece<D, W> &v,
                                                    const Magnitudes<D, W> &mag,
                                                    int group = GROUP) {
    uint32_t top;
    if constexpr (W == 8) {
        top = max2_u16(max2_u16(v.w[0] & mag.m[0], v.w[1] & mag.m[1]),
                       max2_u16(v.w[2] & mag.m[2], v.w[3] & mag.m[3]));
        const uint32_t hi = top >> 16, lo = top & 0xffffu;
        top = hi > lo ? hi : lo;
    } else if constexpr (W == 4) {
        top = v.w[0] & mag.m[0];
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const uint32_t b = v.w[k] & mag.m[k];
            top = b > top ? b : top;
        }
    } else if constexpr (sizeof(v.b) == 2) {
        top = v.b & mag.m[0];
    } else {
        top = __float_as_uint(v.b) & mag.m[0];
    }
    if (group >= GROUP) {
        top = lane_max<GROUP>(top);
    } else if (group >= 2) {  // rows of fewer lanes
        top = lane_max<2>(top);
        if (group >= 4) top = max(top, dpp<kDppXor2>(top));
    }
    if constexpr (std::is_same<D, Bf16>::value)
        return top >> 7;
    else if constexpr (std::is_same<D, Fp16>::value)
        return __float_as_uint(Fp16::to_f32(static_cast<uint16_t>(top))) >> 23;
    else
        return top >> 23;
}

// rint by adding 1.5 * 2^23: the sum's low byte is the code in two's
// complement (the sum is rounded to an integer, half to even).
template <int W>
__device__ __forceinline__ Codes<W> block8_encode(const float (&v)[W], uint32_t E) {
    uint32_t b[W];
    const int e = 133 - static_cast<int>(E);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const float t = __builtin_ldexpf(v[j], e);
        b[j] = __float_as_uint(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f) + 12582912.0f);
    }
    const uint32_t keep = E == 255u ? 0u : ~0u;
    Codes<W> q;
    if constexpr (W == 1) {
        q.w = b[0] & keep;
    } else {
        // v_perm_b32: selector bytes 0-3 take the second operand's bytes, 4-7
        // the first's, 12 zero
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
            q.set4(k, (__builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0c0c0400u) |
                       __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000c0cu)) &
                          keep);
    }
    return q;
}

// Writes a piece's codes and, from the block's first piece, its scale, into a
// row's codes and scales.  c: the piece's first channel in memory; lo: its
// first own channel.
template <int W, bool TAIL, bool NT>
__device__ __forceinline__ void store_block8(const Codes<W> &q, uint32_t E, int8_t *codes,
                                             uint8_t *scales, int c, int lo) {
    int8_t *p = codes + c;
    if (!TAIL || lo == 0) {
        q.template store<NT>(p);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j >= lo) p[j] = static_cast<int8_t>(q.get(j));
    }
    if ((c + lo) % kBlock8 == 0) scales[(c + lo) / kBlock8] = static_cast<uint8_t>(E);
}

}  // namespace gnsilu
