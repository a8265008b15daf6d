// gn_row_passes.hpp -- what the norms over a row's last dimension (layer norm,
// root-mean-square norm) share: a row's lanes and their sums, the loop over a
// row slot's rows, the weight's gradients from partial rows, and the shapes in
// which the host launches them.
//
// A row belongs to TPR lanes (a power of two, of one wave up to 64, of several
// beyond), each holding NV pieces of W channels, so a row's sums are a
// lane-group butterfly and, for several waves, one exchange of the waves' sums
// through LDS.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "gn_host.hpp"
#include "gn_rows.hpp"
#include "gnsilu.h"

namespace gnsilu {
namespace {

// The sums over a row's lanes.  A row of several waves exchanges their sums
// through `red` (its workgroup has kSlots rows' of them); the caller passes a
// different part of it to consecutive sums, so one barrier is enough.  Every
// wave then joins them: in order, or (FOLD) by a butterfly over as many lanes,
// which takes one register instead of one for each wave.
template <int TPR, bool FOLD = false, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *red) {
    constexpr int N = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane_sum<N>(v[k]);
    if constexpr (TPR > 64) {
        constexpr int kWaves = TPR / 64;
        float *mine = red + (threadIdx.x / TPR) * (K * kWaves);
        const int wave = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) mine[k * kWaves + wave] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (FOLD) {
                v[k] = lane_sum<kWaves>(mine[k * kWaves + threadIdx.x % kWaves]);
            } else {
                float s = mine[k * kWaves];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) s += mine[k * kWaves + w];
                v[k] = s;
            }
        }
    }
}

// Where the calling lane's piece p starts in its row and its first own
// channel; W for a lane beyond the row (it reads piece 0 and counts nothing).
template <int W, bool TAIL, class Args>
__device__ __forceinline__ void piece_at(const Args &a, int p, int *c, int *lo) {
    *lo = 0;
    *c = p * W;
    if (p >= a.P) {
        *c = 0;
        *lo = W;
    } else if (TAIL && *c + W > a.C) {
        *lo = *c + W - a.C;
        *c = a.C - W;
    }
}

// The calling lane's row slot; a scalar when whole waves share it.
template <int TPR> __device__ __forceinline__ int row_slot() {
    const int slot = static_cast<int>(threadIdx.x) / TPR;
    return TPR >= 64 ? __builtin_amdgcn_readfirstlane(slot) : slot;
}

// The sum over a piece's own channels of f(i); 0 for a lane beyond the row.
// edge: wave_has_edge.
template <int W, bool TAIL, class F>
__device__ __forceinline__ float own_sum(int lo, bool edge, F &&f) {
    float p = 0.0f;
    if (TAIL && edge) {
#pragma unroll
        for (int i = 0; i < W; ++i) p += i >= lo ? f(i) : 0.0f;
        return p;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) p += f(i);
    return lo < W ? p : 0.0f;
}

// The rows of a row slot: base + slot, then one grid's worth of rows further.
// AHEAD: each row's loads are issued before the row ahead of it is worked on
// (not where a lane's four pieces of fp32 leave no registers for them: the
// backward pass at (2796,12000) took 187 us with them spilt, 87 without).
// Slots behind the last row read that row and do not store (the loop's end is
// the same for the whole workgroup, which has barriers in it).
template <class Row, int SLOTS, bool AHEAD> struct RowLoop {
    int64_t M;
    int slot;
    uint32_t blocks;  // workgroups that share the rows
    Row a, b;
    __device__ __forceinline__ int64_t row(int64_t base) const {
        return base + slot < M ? base + slot : M - 1;
    }
    template <class Fetch> __device__ __forceinline__ void begin(Fetch &&fetch) {
        fetch(a, row(int64_t{blockIdx.x} * SLOTS));
    }
    template <class Fetch, class Work>
    __device__ __forceinline__ void run(Fetch &&fetch, Work &&work) {
        const int64_t step = int64_t{blocks} * SLOTS;
        for (int64_t base = int64_t{blockIdx.x} * SLOTS;;) {
            int64_t next = base + step;
            if constexpr (!AHEAD) {
                work(a, row(base), base + slot < M);
                if (next >= M) break;
                base = next;
                fetch(a, row(base));
                continue;
            }
            if (next < M) fetch(b, row(next));
            work(a, row(base), base + slot < M);
            if (next >= M) break;
            base = next;
            next += step;
            if (next < M) fetch(a, row(next));
            work(b, row(base), base + slot < M);
            if (next >= M) break;
            base = next;
        }
    }
};

// dgamma and dbeta from the K partial rows of C sums: 32 channels and 32 row
// parts per workgroup, each part's rows in order (eight rows' loads in
// flight), then the parts by a fixed tree, in fp64.  K = 0 writes zeros.
// blockIdx.y: 0 dgamma, 1 dbeta.
constexpr int kColLanes = 32, kColParts = 32;
[[maybe_unused]] __global__ __launch_bounds__(kColLanes *kColParts) void gn_column_sums(const float *part,
                                                                        int64_t K, int C,
                                                                        void *dgamma, void *dbeta,
                                                                        int type) {
    __shared__ double red[kColParts][kColLanes];
    void *out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int lane = threadIdx.x % kColLanes, r = threadIdx.x / kColLanes;
    const int c = static_cast<int>(blockIdx.x) * kColLanes + lane;
    const float *p = part + static_cast<int64_t>(blockIdx.y) * K * C + c;
    double s = 0.0;
    if (c < C) {
        constexpr int kBatch = 8;
        for (int64_t k = r; k < K; k += kBatch * kColParts) {
            float v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int64_t ku = k + u * kColParts;
                v[u] = p[(ku < K ? ku : K - 1) * C];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                s += k + u * kColParts < K ? static_cast<double>(v[u]) : 0.0;
        }
    }
    s += __shfl_xor(s, 32, 64);  // the wave's two parts
    red[r][lane] = s;
    __syncthreads();
    for (int h = kColParts / 2; h > 1; h >>= 1) {  // even parts r < h + those at r + h
        if (r < h) red[r][lane] = s += red[r + h][lane];
        __syncthreads();
    }
    if (r == 0 && c < C) store_affine(out, type, c, static_cast<float>(s));
}

// ---- host -----------------------------------------------------------------------
// Workgroups: eight waves' worth of lanes per SIMD of 256 CUs forward; backward,
// where each workgroup writes a partial row, four, or two where a workgroup has
// 512 lanes (two pieces a lane or more, for their registers).
constexpr int64_t kForwardLanes = int64_t{2048} * 256;
constexpr int64_t kBackwardBlocks = 256;  // one per CU, or more when there are
constexpr int64_t kMaxRun = 4096;         // more rows than a slot should add up in fp32

// Lanes of a row: the fewest (a power of two) that hold it with `nv` pieces
// each.  Backward, one piece a lane leaves registers for twice the waves, two
// halve a row's fixed work: one / two took 17.4 / 19.1 us of kernel time at
// (5001,1537) from the checkpoint, 86.7 / 78 at (16384,4096).
struct LnShape {
    int w, tpr, nv;
    bool tail;
    int P;
};

inline LnShape ln_shape(int64_t C, int dtype, bool forward) {
    LnShape s;
    const int w = static_cast<int>(16 / elem_bytes(dtype));
    s.w = C < w ? 1 : w;
    s.tail = C % s.w != 0;
    s.P = static_cast<int>(ceil_div(C, s.w));
    if (forward)
        s.nv = s.P <= 64 ? 1 : (s.P <= 2048 ? 2 : 4);
    else
        s.nv = s.P <= 256 ? 1 : (s.P <= 1024 ? 2 : 4);
    s.tpr = s.w == 1 ? 8 : 1;
    while (s.tpr * s.nv < s.P) s.tpr *= 2;
    return s;
}

template <int V> using IC = std::integral_constant<int, V>;

// Calls f(IC<W>, IC<TAIL>, IC<TPR>, IC<NV>).
template <class D, bool FORWARD, class F>
void with_ln_shape(const LnShape &s, F &&f) {
    constexpr int W = static_cast<int>(16 / sizeof(typename D::storage));
    if (s.w == 1) return f(IC<1>{}, IC<0>{}, IC<8>{}, IC<1>{});
    auto by_tail = [&](auto tail) {
        if (s.nv == 1) {
            switch (s.tpr) {
                case 1: return f(IC<W>{}, IC<0>{}, IC<1>{}, IC<1>{});  // P = 1: C = W
                case 2: return f(IC<W>{}, tail, IC<2>{}, IC<1>{});
                case 4: return f(IC<W>{}, tail, IC<4>{}, IC<1>{});
                case 8: return f(IC<W>{}, tail, IC<8>{}, IC<1>{});
                case 16: return f(IC<W>{}, tail, IC<16>{}, IC<1>{});
                case 32: return f(IC<W>{}, tail, IC<32>{}, IC<1>{});
                case 64: return f(IC<W>{}, tail, IC<64>{}, IC<1>{});
            }
            if constexpr (!FORWARD) {
                if (s.tpr == 128) return f(IC<W>{}, tail, IC<128>{}, IC<1>{});
                return f(IC<W>{}, tail, IC<256>{}, IC<1>{});
            }
        }
        if (s.nv == 2) {
            if constexpr (FORWARD) {
                if (s.tpr == 64) return f(IC<W>{}, tail, IC<64>{}, IC<2>{});
                if (s.tpr == 128) return f(IC<W>{}, tail, IC<128>{}, IC<2>{});
                if (s.tpr == 1024) return f(IC<W>{}, tail, IC<1024>{}, IC<2>{});
            }
            if (s.tpr == 256) return f(IC<W>{}, tail, IC<256>{}, IC<2>{});
            return f(IC<W>{}, tail, IC<512>{}, IC<2>{});
        }
        if constexpr (!FORWARD)
            if (s.tpr == 512) return f(IC<W>{}, tail, IC<512>{}, IC<4>{});
        if constexpr (W == 4) f(IC<W>{}, tail, IC<1024>{}, IC<4>{});
    };
    if (s.tail)
        by_tail(IC<1>{});
    else
        by_tail(IC<0>{});
}

constexpr int forward_threads(int tpr) { return tpr < 256 ? 256 : tpr; }
constexpr int backward_threads(int tpr, int nv) { return nv == 1 || tpr > 512 ? 1024 : 512; }

// Workgroups of a forward pass without loads ahead, whose slots take a row each:
// other rows' waves hide a row's latency, and those that hold one row at a time are
// more.  Measured, us with a row ahead and kForwardLanes / with a row a slot (bf16):
// quantize (16384,4096) 42.0 / 38.3, (8192,2560) 19.4 / 17.3; norm with residual
// into 8 bits 93.0 / 86.9, 36.1 / 32.3, into bf16 104.0 / 96.0, 30.0 / 31.6, the
// last 29.3 with two rows a slot, which share gamma's loads (up to 64 MiB of x: the
// two sizes measured hold 40 and 128).  fp32 rows keep kForwardLanes: up to 8192
// channels they have a row ahead, and wider ones, which have no registers for it,
// took with kForwardLanes / with a row a slot: norm (4096,9000) 50.1 / 58.5 us, into
// 8 bits with residual 93.0 / 102.0, (2048,12288) 58.4 / 66.7, quantize (1500,9000)
// 12.1 / 13.3, and at (16384,12288) the norm 291 / 284, quantize 187 / 171.
constexpr int64_t kOneEachBytes = int64_t{64} << 20;
inline int64_t one_each_blocks(int64_t M, int slots) {
    return std::min(ceil_div(M, slots), int64_t{1} << 21);
}

inline int64_t backward_blocks(const LnShape &s, int64_t M) {
    const int64_t slots = backward_threads(s.tpr, s.nv) / s.tpr;
    return std::max(std::min(ceil_div(M, slots), kBackwardBlocks), ceil_div(M, slots * kMaxRun));
}

template <class F>
void by_type(int dtype, F &&f) {
    switch (x_dtype(dtype)) {
        case GN_DTYPE_F16: f(Fp16{}); break;
        case GN_DTYPE_F32: f(F32{}); break;
        default: f(Bf16{}); break;
    }
}

inline bool overflows(int64_t M, int64_t stride, int64_t C) {
    return M > 0 && stride > 0 && M > (INT64_MAX / 4 - C) / stride;
}

inline bool misaligned(const void *p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

// The checks that row passes share; in_strides: row strides of inputs (0: one
// row for all), out_strides: of outputs.
inline gn_status check_rows(int64_t M, int64_t C, int dtype, const int64_t *in_strides, int n_in,
                            const int64_t *out_strides, int n_out) {
    if (!valid_dtype(dtype)) return GN_INVALID_ARGUMENT;
    if (M < 0 || C <= 0) return GN_INVALID_ARGUMENT;
    if (overflows(M, C, C)) return GN_INVALID_ARGUMENT;
    for (int i = 0; i < n_in; ++i)
        if (in_strides[i] < 0 || overflows(M, in_strides[i], C)) return GN_INVALID_ARGUMENT;
    for (int i = 0; i < n_out; ++i) {
        if (out_strides[i] < 0 || (M > 1 && out_strides[i] < C)) return GN_INVALID_ARGUMENT;
        if (overflows(M, out_strides[i], C)) return GN_INVALID_ARGUMENT;
    }
    if (C > GN_LAYER_NORM_MAX_CHANNELS) return GN_UNSUPPORTED;
    return GN_OK;
}

}  // namespace
}  // namespace gnsilu
