// gn_rms_norm.hip -- root-mean-square norm over the last dimension of rows, with
// the residual's addition in front and an output in 8 bits, and its backward
// pass, for MI355X (gfx950).
//
//   forward    h = x + residual (rounded to the rows' type; h = x without one)
//              rstd = 1/sqrt(sum(h^2)/C + eps), y = gamma*(h*rstd)
//              or, in 8 bits with a scale for the row, t = gamma*h in fp32,
//              q = rint(127*t/max|t|), scale = max|t|/127*rstd
//   backward   n = h*rstd, g = dy*gamma,
//              dx = rstd*(g - n*sum(g*n)/C) + dh, dgamma[c] = sum over rows of dy*n
//
// As layer norm the passes are bound by HBM: a row is read once, held in
// registers and written once.  One sum is enough (no mean is taken off, so
// nothing cancels), and in 8 bits the row's maximum goes through the same exchange
// as its sum: rstd is a factor of the whole row and drops out of the codes, so
// that both are taken of values that are known before any sum.  The sum of squares
// goes over the lanes times 2^-6: 16384 squares of 1e18 then stay below fp32's
// largest number (2^127.6) and one square of 1e-18 above its smallest normal one
// (2^-125.6).  A lane's own are at most 16.
//
// dh is the gradient that reaches h past the norm, through the residual stream:
// added here it costs one read, where a kernel of its own would read both and
// write again.
//
// Measured on MI355X: (16384,4096) bf16 with a residual 93 us (5.8 TB/s), backward
// with dh 95 us (5.65 TB/s) and column sums 4.9; (4099,1003) fp16 with a residual
// into 8 bits 9.6 us; backward (5001,1537) from the checkpoint 14.7 us and 3.9 (its
// start and end and five rows a slot; three rows ahead instead of one took 10%
// longer); fp32 with a residual (4096,8192) 104 us (5.2 TB/s), (16384,12288) 590 us
// (5.5 TB/s), (5003,1001) 13.6 us; into 8 bits (2048,12288) 58 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gn_row_passes.hpp"
#include "gn_rows8.hpp"
#include "gnsilu.h"

namespace gnsilu {
namespace {

struct RmsArgs {
    const void *x;          // backward: rows of h, or null when codes/scales hold them
    const void *res;        // forward: the residual, or null
    const int8_t *codes;    // backward: checkpoint of h, [M][C]
    const uint8_t *scales;  // [M][ceil(C / 32)]
    const void *dy, *dh;    // backward; dh or null
    void *y;                // forward: y or null; backward: dx
    void *h;                // forward: x + residual
    int8_t *codes_out;      // forward: y in 8 bits, row m at m * codes_stride
    float *scales_out;      // [M]
    float *rstd;            // [M]; forward: written unless null, backward: read
    float *part;            // backward: [blocks][C] partial dgamma, or null
    uint32_t rows_end;      // backward of few rows: workgroups from here on take columns
    void *dgamma;
    int64_t M, x_stride, res_stride, y_stride, h_stride, codes_stride, dy_stride, dh_stride;
    int C, P;
    float eps, inv_c;
    Affine af;
};

// A row's sum of squares and, as bits, its largest magnitude, over its lanes.
template <int TPR, bool MAX>
__device__ __forceinline__ void row_sum_max(float &s, uint32_t &top, float *red) {
    constexpr int N = TPR < 64 ? TPR : 64;
    s = lane_sum<N>(s);
    if constexpr (MAX) top = lane_max<N>(top);
    if constexpr (TPR > 64) {
        constexpr int kWaves = TPR / 64, kEach = MAX ? 2 : 1;
        float *mine = red + (threadIdx.x / TPR) * (kEach * kWaves);
        const int wave = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0) {
            mine[wave] = s;
            if constexpr (MAX) mine[kWaves + wave] = __uint_as_float(top);
        }
        __syncthreads();
        s = lane_sum<kWaves>(mine[threadIdx.x % kWaves]);
        if constexpr (MAX) top = lane_max<kWaves>(__float_as_uint(mine[kWaves + threadIdx.x % kWaves]));
    }
}

// What a lane's sum of squares is multiplied by on its way to the row's; exact.
constexpr float kSquares = 0x1p-6f;

// ---------------------------------------------------------------------------
// Forward.  RES: with a residual; CODES: y in 8 bits.
// ---------------------------------------------------------------------------
template <class D, int W, int NV, bool RES> struct RmsForwardRow {
    Piece<D, W> v[NV], r[RES ? NV : 1];
};

template <class D, int W, bool TAIL, int TPR, int NV, int THREADS, bool RES, bool CODES>
__global__ __launch_bounds__(THREADS) void gn_rms_norm(RmsArgs a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    constexpr int kRed = TPR > 64 ? 2 * (THREADS / 64) : 1;
    __shared__ float red[2 * kRed];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    const T *x = static_cast<const T *>(a.x);
    const T *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = static_cast<T *>(a.h);
    int c[NV], lo[NV];
    bool edge[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
        edge[j] = wave_has_edge<W, TAIL>(lo[j]);
    }
    using Row = RmsForwardRow<D, W, NV, RES>;
    auto fetch = [&](Row &r, int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            r.v[j].template load<false>(x + m * a.x_stride + c[j]);
            if constexpr (RES) r.r[j].template load<false>(res + m * a.res_stride + c[j]);
        }
    };
    RowLoop<Row, kSlots, sizeof(T) == 4 && NV < 4> loop{a.M, slot, gridDim.x};
    loop.begin(fetch);
    float ga[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_affine<W>(a.af.gamma, a.af.type, c[j], 1.0f, ga[j]);
    const float fc = static_cast<float>(a.C) * kSquares;
    int par = 0;
    loop.run(fetch, [&](Row &r, int64_t m, bool live) {
        float s = 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (RES) {
                float o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = r.v[j].get(i) + r.r[j].get(i);
                r.v[j].set(o);
            }
            s += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) { return r.v[j].get(i) * r.v[j].get(i); });
            if constexpr (CODES) {
#pragma unroll
                for (int i = 0; i < W; ++i)  // channels counted twice change no maximum
                    top = max(top, __float_as_uint(r.v[j].get(i) * ga[j][i]) & 0x7fffffffu);
            }
        }
        s *= kSquares;
        row_sum_max<TPR, CODES>(s, top, red + par * kRed);
        par ^= 1;
        if (!live) return;  // no barrier from here on
        const float rstd = 1.0f / sqrtf(s / fc + a.eps);
        if (t == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
        if constexpr (CODES) {
            const Rows8Scale sc(top);
            if (t == 0) a.scales_out[m] = Rows8Scale::step(top, rstd);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (lo[j] >= W) continue;
                float o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = r.v[j].get(i) * ga[j][i];
                rows8_encode<W>(o, sc).template store<false>(a.codes_out + m * a.codes_stride + c[j]);
                if constexpr (RES) r.v[j].put(h + m * a.h_stride + c[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (lo[j] >= W) continue;
                float o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = r.v[j].get(i) * rstd * ga[j][i];
                // A last piece's foreign channels get the value that their owner
                // writes, computed alike.
                Piece<D, W>::template store<false>(y + m * a.y_stride + c[j], o);
                if constexpr (RES) r.v[j].put(h + m * a.h_stride + c[j]);
            }
        }
    });
}

// ---------------------------------------------------------------------------
// Backward.  SAVED: h comes from its 8-bit checkpoint.
// ---------------------------------------------------------------------------
template <class D, int W, bool TAIL, int NV, bool SAVED> struct RmsBackwardRow {
    Piece<D, W> vx[SAVED ? 1 : NV], vy[NV];
    Piece8<W, TAIL> v8[SAVED ? NV : 1];
    float rstd;
    __device__ __forceinline__ void widen(int j, int c, bool edge, float (&o)[W]) const {
        if constexpr (SAVED) {
            v8[j].widen(c, edge, o);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = vx[j].get(i);
        }
    }
    // Hides from the compiler that the row's values are those it has used, so
    // that it does not keep what it made of them.
    __device__ __forceinline__ void opaque() {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (SAVED)
                v8[j].opaque();
            else
                vx[j].opaque();
            vy[j].opaque();
        }
    }
};

// dgamma of 16 pieces' channels over all rows, by a workgroup of THREADS lanes:
// THREADS / 16 row slots, four rows' loads of a slot in flight; the slots of a
// wave by a butterfly, then the waves in order.
constexpr int kRmsColPieces = 16;
template <class D, int W, bool TAIL, int THREADS, bool SAVED>
__device__ __forceinline__ void rms_few_rows_columns(const RmsArgs &a, int block) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / kRmsColPieces, kWaves = THREADS / 64, kBatch = 4;
    __shared__ float red[kWaves][kRmsColPieces * W];
    const int t = threadIdx.x % kRmsColPieces, slot = threadIdx.x / kRmsColPieces;
    int c, lo;
    piece_at<W, TAIL>(a, block * kRmsColPieces + t, &c, &lo);
    const bool edge = SAVED && wave_has_edge<W, TAIL>(lo);
    const int64_t nsb = (a.C + kBlock8 - 1) / kBlock8;
    const T *x = static_cast<const T *>(a.x);
    const T *dy = static_cast<const T *>(a.dy);
    using Row = RmsBackwardRow<D, W, TAIL, 1, SAVED>;
    float g[W];
#pragma unroll
    for (int i = 0; i < W; ++i) g[i] = 0.0f;
    for (int64_t base = slot; base < a.M; base += kBatch * kSlots) {
        Row r[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t m = base + u * kSlots < a.M ? base + u * kSlots : a.M - 1;
            if constexpr (SAVED)
                r[u].v8[0].load(Piece8At<W, TAIL>(a.codes, a.scales, 0, a.C, c), m * a.C, m * nsb);
            else
                r[u].vx[0].template load<false>(x + m * a.x_stride + c);
            r[u].vy[0].template load<false>(dy + m * a.dy_stride + c);
            r[u].rstd = a.rstd[m];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * kSlots >= a.M) break;
            float v[W];
            r[u].widen(0, c, edge, v);
#pragma unroll
            for (int i = 0; i < W; ++i) g[i] = fmaf(r[u].vy[0].get(i) * r[u].rstd, v[i], g[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int o = kRmsColPieces; o < 64; o <<= 1) g[i] += __shfl_xor(g[i], o, 64);
        if ((threadIdx.x & 63) < kRmsColPieces) red[threadIdx.x >> 6][t * W + i] = g[i];
    }
    __syncthreads();
    const int e = threadIdx.x;  // channel
    if (e >= kRmsColPieces * W) return;
    piece_at<W, TAIL>(a, block * kRmsColPieces + e / W, &c, &lo);
    if (e % W < lo) return;
    float s = red[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[w][e];
    store_affine(a.dgamma, a.af.type, c + e % W, s);
}

// FEW: few rows.  Workgroups up to rows_end make dx alone, the others dgamma
// from h and dy again, as in layer norm's backward pass.
template <class D, int W, bool TAIL, int TPR, int NV, int THREADS, bool SAVED, bool FEW>
__global__ __launch_bounds__(THREADS) void gn_rms_norm_backward(RmsArgs a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    if constexpr (FEW) {
        if (blockIdx.x >= a.rows_end) {
            rms_few_rows_columns<D, W, TAIL, THREADS, SAVED>(
                a, static_cast<int>(blockIdx.x - a.rows_end));
            return;
        }
    }
    constexpr int kRed = TPR > 64 ? THREADS / 64 : 1;
    __shared__ float red[2 * kRed];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    const T *x = static_cast<const T *>(a.x);
    const T *dy = static_cast<const T *>(a.dy);
    const T *dh = static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.y);
    int c[NV], lo[NV];
    bool edge[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
        edge[j] = wave_has_edge<W, TAIL>(lo[j]);
    }
    const int64_t nsb = (a.C + kBlock8 - 1) / kBlock8;
    using Row = RmsBackwardRow<D, W, TAIL, NV, SAVED>;
    auto at8 = [&](int j) { return Piece8At<W, TAIL>(a.codes, a.scales, 0, a.C, c[j]); };
    auto fetch = [&](Row &r, int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (SAVED)
                r.v8[j].load(at8(j), m * a.C, m * nsb);
            else
                r.vx[j].template load<false>(x + m * a.x_stride + c[j]);
            r.vy[j].template load<false>(dy + m * a.dy_stride + c[j]);
        }
        r.rstd = a.rstd[m];
    };
    RowLoop<Row, kSlots, sizeof(T) == 2 || NV < 4> loop{a.M, slot, FEW ? a.rows_end : gridDim.x};
    loop.begin(fetch);
    float ga[NV][W], dg[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load_affine<W>(a.af.gamma, a.af.type, c[j], 1.0f, ga[j]);
#pragma unroll
        for (int i = 0; i < W; ++i) dg[j][i] = 0.0f;
    }
    int par = 0;
    loop.run(fetch, [&](Row &r, int64_t m, bool live) {
        // dh is wanted after the sum only: its loads are on their way meanwhile
        Piece<D, W> vh[NV];
        if (dh != nullptr) {
#pragma unroll
            for (int j = 0; j < NV; ++j) vh[j].template load<false>(dh + m * a.dh_stride + c[j]);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float v[W];
            r.widen(j, c[j], edge[j], v);
            s[0] += own_sum<W, TAIL>(lo[j], edge[j],
                                     [&](int i) { return r.vy[j].get(i) * ga[j][i] * v[i]; });
        }
        row_sum<TPR, true>(s, red + par * kRed);
        par ^= 1;
        if (!live) return;  // no barrier from here on
        if constexpr (NV > 1) r.opaque();
        // rstd by rstd, not their square, which leaves fp32's range where dx does not
        const float s1 = r.rstd * (r.rstd * (s[0] * a.inv_c));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float v[W], o[W];
            r.widen(j, c[j], edge[j], v);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = r.vy[j].get(i);
                o[i] = r.rstd * fmaf(-v[i], s1, d * ga[j][i]);
                if constexpr (!FEW) dg[j][i] = fmaf(d * r.rstd, v[i], dg[j][i]);
            }
            if (dh != nullptr) {
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] += vh[j].get(i);
            }
            if (lo[j] >= W) continue;
            T *p = dx + m * a.y_stride + c[j];
            // dx may be dh, whose loads no barrier waits for: a last piece's
            // foreign channels, which their owner may have written by then, are
            // left to it.
            if (!TAIL || lo[j] == 0)
                Piece<D, W>::template store<!TAIL>(p, o);
            else
                store_from<D, W>(p, o, lo[j]);
        }
    });
    if (FEW || a.part == nullptr) return;
    // The row slots of the workgroup: within a wave by butterflies over the
    // lanes that hold the same channels, then slot by slot (wave by wave)
    // through LDS.
    float *pg = a.part + int64_t{blockIdx.x} * a.C;
    if constexpr (TPR >= 64) {
        constexpr int kPer = NV * W;
        __shared__ float comb[kSlots > 1 ? kPer * TPR : 1];
#pragma unroll 1
        for (int w = 0; w < kSlots; ++w) {
            if (slot == w) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const int e = (j * W + i) * TPR + t;
                        if constexpr (kSlots > 1) {
                            if (w > 0) dg[j][i] += comb[e];
                            if (w + 1 < kSlots) comb[e] = dg[j][i];
                        }
                        if (w + 1 == kSlots && i >= lo[j]) pg[c[j] + i] = dg[j][i];
                    }
            }
            if constexpr (kSlots > 1) __syncthreads();
        }
    } else {
        static_assert(NV == 1, "rows of fewer lanes than a wave have one piece per lane");
        constexpr int kWaves = THREADS / 64;
        __shared__ float comb[kWaves][W][TPR];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float g = dg[0][i];
#pragma unroll
            for (int o = TPR; o < 64; o <<= 1) g += __shfl_xor(g, o, 64);
            if ((threadIdx.x & 63) < TPR) comb[threadIdx.x >> 6][i][t] = g;
        }
        __syncthreads();
        if (threadIdx.x < TPR) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                float g = comb[0][i][t];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) g += comb[w][i][t];
                if (i >= lo[0]) pg[c[0] + i] = g;
            }
        }
    }
}

// ---- host -----------------------------------------------------------------------
template <class D>
void launch_rms_forward(const LnShape &s, const RmsArgs &a, hipStream_t st) {
    const int nt = forward_threads(s.tpr);
    constexpr int64_t kBytes = sizeof(typename D::storage);
    int64_t blocks = one_each_blocks(a.M, nt / s.tpr);
    if (kBytes == 4)  // one_each_blocks' comment
        blocks = std::min(blocks, kForwardLanes / nt);
    else if (a.codes_out == nullptr && a.M <= kOneEachBytes / (a.C * kBytes))
        blocks = std::min(blocks, 2 * kForwardLanes / nt);
    with_ln_shape<D, true>(s, [&](auto w, auto tail, auto tpr, auto nv) {
        constexpr int W = decltype(w)::value, TPR = decltype(tpr)::value;
        constexpr int NV = decltype(nv)::value, NT = forward_threads(TPR);
        constexpr bool TAIL = decltype(tail)::value != 0;
        const dim3 grid(static_cast<unsigned>(blocks)), block(NT);
        auto go = [&](auto res, auto codes) {
            gn_rms_norm<D, W, TAIL, TPR, NV, NT, decltype(res)::value != 0,
                        decltype(codes)::value != 0><<<grid, block, 0, st>>>(a);
        };
        if (a.res != nullptr)
            a.codes_out != nullptr ? go(IC<1>{}, IC<1>{}) : go(IC<1>{}, IC<0>{});
        else
            a.codes_out != nullptr ? go(IC<0>{}, IC<1>{}) : go(IC<0>{}, IC<0>{});
    });
}

// Up to this many rows the columns' workgroups read h and dy again instead of
// adding up partial rows (layer norm's limit, whose pass moves the same bytes).
constexpr int64_t kRmsFewRows = 1024;

template <class D>
void launch_rms_backward(const LnShape &s, RmsArgs a, hipStream_t st) {
    const int64_t blocks = backward_blocks(s, a.M);
    const bool few = a.M <= kRmsFewRows;
    a.rows_end = static_cast<uint32_t>(blocks);
    with_ln_shape<D, false>(s, [&](auto w, auto tail, auto tpr, auto nv) {
        constexpr int W = decltype(w)::value, TPR = decltype(tpr)::value;
        constexpr int NV = decltype(nv)::value, NT = backward_threads(TPR, NV);
        constexpr bool TAIL = decltype(tail)::value != 0;
        const unsigned rows = static_cast<unsigned>(blocks);
        const unsigned cols = few && a.dgamma != nullptr
                                  ? static_cast<unsigned>(ceil_div(s.P, kRmsColPieces))
                                  : 0u;
        auto launch = [&](auto saved, auto fewc, unsigned grid) {
            gn_rms_norm_backward<D, W, TAIL, TPR, NV, NT, decltype(saved)::value != 0,
                                 decltype(fewc)::value != 0><<<grid, NT, 0, st>>>(a);
        };
        auto go = [&](auto saved) {
            if (!few) return launch(saved, IC<0>{}, rows);
            if (cols > 0 && (a.y == a.x || a.y == a.dy)) {
                // in place: the columns before any row is overwritten
                a.rows_end = 0;
                launch(saved, IC<1>{}, cols);
                a.rows_end = rows;
                return launch(saved, IC<1>{}, rows);
            }
            launch(saved, IC<1>{}, rows + cols);
        };
        if (a.codes != nullptr)
            go(IC<1>{});
        else
            go(IC<0>{});
    });
}

size_t rms_backward_workspace(int64_t M, int64_t C, int dtype) {
    if (M <= kRmsFewRows) return 0;
    return sizeof(float) * static_cast<size_t>(backward_blocks(ln_shape(C, dtype, false), M)) *
           static_cast<size_t>(C);
}

}  // namespace
}  // namespace gnsilu

using namespace gnsilu;

extern "C" {

gn_status gn_rms_norm_rows(const void *x, int64_t x_stride, const void *residual,
                           int64_t residual_stride, const void *gamma, void *h, int64_t h_stride,
                           void *y, int64_t y_stride, void *codes, int64_t codes_stride,
                           float *scales, float *rstd_out, int64_t M, int64_t C, float eps,
                           int dtype, void *stream) {
    if (x == nullptr || (y == nullptr) == (codes == nullptr)) return GN_INVALID_ARGUMENT;
    if ((codes == nullptr) != (scales == nullptr) || (residual == nullptr) != (h == nullptr))
        return GN_INVALID_ARGUMENT;
    if (y != nullptr && y == h) return GN_INVALID_ARGUMENT;  // two outputs
    if (!(eps >= 0.0f) || std::isinf(eps)) return GN_INVALID_ARGUMENT;
    const int64_t in[2] = {x_stride, residual == nullptr ? 0 : residual_stride};
    const int64_t out[2] = {y == nullptr ? codes_stride : y_stride, h == nullptr ? C : h_stride};
    gn_status st = check_rows(M, C, dtype, in, 2, out, 2);
    if (st == GN_OK) st = check_affine(gamma, nullptr, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(x, es) || misaligned(residual, es) || misaligned(h, es) || misaligned(y, es) ||
        misaligned(scales, 4) || misaligned(rstd_out, 4))
        return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    Call c;
    st = begin_call(stream, {x, residual, gamma, h, y, codes, scales, rstd_out}, &c);
    if (st != GN_OK) return st;
    const LnShape s = ln_shape(C, dtype, true);
    RmsArgs a{};
    a.x = x;
    a.res = residual;
    a.h = h;
    a.y = y;
    a.codes_out = static_cast<int8_t *>(codes);
    a.scales_out = scales;
    a.rstd = rstd_out;
    a.M = M;
    a.x_stride = x_stride;
    a.res_stride = residual_stride;
    a.h_stride = h_stride;
    a.y_stride = y_stride;
    a.codes_stride = codes_stride;
    a.C = static_cast<int>(C);
    a.P = s.P;
    a.eps = eps;
    a.af = Affine{gamma, nullptr, affine_type(dtype)};
    by_type(dtype, [&](auto d) { launch_rms_forward<decltype(d)>(s, a, c.stream); });
    return finish_launch();
}

gn_status gn_rms_norm_rows_backward_workspace(int64_t M, int64_t C, int dtype,
                                              int64_t *bytes_out) {
    if (bytes_out == nullptr) return GN_INVALID_ARGUMENT;
    const gn_status st = check_rows(M, C, dtype, nullptr, 0, nullptr, 0);
    if (st != GN_OK) return st;
    if (M > 0 && backward_blocks(ln_shape(C, dtype, false), M) >= int64_t{1} << 22)
        return GN_UNSUPPORTED;
    *bytes_out = static_cast<int64_t>(rms_backward_workspace(M, C, dtype));
    return GN_OK;
}

gn_status gn_rms_norm_rows_backward(const void *dy, int64_t dy_stride, const void *x,
                                    int64_t x_stride, const void *codes, const void *scales,
                                    const float *rstd, const void *gamma, const void *dh,
                                    int64_t dh_stride, void *dx, int64_t dx_stride, void *dgamma,
                                    int64_t M, int64_t C, int dtype, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
    if (dy == nullptr || dx == nullptr || rstd == nullptr) return GN_INVALID_ARGUMENT;
    // h, or its checkpoint, not both
    if ((codes == nullptr) != (scales == nullptr) || (x == nullptr) == (codes == nullptr))
        return GN_INVALID_ARGUMENT;
    const int64_t in[3] = {dy_stride, x == nullptr ? 0 : x_stride, dh == nullptr ? 0 : dh_stride};
    gn_status st = check_rows(M, C, dtype, in, 3, &dx_stride, 1);
    if (st == GN_OK) st = check_affine(gamma, dgamma, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(dy, es) || misaligned(x, es) || misaligned(dh, es) || misaligned(dx, es) ||
        misaligned(rstd, 4) || misaligned(workspace, 4))
        return GN_UNSUPPORTED;
    if (M == 0 && dgamma == nullptr) return GN_OK;
    const size_t need = dgamma != nullptr ? rms_backward_workspace(M, C, dtype) : 0;
    if (M > 0 && backward_blocks(ln_shape(C, dtype, false), M) >= int64_t{1} << 22)
        return GN_UNSUPPORTED;  // a dispatch holds fewer than 2^32 work-items
    if (need > 0 && workspace == nullptr) return GN_INVALID_ARGUMENT;
    if (need > 0 && (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < need))
        return GN_SCRATCH_TOO_SMALL;
    Call c;
    st = begin_call(stream,
                    {dy, x, codes, scales, rstd, gamma, dh, dx, dgamma,
                     need > 0 ? workspace : nullptr},
                    &c);
    if (st != GN_OK) return st;
    const LnShape s = ln_shape(C, dtype, false);
    RmsArgs a{};
    a.x = x;
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.dy = dy;
    a.dh = dh;
    a.y = dx;
    a.rstd = const_cast<float *>(rstd);
    a.part = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.dgamma = dgamma;
    a.M = M;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.dh_stride = dh_stride;
    a.y_stride = dx_stride;
    a.C = static_cast<int>(C);
    a.P = s.P;
    a.inv_c = 1.0f / static_cast<float>(C);
    a.af = Affine{gamma, nullptr, affine_type(dtype)};
    if (M > 0) by_type(dtype, [&](auto d) { launch_rms_backward<decltype(d)>(s, a, c.stream); });
    if (need > 0 || M == 0)  // M = 0: zeros
        gn_column_sums<<<dim3(static_cast<unsigned>(ceil_div(C, kColLanes)), 1),
                         kColLanes * kColParts, 0, c.stream>>>(
            a.part, M > 0 ? backward_blocks(s, M) : 0, a.C, dgamma, nullptr, a.af.type);
    return finish_launch();
}

}  // extern "C"
