// gn_layer_norm.hip -- layer norm over the last dimension of rows, forward and
// backward, for MI355X (gfx950).
//
//   forward    mean = sum(x)/C, var = sum((x-mean)^2)/C, rstd = 1/sqrt(var+eps),
//              y = gamma*(x-mean)*rstd + beta
//   backward   h = (x-mean)*rstd, g = dy*gamma,
//              dx = rstd*(g - sum(g)/C - h*sum(g*h)/C),
//              dgamma[c] = sum over rows of dy*h, dbeta[c] = sum over rows of dy
//
// Both passes are bound by HBM: a row is read once, held in registers and
// written once, and the next row's loads are in flight meanwhile.  A row
// belongs to TPR lanes (a power of two, of one wave up to 64, of several
// beyond), each holding NV pieces of W channels, so a row's sums are a
// lane-group butterfly and, for several waves, one exchange of the waves' sums
// through LDS.  The mean is taken first and the variance from the differences:
// with the row in registers the second sum costs no memory traffic, and no
// channel far from the rest can cancel it.  The first sum is off by a few times
// 2^-24 of the row's size, which in fp32 rows can be more than their spread (of
// 12288 times 10000.1 the mean came out 0.002 too large, twice the root of
// eps = 1e-6): there the mean and the variance are corrected by the sum of the
// differences themselves, taken beside that of their squares (1 to 3% of the
// time: (8192,4096) 43.6 to 44.3 us, (300000,100) 44.4 to 45.8).  A row of a
// 16-bit type whose values lie far from zero, within a power of two, has a sum
// of at most 25 bits: exact, or as good as the quotient's own rounding.
//
// The weight's gradients run down the columns.  A lane keeps the same channels
// for every row it works on, so their sums stay in its registers over all of a
// workgroup's rows; the workgroup adds its row slots in a fixed order and
// writes one partial row of C sums, and a second kernel adds the partial rows
// (in fp64) in a fixed order: no atomics, the same bits on every call.
//
// Measured on MI355X, bf16 (a 1 GiB copy reads and writes 5.1 TB/s there):
// (16384,4096) forward 45.9 us (5.85 TB/s), backward 78.3 us (5.25 TB/s) and
// column sums 4.8 us; forward with the checkpoint (8192,2560) 22.4 us; backward
// from the checkpoint (5001,1537) 16.2 us (five rows a slot: their latencies
// and the sums' instructions bound it) and 3.8 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gn_host.hpp"
#include "gn_rows.hpp"
#include "gnsilu.h"

namespace gnsilu {
namespace {

struct LnArgs {
    const void *x;          // rows of x, or null when codes/scales hold them
    const int8_t *codes;    // [M][C]
    const uint8_t *scales;  // [M][ceil(C / 32)]
    const void *dy;
    void *y;                // forward: y; backward: dx
    int8_t *codes_out;      // forward: the checkpoint, or null
    uint8_t *scales_out;
    float *mean, *rstd;     // [M]; forward: written unless null, backward: read
    float *part;            // backward: [2][blocks][C] partial dgamma, dbeta, or null
    uint32_t rows_end;      // backward of few rows: workgroups from here on take columns
    void *dgamma, *dbeta;   // (those workgroups' results)
    int64_t M, x_stride, dy_stride, y_stride;
    int C, P;
    float eps, inv_c;       // inv_c: 1 / C
    Affine af;
};

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
template <int W, bool TAIL>
__device__ __forceinline__ void piece_at(const LnArgs &a, int p, int *c, int *lo) {
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

// ---------------------------------------------------------------------------
// Forward.  Row slots per workgroup: THREADS / TPR.
// ---------------------------------------------------------------------------
template <class D, int W, int NV> struct ForwardRow {
    Piece<D, W> v[NV];
};

template <class D, int W, bool TAIL, int TPR, int NV, int THREADS, bool SAVE>
__global__ __launch_bounds__(THREADS) void gn_layer_norm(LnArgs a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    constexpr int kRed = TPR > 64 ? THREADS / 64 : 1;
    constexpr int kGroup = TPR < kBlock8 / W ? TPR : kBlock8 / W;
    // fp32 rows: the mean is corrected by the mean difference from it
    constexpr bool kCorrect = sizeof(T) == 4;
    constexpr int kSums = kCorrect ? 2 : 1;
    __shared__ float red[(1 + kSums) * kRed];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    int c[NV], lo[NV];
    bool edge[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
        edge[j] = wave_has_edge<W, TAIL>(lo[j]);
    }
    using Row = ForwardRow<D, W, NV>;
    auto fetch = [&](Row &r, int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) r.v[j].template load<false>(x + m * a.x_stride + c[j]);
    };
    RowLoop<Row, kSlots, sizeof(T) == 2 || NV < 4> loop{a.M, slot, gridDim.x};
    loop.begin(fetch);
    float ga[NV][W], be[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load_affine<W>(a.af.gamma, a.af.type, c[j], 1.0f, ga[j]);
        load_affine<W>(a.af.beta, a.af.type, c[j], 0.0f, be[j]);
    }
    const float fc = static_cast<float>(a.C);
    const int64_t nsb = (a.C + kBlock8 - 1) / kBlock8;
    loop.run(fetch, [&](const Row &r, int64_t m, bool live) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            s[0] += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) { return r.v[j].get(i); });
        row_sum<TPR>(s, red);
        const float mean = s[0] / fc;
        float q[kSums] = {};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            q[0] += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) {
                const float d = r.v[j].get(i) - mean;
                return d * d;
            });
            if constexpr (kCorrect)
                q[1] += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) { return r.v[j].get(i) - mean; });
        }
        row_sum<TPR, kCorrect>(q, red + kRed);
        float shift = 0.0f, var = q[0] / fc;
        if constexpr (kCorrect) {
            shift = q[1] / fc;
            // an fma: its product is not infinite where var is
            var = fmaf(-shift, shift, var);
            var = var < 0.0f ? 0.0f : var;  // a NaN stays
        }
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (live && t == 0) {
            if (a.mean != nullptr) a.mean[m] = mean + shift;
            if (a.rstd != nullptr) a.rstd[m] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[W], o[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                f[i] = r.v[j].get(i);
                float d = f[i] - mean;
                if constexpr (kCorrect) d -= shift;
                o[i] = fmaf(d * rstd, ga[j][i], be[j][i]);
            }
            uint32_t E = 0;
            if constexpr (SAVE)
                E = block8_exponent<D, W, kGroup>(r.v[j], Magnitudes<D, W>(lo[j]));
            if (!live || lo[j] >= W) continue;
            // A last piece's foreign channels get the value that their owner
            // writes, computed alike.  Nontemporal only beside a checkpoint of
            // 16-byte rows, as measured: y alone (16384,4096) 49.5 us, 46.0
            // plain; with a checkpoint (8192,2560) 22.9, 24.8 plain; rows off
            // 16-byte boundaries, whose partial lines the L2 joins, with a
            // checkpoint and its restore (33520,1001) 61.5, 53.8 plain,
            // (8001,4097) 79.6, 75.0 plain, (100001,257) 73, 66 plain.
            Piece<D, W>::template store<SAVE && !TAIL>(y + m * a.y_stride + c[j], o);
            if constexpr (SAVE)
                store_block8<W, TAIL, !TAIL>(block8_encode<W>(f, E), E, a.codes_out + m * a.C,
                                            a.scales_out + m * nsb, c[j], lo[j]);
        }
    });
}

// ---------------------------------------------------------------------------
// Backward.  SAVED: x comes from its 8-bit checkpoint.
// ---------------------------------------------------------------------------
template <class D, int W, bool TAIL, int NV, bool SAVED> struct BackwardRow {
    Piece<D, W> vx[SAVED ? 1 : NV], vy[NV];
    Piece8<W, TAIL> v8[SAVED ? NV : 1];
    float mean, rstd;
    // x - mean
    __device__ __forceinline__ void centred(int j, int c, bool edge, float (&o)[W]) const {
        if constexpr (SAVED) {
            float mu[W];
#pragma unroll
            for (int i = 0; i < W; ++i) mu[i] = mean;
            v8[j].widen_less(c, mu, edge, o);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = vx[j].get(i) - mean;
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
        asm volatile("" : "+v"(mean));
    }
};

// dgamma and dbeta of 16 pieces' channels over all rows, by a workgroup of
// THREADS lanes: THREADS / 16 row slots, four rows' loads of a slot in flight;
// the slots of a wave by a butterfly, then the waves in order.
constexpr int kColPieces = 16;
template <class D, int W, bool TAIL, int THREADS, bool SAVED>
__device__ __forceinline__ void few_rows_columns(const LnArgs &a, int block) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / kColPieces, kWaves = THREADS / 64, kBatch = 4;
    __shared__ float red[2][kWaves][kColPieces * W];
    const int t = threadIdx.x % kColPieces, slot = threadIdx.x / kColPieces;
    int c, lo;
    piece_at<W, TAIL>(a, block * kColPieces + t, &c, &lo);
    const bool edge = SAVED && wave_has_edge<W, TAIL>(lo);
    const int64_t nsb = (a.C + kBlock8 - 1) / kBlock8;
    const T *x = static_cast<const T *>(a.x);
    const T *dy = static_cast<const T *>(a.dy);
    using Row = BackwardRow<D, W, TAIL, 1, SAVED>;
    float g[W], b[W];
#pragma unroll
    for (int i = 0; i < W; ++i) g[i] = b[i] = 0.0f;
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
            r[u].mean = a.mean[m];
            r[u].rstd = a.rstd[m];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * kSlots >= a.M) break;
            float v[W];
            r[u].centred(0, c, edge, v);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = r[u].vy[0].get(i);
                g[i] = fmaf(d * r[u].rstd, v[i], g[i]);
                b[i] += d;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int o = kColPieces; o < 64; o <<= 1) {
            g[i] += __shfl_xor(g[i], o, 64);
            b[i] += __shfl_xor(b[i], o, 64);
        }
        if ((threadIdx.x & 63) < kColPieces) {
            red[0][threadIdx.x >> 6][t * W + i] = g[i];
            red[1][threadIdx.x >> 6][t * W + i] = b[i];
        }
    }
    __syncthreads();
    // thread (which, piece, channel)
    const int e = threadIdx.x % (kColPieces * W), which = threadIdx.x / (kColPieces * W);
    if (which >= 2) return;
    piece_at<W, TAIL>(a, block * kColPieces + e / W, &c, &lo);
    void *out = which == 0 ? a.dgamma : a.dbeta;
    if (out == nullptr || e % W < lo) return;
    float s = red[which][0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[which][w][e];
    store_affine(out, a.af.type, c + e % W, s);
}

// FEW: few rows.  Workgroups up to rows_end make dx alone, the others dgamma
// and dbeta from x and dy again: one launch and no partial rows, and what is
// read twice comes from a cache.
template <class D, int W, bool TAIL, int TPR, int NV, int THREADS, bool SAVED, bool FEW>
__global__ __launch_bounds__(THREADS) void gn_layer_norm_backward(LnArgs a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    if constexpr (FEW) {
        if (blockIdx.x >= a.rows_end) {
            few_rows_columns<D, W, TAIL, THREADS, SAVED>(
                a, static_cast<int>(blockIdx.x - a.rows_end));
            return;
        }
    }
    constexpr int kRed = TPR > 64 ? 2 * (THREADS / 64) : 1;
    __shared__ float red[2 * kRed];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    const T *x = static_cast<const T *>(a.x);
    const T *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.y);
    int c[NV], lo[NV];
    bool edge[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
        edge[j] = wave_has_edge<W, TAIL>(lo[j]);
    }
    const int64_t nsb = (a.C + kBlock8 - 1) / kBlock8;
    using Row = BackwardRow<D, W, TAIL, NV, SAVED>;
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
        r.mean = a.mean[m];
        r.rstd = a.rstd[m];
    };
    RowLoop<Row, kSlots, sizeof(T) == 2 || NV < 4> loop{a.M, slot, FEW ? a.rows_end : gridDim.x};
    loop.begin(fetch);
    float ga[NV][W], dg[NV][W], db[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        load_affine<W>(a.af.gamma, a.af.type, c[j], 1.0f, ga[j]);
#pragma unroll
        for (int i = 0; i < W; ++i) dg[j][i] = db[j][i] = 0.0f;
    }
    int par = 0;
    loop.run(fetch, [&](Row &r, int64_t m, bool live) {
        // sums of g and of g*(x-mean); h = (x-mean)*rstd
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[W];
            r.centred(j, c[j], edge[j], x);
            float g[W];
#pragma unroll
            for (int i = 0; i < W; ++i) g[i] = r.vy[j].get(i) * ga[j][i];
            s[0] += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) { return g[i]; });
            s[1] += own_sum<W, TAIL>(lo[j], edge[j], [&](int i) { return g[i] * x[i]; });
        }
        row_sum<TPR>(s, red + par * kRed);
        par ^= 1;
        if (!live) return;  // no barrier from here on
        // With two pieces or more the widened values are made again rather than
        // kept across the sums, for their registers.
        if constexpr (NV > 1) r.opaque();
        // rstd by rstd, not their square, which leaves fp32's range where dx does not
        const float s0 = s[0] * a.inv_c, s1 = r.rstd * (r.rstd * (s[1] * a.inv_c));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[W], o[W];
            r.centred(j, c[j], edge[j], x);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = r.vy[j].get(i);
                o[i] = r.rstd * fmaf(-x[i], s1, fmaf(d, ga[j][i], -s0));
                if constexpr (!FEW) {
                    dg[j][i] = fmaf(d * r.rstd, x[i], dg[j][i]);
                    db[j][i] += d;
                }
            }
            // Rows off 16-byte boundaries: from the checkpoint nontemporal, from x
            // itself plain.  Measured, us nontemporal / plain, with dx in new
            // memory each call (and in the memory of the call before): saved
            // (12000,1001) 23.5/24.8, (33520,1001) 53.3/55.1 (52.3/51.7),
            // (40001,1537) 99/102.6 (97.8/100.2), fp32 (8001,1001) 19.5/22.3; x
            // itself (12000,1001) 23.6/26.9 (24.0/23.9), (33520,1001) 55.7/57.2
            // (55.0/53.5), (40001,1537) 103/106 (102/104), (100001,257) 64.3/63.5
            // (64.4/62.0): plain gains where the caches still hold dx's lines.
            if (lo[j] < W)
                Piece<D, W>::template store<!TAIL || SAVED>(dx + m * a.y_stride + c[j], o);
        }
    });
    if (FEW || a.part == nullptr) return;
    // The row slots of the workgroup: within a wave by butterflies over the
    // lanes that hold the same channels, then slot by slot (wave by wave)
    // through LDS.
    float *pg = a.part + int64_t{blockIdx.x} * a.C;
    float *pb = pg + int64_t{gridDim.x} * a.C;
    if constexpr (TPR >= 64) {
        constexpr int kPer = NV * W;
        __shared__ float comb[kSlots > 1 ? 2 * kPer * TPR : 1];
#pragma unroll 1
        for (int w = 0; w < kSlots; ++w) {
            if (slot == w) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const int e = (j * W + i) * TPR + t;
                        if constexpr (kSlots > 1) {
                            if (w > 0) {
                                dg[j][i] += comb[e];
                                db[j][i] += comb[kPer * TPR + e];
                            }
                            if (w + 1 < kSlots) {
                                comb[e] = dg[j][i];
                                comb[kPer * TPR + e] = db[j][i];
                            }
                        }
                        if (w + 1 == kSlots && i >= lo[j]) {
                            pg[c[j] + i] = dg[j][i];
                            pb[c[j] + i] = db[j][i];
                        }
                    }
            }
            if constexpr (kSlots > 1) __syncthreads();
        }
    } else {
        static_assert(NV == 1, "rows of fewer lanes than a wave have one piece per lane");
        constexpr int kWaves = THREADS / 64;
        __shared__ float comb[2][kWaves][W][TPR];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float g = dg[0][i], b = db[0][i];
#pragma unroll
            for (int o = TPR; o < 64; o <<= 1) {
                g += __shfl_xor(g, o, 64);
                b += __shfl_xor(b, o, 64);
            }
            if ((threadIdx.x & 63) < TPR) {
                comb[0][threadIdx.x >> 6][i][t] = g;
                comb[1][threadIdx.x >> 6][i][t] = b;
            }
        }
        __syncthreads();
        if (threadIdx.x < TPR) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                float g = comb[0][0][i][t], b = comb[1][0][i][t];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) {
                    g += comb[0][w][i][t];
                    b += comb[1][w][i][t];
                }
                if (i >= lo[0]) {
                    pg[c[0] + i] = g;
                    pb[c[0] + i] = b;
                }
            }
        }
    }
}

// dgamma and dbeta from the K partial rows of C sums: 32 channels and 32 row
// parts per workgroup, each part's rows in order (eight rows' loads in
// flight), then the parts by a fixed tree, in fp64.  K = 0 writes zeros.
// blockIdx.y: 0 dgamma, 1 dbeta.
constexpr int kColLanes = 32, kColParts = 32;
__global__ __launch_bounds__(kColLanes *kColParts) void gn_column_sums(const float *part,
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

LnShape ln_shape(int64_t C, int dtype, bool forward) {
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

template <class D>
void launch_forward(const LnShape &s, const LnArgs &a, hipStream_t st) {
    const int nt = forward_threads(s.tpr);
    const int64_t blocks = std::min(ceil_div(a.M, nt / s.tpr), kForwardLanes / nt);
    with_ln_shape<D, true>(s, [&](auto w, auto tail, auto tpr, auto nv) {
        constexpr int W = decltype(w)::value, TPR = decltype(tpr)::value;
        constexpr int NV = decltype(nv)::value, NT = forward_threads(TPR);
        constexpr bool TAIL = decltype(tail)::value != 0;
        const dim3 grid(static_cast<unsigned>(blocks)), block(NT);
        if (a.codes_out != nullptr)
            gn_layer_norm<D, W, TAIL, TPR, NV, NT, true><<<grid, block, 0, st>>>(a);
        else
            gn_layer_norm<D, W, TAIL, TPR, NV, NT, false><<<grid, block, 0, st>>>(a);
    });
}

int64_t backward_blocks(const LnShape &s, int64_t M) {
    const int64_t slots = backward_threads(s.tpr, s.nv) / s.tpr;
    return std::max(std::min(ceil_div(M, slots), kBackwardBlocks), ceil_div(M, slots * kMaxRun));
}

// Up to this many rows the columns' workgroups read x and dy again instead of
// adding up partial rows.  Measured on MI355X, bf16, partial rows / again:
// (1024,1024) 22.4/17.5 us a call, (2048,1024) 22.3/24.5, (4096,256) 22.1/41.4.
constexpr int64_t kFewRows = 1024;

template <class D>
void launch_backward(const LnShape &s, LnArgs a, bool grads, hipStream_t st) {
    const int64_t blocks = backward_blocks(s, a.M);
    const bool few = a.M <= kFewRows;
    a.rows_end = static_cast<uint32_t>(blocks);
    with_ln_shape<D, false>(s, [&](auto w, auto tail, auto tpr, auto nv) {
        constexpr int W = decltype(w)::value, TPR = decltype(tpr)::value;
        constexpr int NV = decltype(nv)::value, NT = backward_threads(TPR, NV);
        constexpr bool TAIL = decltype(tail)::value != 0;
        const unsigned rows = static_cast<unsigned>(blocks);
        const unsigned cols =
            few && grads ? static_cast<unsigned>(ceil_div(s.P, kColPieces)) : 0u;
        auto launch = [&](auto saved, auto fewc, unsigned grid) {
            gn_layer_norm_backward<D, W, TAIL, TPR, NV, NT, decltype(saved)::value != 0,
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

template <class F>
void by_type(int dtype, F &&f) {
    switch (x_dtype(dtype)) {
        case GN_DTYPE_F16: f(Fp16{}); break;
        case GN_DTYPE_F32: f(F32{}); break;
        default: f(Bf16{}); break;
    }
}

bool overflows(int64_t M, int64_t stride, int64_t C) {
    return M > 0 && stride > 0 && M > (INT64_MAX / 4 - C) / stride;
}

bool misaligned(const void *p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

// The checks both passes share; in_strides: row strides of inputs (0: one row
// for all), out_stride: of the output.
gn_status check_ln(int64_t M, int64_t C, int dtype, const int64_t *in_strides, int n_in,
                   int64_t out_stride) {
    if (!valid_dtype(dtype)) return GN_INVALID_ARGUMENT;
    if (M < 0 || C <= 0) return GN_INVALID_ARGUMENT;
    if (overflows(M, C, C)) return GN_INVALID_ARGUMENT;
    for (int i = 0; i < n_in; ++i) {
        if (in_strides[i] < 0) return GN_INVALID_ARGUMENT;
        if (overflows(M, in_strides[i], C)) return GN_INVALID_ARGUMENT;
    }
    if (out_stride < 0 || (M > 1 && out_stride < C)) return GN_INVALID_ARGUMENT;
    if (overflows(M, out_stride, C)) return GN_INVALID_ARGUMENT;
    if (C > GN_LAYER_NORM_MAX_CHANNELS) return GN_UNSUPPORTED;
    return GN_OK;
}

size_t backward_workspace(int64_t M, int64_t C, int dtype) {
    if (M <= kFewRows) return 0;
    return sizeof(float) * 2 * static_cast<size_t>(backward_blocks(ln_shape(C, dtype, false), M)) *
           static_cast<size_t>(C);
}

}  // namespace
}  // namespace gnsilu

using namespace gnsilu;

extern "C" {

gn_status gn_layer_norm_rows(const void *x, int64_t x_stride, const void *gamma, const void *beta,
                             void *y, int64_t y_stride, int64_t M, int64_t C, float eps, int dtype,
                             float *mean_out, float *rstd_out, void *codes_out, void *scales_out,
                             void *stream) {
    if (x == nullptr || y == nullptr) return GN_INVALID_ARGUMENT;
    if ((codes_out == nullptr) != (scales_out == nullptr)) return GN_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || std::isinf(eps)) return GN_INVALID_ARGUMENT;
    gn_status st = check_ln(M, C, dtype, &x_stride, 1, y_stride);
    if (st == GN_OK) st = check_affine(gamma, beta, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(x, es) || misaligned(y, es) || misaligned(mean_out, 4) ||
        misaligned(rstd_out, 4))
        return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    Call c;
    st = begin_call(stream,
                    {x, gamma, beta, y, mean_out, rstd_out, codes_out, scales_out}, &c);
    if (st != GN_OK) return st;
    const LnShape s = ln_shape(C, dtype, true);
    LnArgs a{};
    a.x = x;
    a.y = y;
    a.codes_out = static_cast<int8_t *>(codes_out);
    a.scales_out = static_cast<uint8_t *>(scales_out);
    a.mean = mean_out;
    a.rstd = rstd_out;
    a.M = M;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.C = static_cast<int>(C);
    a.P = s.P;
    a.eps = eps;
    a.af = Affine{gamma, beta, affine_type(dtype)};
    by_type(dtype, [&](auto d) { launch_forward<decltype(d)>(s, a, c.stream); });
    return finish_launch();
}

gn_status gn_layer_norm_rows_backward_workspace(int64_t M, int64_t C, int dtype,
                                                int64_t *bytes_out) {
    if (bytes_out == nullptr) return GN_INVALID_ARGUMENT;
    const gn_status st = check_ln(M, C, dtype, nullptr, 0, C);
    if (st != GN_OK) return st;
    if (M > 0 && backward_blocks(ln_shape(C, dtype, false), M) >= int64_t{1} << 22)
        return GN_UNSUPPORTED;
    *bytes_out = static_cast<int64_t>(backward_workspace(M, C, dtype));
    return GN_OK;
}

gn_status gn_layer_norm_rows_backward(const void *dy, int64_t dy_stride, const void *x,
                                      int64_t x_stride, const void *codes, const void *scales,
                                      const float *mean, const float *rstd, const void *gamma,
                                      void *dx, int64_t dx_stride, void *dgamma, void *dbeta,
                                      int64_t M, int64_t C, int dtype, void *workspace,
                                      int64_t workspace_bytes, void *stream) {
    if (dy == nullptr || dx == nullptr || mean == nullptr || rstd == nullptr)
        return GN_INVALID_ARGUMENT;
    // x, or its checkpoint, not both
    if ((codes == nullptr) != (scales == nullptr) || (x == nullptr) == (codes == nullptr))
        return GN_INVALID_ARGUMENT;
    const int64_t strides[2] = {dy_stride, x == nullptr ? 0 : x_stride};
    gn_status st = check_ln(M, C, dtype, strides, 2, dx_stride);
    if (st == GN_OK) st = check_affine(gamma, nullptr, dtype);
    if (st == GN_OK) st = check_affine(dgamma, dbeta, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(dy, es) || misaligned(x, es) || misaligned(dx, es) || misaligned(mean, 4) ||
        misaligned(rstd, 4) || misaligned(workspace, 4))
        return GN_UNSUPPORTED;
    const bool grads = dgamma != nullptr || dbeta != nullptr;
    if (M == 0 && !grads) return GN_OK;
    const size_t need = grads ? backward_workspace(M, C, dtype) : 0;
    if (M > 0 && backward_blocks(ln_shape(C, dtype, false), M) >= int64_t{1} << 22)
        return GN_UNSUPPORTED;  // a dispatch holds fewer than 2^32 work-items
    if (need > 0 && workspace == nullptr) return GN_INVALID_ARGUMENT;
    if (need > 0 && (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < need))
        return GN_SCRATCH_TOO_SMALL;
    Call c;
    st = begin_call(stream,
                    {dy, x, codes, scales, mean, rstd, gamma, dx, dgamma, dbeta,
                     need > 0 ? workspace : nullptr},
                    &c);
    if (st != GN_OK) return st;
    const LnShape s = ln_shape(C, dtype, false);
    LnArgs a{};
    a.x = x;
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.dy = dy;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.part = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.M = M;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.y_stride = dx_stride;
    a.C = static_cast<int>(C);
    a.P = s.P;
    a.inv_c = 1.0f / static_cast<float>(C);
    a.af = Affine{gamma, nullptr, affine_type(dtype)};
    if (M > 0)
        by_type(dtype, [&](auto d) { launch_backward<decltype(d)>(s, a, grads, c.stream); });
    if (need > 0 || M == 0)  // M = 0: zeros
        gn_column_sums<<<dim3(static_cast<unsigned>(ceil_div(C, kColLanes)), 2),
                         kColLanes * kColParts, 0, c.stream>>>(a.part,
                                     M > 0 ? backward_blocks(s, M) : 0, a.C, dgamma, dbeta,
                                     a.af.type);
    return finish_launch();
}

}  // extern "C"
