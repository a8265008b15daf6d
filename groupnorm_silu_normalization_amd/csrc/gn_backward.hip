// gn_backward.hip -- the backward pass of GroupNorm(+SiLU) over (N, L, C)
// rows, the apply step that keeps its input in 8 bits, and the 8-bit
// checkpoints themselves, for MI355X (gfx950).
//
//   h = (x-mean)*rstd, t = gamma*h + beta, s = 1/(1+exp(-t)),
//   dt = dy*s*(1 + t*(1-s))                       (dt = dy without SiLU)
//   dbeta[c]  = sum over n, l of dt,   dgamma[c] = sum over n, l of dt*h
//   a = sum over the group of gamma*dt / M,  b = ... of gamma*dt*h / M, M = L*Cg
//   dx = rstd*(gamma*dt - a - h*b)
//
// The group sums are sums over channels of gamma times the channel sums, so
// one pass over x and dy that keeps two sums per channel gives everything
// (pass 1); a small kernel finishes the sums; a second pass over x and dy
// writes dx (pass 2).  Both passes are bound by memory and by the vector ALU
// (about sixteen instructions per value, SiLU's exponential and reciprocal
// among them), so t is one fma, its exponential and reciprocal the hardware's,
// and dx two fmas and a product on dt and x-mean.
//
// A lane keeps one piece of W consecutive channels for all its rows: a tile is
// R rows of Pc pieces over the workgroup's lanes, and a longer row is cut into
// column blocks.  Channel parameters and sums stay in registers.  The
// workgroups advance through a sample together, a batch of tiles each, with the
// next batch's loads in flight; small samples go in one launch instead
// (gn_grad_strip).
//
// Measured on MI355X, bf16 (a 1 GiB copy reads and writes 5.1 TB/s there):
// (1,1048576,256) pass 1 191 us (5.6 TB/s, VALU 76% busy), finish 5.8 us, pass
// 2 284 us (5.7 TB/s); from the checkpoint, (1,65536,512), 28.7, 5.6 and 31.5
// us (pass 1 bound by the VALU and its start and end, pass 2 by its stores);
// apply that saves, (1,262144,512), 130 us (5.2 TB/s), restored 71.6 us (5.7).
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

constexpr int kLanes = 256;
// Lanes of pass 1's workgroups beyond kSmallBytes: 256/512/1024 lanes took
// 204/193/196 us at (1,1048576,256), and 7.0/8.3/11.9 at (1,4096,128).  Many
// samples that one batch of 256 lanes holds stay with 256: 256/512 took 93/162
// us at (10000,64,64), 799/1540 at (100000,16,32).
constexpr int kSumLanes = 512;
// Tiles per batch; two batches of loads are in flight.  Pass 2 from x itself
// takes more: 2/4/6 took 295/282/290 us at (1,1048576,256); from a checkpoint
// 2/4 took 32.9/35.4 us at (1,65536,512).
constexpr int kUnroll = 2;
constexpr int kInputUnroll = 4;

struct Tiles {
    int64_t L;        // rows per sample
    int64_t batches;  // batches of U tiles per sample (the last one may be partial)
    int64_t K;        // workgroups per sample and column block: every K-th batch is one's own
    int C, P;         // channels and pieces of a row
    int ncb, Pc;      // column blocks of a row and their pieces
    int R;            // rows per tile
};

struct RowArgs {
    const void *x;
    const int8_t *codes;
    const uint8_t *scales;
    const void *dy;
    void *y;  // y, dx, or the restored rows
    int8_t *codes_out;
    uint8_t *scales_out;
    const float *mean, *rstd;  // [N][G]
    float *part;               // [N][K][2][C]: pass 1's sums of dt and of dt*(x-mean)
    const float *coef;         // [N][G][2]: a and b
    int64_t x_stride, y_stride;  // elements between rows
    int G, Cg;
    Affine af;
    Tiles tl;
    // pass 2 of several samples: the first workgroups, beside the others, add up
    // dgamma and dbeta
    uint32_t sample_blocks;
    int64_t N;
    const float *sums;  // [N][2][C]
    void *dgamma, *dbeta;
};

// The calling lane's sample, workgroup of the sample, row slot and piece.
template <int W, bool TAIL> struct Place {
    int64_t n, k;
    int r, c, lo;
    bool active;
    __device__ __forceinline__ explicit Place(const Tiles &t, uint32_t b = blockIdx.x) {
        const uint32_t nk = b / static_cast<uint32_t>(t.ncb);
        const int cb = static_cast<int>(b - nk * static_cast<uint32_t>(t.ncb));
        const uint32_t ns = nk / static_cast<uint32_t>(t.K);
        k = nk - ns * static_cast<uint32_t>(t.K);
        n = ns;
        r = static_cast<int>(threadIdx.x) / t.Pc;
        const int p = cb * t.Pc + static_cast<int>(threadIdx.x) - r * t.Pc;
        active = r < t.R && p < t.P;
        c = active ? p * W : 0;
        lo = 0;
        if (TAIL && c + W > t.C) {
            lo = c + W - t.C;
            c = t.C - W;
        }
    }
};

// A workgroup's batches k, k + K, ...: the workgroups together move through
// the sample as one front, and while a batch is worked on the next one's
// loads are in flight.  load(v, d) and work(v, d, live) take the row that lies
// d rows behind the lane's row slot; rows behind the sample's last one are
// read as that one and not live.  BACK: from the sample's end.
template <bool BACK, int U, class V> struct Stream {
    const Tiles &tl;
    int64_t r;
    V a[U], b[U];
    __device__ __forceinline__ Stream(const Tiles &t, int row_slot) : tl(t), r(row_slot) {}
    __device__ __forceinline__ int64_t first(int64_t i) const {
        return (BACK ? tl.batches - 1 - i : i) * (U * tl.R);
    }
    template <class Load>
    __device__ __forceinline__ void fetch(V (&v)[U], int64_t i, Load &&load) {
        const int64_t d = first(i);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t l = d + u * tl.R + r;
            load(v[u], (l < tl.L ? l : tl.L - 1) - r);
        }
    }
    template <class Work>
    __device__ __forceinline__ void work(const V (&v)[U], int64_t i, Work &&w) {
        const int64_t d = first(i);
#pragma unroll
        for (int u = 0; u < U; ++u) w(v[u], d + u * tl.R, d + u * tl.R + r < tl.L);
    }
    // The first batch's loads; before the loads of the channel parameters, so
    // that their round trips overlap.
    template <class Load> __device__ __forceinline__ void begin(int64_t k, Load &&load) {
        fetch(a, k, load);
    }
    template <class Load, class Work>
    __device__ __forceinline__ void run(int64_t k, Load &&load, Work &&w) {
        for (int64_t i = k;;) {
            int64_t n = i + tl.K;
            if (n < tl.batches) fetch(b, n, load);
            work(a, i, w);
            if (n >= tl.batches) break;
            i = n;
            n += tl.K;
            if (n < tl.batches) fetch(a, n, load);
            work(b, i, w);
            if (n >= tl.batches) break;
            i = n;
        }
    }
};

// A lane's W channels of sample n: mean and rstd, scale = gamma*rstd, beta.
template <int W> struct Channels {
    float mu[W], rs[W], sc[W], be[W];
    __device__ __forceinline__ void load(const RowArgs &a, int64_t n, int c) {
        load_affine<W>(a.af.gamma, a.af.type, c, 1.0f, sc);
        load_affine<W>(a.af.beta, a.af.type, c, 0.0f, be);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t g = n * a.G + (c + i) / a.Cg;
            mu[i] = a.mean[g];
            rs[i] = a.rstd[g];
        }
#pragma unroll
        for (int i = 0; i < W; ++i) sc[i] *= rs[i];
    }
};

// dt = dy * d/dt(t*sigmoid(t)); with u = t*s the derivative is s + u*(1-s).
__device__ __forceinline__ float silu_grad(float t, float dy) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.4426950408889634f));
    return dy * fmaf(t * s, 1.0f - s, s);
}

// dx = dt*scale + rstd*((x-mean)*k1 + k0), k1 = -rstd*b, k0 = -a.  The outer
// rstd stays a product of its own: rstd*k1 leaves fp32's range (rstd above
// 1e19, below 1e-19) where dx does not.
__device__ __forceinline__ float input_grad(float dt, float x, float sc, float rs, float k1,
                                            float k0) {
    return fmaf(dt, sc, rs * fmaf(x, k1, k0));
}

// One row's piece of x (or its saved codes) and dy.
template <class D, int W, bool TAIL, bool SAVED> struct Pair {
    using T = typename D::storage;
    Piece<D, W> vx, vy;
    Piece8<W, TAIL> v8;
    // The lane's piece of its row slot's first row; d rows further is a scalar
    // away.
    struct From {
        const T *x, *dy;
        Piece8At<W, TAIL> at8;
        int64_t C, nsb;
        __device__ __forceinline__ From(const RowArgs &a, int64_t row, int c)
            : x(static_cast<const T *>(a.x) + row * a.tl.C + c),
              dy(static_cast<const T *>(a.dy) + row * a.tl.C + c),
              at8(a.codes, a.scales, row, a.tl.C, c), C(a.tl.C),
              nsb((a.tl.C + kBlock8 - 1) / kBlock8) {}
    };
    __device__ __forceinline__ void load(const From &f, int64_t d) {
        if constexpr (SAVED)
            v8.load(f.at8, d * f.C, d * f.nsb);
        else
            vx.template load<false>(f.x + d * f.C);
        vy.template load<false>(f.dy + d * f.C);
    }
    // x - mean: a saved value is widened and shifted in one fma
    __device__ __forceinline__ void centred(int c, const float (&mu)[W], bool edge,
                                            float (&o)[W]) const {
        if constexpr (SAVED) {
            v8.widen_less(c, mu, edge, o);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = vx.get(i) - mu[i];
        }
    }
};

// Adds the tile's R row slots' values by a fixed tree, into slot 0.
template <int W, int NT>
__device__ __forceinline__ void slot_tree(float (&red)[W][NT], int r, int R, int Pc,
                                          float (&s)[W]) {
    if (R == 1) return;
    int p2 = 1;
    while (p2 < R) p2 <<= 1;
    __syncthreads();  // red is free
#pragma unroll
    for (int i = 0; i < W; ++i) red[i][threadIdx.x] = s[i];
    for (int h = p2 >> 1; h > 0; h >>= 1) {
        __syncthreads();
        if (r < h && r + h < R) {
            const int o = static_cast<int>(threadIdx.x) + h * Pc;
#pragma unroll
            for (int i = 0; i < W; ++i) red[i][threadIdx.x] = s[i] += red[i][o];
        }
    }
}

// Pass 1, by workgroups of NT lanes.
template <class D, int W, bool TAIL, bool SILU, bool SAVED, int NT>
__global__ __launch_bounds__(NT) void gn_grad_sums(RowArgs a) {
    __shared__ float red[W][NT];
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    const int64_t row0 = at.n * tl.L + at.r;
    using V = Pair<D, W, TAIL, SAVED>;
    const typename V::From from(a, row0, at.c);
    auto load = [&](V &v, int64_t d) { v.load(from, d); };
    const bool edge = SAVED && wave_has_edge<W, TAIL>(at.lo);
    Stream<false, kUnroll, V> st(tl, at.r);
    st.begin(at.k, load);
    Channels<W> ch;
    ch.load(a, at.n, at.c);
    float s1[W], s2[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s1[i] = s2[i] = 0.0f;
    st.run(at.k, load, [&](const V &v, int64_t, bool live) {
        if (!live) return;
        float x[W];
        v.centred(at.c, ch.mu, edge, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float d = v.vy.get(i);
            if constexpr (SILU) d = silu_grad(fmaf(x[i], ch.sc[i], ch.be[i]), d);
            s1[i] += d;
            s2[i] = fmaf(d, x[i], s2[i]);
        }
    });
    slot_tree<W, NT>(red, at.r, tl.R, tl.Pc, s1);
    slot_tree<W, NT>(red, at.r, tl.R, tl.Pc, s2);
    if (at.active && at.r == 0) {
        float *p = a.part + (at.n * tl.K + at.k) * 2 * tl.C + at.c;
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i >= at.lo) {
                p[i] = s1[i];
                p[tl.C + i] = s2[i];
            }
    }
}

// Finishes pass 1: channel sums over the K partials, in fp64.  A workgroup
// takes tile_c channels of one sample: its 1024 threads are 2^width lanes of
// channels by 2^(10-width) parts of the partials, each part's partials added
// in order, then the parts by fixed trees.  sums[N][2][C] receives sum dt and
// sum dt*h.  A tile of whole groups (Cg <= 64) also gives their a and b; one
// sample alone its dgamma and dbeta.  The narrowest tile that holds a group
// (16 to 64 channels) has the most parts and so the shortest chain of loads.
// FEW: no more partials than a part has loads in flight, as in many small
// samples: each of four waves takes a tile of up to 64 channels.  1024 threads a
// tile took (200,3,8192) 559 us, (10000,64,64) 486 and (500,256,320) 176.
constexpr int kFinishThreads = 1024, kFinishBatch = 8, kFewThreads = 256;
struct FinishArgs {
    const float *part;
    const float *rstd;
    float *sums, *coef;
    void *dgamma, *dbeta;  // null unless N = 1 and wanted
    int64_t K, all_tiles;  // all_tiles: of the samples together
    int C, G, Cg, tile_c, tiles, width;
    double inv_m;
    Affine af;
};
template <bool FEW>
__global__ __launch_bounds__(FEW ? kFewThreads : kFinishThreads) void gn_grad_finish(FinishArgs a) {
    const int tid = FEW ? threadIdx.x & 63 : threadIdx.x;
    const int wide = FEW ? 64 : 1 << a.width, parts = FEW ? 1 : kFinishThreads >> a.width;
    const int lane = tid & (wide - 1), r = FEW ? 0 : tid >> a.width;
    const uint32_t tile = FEW ? blockIdx.x * (kFewThreads / 64) + (threadIdx.x >> 6) : blockIdx.x;
    if (FEW && tile >= a.all_tiles) return;
    const int64_t n = tile / static_cast<uint32_t>(a.tiles);
    const int c = static_cast<int>(tile % static_cast<uint32_t>(a.tiles)) * a.tile_c + lane;
    const bool live = lane < a.tile_c && c < a.C;
    double s1 = 0.0, s2 = 0.0;
    float ga[1] = {0.0f}, rs = 0.0f;
    if (live) {
        // used at the end; their round trips overlap the partials'
        rs = a.rstd[n * a.G + c / a.Cg];
        load_affine<1>(a.af.gamma, a.af.type, c, 1.0f, ga);
        const float *p = a.part + n * a.K * 2 * a.C + c;
        // the loads of a batch in flight (the last ones clamped, not added)
        constexpr int kBatch = kFinishBatch;
        const int64_t step = 2 * static_cast<int64_t>(a.C);
        for (int64_t k = r; k < a.K; k += kBatch * parts) {
            float v1[kBatch], v2[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int64_t ku = k + u * parts < a.K ? k + u * parts : a.K - 1;
                v1[u] = p[ku * step];
                v2[u] = p[ku * step + a.C];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool in = k + u * parts < a.K;
                s1 += in ? static_cast<double>(v1[u]) : 0.0;
                s2 += in ? static_cast<double>(v2[u]) : 0.0;
            }
        }
    }
    if constexpr (!FEW) {
        // the parts within a wave by a butterfly, then the 16 waves' sums: wave
        // 0 adds each channel's in `per` interleaved runs and joins those
        __shared__ double red[2][kFinishThreads];
        const int per = 64 >> a.width;
        for (int o = wide; o < 64; o <<= 1) {
            s1 += __shfl_xor(s1, o, 64);
            s2 += __shfl_xor(s2, o, 64);
        }
        if ((tid & 63) < wide) {
            red[0][(tid >> 6) * wide + lane] = s1;
            red[1][(tid >> 6) * wide + lane] = s2;
        }
        __syncthreads();
        if (tid >= 64) return;
        s1 = s2 = 0.0;
#pragma unroll 4
        for (int w = r; w < kFinishThreads / 64; w += per) {
            s1 += red[0][w * wide + lane];
            s2 += red[1][w * wide + lane];
        }
        for (int o = wide; o < 64; o <<= 1) {
            s1 += __shfl_xor(s1, o, 64);
            s2 += __shfl_xor(s2, o, 64);
        }
    }
    s2 *= static_cast<double>(rs);
    if (live && r == 0) {
        a.sums[n * 2 * a.C + c] = static_cast<float>(s1);
        a.sums[n * 2 * a.C + a.C + c] = static_cast<float>(s2);
        if (a.dbeta != nullptr) store_affine(a.dbeta, a.af.type, c, static_cast<float>(s1));
        if (a.dgamma != nullptr) store_affine(a.dgamma, a.af.type, c, static_cast<float>(s2));
    }
    if (a.coef == nullptr) return;
    s1 *= static_cast<double>(ga[0]);
    s2 *= static_cast<double>(ga[0]);
    // The sums of lanes lane .. lane + Cg - 1, the group that starts at the
    // lane, from runs of 1, 2, 4, ... lanes (a group of 64 lanes, lane by lane:
    // 677 us at (8192,1,2048) with 64 channels a group).
    double ta = 0.0, tb = 0.0;
    for (int run = 1, at = lane; run <= a.Cg; run <<= 1) {
        if (a.Cg & run) {
            ta += __shfl(s1, at, 64);
            tb += __shfl(s2, at, 64);
            at += run;
        }
        s1 += __shfl(s1, lane + run, 64);
        s2 += __shfl(s2, lane + run, 64);
    }
    if (live && r == 0 && lane % a.Cg == 0) {
        float *o = a.coef + 2 * (n * a.G + c / a.Cg);
        o[0] = static_cast<float>(ta * a.inv_m);
        o[1] = static_cast<float>(tb * a.inv_m);
    }
}

// a and b of a group of more than 64 channels, from the channel sums.
__global__ __launch_bounds__(kLanes) void gn_grad_groups(FinishArgs a) {
    __shared__ double red[2][kLanes];
    const int64_t n = blockIdx.x / a.G;
    const int g = static_cast<int>(blockIdx.x % a.G);
    const int tid = threadIdx.x;
    double ta = 0.0, tb = 0.0;
    for (int i = tid; i < a.Cg; i += kLanes) {
        const int c = g * a.Cg + i;
        float ga[1];
        load_affine<1>(a.af.gamma, a.af.type, c, 1.0f, ga);
        ta += static_cast<double>(ga[0]) * static_cast<double>(a.sums[n * 2 * a.C + c]);
        tb += static_cast<double>(ga[0]) * static_cast<double>(a.sums[n * 2 * a.C + a.C + c]);
    }
    red[0][tid] = ta;
    red[1][tid] = tb;
    __syncthreads();
    for (int h = kLanes / 2; h > 0; h >>= 1) {
        if (tid < h) {
            red[0][tid] += red[0][tid + h];
            red[1][tid] += red[1][tid + h];
        }
        __syncthreads();
    }
    if (tid == 0) {
        float *o = a.coef + 2 * blockIdx.x;
        o[0] = static_cast<float>(red[0][0] * a.inv_m);
        o[1] = static_cast<float>(red[1][0] * a.inv_m);
    }
}

// dgamma and dbeta of N samples (zeros for none): a workgroup takes 16 channels
// and 16 parts of the samples, each part's in order with eight samples' loads
// in flight, then the parts in a fixed order, in fp64.  One lane a channel, a
// sample at a time, took 0.27 us a sample: 72.5 us of pass 2's launch at
// (300,3,32), 5.6 so.
constexpr int kSampleLanes = 16, kSampleParts = kLanes / kSampleLanes;
__device__ __forceinline__ void add_samples(const float *sums, int64_t N, int C, int block,
                                            void *dgamma, void *dbeta, int type) {
    constexpr int kWaves = kLanes / 64, kBatch = 8;
    __shared__ double red[2][kWaves][kSampleLanes];
    const int lane = threadIdx.x % kSampleLanes, part = threadIdx.x / kSampleLanes;
    const int c = block * kSampleLanes + lane;
    double s1 = 0.0, s2 = 0.0;
    if (c < C) {
        const float *p = sums + c;
        const int64_t step = 2 * static_cast<int64_t>(C);
        for (int64_t n = part; n < N; n += kBatch * kSampleParts) {
            float v1[kBatch], v2[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int64_t m = n + u * kSampleParts < N ? n + u * kSampleParts : N - 1;
                v1[u] = p[m * step];
                v2[u] = p[m * step + C];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool in = n + u * kSampleParts < N;
                s1 += in ? static_cast<double>(v1[u]) : 0.0;
                s2 += in ? static_cast<double>(v2[u]) : 0.0;
            }
        }
    }
#pragma unroll
    for (int o = kSampleLanes; o < 64; o <<= 1) {
        s1 += __shfl_xor(s1, o, 64);
        s2 += __shfl_xor(s2, o, 64);
    }
    if ((threadIdx.x & 63) < kSampleLanes) {
        red[0][threadIdx.x >> 6][lane] = s1;
        red[1][threadIdx.x >> 6][lane] = s2;
    }
    __syncthreads();
    if (part > 0 || c >= C) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        s1 += red[0][w][lane];
        s2 += red[1][w][lane];
    }
    if (dbeta != nullptr) store_affine(dbeta, type, c, static_cast<float>(s1));
    if (dgamma != nullptr) store_affine(dgamma, type, c, static_cast<float>(s2));
}
__global__ __launch_bounds__(kLanes) void gn_grad_samples(const float *sums, int64_t N, int C,
                                                          void *dgamma, void *dbeta, int type) {
    add_samples(sums, N, C, static_cast<int>(blockIdx.x), dgamma, dbeta, type);
}

// Pass 2: dx from the rows that pass 1 read last to those that it read first,
// so that what the Infinity Cache still holds of x and dy is read before it is
// replaced; dx is stored nontemporally for the same reason.
template <class D, int W, bool TAIL, bool SILU, bool SAVED>
__global__ __launch_bounds__(kLanes) void gn_grad_input(RowArgs a) {
    using T = typename D::storage;
    if (blockIdx.x < a.sample_blocks) {
        add_samples(a.sums, a.N, a.tl.C, static_cast<int>(blockIdx.x), a.dgamma, a.dbeta,
                    a.af.type);
        return;
    }
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl, blockIdx.x - a.sample_blocks);
    const int64_t row0 = at.n * tl.L + at.r;
    using V = Pair<D, W, TAIL, SAVED>;
    const typename V::From from(a, row0, at.c);
    auto load = [&](V &v, int64_t d) { v.load(from, d); };
    const bool edge = SAVED && wave_has_edge<W, TAIL>(at.lo);
    Stream<true, SAVED ? kUnroll : kInputUnroll, V> st(tl, at.r);
    st.begin(at.k, load);
    Channels<W> ch;
    ch.load(a, at.n, at.c);
    float k0[W], k1[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float *co = a.coef + 2 * (at.n * a.G + (at.c + i) / a.Cg);
        k0[i] = -co[0];
        k1[i] = -ch.rs[i] * co[1];
    }
    T *dx = static_cast<T *>(a.y) + row0 * tl.C + at.c;
    st.run(at.k, load, [&](const V &v, int64_t d, bool live) {
        if (!live || !at.active) return;
        float x[W], o[W];
        v.centred(at.c, ch.mu, edge, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float g = v.vy.get(i);
            if constexpr (SILU) g = silu_grad(fmaf(x[i], ch.sc[i], ch.be[i]), g);
            o[i] = input_grad(g, x[i], ch.sc[i], ch.rs[i], k1[i], k0[i]);
        }
        T *p = dx + d * tl.C;
        // dx may be dy or x: a lane writes only channels that no other reads
        if (!TAIL || at.lo == 0)
            Piece<D, W>::template store<true>(p, o);
        else
            store_from<D, W>(p, o, at.lo);
    });
}

// The whole backward pass in one launch, for samples small enough: a workgroup
// takes a strip of whole groups of one sample (P pieces of a row: the least
// common multiple of a group and a piece) and holds its x and dy in registers,
// NP pieces each per lane, so both are read once.  Its channels' sums: for P a
// power of two up to 32 (POW2) the lanes of a wave that hold the same piece by
// a butterfly, then the waves in order; else the row slots by a tree in LDS.
// dx is stored through the L2: strips narrower than a cache line write parts
// of lines, which neighbouring strips on the same XCD complete there
// ((1,4096,128): 22.0 us of kernel time with nontemporal stores and strips
// dealt over the XCDs, 16.7 so).
constexpr int kStripLanes = 1024;
constexpr int kStripMaxPieces = 4;    // NP
constexpr int kStripMaxRow = 128;     // P
constexpr int kStripMaxPow2Row = 32;  // P of the butterfly
struct StripArgs {
    RowArgs r;      // tl.L and tl.C
    float *sums;    // [N][2][C] to write, or null
    int P, shift;   // pieces of a strip's row; log2 for POW2
    int strips;     // per sample
    int xcd;        // the grid is a multiple of 8
    double inv_m;
};

// v plus its value in the lane whose number differs in the bits >= P of 63;
// P a power of two, the same for all lanes.  (A rotation by 8 within 16 lanes
// exchanges the halves; after it one by 4 exchanges the quads.)
__device__ __forceinline__ float fold_from(float v, int P) {
    auto add = [&](uint32_t o) { v += __uint_as_float(o); };
    if (P <= 1) add(dpp<kDppXor1>(__float_as_uint(v)));
    if (P <= 2) add(dpp<kDppXor2>(__float_as_uint(v)));
    if (P <= 8) add(dpp<kDppRor8>(__float_as_uint(v)));
    if (P <= 4) add(dpp<kDppRor4>(__float_as_uint(v)));
    if (P <= 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v),
                                                        false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <class D, int W, bool SILU, bool SAVED, int NP, bool POW2>
__global__ __launch_bounds__(kStripLanes) void gn_grad_strip(StripArgs sa) {
    using T = typename D::storage;
    constexpr int kWaves = kStripLanes / 64;
    static_assert(2 * kWaves * kStripMaxPow2Row == kStripLanes, "the waves' sums fill red");
    const RowArgs &a = sa.r;
    __shared__ float red[W][kStripLanes];
    __shared__ float total[2][kStripMaxRow * W];  // per channel: sums, then times gamma
    __shared__ float coef[2][W];                  // a and b of the strip's groups
    const int tid = threadIdx.x;
    // Workgroups go to the 8 XCDs in turn; neighbouring strips, whose rows share
    // cache lines, are given to workgroups of one XCD (one L2).
    const uint32_t wg = sa.xcd ? (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
    const int64_t n = wg / static_cast<uint32_t>(sa.strips);
    const int strip = static_cast<int>(wg % static_cast<uint32_t>(sa.strips));
    const int r = POW2 ? tid >> sa.shift : tid / sa.P;
    const int R = POW2 ? kStripLanes >> sa.shift : kStripLanes / sa.P;
    const int pc = tid - r * sa.P;
    const bool active = POW2 || r < R;
    const int c0 = strip * sa.P * W, c = c0 + pc * W, wide = sa.P * W;
    const int64_t row0 = n * a.tl.L;
    using V = Pair<D, W, false, SAVED>;
    const typename V::From from(a, row0, c);
    V v[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) {
        const int64_t l = r + int64_t{u} * R;
        v[u].load(from, l < a.tl.L ? l : a.tl.L - 1);
    }
    Channels<W> ch;
    ch.load(a, n, c);
    float s1[W], s2[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s1[i] = s2[i] = 0.0f;
    auto gradient = [&](const V &p, float (&x)[W], float (&g)[W]) {
        p.centred(c, ch.mu, false, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            g[i] = p.vy.get(i);
            if constexpr (SILU) g[i] = silu_grad(fmaf(x[i], ch.sc[i], ch.be[i]), g[i]);
        }
    };
#pragma unroll
    for (int u = 0; u < NP; ++u) {
        if (!active || r + int64_t{u} * R >= a.tl.L) break;
        float x[W], g[W];
        gradient(v[u], x, g);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s1[i] += g[i];
            s2[i] = fmaf(g[i], x[i], s2[i]);
        }
    }
    float t1 = 0.0f, t2 = 0.0f;  // thread tid's channel, tid < wide
    if constexpr (POW2) {
        float *const flat = &red[0][0];  // [2][kWaves][P * W]
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s1[i] = fold_from(s1[i], sa.P);
            s2[i] = fold_from(s2[i], sa.P);
        }
        if ((tid & 63) < sa.P) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                flat[(tid >> 6) * wide + pc * W + i] = s1[i];
                flat[(kWaves + (tid >> 6)) * wide + pc * W + i] = s2[i];
            }
        }
        __syncthreads();
        if (tid < wide) {
            t1 = flat[tid];
            t2 = flat[kWaves * wide + tid];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                t1 += flat[w * wide + tid];
                t2 += flat[(kWaves + w) * wide + tid];
            }
        }
    } else {
        slot_tree<W, kStripLanes>(red, r, R, sa.P, s1);
        slot_tree<W, kStripLanes>(red, r, R, sa.P, s2);
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                total[0][pc * W + i] = s1[i];
                total[1][pc * W + i] = s2[i];
            }
        }
        __syncthreads();
        if (tid < wide) {
            t1 = total[0][tid];
            t2 = total[1][tid];
        }
    }
    if (tid < wide) {
        const int cc = c0 + tid;
        t2 *= a.rstd[n * a.G + cc / a.Cg];
        if (sa.sums != nullptr) {
            sa.sums[n * 2 * a.tl.C + cc] = t1;
            sa.sums[n * 2 * a.tl.C + a.tl.C + cc] = t2;
        } else {
            if (a.dbeta != nullptr) store_affine(a.dbeta, a.af.type, cc, t1);
            if (a.dgamma != nullptr) store_affine(a.dgamma, a.af.type, cc, t2);
        }
        float ga[1];
        load_affine<1>(a.af.gamma, a.af.type, cc, 1.0f, ga);
        total[0][tid] = t1 * ga[0];
        total[1][tid] = t2 * ga[0];
    }
    __syncthreads();
    // the groups' sums in fp64, a wave each
    const int groups = wide / a.Cg;
    const int wave = tid >> 6, lane = tid & 63;
    if (wave < groups) {
        double ta = 0.0, tb = 0.0;
        for (int e = lane; e < a.Cg; e += 64) {
            ta += static_cast<double>(total[0][wave * a.Cg + e]);
            tb += static_cast<double>(total[1][wave * a.Cg + e]);
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            ta += __shfl_xor(ta, o, 64);
            tb += __shfl_xor(tb, o, 64);
        }
        if (lane == 0) {
            coef[0][wave] = static_cast<float>(ta * sa.inv_m);
            coef[1][wave] = static_cast<float>(tb * sa.inv_m);
        }
    }
    __syncthreads();
    if (!active) return;
    float k0[W], k1[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int g = (pc * W + i) / a.Cg;
        k0[i] = -coef[0][g];
        k1[i] = -ch.rs[i] * coef[1][g];
    }
    T *dx = static_cast<T *>(a.y) + row0 * a.tl.C + c;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
        const int64_t l = r + int64_t{u} * R;
        if (l >= a.tl.L) break;
        float x[W], g[W], o[W];
        gradient(v[u], x, g);
#pragma unroll
        for (int i = 0; i < W; ++i)
            o[i] = input_grad(g[i], x[i], ch.sc[i], ch.rs[i], k1[i], k0[i]);
        Piece<D, W>::template store<false>(dx + l * a.tl.C, o);
    }
}

// The apply step that also saves x (kApply, kApplySilu), or x saved alone
// (kSave).  A block of the format lies in consecutive lanes of one row: the
// plan makes Pc a multiple of the lanes that hold a block, or for shorter rows
// a power of two.  What is stored is read much later, if at all, so it goes
// past the caches -- but through the L2 where rows start off 16-byte
// boundaries (TAIL), which joins their partial lines there: (2,16760,1001) bf16
// with its restore took 65 us nontemporally, 57 so.
enum { kApply = 0, kApplySilu = 1, kSave = 2 };
template <class D, int W, bool TAIL, int MODE>
__global__ __launch_bounds__(kLanes) void gn_rows_save(RowArgs a) {
    using T = typename D::storage;
    constexpr int kGroup = W == 1 ? 8 : kBlock8 / W;
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L + at.r;
    using V = Piece<D, W>;
    const T *x0 = static_cast<const T *>(a.x) + row0 * a.x_stride + at.c;
    auto load = [&](V &v, int64_t d) { v.template load<false>(x0 + d * a.x_stride); };
    Stream<false, kUnroll, V> st(tl, at.r);
    st.begin(at.k, load);
    float sc[W], sh[W];
    if constexpr (MODE != kSave) {  // scale and shift as the apply step folds them
        Channels<W> ch;
        ch.load(a, at.n, at.c);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            sc[i] = ch.sc[i];
            sh[i] = fmaf(-ch.mu[i], ch.sc[i], ch.be[i]);
        }
    }
    const Magnitudes<D, W> mag(at.active ? at.lo : W);
    int8_t *codes0 = a.codes_out + row0 * tl.C;
    uint8_t *scales0 = a.scales_out + row0 * nsb;
    T *y0 = static_cast<T *>(a.y) + row0 * a.y_stride + at.c;
    // every lane of the workgroup takes part in the blocks' maxima
    st.run(at.k, load, [&](const V &v, int64_t d, bool live) {
        float x[W];
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = v.get(i);
        const uint32_t E = block8_exponent<D, W, kGroup>(v, mag, tl.Pc);
        if (!live || !at.active) return;
        if constexpr (MODE != kSave) {
            float o[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float t = fmaf(x[i], sc[i], sh[i]);
                o[i] = MODE == kApplySilu ? silu_f32(t) : t;
            }
            T *p = y0 + d * a.y_stride;
            if (!TAIL || at.lo == 0)  // y may be x: only the lane's own channels
                Piece<D, W>::template store<!TAIL>(p, o);
            else
                store_from<D, W>(p, o, at.lo);
        }
        store_block8<W, TAIL, !TAIL>(block8_encode<W>(x, E), E, codes0 + d * tl.C,
                                    scales0 + d * nsb, at.c, at.lo);
    });
}

// Saved rows widened again.
template <class D, int W, bool TAIL>
__global__ __launch_bounds__(kLanes) void gn_rows_restore(RowArgs a) {
    using T = typename D::storage;
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L + at.r;
    using V = Piece8<W, TAIL>;
    const Piece8At<W, TAIL> from(a.codes, a.scales, row0, tl.C, at.c);
    auto load = [&](V &v, int64_t d) { v.load(from, d * tl.C, d * nsb); };
    const bool edge = wave_has_edge<W, TAIL>(at.lo);
    T *y0 = static_cast<T *>(a.y) + row0 * a.y_stride + at.c;
    Stream<false, kUnroll, V> st(tl, at.r);
    st.begin(at.k, load);
    st.run(at.k, load, [&](const V &v, int64_t d, bool live) {
        if (!live || !at.active) return;
        float o[W];
        v.widen(at.c, edge, o);
        Piece<D, W>::template store<!TAIL>(y0 + d * a.y_stride, o);
    });
}

// ---- host -----------------------------------------------------------------------
constexpr int64_t kSumBlocks = 512;         // pass 1: 2 per CU, each with its partial sums
constexpr int64_t kStreamBlocks = 2048;     // the other passes (pass 2 at (1,1048576,256) with
                                            // 1024/1280/2048/4096: 294/288/283/285 us)
constexpr int64_t kSmallBytes = int64_t{16} << 20;  // x at most this: latency rules
constexpr int64_t kMaxRun = 1024;           // rows a lane adds up in fp32

// whole: lanes that must stay in one row together (a block of the format when
// saving, else 1).  A row is cut into column blocks of at most 64 pieces (a
// KiB), so that a workgroup's lanes cover several rows: its row slots add up
// before anything is written, and pieces and lanes fit each other better.  Rows
// that start off 16-byte boundaries are cut at 128: each cut costs them two
// partial cache lines.  Measured on MI355X, backward of 2^25 bf16 values in two
// samples, cut at 16/32/64/128/256: C = 2560 79/79/80/80/94 us, C = 8192
// 80/79/79/81/89, C = 1001 99/89/83/80/80.
constexpr int kMaxPieces = 64, kMaxPiecesTail = 128;
Tiles make_tiles(int64_t N, int64_t L, int64_t C, int w, int whole, int64_t blocks,
                 int64_t max_run = 0, int lanes = kLanes, int unroll = kUnroll) {
    Tiles t{};
    t.L = L;
    t.C = static_cast<int>(C);
    t.P = static_cast<int>(ceil_div(C, w));
    int best = 0;
    const int least = static_cast<int>(ceil_div(t.P, C % w == 0 ? kMaxPieces : kMaxPiecesTail));
    for (int ncb = least; ncb <= least + 3; ++ncb) {
        int pc = static_cast<int>(ceil_div(t.P, ncb));
        int part = whole;
        while (part / 2 >= pc) part /= 2;
        pc = static_cast<int>(ceil_div(pc, part)) * part;
        const int used = static_cast<int>(static_cast<int64_t>(lanes / pc) * t.P * 1024 /
                                          (int64_t{lanes} * ceil_div(t.P, pc)));
        if (used > best) {  // lanes at work, in 1024ths
            best = used;
            t.Pc = pc;
        }
        if (best >= 960 || pc <= 16) break;
    }
    t.ncb = static_cast<int>(ceil_div(t.P, t.Pc));
    t.R = lanes / t.Pc;
    t.batches = std::max<int64_t>(1, ceil_div(L, int64_t{t.R} * unroll));
    int64_t k = std::max<int64_t>(1, blocks / std::max<int64_t>(1, N * t.ncb));
    if (max_run > 0) k = std::max(k, ceil_div(t.batches * unroll, max_run));
    t.K = std::min(k, t.batches);
    return t;
}

int piece_width(int64_t C, int dtype) {
    const int w = static_cast<int>(16 / elem_bytes(dtype));
    return C < w ? 1 : w;
}
int block_lanes(int w) { return w == 1 ? 8 : kBlock8 / w; }

template <int V> using IC = std::integral_constant<int, V>;

// Calls f(D{}, IC<W>, IC<TAIL>).
template <class F>
void with_pieces(int64_t C, int dtype, F &&f) {
    auto by_w = [&](auto d) {
        using D = decltype(d);
        constexpr int W = static_cast<int>(16 / sizeof(typename D::storage));
        if (C < W)
            f(d, IC<1>{}, IC<0>{});
        else if (C % W != 0)
            f(d, IC<W>{}, IC<1>{});
        else
            f(d, IC<W>{}, IC<0>{});
    };
    switch (x_dtype(dtype)) {
        case GN_DTYPE_F16: by_w(Fp16{}); break;
        case GN_DTYPE_F32: by_w(F32{}); break;
        default: by_w(Bf16{}); break;
    }
}

dim3 grid_of(int64_t N, const Tiles &t) {
    return dim3(static_cast<unsigned>(N * t.K * t.ncb));
}
// A dispatch holds fewer than 2^32 work-items.
bool grid_fits(int64_t N, const Tiles &t, int lanes = kLanes) {
    const int64_t most = (int64_t{1} << 32) / lanes - GN_MAX_CHANNELS;  // and pass 2's sums
    return N < most && t.K < most && N * t.K < most && N * t.K * t.ncb < most;
}

bool misaligned(const void *p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

// Shape checks of the GroupNorm forms; dense rows.
gn_status check_group_rows(int64_t N, int64_t L, int64_t C, int64_t G, int apply_silu, int dtype) {
    if (!valid_dtype(dtype)) return GN_INVALID_ARGUMENT;
    if (N < 0 || L < 0 || C <= 0 || G <= 0 || C % G != 0) return GN_INVALID_ARGUMENT;
    if (apply_silu != 0 && apply_silu != 1) return GN_INVALID_ARGUMENT;
    if (L > 0 && N > INT64_MAX / L) return GN_INVALID_ARGUMENT;
    if (N * L > 0 && C > INT64_MAX / (N * L) / 4) return GN_INVALID_ARGUMENT;
    if (C > GN_MAX_CHANNELS) return GN_UNSUPPORTED;
    return GN_OK;
}

// The single launch: rows of whole pieces, a strip's row of at most
// kStripMaxRow pieces and its rows within kStripMaxPieces per lane, at most
// kStripMaxBlocks workgroups (so x at most 16 MiB).  A strip of one piece
// fetches eight times what it uses of each line, so these take x of at most
// kStripNarrowBytes.  Measured on MI355X, bf16, G = 32, us in a captured graph
// (eager calls, where a launch costs 3 us of host time), single launch / three:
// one piece (1,4096,128) 19.9/16.1 (19.9/24.5), (4,4096,128) 21.6/20.4
// (22.3/24.4), beyond the limit (5,4096,128) 25.2/22.3 (24.6/24.0),
// (8,4096,128) 24.7/24.3 (24.5/24.8); two (2,2048,512) 20.3/20.4 (20.6/24.1),
// (8,2048,512) 26.3/33.1 (25.7/32.8); four (8,1024,1024) 25.7/33.4 (25.1/33.6);
// more (1,256,512) 7.9/14.9 (16.3/23.8), (4,64,8192) 15/29.6.
constexpr int64_t kStripMaxBlocks = 256;
constexpr int64_t kStripNarrowBytes = int64_t{4} << 20;
struct StripPlan {
    int P = 0, shift = 0, np = 0, strips = 0;  // np = 0: not taken
    bool pow2 = false;
};
StripPlan strip_plan(int64_t N, int64_t L, int64_t C, int64_t G, int w) {
    StripPlan s;
    const int64_t cg = C / G;
    if (w == 1 || C % w != 0) return s;
    int64_t wide = cg;  // least common multiple with w, a power of two
    while (wide % w != 0) wide *= 2;
    const int64_t P = wide / w;
    if (P > kStripMaxRow || N * (C / wide) > kStripMaxBlocks) return s;
    const int64_t np = ceil_div(L, kStripLanes / P);
    if (np > kStripMaxPieces) return s;
    if (P == 1 && N * L * C * (16 / w) > kStripNarrowBytes) return s;
    s.P = static_cast<int>(P);
    s.pow2 = P <= kStripMaxPow2Row && (P & (P - 1)) == 0;
    while (s.pow2 && (1 << s.shift) < s.P) ++s.shift;
    s.np = np <= 1 ? 1 : (np <= 2 ? 2 : 4);
    s.strips = static_cast<int>(C / wide);
    return s;
}

struct BackwardPlan {
    StripPlan strip;
    Tiles sums, input;
    int lanes;  // of pass 1's workgroups
    bool few;   // partials
    int tile_c, tiles, width;
    size_t part, total;  // floats
};
BackwardPlan backward_plan(int64_t N, int64_t L, int64_t C, int64_t G, int dtype, bool saved) {
    BackwardPlan p{};
    const int w = piece_width(C, dtype);
    p.strip = strip_plan(N, L, C, G, w);
    if (p.strip.np > 0) {
        p.total = N > 1 ? static_cast<size_t>(N) * 2 * C : 0;
        return p;
    }
    const bool small = N * L * C * elem_bytes(dtype) <= kSmallBytes;
    const bool one_batch = L * std::min<int64_t>(ceil_div(C, w), kMaxPieces) <= kLanes * kUnroll;
    p.lanes = small || one_batch ? kLanes : kSumLanes;
    p.sums = make_tiles(N, L, C, w, 1, kSumBlocks, kMaxRun, p.lanes);
    p.input = make_tiles(N, L, C, w, 1, kStreamBlocks, 0, kLanes,
                         saved ? kUnroll : kInputUnroll);
    const int64_t cg = C / G;
    p.few = p.sums.K <= kFinishBatch;
    p.width = p.few ? 6 : (cg <= 16 || cg > 64 ? 4 : (cg <= 32 ? 5 : 6));
    const int64_t wide = int64_t{1} << p.width;
    p.tile_c = static_cast<int>(cg <= 64 ? wide / cg * cg : wide);
    p.tiles = static_cast<int>(ceil_div(C, p.tile_c));
    p.part = static_cast<size_t>(N) * p.sums.K * 2 * C;
    p.total = p.part + static_cast<size_t>(N) * 2 * (C + G);
    return p;
}
bool backward_fits(int64_t N, const BackwardPlan &p) {
    if (p.strip.np > 0) return true;
    return grid_fits(N, p.sums, p.lanes) && grid_fits(N, p.input) && N * p.tiles < (int64_t{1} << 22) &&
           N * p.sums.C < (int64_t{1} << 40);
}

void launch_strip(const StripArgs &sa, unsigned grid, const StripPlan &p, bool silu, bool saved,
                  int dtype, hipStream_t st) {
    auto by_np = [&](auto d, auto siluc, auto savedc, auto pow2c) {
        using D = decltype(d);
        constexpr int W = static_cast<int>(16 / sizeof(typename D::storage));
        constexpr bool SILU = decltype(siluc)::value != 0, SAVED = decltype(savedc)::value != 0;
        constexpr bool POW2 = decltype(pow2c)::value != 0;
        if (p.np == 1)
            gn_grad_strip<D, W, SILU, SAVED, 1, POW2><<<grid, kStripLanes, 0, st>>>(sa);
        else if (p.np == 2)
            gn_grad_strip<D, W, SILU, SAVED, 2, POW2><<<grid, kStripLanes, 0, st>>>(sa);
        else
            gn_grad_strip<D, W, SILU, SAVED, 4, POW2><<<grid, kStripLanes, 0, st>>>(sa);
    };
    auto by_row = [&](auto d, auto siluc, auto savedc) {
        if (p.pow2)
            by_np(d, siluc, savedc, IC<1>{});
        else
            by_np(d, siluc, savedc, IC<0>{});
    };
    auto by_flags = [&](auto d) {
        if (silu)
            saved ? by_row(d, IC<1>{}, IC<1>{}) : by_row(d, IC<1>{}, IC<0>{});
        else
            saved ? by_row(d, IC<0>{}, IC<1>{}) : by_row(d, IC<0>{}, IC<0>{});
    };
    switch (x_dtype(dtype)) {
        case GN_DTYPE_F16: by_flags(Fp16{}); break;
        case GN_DTYPE_F32: by_flags(F32{}); break;
        default: by_flags(Bf16{}); break;
    }
}

// Row forms with a stride (the checkpoints).
gn_status check_saved_rows(int64_t M, int64_t C, int64_t stride, bool out, int dtype) {
    if (!valid_dtype(dtype)) return GN_INVALID_ARGUMENT;
    if (M < 0 || C <= 0 || stride < 0) return GN_INVALID_ARGUMENT;
    if (out && M > 1 && stride < C) return GN_INVALID_ARGUMENT;
    const int64_t step = std::max(stride, C);
    if (M > 0 && (step > INT64_MAX / 8 || M > (INT64_MAX / 4 - C) / step))
        return GN_INVALID_ARGUMENT;
    if (C > GN_LAYER_NORM_MAX_CHANNELS) return GN_UNSUPPORTED;
    return GN_OK;
}

}  // namespace
}  // namespace gnsilu

using namespace gnsilu;

extern "C" {

gn_status gn_checkpoint_rows(const void *x, int64_t x_stride, void *codes, void *scales, int64_t M,
                             int64_t C, int dtype, void *stream) {
    if (x == nullptr || codes == nullptr || scales == nullptr) return GN_INVALID_ARGUMENT;
    gn_status st = check_saved_rows(M, C, x_stride, false, dtype);
    if (st != GN_OK) return st;
    if (misaligned(x, elem_bytes(dtype))) return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    const int w = piece_width(C, dtype);
    RowArgs a{};
    a.tl = make_tiles(1, M, C, w, block_lanes(w), kStreamBlocks);
    if (!grid_fits(1, a.tl)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    a.x = x;
    a.codes_out = static_cast<int8_t *>(codes);
    a.scales_out = static_cast<uint8_t *>(scales);
    a.x_stride = x_stride;
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        gn_rows_save<decltype(d), decltype(wc)::value, decltype(tail)::value != 0, kSave>
            <<<grid_of(1, a.tl), kLanes, 0, c.stream>>>(a);
    });
    return finish_launch();
}

gn_status gn_restore_rows(const void *codes, const void *scales, void *x, int64_t x_stride,
                          int64_t M, int64_t C, int dtype, void *stream) {
    if (x == nullptr || codes == nullptr || scales == nullptr) return GN_INVALID_ARGUMENT;
    gn_status st = check_saved_rows(M, C, x_stride, true, dtype);
    if (st != GN_OK) return st;
    if (misaligned(x, elem_bytes(dtype))) return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    const int w = piece_width(C, dtype);
    RowArgs a{};
    a.tl = make_tiles(1, M, C, w, 1, kStreamBlocks);
    if (!grid_fits(1, a.tl)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.y = x;
    a.y_stride = x_stride;
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        gn_rows_restore<decltype(d), decltype(wc)::value, decltype(tail)::value != 0>
            <<<grid_of(1, a.tl), kLanes, 0, c.stream>>>(a);
    });
    return finish_launch();
}

gn_status gn_apply_rows_save(const void *x, const float *mean, const float *rstd,
                             const void *gamma, const void *beta, void *y, void *codes,
                             void *scales, int64_t N, int64_t L, int64_t C, int64_t G,
                             int apply_silu, int dtype, void *stream) {
    if (x == nullptr || y == nullptr || mean == nullptr || rstd == nullptr || codes == nullptr ||
        scales == nullptr)
        return GN_INVALID_ARGUMENT;
    gn_status st = check_group_rows(N, L, C, G, apply_silu, dtype);
    if (st == GN_OK) st = check_affine(gamma, beta, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(x, es) || misaligned(y, es) || misaligned(mean, 4) || misaligned(rstd, 4))
        return GN_UNSUPPORTED;
    if (N * L == 0) return GN_OK;
    const int w = piece_width(C, dtype);
    RowArgs a{};
    a.tl = make_tiles(N, L, C, w, block_lanes(w), kStreamBlocks);
    if (!grid_fits(N, a.tl)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {x, mean, rstd, gamma, beta, y, codes, scales}, &c);
    if (st != GN_OK) return st;
    a.x = x;
    a.y = y;
    a.codes_out = static_cast<int8_t *>(codes);
    a.scales_out = static_cast<uint8_t *>(scales);
    a.mean = mean;
    a.rstd = rstd;
    a.x_stride = a.y_stride = C;
    a.G = static_cast<int>(G);
    a.Cg = static_cast<int>(C / G);
    a.af = Affine{gamma, beta, affine_type(dtype)};
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        using D = decltype(d);
        constexpr int W = decltype(wc)::value;
        constexpr bool TAIL = decltype(tail)::value != 0;
        if (apply_silu)
            gn_rows_save<D, W, TAIL, kApplySilu>
                <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
        else
            gn_rows_save<D, W, TAIL, kApply>
                <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
    });
    return finish_launch();
}

gn_status gn_silu_rows_backward_workspace(int64_t N, int64_t L, int64_t C, int64_t G, int dtype,
                                          int64_t *bytes_out) {
    if (bytes_out == nullptr) return GN_INVALID_ARGUMENT;
    const gn_status st = check_group_rows(N, L, C, G, 0, dtype);
    if (st != GN_OK) return st;
    if (N * L == 0) {
        *bytes_out = 0;
        return GN_OK;
    }
    const BackwardPlan p = backward_plan(N, L, C, G, dtype, false);
    if (!backward_fits(N, p)) return GN_UNSUPPORTED;
    *bytes_out = static_cast<int64_t>(sizeof(float) * p.total);
    return GN_OK;
}

gn_status gn_silu_rows_backward(const void *dy, const void *x, const void *codes,
                                const void *scales, const float *mean, const float *rstd,
                                const void *gamma, const void *beta, void *dx, void *dgamma,
                                void *dbeta, int64_t N, int64_t L, int64_t C, int64_t G,
                                int apply_silu, int dtype, void *workspace,
                                int64_t workspace_bytes, void *stream) {
    if (dy == nullptr || dx == nullptr || mean == nullptr || rstd == nullptr)
        return GN_INVALID_ARGUMENT;
    // x, or its checkpoint, not both
    if ((codes == nullptr) != (scales == nullptr) || (x == nullptr) == (codes == nullptr))
        return GN_INVALID_ARGUMENT;
    gn_status st = check_group_rows(N, L, C, G, apply_silu, dtype);
    if (st == GN_OK) st = check_affine(gamma, beta, dtype);
    if (st == GN_OK) st = check_affine(dgamma, dbeta, dtype);
    if (st != GN_OK) return st;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(dy, es) || misaligned(x, es) || misaligned(dx, es) || misaligned(mean, 4) ||
        misaligned(rstd, 4) || misaligned(workspace, 4))
        return GN_UNSUPPORTED;
    const bool grads = dgamma != nullptr || dbeta != nullptr;
    const bool empty = N * L == 0;
    if (empty && !grads) return GN_OK;
    BackwardPlan p{};
    if (!empty) {
        p = backward_plan(N, L, C, G, dtype, codes != nullptr);
        if (!backward_fits(N, p)) return GN_UNSUPPORTED;
        if (p.total > 0 && workspace == nullptr) return GN_INVALID_ARGUMENT;
        if (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < sizeof(float) * p.total)
            return GN_SCRATCH_TOO_SMALL;
    }
    Call c;
    st = begin_call(stream,
                    {dy, x, codes, scales, mean, rstd, gamma, beta, dx, dgamma, dbeta,
                     p.total > 0 ? workspace : nullptr},
                    &c);
    if (st != GN_OK) return st;
    const unsigned sgrid = static_cast<unsigned>(ceil_div(C, kSampleLanes));
    const int atype = affine_type(dtype);
    if (empty) {
        gn_grad_samples<<<sgrid, kLanes, 0, c.stream>>>(nullptr, 0, static_cast<int>(C), dgamma,
                                                        dbeta, atype);
        return finish_launch();
    }
    float *ws = static_cast<float *>(workspace);
    RowArgs a{};
    a.dy = dy;
    a.x = x;
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.y = dx;
    a.mean = mean;
    a.rstd = rstd;
    a.part = ws;
    a.G = static_cast<int>(G);
    a.Cg = static_cast<int>(C / G);
    a.af = Affine{gamma, beta, atype};
    FinishArgs f{};
    f.part = ws;
    f.rstd = rstd;
    f.sums = ws + p.part;
    float *coef = f.sums + static_cast<size_t>(N) * 2 * C;
    f.dgamma = N == 1 ? dgamma : nullptr;
    f.dbeta = N == 1 ? dbeta : nullptr;
    f.K = p.sums.K;
    f.C = static_cast<int>(C);
    f.G = a.G;
    f.Cg = a.Cg;
    f.tile_c = p.tile_c;
    f.tiles = p.tiles;
    f.all_tiles = N * p.tiles;
    f.width = p.width;
    f.inv_m = 1.0 / (static_cast<double>(L) * static_cast<double>(a.Cg));
    f.af = a.af;
    f.coef = a.Cg <= 64 ? coef : nullptr;
    a.coef = coef;
    a.N = N;
    a.sums = f.sums;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    if (p.strip.np > 0) {
        a.tl.L = L;
        a.tl.C = f.C;
        StripArgs sa{};
        sa.r = a;
        sa.sums = grads && N > 1 ? ws : nullptr;
        sa.P = p.strip.P;
        sa.shift = p.strip.shift;
        sa.strips = p.strip.strips;
        sa.xcd = N * p.strip.strips % 8 == 0;
        sa.inv_m = f.inv_m;
        launch_strip(sa, static_cast<unsigned>(N * p.strip.strips), p.strip, apply_silu != 0,
                     codes != nullptr, dtype, c.stream);
        if (sa.sums != nullptr)
            gn_grad_samples<<<sgrid, kLanes, 0, c.stream>>>(ws, N, f.C, dgamma, dbeta, atype);
        return finish_launch();
    }
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        using D = decltype(d);
        constexpr int W = decltype(wc)::value;
        constexpr bool TAIL = decltype(tail)::value != 0;
        auto passes = [&](auto silu, auto saved) {
            constexpr bool SILU = decltype(silu)::value != 0;
            constexpr bool SAVED = decltype(saved)::value != 0;
            a.tl = p.sums;
            if (p.lanes == kLanes)
                gn_grad_sums<D, W, TAIL, SILU, SAVED, kLanes>
                    <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
            else
                gn_grad_sums<D, W, TAIL, SILU, SAVED, kSumLanes>
                    <<<grid_of(N, a.tl), kSumLanes, 0, c.stream>>>(a);
            const int64_t per = p.few ? kFewThreads / 64 : 1;
            const unsigned tiles = static_cast<unsigned>(ceil_div(f.all_tiles, per));
            if (p.few)
                gn_grad_finish<true><<<tiles, kFewThreads, 0, c.stream>>>(f);
            else
                gn_grad_finish<false><<<tiles, kFinishThreads, 0, c.stream>>>(f);
            if (f.coef == nullptr) {
                FinishArgs g = f;
                g.coef = coef;
                gn_grad_groups<<<dim3(static_cast<unsigned>(N * G)), kLanes, 0, c.stream>>>(g);
            }
            a.tl = p.input;
            dim3 grid = grid_of(N, a.tl);
            a.sample_blocks = grads && N > 1 ? sgrid : 0;
            grid.x += a.sample_blocks;
            gn_grad_input<D, W, TAIL, SILU, SAVED><<<grid, kLanes, 0, c.stream>>>(a);
        };
        auto by_saved = [&](auto silu) {
            if (codes != nullptr)
                passes(silu, IC<1>{});
            else
                passes(silu, IC<0>{});
        };
        if (apply_silu)
            by_saved(IC<1>{});
        else
            by_saved(IC<0>{});
    });
    return finish_launch();
}

}  // extern "C"
