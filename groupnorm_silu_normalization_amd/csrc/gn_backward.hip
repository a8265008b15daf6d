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
// (about twenty instruction slots per element, SiLU's exponential and
// reciprocal counting four each), so t is one fma, its exponential and
// reciprocal the hardware's, and dx two fmas on dt and x-mean.
//
// A lane keeps one piece of W consecutive channels for all its rows: a tile is
// R rows of Pc pieces over the 256 lanes, and a row of more than 256 pieces is
// cut into column blocks.  Channel parameters and sums stay in registers.
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

struct Tiles {
    int64_t L;    // rows per sample
    int64_t K;    // chunks per sample
    int64_t rpc;  // rows per chunk (the last one may be shorter)
    int C, P;     // channels and pieces of a row
    int ncb, Pc;  // column blocks of a row and their pieces
    int R;        // rows per tile
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
};

// The calling lane's rows and piece.
template <int W, bool TAIL> struct Place {
    int64_t n, k, l, l1;  // sample, chunk, first row, end of the chunk's rows
    int r, c, lo;
    bool active;
    __device__ __forceinline__ explicit Place(const Tiles &t) {
        const int64_t b = blockIdx.x;
        const int cb = static_cast<int>(b % t.ncb);
        const int64_t nk = b / t.ncb;
        k = nk % t.K;
        n = nk / t.K;
        r = static_cast<int>(threadIdx.x) / t.Pc;
        const int pc = static_cast<int>(threadIdx.x) % t.Pc;
        const int p = cb * t.Pc + pc;
        active = r < t.R && p < t.P;
        c = active ? p * W : 0;
        lo = 0;
        if (TAIL && c + W > t.C) {
            lo = c + W - t.C;
            c = t.C - W;
        }
        l = k * t.rpc;
        l1 = l + t.rpc < t.L ? l + t.rpc : t.L;
        l += r;
    }
};

// scale = gamma*rstd and shift = beta - mean*scale as the apply step folds
// them, and the statistics, for a lane's W channels of sample n.
template <int W> struct Channels {
    float mu[W], rs[W], sc[W], sh[W];
    __device__ __forceinline__ void load(const RowArgs &a, int64_t n, int c) {
        float be[W];
        load_affine<W>(a.af.gamma, a.af.type, c, 1.0f, sc);
        load_affine<W>(a.af.beta, a.af.type, c, 0.0f, be);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t g = n * a.G + (c + i) / a.Cg;
            mu[i] = a.mean[g];
            rs[i] = a.rstd[g];
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            sc[i] *= rs[i];
            sh[i] = fmaf(-mu[i], sc[i], be[i]);
        }
    }
};

// dt = dy * d/dt(t*sigmoid(t)); with u = t*s the derivative is s + u*(1-s).
__device__ __forceinline__ float silu_grad(float t, float dy) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.4426950408889634f));
    return dy * fmaf(t * s, 1.0f - s, s);
}

// One row's piece of x (or its saved codes) and dy.
template <class D, int W, bool TAIL, bool SAVED> struct Pair {
    using T = typename D::storage;
    Piece<D, W> vx, vy;
    Piece8<W, TAIL> v8;
    __device__ __forceinline__ void load(const RowArgs &a, int64_t row, int64_t nsb, int c) {
        if constexpr (SAVED)
            v8.load(a.codes, a.scales, row * a.tl.C, row * nsb, c);
        else
            vx.template load<false>(static_cast<const T *>(a.x) + row * a.tl.C + c);
        vy.template load<false>(static_cast<const T *>(a.dy) + row * a.tl.C + c);
    }
    __device__ __forceinline__ void x(int c, float (&o)[W]) const {
        if constexpr (SAVED) {
            v8.widen(c, o);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = vx.get(i);
        }
    }
};

// Pass 1.  U rows of a lane in flight.
template <class D, int W, bool TAIL, bool SILU, bool SAVED, int U>
__global__ __launch_bounds__(kLanes) void gn_grad_sums(RowArgs a) {
    __shared__ float red[2 * W][kLanes];
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    Channels<W> ch;
    ch.load(a, at.n, at.c);
    float s1[W], s2[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s1[i] = s2[i] = 0.0f;
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L;
    using V = Pair<D, W, TAIL, SAVED>;
    auto add = [&](const V &v) {
        float x[W];
        v.x(at.c, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float d = v.vy.get(i);
            if constexpr (SILU) d = silu_grad(fmaf(x[i], ch.sc[i], ch.sh[i]), d);
            s1[i] += d;
            s2[i] = fmaf(d, x[i] - ch.mu[i], s2[i]);
        }
    };
    if (at.active) {
        int64_t l = at.l;
        for (; l + (U - 1) * int64_t{tl.R} < at.l1; l += U * int64_t{tl.R}) {
            V v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(a, row0 + l + u * int64_t{tl.R}, nsb, at.c);
#pragma unroll
            for (int u = 0; u < U; ++u) add(v[u]);
        }
        for (; l < at.l1; l += tl.R) {
            V v;
            v.load(a, row0 + l, nsb, at.c);
            add(v);
        }
    }
    // the R row slots, by a fixed tree
    int p2 = 1;
    while (p2 < tl.R) p2 <<= 1;
    if (tl.R > 1) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            red[i][threadIdx.x] = s1[i];
            red[W + i][threadIdx.x] = s2[i];
        }
        __syncthreads();
        for (int h = p2 >> 1; h > 0; h >>= 1) {
            if (at.r < h && at.r + h < tl.R) {
                const int o = static_cast<int>(threadIdx.x) + h * tl.Pc;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    red[i][threadIdx.x] = s1[i] += red[i][o];
                    red[W + i][threadIdx.x] = s2[i] += red[W + i][o];
                }
            }
            __syncthreads();
        }
    }
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

// Finishes pass 1: channel sums over the K chunks (16 parts of chunks per
// workgroup, each in order, then the parts in order, in fp64), tile_c channels
// of one sample per workgroup.  sums[N][2][C] receives sum dt and sum dt*h.
// A tile of whole groups (Cg <= 64) also gives their a and b; one sample alone
// its dgamma and dbeta.
constexpr int kParts = 16;
struct FinishArgs {
    const float *part;
    const float *rstd;
    float *sums, *coef;
    void *dgamma, *dbeta;  // null unless N = 1 and wanted
    int64_t K;
    int C, G, Cg, tile_c, tiles;
    double inv_m;
    Affine af;
};
__global__ __launch_bounds__(64 * kParts) void gn_grad_finish(FinishArgs a) {
    __shared__ double red[2][kParts][64];
    const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
    const int64_t n = blockIdx.x / a.tiles;
    const int c = static_cast<int>(blockIdx.x % a.tiles) * a.tile_c + lane;
    const bool live = lane < a.tile_c && c < a.C;
    double s1 = 0.0, s2 = 0.0;
    if (live) {
        const float *p = a.part + n * a.K * 2 * a.C + c;
#pragma unroll 4
        for (int64_t k = r; k < a.K; k += kParts) {
            s1 += static_cast<double>(p[k * 2 * a.C]);
            s2 += static_cast<double>(p[k * 2 * a.C + a.C]);
        }
    }
    red[0][r][lane] = s1;
    red[1][r][lane] = s2;
    __syncthreads();
    if (r != 0) return;
#pragma unroll
    for (int i = 1; i < kParts; ++i) {
        s1 += red[0][i][lane];
        s2 += red[1][i][lane];
    }
    float ga[1] = {0.0f};
    if (live) {
        s2 *= static_cast<double>(a.rstd[n * a.G + c / a.Cg]);
        a.sums[n * 2 * a.C + c] = static_cast<float>(s1);
        a.sums[n * 2 * a.C + a.C + c] = static_cast<float>(s2);
        if (a.dbeta != nullptr) store_affine(a.dbeta, a.af.type, c, static_cast<float>(s1));
        if (a.dgamma != nullptr) store_affine(a.dgamma, a.af.type, c, static_cast<float>(s2));
        load_affine<1>(a.af.gamma, a.af.type, c, 1.0f, ga);
    }
    if (a.coef == nullptr) return;
    // one wave is left: its LDS accesses are in order
    red[0][0][lane] = s1 * static_cast<double>(ga[0]);
    red[1][0][lane] = s2 * static_cast<double>(ga[0]);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    if (live && lane % a.Cg == 0) {
        double ta = 0.0, tb = 0.0;
        for (int i = 0; i < a.Cg; ++i) {
            ta += red[0][0][lane + i];
            tb += red[1][0][lane + i];
        }
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

// dgamma and dbeta of N samples (zeros for none).
__global__ __launch_bounds__(kLanes) void gn_grad_samples(const float *sums, int64_t N, int C,
                                                          void *dgamma, void *dbeta, int type) {
    const int c = static_cast<int>(blockIdx.x) * kLanes + static_cast<int>(threadIdx.x);
    if (c >= C) return;
    double s1 = 0.0, s2 = 0.0;
    for (int64_t n = 0; n < N; ++n) {
        s1 += static_cast<double>(sums[n * 2 * C + c]);
        s2 += static_cast<double>(sums[n * 2 * C + C + c]);
    }
    if (dbeta != nullptr) store_affine(dbeta, type, c, static_cast<float>(s1));
    if (dgamma != nullptr) store_affine(dgamma, type, c, static_cast<float>(s2));
}

// Pass 2: dx = dt*scale - (x-mean)*rstd^2*b - rstd*a.
template <class D, int W, bool TAIL, bool SILU, bool SAVED, int U>
__global__ __launch_bounds__(kLanes) void gn_grad_input(RowArgs a) {
    using T = typename D::storage;
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    if (!at.active) return;
    Channels<W> ch;
    ch.load(a, at.n, at.c);
    float k0[W], k1[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float *co = a.coef + 2 * (at.n * a.G + (at.c + i) / a.Cg);
        k0[i] = -ch.rs[i] * co[0];
        k1[i] = -ch.rs[i] * ch.rs[i] * co[1];
    }
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L;
    using V = Pair<D, W, TAIL, SAVED>;
    auto finish = [&](const V &v, int64_t row) {
        float x[W], o[W];
        v.x(at.c, x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float d = v.vy.get(i);
            if constexpr (SILU) d = silu_grad(fmaf(x[i], ch.sc[i], ch.sh[i]), d);
            o[i] = fmaf(d, ch.sc[i], fmaf(x[i] - ch.mu[i], k1[i], k0[i]));
        }
        T *p = static_cast<T *>(a.y) + row * tl.C + at.c;
        // dx may be dy or x: a lane writes only channels that no other reads
        if (!TAIL || at.lo == 0)
            Piece<D, W>::template store<false>(p, o);
        else
            store_from<D, W>(p, o, at.lo);
    };
    int64_t l = at.l;
    for (; l + (U - 1) * int64_t{tl.R} < at.l1; l += U * int64_t{tl.R}) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].load(a, row0 + l + u * int64_t{tl.R}, nsb, at.c);
#pragma unroll
        for (int u = 0; u < U; ++u) finish(v[u], row0 + l + u * int64_t{tl.R});
    }
    for (; l < at.l1; l += tl.R) {
        V v;
        v.load(a, row0 + l, nsb, at.c);
        finish(v, row0 + l);
    }
}

// The apply step that also saves x (kApply, kApplySilu), or x saved alone
// (kSave).  A block of the format lies in consecutive lanes of one row: the
// plan makes Pc a multiple of the lanes that hold a block.
enum { kApply = 0, kApplySilu = 1, kSave = 2 };
template <class D, int W, bool TAIL, int MODE, int U>
__global__ __launch_bounds__(kLanes) void gn_rows_save(RowArgs a) {
    using T = typename D::storage;
    constexpr int kGroup = W == 1 ? 8 : kBlock8 / W;
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    Channels<W> ch;
    if constexpr (MODE != kSave) ch.load(a, at.n, at.c);
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L;
    const int lo = at.active ? at.lo : W;
    // every lane of the workgroup takes part in the blocks' maxima
    for (int64_t l = at.l - at.r; l < at.l1; l += U * int64_t{tl.R}) {
        Piece<D, W> v[U];
        int64_t row[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t lu = l + at.r + u * int64_t{tl.R};
            live[u] = at.active && lu < at.l1;
            row[u] = row0 + (live[u] ? lu : at.l1 - 1);
            v[u].template load<false>(static_cast<const T *>(a.x) + row[u] * a.x_stride + at.c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[W];
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = v[u].get(i);
            if constexpr (MODE != kSave) {
                float o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float t = fmaf(x[i], ch.sc[i], ch.sh[i]);
                    o[i] = MODE == kApplySilu ? silu_f32(t) : t;
                }
                T *p = static_cast<T *>(a.y) + row[u] * a.y_stride + at.c;
                if (live[u]) {  // y may be x: only the lane's own channels
                    if (!TAIL || at.lo == 0)
                        Piece<D, W>::template store<false>(p, o);
                    else
                        store_from<D, W>(p, o, at.lo);
                }
            }
            const uint32_t E = block8_exponent<W, kGroup>(x, lo);
            const Codes<W> q = block8_encode<W>(x, E);
            if (live[u])
                store_block8<W, TAIL>(q, E, a.codes_out, a.scales_out, row[u] * tl.C,
                                      row[u] * nsb, at.c, at.lo);
        }
    }
}

// Saved rows widened again.
template <class D, int W, bool TAIL, int U>
__global__ __launch_bounds__(kLanes) void gn_rows_restore(RowArgs a) {
    using T = typename D::storage;
    const Tiles &tl = a.tl;
    const Place<W, TAIL> at(tl);
    if (!at.active) return;
    const int64_t nsb = (tl.C + kBlock8 - 1) / kBlock8;
    const int64_t row0 = at.n * tl.L;
    auto put = [&](const Piece8<W, TAIL> &v, int64_t row) {
        float o[W];
        v.widen(at.c, o);
        Piece<D, W>::template store<false>(static_cast<T *>(a.y) + row * a.y_stride + at.c, o);
    };
    int64_t l = at.l;
    for (; l + (U - 1) * int64_t{tl.R} < at.l1; l += U * int64_t{tl.R}) {
        Piece8<W, TAIL> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + l + u * int64_t{tl.R};
            v[u].load(a.codes, a.scales, row * tl.C, row * nsb, at.c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) put(v[u], row0 + l + u * int64_t{tl.R});
    }
    for (; l < at.l1; l += tl.R) {
        Piece8<W, TAIL> v;
        const int64_t row = row0 + l;
        v.load(a.codes, a.scales, row * tl.C, row * nsb, at.c);
        put(v, row);
    }
}

// ---- host -----------------------------------------------------------------------
constexpr int kUnroll = 4;                  // rows of a lane in flight
constexpr int64_t kSumBlocks = 512;         // pass 1: workgroups, 2 per CU
constexpr int64_t kStreamBlocks = 2048;     // the other passes
constexpr int64_t kMaxRun = 1024;           // rows a lane adds up in fp32

// whole: lanes that must stay in one row together (a block of the format when
// saving, else 1).
Tiles make_tiles(int64_t N, int64_t L, int64_t C, int w, int whole, int64_t blocks,
                 int64_t max_run) {
    Tiles t{};
    t.L = L;
    t.C = static_cast<int>(C);
    t.P = static_cast<int>(ceil_div(C, w));
    t.ncb = static_cast<int>(ceil_div(t.P, kLanes));
    t.Pc = static_cast<int>(ceil_div(ceil_div(t.P, t.ncb), whole)) * whole;
    t.R = kLanes / t.Pc;
    const int64_t tiles = std::max<int64_t>(1, ceil_div(L, t.R));
    int64_t k = std::max<int64_t>(1, blocks / std::max<int64_t>(1, N * t.ncb));
    k = std::min(k, ceil_div(tiles, kUnroll));
    if (max_run > 0) k = std::max(k, ceil_div(tiles, max_run));
    t.rpc = ceil_div(tiles, k) * t.R;
    t.K = std::max<int64_t>(1, ceil_div(L, t.rpc));
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
bool grid_fits(int64_t N, const Tiles &t) {
    return N < (int64_t{1} << 24) && t.K < (int64_t{1} << 24) &&
           N * t.K < (int64_t{1} << 24) && N * t.K * t.ncb < (int64_t{1} << 24);
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

struct BackwardPlan {
    Tiles sums, input;
    int tile_c, tiles;
    size_t part, total;  // floats
};
BackwardPlan backward_plan(int64_t N, int64_t L, int64_t C, int64_t G, int dtype) {
    BackwardPlan p;
    const int w = piece_width(C, dtype);
    p.sums = make_tiles(N, L, C, w, 1, kSumBlocks, kMaxRun);
    p.input = make_tiles(N, L, C, w, 1, kStreamBlocks, 0);
    const int64_t cg = C / G;
    p.tile_c = static_cast<int>(cg <= 64 ? 64 / cg * cg : 64);
    p.tiles = static_cast<int>(ceil_div(C, p.tile_c));
    p.part = static_cast<size_t>(N) * p.sums.K * 2 * C;
    p.total = p.part + static_cast<size_t>(N) * 2 * (C + G);
    return p;
}
bool backward_fits(int64_t N, const BackwardPlan &p) {
    return grid_fits(N, p.sums) && grid_fits(N, p.input) && N * p.tiles < (int64_t{1} << 22) &&
           N * p.sums.C < (int64_t{1} << 40);
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
    a.tl = make_tiles(1, M, C, w, block_lanes(w), kStreamBlocks, 0);
    if (!grid_fits(1, a.tl)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    a.x = x;
    a.codes_out = static_cast<int8_t *>(codes);
    a.scales_out = static_cast<uint8_t *>(scales);
    a.x_stride = x_stride;
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        gn_rows_save<decltype(d), decltype(wc)::value, decltype(tail)::value != 0, kSave, kUnroll>
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
    a.tl = make_tiles(1, M, C, w, 1, kStreamBlocks, 0);
    if (!grid_fits(1, a.tl)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.y = x;
    a.y_stride = x_stride;
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        gn_rows_restore<decltype(d), decltype(wc)::value, decltype(tail)::value != 0, kUnroll>
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
    a.tl = make_tiles(N, L, C, w, block_lanes(w), kStreamBlocks, 0);
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
            gn_rows_save<D, W, TAIL, kApplySilu, kUnroll>
                <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
        else
            gn_rows_save<D, W, TAIL, kApply, kUnroll>
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
    const BackwardPlan p = backward_plan(N, L, C, G, dtype);
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
        p = backward_plan(N, L, C, G, dtype);
        if (!backward_fits(N, p)) return GN_UNSUPPORTED;
        if (workspace == nullptr) return GN_INVALID_ARGUMENT;
        if (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < sizeof(float) * p.total)
            return GN_SCRATCH_TOO_SMALL;
    }
    Call c;
    st = begin_call(stream,
                    {dy, x, codes, scales, mean, rstd, gamma, beta, dx, dgamma, dbeta,
                     empty ? nullptr : workspace},
                    &c);
    if (st != GN_OK) return st;
    const dim3 sgrid(static_cast<unsigned>(ceil_div(C, kLanes)));
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
    f.inv_m = 1.0 / (static_cast<double>(L) * static_cast<double>(a.Cg));
    f.af = a.af;
    f.coef = a.Cg <= 64 ? coef : nullptr;
    a.coef = coef;
    with_pieces(C, dtype, [&](auto d, auto wc, auto tail) {
        using D = decltype(d);
        constexpr int W = decltype(wc)::value;
        constexpr bool TAIL = decltype(tail)::value != 0;
        auto passes = [&](auto silu, auto saved) {
            constexpr bool SILU = decltype(silu)::value != 0;
            constexpr bool SAVED = decltype(saved)::value != 0;
            a.tl = p.sums;
            gn_grad_sums<D, W, TAIL, SILU, SAVED, kUnroll>
                <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
            gn_grad_finish<<<dim3(static_cast<unsigned>(N * p.tiles)), 64 * kParts, 0, c.stream>>>(
                f);
            if (f.coef == nullptr) {
                FinishArgs g = f;
                g.coef = coef;
                gn_grad_groups<<<dim3(static_cast<unsigned>(N * G)), kLanes, 0, c.stream>>>(g);
            }
            a.tl = p.input;
            gn_grad_input<D, W, TAIL, SILU, SAVED, kUnroll>
                <<<grid_of(N, a.tl), kLanes, 0, c.stream>>>(a);
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
    if (grads && N > 1)
        gn_grad_samples<<<sgrid, kLanes, 0, c.stream>>>(f.sums, N, f.C, dgamma, dbeta, atype);
    return finish_launch();
}

}  // extern "C"
