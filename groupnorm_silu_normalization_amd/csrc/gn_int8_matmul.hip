// gn_int8_matmul.hip -- products of rows in 8 bits with weights in 8 bits, a scale
// for each row (token) and for each output channel, for MI355X (gfx950).
//
//   z[m][n] = (sum_k a[m][k]*b[n][k]) * sa[m] * sb[n] + bias[n] + res[m][n]
//
// The sums are int32 on the matrix cores (v_mfma_i32_*_i8), exact up to
// GN_INT8_MAX_K, so any split of K gives the same bits; the scales, the bias and
// the residual are applied to them in fp32 and z is rounded once.
//
// Weights are packed once: per 16 output channels and 64 input channels the
// 1024 bytes that one product instruction takes, lane by lane (lane l: channel
// l % 16, inputs 16*(l/16) to +15), zero beyond N and K.  A wave's load of a
// fragment is then 1024 contiguous bytes, and whatever the rows hold behind K
// is multiplied by zero.  Rows are read as they lie and turned in LDS.  The weights
// are the first operand, so that a lane's four results are neighbours in a row of z.
//
// Measured on MI355X, bf16, us and TOP/s (a library product without scales in
// brackets): (16384,4096,4096) 253, 2170 (244), (4096,4096,4096) 67 (66),
// (1024,4096,4096) 24 (25), (256,4096,4096) 9.8 (10.8), (1001,1537,2003) 10.2,
// (48,10240,2560) 6.4 to 7 (8.1), (1,4096,4096) 4.0, all with weights in the caches;
// from HBM, a new copy of 640 MiB of them each time, the last two take 10.1 and 6.4.
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

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct MatmulArgs {
    const int8_t *a;      // [M][K], rows a_stride apart, any alignment
    const float *sa;      // [M]
    const int8_t *b;      // packed weights
    const float *sb;      // [N]
    const void *bias;     // [N] or null
    const void *res;      // or null
    void *z;
    int64_t M, a_stride, res_stride, z_stride;
    int N, K;
    int kb;               // blocks of 64 input channels, even
    int nb;               // blocks of 16 output channels
    int bias_type;
    int mt, nt;           // tiles of rows and of channels
};

constexpr int kKBlock = 64, kNBlock = 16, kFragment = 1024;

// ---- packing ---------------------------------------------------------------------
// A lane makes 16 bytes of a fragment at a time; the grid goes through all of them
// (up to 2^32, more than a dispatch holds lanes).  Its 16 loads of a byte bound it:
// (4096,4096) takes 31 us, five times a copy, once for a weight's life.
constexpr int64_t kPackBlocks = 1 << 16;
__global__ __launch_bounds__(256) void gn_int8_pack(const int8_t *w, int64_t stride, int8_t *packed,
                                                    int N, int K, int kb, int64_t pieces) {
    for (int64_t i = int64_t{blockIdx.x} * 256 + threadIdx.x; i < pieces;
         i += int64_t{gridDim.x} * 256) {
        const int lane = static_cast<int>(i & 63);
        const int64_t f = i >> 6;
        const int64_t n = f / kb * kNBlock + (lane & 15);
        const int64_t k = f % kb * kKBlock + (lane >> 4) * 16;
        uint32_t v[4] = {0, 0, 0, 0};
        if (n < N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k + j < K)
                    v[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(w[n * stride + k + j]))
                                 << (8 * (j & 3));
        }
        u32x4 o = {v[0], v[1], v[2], v[3]};
        reinterpret_cast<u32x4 *>(packed)[i] = o;
    }
}

// ---- the end of a product ----------------------------------------------------------
template <class D> __device__ __forceinline__ void store4(typename D::storage *p, const float (&o)[4]) {
    if constexpr (sizeof(typename D::storage) == 4) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(o[j]);
        *reinterpret_cast<u32x4_a4 *>(p) = v;
    } else {
        u32x2 v = {D::pack2(o[0], o[1]), D::pack2(o[2], o[3])};
        *reinterpret_cast<u32x2_a2 *>(p) = v;
    }
}
template <class D> __device__ __forceinline__ void load4(const typename D::storage *p, float (&o)[4]) {
    if constexpr (sizeof(typename D::storage) == 4) {
        const u32x4 v = *reinterpret_cast<const u32x4_a4 *>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __uint_as_float(v[j]);
    } else {
        const u32x2 v = *reinterpret_cast<const u32x2_a2 *>(p);
        o[0] = D::lo(v[0]), o[1] = D::hi(v[0]), o[2] = D::lo(v[1]), o[3] = D::hi(v[1]);
    }
}

// W sums times their scales, plus b.  A sum is at most 2^30, so that times a row's
// scale below 2^97 it is in fp32's range; with a larger one, which the channel's
// scale may bring back, all is taken 2^-32-fold until the end (in fp64 instead, the
// widest tiles spilt 60 registers).
template <int W, class Sums>
__device__ __forceinline__ void scaled(const Sums &acc, float sa, const float (&sb)[W],
                                       const float (&b)[W], float (&o)[W]) {
    if (fabsf(sa) >= 0x1p97f) {
        sa *= 0x1p-32f;
#pragma unroll
        for (int j = 0; j < W; ++j)
            o[j] = fmaf(static_cast<float>(acc(j)) * sa, sb[j], b[j] * 0x1p-32f) * 0x1p32f;
        return;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) o[j] = fmaf(static_cast<float>(acc(j)) * sa, sb[j], b[j]);
}

// Four neighbouring sums of row m from channel n on, scaled and stored.
template <class D>
__device__ __forceinline__ void finish4(const MatmulArgs &a, int64_t m, int n, const i32x4 &acc) {
    using T = typename D::storage;
    if (m >= a.M || n >= a.N) return;
    const float sa = a.sa[m];
    T *z = static_cast<T *>(a.z) + m * a.z_stride + n;
    const T *res = static_cast<const T *>(a.res) + m * a.res_stride + n;
    if (n + 4 <= a.N) {
        float sb[4], b[4], r[4] = {0.0f, 0.0f, 0.0f, 0.0f}, o[4];
        load4<F32>(a.sb + n, sb);
        load_affine<4>(a.bias, a.bias_type, n, 0.0f, b);
        if (a.res != nullptr) load4<D>(res, r);
        scaled<4>([&](int j) { return acc[j]; }, sa, sb, b, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += r[j];
        store4<D>(z, o);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= a.N) break;
        float b[1], o[1];
        const float sb[1] = {a.sb[n + j]};
        load_affine<1>(a.bias, a.bias_type, n + j, 0.0f, b);
        scaled<1>([&](int) { return acc[j]; }, sa, sb, b, o);
        if (a.res != nullptr) o[0] += D::to_f32(res[j]);
        z[j] = D::from_f32(o[0]);
    }
}

// Between one wave's accesses to LDS that its other lanes made or will make: LDS
// works in order, the compiler is told to.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The tile of a workgroup: consecutive workgroups go to the eight XCDs in turn,
// each of which takes a run of tiles, in strips of kStrip rows of tiles, so
// that the tiles it works on at one time share rows and weights in its L2 (strips
// of 8 or 16 take the same time within 2%: the products' power bounds large ones).
constexpr int kStrip = 4;
__device__ __forceinline__ void tile_of(int b, int tiles, int mt, int nt, int *tm, int *tn) {
    const int xcd = b & 7, per = tiles >> 3, rest = tiles & 7;
    const int t = xcd * per + (xcd < rest ? xcd : rest) + (b >> 3);
    const int strip = t / (kStrip * nt);
    const int rows = mt - strip * kStrip < kStrip ? mt - strip * kStrip : kStrip;
    const int in = t - strip * kStrip * nt;
    *tm = strip * kStrip + in % rows;
    *tn = in / rows;
}

// 16 bytes of a row from k on.  What lies behind K is multiplied by packed zeros:
// any bytes will do that may be read, the next row's or, from `end` on (behind
// the last row), none.  last: the block may reach behind K.
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
__device__ __forceinline__ i32x4 load16(const int8_t *row, int k, int K, const int8_t *end, bool last) {
    const int8_t *p = row + k;
    if (!last || (k < K && end - p >= 16))
        return __builtin_bit_cast(i32x4, *reinterpret_cast<const u32x4_a1 *>(p));
    uint64_t w[2] = {0, 0};
#pragma unroll 1
    for (int j = 0; k + j < K && j < 16; ++j) {
        const uint64_t v = static_cast<uint64_t>(static_cast<uint8_t>(p[j])) << (8 * (j & 7));
        if (j < 8)
            w[0] |= v;
        else
            w[1] |= v;
    }
    return i32x4{static_cast<int>(w[0]), static_cast<int>(w[0] >> 32), static_cast<int>(w[1]),
                 static_cast<int>(w[1] >> 32)};
}

// ---- few rows ------------------------------------------------------------------------
// A workgroup takes 16*MT rows and 16*NT channels; its waves take the steps of
// 128 input channels in turn and join their sums through LDS at the end, so that
// nothing waits for another wave before.  A wave loads eight rows' 128 bytes an
// instruction (16 rows' 64 bytes, as products want them, come at a third of the
// rate) and turns them in a corner of LDS of its own; weights come as products
// want them.  The next step's loads are on their way while one is multiplied.
template <class D, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gn_int8_rows(MatmulArgs a) {
    constexpr int kTiles = MT * NT, kOwn = 64 * (kTiles > 2 * MT ? kTiles : 2 * MT);
    __shared__ i32x4 lds[WAVES][kOwn];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    i32x4 *own = lds[wave];
    int tm, tn;
    tile_of(blockIdx.x, a.mt * a.nt, a.mt, a.nt, &tm, &tn);
    const int64_t m0 = int64_t{tm} * (16 * MT);
    const int nb0 = tn * NT;
    const int8_t *end = a.a + (a.M - 1) * a.a_stride + a.K;
    const int8_t *ap[2 * MT], *bp[NT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int64_t m = m0 + i * 8 + (lane >> 3);
        ap[i] = a.a + (m < a.M ? m : a.M - 1) * a.a_stride;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int nb = nb0 + j < a.nb ? nb0 + j : a.nb - 1;
        bp[j] = a.b + int64_t{nb} * a.kb * kFragment + lane * 16;
    }
    // piece p of row r lies at place p ^ (r / 2 % 8): a lane's row is i*8 + lane/8
    const int piece[2] = {(lane & 7) ^ (lane >> 4), (lane & 7) ^ (lane >> 4) ^ 4};
    const int steps = a.kb / 2;
    i32x4 sa[2 * MT], fb[2][NT];
    auto load_rows = [&](int it) {
        const bool last = (it + 1) * 2 * kKBlock > a.K;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            sa[i] = load16(ap[i], it * 128 + piece[i & 1] * 16, a.K, end, last);
    };
    auto load_weights = [&](int it, int u) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
            fb[u][j] = *reinterpret_cast<const i32x4 *>(bp[j] + int64_t{it * 2 + u} * kFragment);
    };
    i32x4 acc[MT][NT] = {};
    int it = wave;
    if (it < steps) {
        load_rows(it);
        load_weights(it, 0);
        load_weights(it, 1);
    }
    for (; it < steps; it += WAVES) {
        const bool more = it + WAVES < steps;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) own[i * 64 + lane] = sa[i];
        wave_sync();
        if (more) load_rows(it + WAVES);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            i32x4 fa[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = i * 16 + (lane & 15);
                fa[i] = own[r * 8 + ((u * 4 + (lane >> 4)) ^ (r >> 1 & 7))];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][j], fa[i], acc[i][j], 0,
                                                                       0, 0);
            if (more) load_weights(it + WAVES, u);
            __builtin_amdgcn_sched_barrier(0);
        }
        wave_sync();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) own[(i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int tile = wave; tile < kTiles; tile += WAVES) {
        i32x4 s = lds[0][tile * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += lds[w][tile * 64 + lane];
        finish4<D>(a, m0 + tile / NT * 16 + (lane & 15),
                   (nb0 + tile % NT) * kNBlock + (lane >> 4) * 4, s);
    }
}

// ---- tiles -----------------------------------------------------------------------
// The end of a wave's TM x TN products of 32 x 32.  Each leaves four neighbouring
// channels of 32 rows in an instruction's lanes, 8 bytes of z: turned in the wave's
// own part of LDS, 32 rows at a time, lanes next to each other hold a row's
// neighbouring 16 bytes of z instead, so that residual and z move in runs of 64 to
// 256 bytes.  All of the residual is on its way before the first row is turned.
template <class D, int TM, int TN, class Acc>
__device__ __forceinline__ void finish_tile(const MatmulArgs &a, int64_t m0, int n0, const Acc &acc,
                                            i32x4 *own, int lane) {
    using T = typename D::storage;
    constexpr int W = 16 / sizeof(T), kLanes = 32 * TN / W;  // lanes of a row
    constexpr int kRows = 64 / kLanes, kTimes = 32 / kRows;  // rows at a time, times for 32
    constexpr int kPitch = 8 * TN + 1;                       // pieces of 4 sums from row to row
    const int n = n0 + lane % kLanes * W, r0 = lane / kLanes;
    const bool whole = n + W <= a.N;
    T *z = static_cast<T *>(a.z) + n;
    const T *res = static_cast<const T *>(a.res) + n;
    // (half of it for fp32, for the registers)
    constexpr int kAhead = sizeof(T) == 2 ? TM : TM / 2;
    Piece<D, W> pr[kAhead][kTimes];
    auto load_residual = [&](int i) {
        if (a.res == nullptr || !whole) return;
#pragma unroll
        for (int t = 0; t < kTimes; ++t) {
            const int64_t m = m0 + i * 32 + t * kRows + r0;
            if (m < a.M) pr[i % kAhead][t].template load<false>(res + m * a.res_stride);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_residual(i);
    float s[W], b[W];
    if (whole) {
        load_affine<W>(a.sb, Affine::kF32, n, 1.0f, s);
        load_affine<W>(a.bias, a.bias_type, n, 0.0f, b);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {  // channels behind N count nothing
            const int c = n + j < a.N ? n + j : a.N - 1;
            float v[1];
            load_affine<1>(a.bias, a.bias_type, c, 0.0f, v);
            s[j] = a.sb[c];
            b[j] = v[0];
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                own[(lane & 31) * kPitch + j * 8 + g * 2 + (lane >> 5)] =
                    i32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                          acc[i][j][4 * g + 3]};
        wave_sync();
        i32x4 v[kTimes][W / 4];
#pragma unroll
        for (int t = 0; t < kTimes; ++t)
#pragma unroll
            for (int k = 0; k < W / 4; ++k)
                v[t][k] = own[(t * kRows + r0) * kPitch + lane % kLanes * (W / 4) + k];
        wave_sync();
#pragma unroll
        for (int t = 0; t < kTimes; ++t) {
            const int64_t m = m0 + i * 32 + t * kRows + r0;
            if (m >= a.M || n >= a.N) continue;
            const float sa = a.sa[m];
            float o[W];
            scaled<W>([&](int j) { return v[t][j / 4][j % 4]; }, sa, s, b, o);
            if (whole) {
                if (a.res != nullptr) {
#pragma unroll
                    for (int j = 0; j < W; ++j) o[j] += pr[i % kAhead][t].get(j);
                }
                Piece<D, W>::template store<false>(z + m * a.z_stride, o);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    if (n + j >= a.N) break;
                    if (a.res != nullptr) o[j] += D::to_f32(res[m * a.res_stride + j]);
                    z[m * a.z_stride + j] = D::from_f32(o[j]);
                }
            }
        }
        if (i + kAhead < TM) load_residual(i + kAhead);
    }
}

// A workgroup of WN waves takes BM = 32*TM rows and BN = 32*TN*WN channels, a wave
// all the rows and 32*TN of the channels, as products of 32 x 32 x 32.  Rows go
// through LDS, 128 input channels at a time: 16-byte pieces, piece p of row r at
// place p ^ (r / 2 % 8) of its 128 bytes, so that the 16 lanes that read one piece
// of 16 rows find them on different banks.  Weights come straight from memory, in
// the order in which the lanes hold them, and as no two waves share channels they
// are read once: what a CU gets from its L2 (about 40 bytes a clock) bounds these
// tiles, not the products.
template <class D, int WN, int TM, int TN, int AHEAD>
__global__ __launch_bounds__(WN * 64, 2) void gn_int8_tiles(MatmulArgs a) {
    constexpr int kThreads = WN * 64, BM = 32 * TM, BN = 32 * TN * WN;
    constexpr int kStage = BM * 8 / kThreads;  // 16-byte pieces that a lane copies
    constexpr int kStep = kThreads / 8;        // rows from one of them to the next
    static_assert(kStep % 16 == 0, "a lane's pieces have one place");
    static_assert(kStage % 2 == 0, "half of them in each half of a step");
    __shared__ i32x4 rows[3][BM * 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tm, tn;
    tile_of(blockIdx.x, a.mt * a.nt, a.mt, a.nt, &tm, &tn);
    const int64_t m0 = int64_t{tm} * BM;
    const int n0 = tn * BN + wave * TN * 32;
    const int steps = a.kb / 2;  // of 128 input channels

    // Addresses: one of the tile's rows and one of its weights, the same for all
    // lanes, and 32-bit distances from them.
    const int8_t *arow = a.a + m0 * a.a_stride;
    const int8_t *end = a.a + (a.M - 1) * a.a_stride + a.K;
    const int srow = tid >> 3;
    const int piece = (tid & 7) ^ (srow >> 1 & 7);
    uint32_t aoff[kStage];
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
        const int64_t r = srow + i * kStep;
        aoff[i] = static_cast<uint32_t>((m0 + r < a.M ? r : a.M - 1 - m0) * a.a_stride);
    }
    const int nb0 = n0 / kNBlock < a.nb ? n0 / kNBlock : a.nb - 1;
    const int8_t *brow = a.b + int64_t{nb0} * a.kb * kFragment;
    uint32_t boff[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int nb = j * 2 + (lane >> 4 & 1);
        boff[j] = static_cast<uint32_t>(nb0 + nb < a.nb ? nb : a.nb - 1 - nb0) *
                      static_cast<uint32_t>(a.kb * kFragment) +
                  static_cast<uint32_t>((lane >> 5) * 256 + (lane & 15) * 16);
    }
    i32x4 sa[AHEAD][kStage];
    i32x4 fb[AHEAD][4][TN];
    // FULL: a step that lies wholly inside K, as all but the last are
    auto load_row = [&](auto full, int q, int i, int it) {
        sa[q][i] = load16(arow + aoff[i], it * 128 + piece * 16, a.K, end,
                          !decltype(full)::value && it + 1 == steps);
    };
    auto load_weight = [&](int q, int ks, int j, int it) {
        fb[q][ks][j] = *reinterpret_cast<const i32x4 *>(brow + int64_t{it} * (2 * kFragment) +
                                                        boff[j] + ks * 512);
    };
    auto store_row = [&](int q, int i, int buf) { rows[buf][tid + i * kThreads] = sa[q][i]; };
    // a lane's piece of its row among rows 32*t and up, for product step ks
    auto frag = [&](int buf, int t, int ks) {
        const int r = t * 32 + (lane & 31);
        return rows[buf][r * 8 + ((ks * 2 + (lane >> 5)) ^ (r >> 1 & 7))];
    };
    typedef int i32x16 __attribute__((ext_vector_type(16)));
    i32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
    // One step, `it` with it % AHEAD = q.  The next one's rows go from registers to
    // LDS in its first half, and in the second those of the step AHEAD after it
    // start on their way; each product's operands are read while the products
    // before it run, and once used its weights are replaced by those of the step
    // AHEAD of this one.  `full`: all these steps exist and lie wholly inside K.
    // With three buffers one barrier is enough, in the middle, where no wave waits
    // for it long: what is written here was last read two steps ago.
    // The order is the one written here, one memory access after each product or
    // two: the compiler would move the loads next to their use, and a wave that
    // issues several at once waits for the memory pipe while its matrix core idles.
    i32x4 fa[2][TM];
    int cur = 0;
    constexpr int kHalf = kStage / 2;
    auto step = [&](auto full, int q, int it) {
        constexpr bool kFull = decltype(full)::value != 0;
        const int next = cur == 2 ? 0 : cur + 1, qn = (q + 1) % AHEAD;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            constexpr int kOther = TM + kHalf, kProducts = TM * TN;
#pragma unroll
            for (int m = 0; m < kProducts; ++m) {
                const int i = m % TM, j = m / TM;
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[q][ks][j], fa[ks & 1][i],
                                                                   acc[i][j], 0, 0, 0);
#pragma unroll
                for (int o = m * kOther / kProducts; o < (m + 1) * kOther / kProducts; ++o) {
                    if (o < TM) {
                        if (ks < 3)
                            fa[(ks + 1) & 1][o] = frag(cur, o, ks + 1);
                        else if (kFull || it + 1 < steps)
                            fa[0][o] = frag(next, o, 0);
                    } else if (ks < 2) {
                        if (kFull || it + 1 < steps) store_row(qn, ks * kHalf + o - TM, next);
                    } else if (kFull || it + 1 + AHEAD < steps) {
                        load_row(full, qn, (ks - 2) * kHalf + o - TM, it + 1 + AHEAD);
                    }
                }
                if (i == TM - 1 && (kFull || it + AHEAD < steps)) load_weight(q, ks, j, it + AHEAD);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (ks == 1) __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
        }
        cur = next;
    };
    typedef std::integral_constant<int, 0> Any;
    typedef std::integral_constant<int, 1> Full;
    // Before the first step: its rows in LDS, its weights and what the next ones need
    // on its way, in the order of a step, so that a wait for one is none for those
    // after it (nor may a load be left out on the way to the full steps).
    auto begin = [&](auto full) {
        constexpr bool kFull = decltype(full)::value != 0;
#pragma unroll
        for (int i = 0; i < kStage; ++i) load_row(full, 0, i, 0);
#pragma unroll
        for (int i = 0; i < kStage; ++i) store_row(0, i, 0);
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                __builtin_amdgcn_sched_barrier(0);
                if (ks >= 2 && (kFull || q + 1 < steps)) {
#pragma unroll
                    for (int i = 0; i < kHalf; ++i)
                        load_row(full, (q + 1) % AHEAD, (ks - 2) * kHalf + i, q + 1);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (kFull || q < steps) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) load_weight(q, ks, j, q);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[0][i] = frag(0, i, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    int it = 0;
    if (it + 2 * AHEAD + 1 < steps) {
        begin(Full{});
        for (; it + 2 * AHEAD + 1 < steps; it += AHEAD) {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) step(Full{}, q, it + q);
        }
    } else {
        begin(Any{});
    }
    for (; it < steps; it += AHEAD) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (it + q < steps) step(Any{}, q, it + q);
    }
    __syncthreads();  // rows' buffers are free
    constexpr int kOwn = 3 * BM * 8 / WN;
    static_assert(kOwn >= 32 * (8 * TN + 1), "32 rows of a wave's sums");
    finish_tile<D, TM, TN>(a, m0, n0, acc, &rows[0][0] + wave * kOwn, lane);
}

// ---- host -----------------------------------------------------------------------
template <int V> using IC = std::integral_constant<int, V>;

template <class F> void by_type(int dtype, F &&f) {
    switch (x_dtype(dtype)) {
        case GN_DTYPE_F16: f(Fp16{}); break;
        case GN_DTYPE_F32: f(F32{}); break;
        default: f(Bf16{}); break;
    }
}

bool misaligned(const void *p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

bool overflows(int64_t rows, int64_t stride, int64_t n) {
    return rows > 0 && stride > 0 && rows > (INT64_MAX / 4 - n) / stride;
}

int64_t k_blocks(int64_t K) { return ceil_div(K, 2 * kKBlock) * 2; }
int64_t n_blocks(int64_t N) { return ceil_div(N, kNBlock); }

gn_status check_nk(int64_t N, int64_t K) {
    if (N <= 0 || K <= 0) return GN_INVALID_ARGUMENT;
    if (K > GN_INT8_MAX_K || N > GN_INT8_MAX_N) return GN_UNSUPPORTED;
    return GN_OK;
}

constexpr int64_t kMaxTiles = int64_t{1} << 23;  // a dispatch holds fewer than 2^32 work-items

// Which kernel takes a product, and in what tiles.
struct MatmulPlan {
    int bm, bn;   // rows and channels of a tile
    bool rows;    // gn_int8_rows, else gn_int8_tiles
    int mt, nt;
};

// The kernel and tile with the least estimated time: the tiles that the busiest of
// the 256 CUs gets, times what one costs, which is proportional to K.  `cost` is in
// tenths of a microsecond at K = 4096.  A tile of the rows kernel is bound by its
// CU's traffic with the L2 and costs its rows and channels, about 1 us for 16 of
// them; the tiles kernel's were measured.  Measured, us for 1 / 2 / 4 / 8 tiles a
// CU (bf16, K = 4096): rows 16x16 5.8 / 7 / 9.1 / 15, 32x32 7.4 / 9.4 / 16 / 29,
// 32x64 8.2 / 14 / 26 / 47, 64x64 11.3 / 20 / 36 / 69; tiles 64x128 15.6 / 25 / 45 /
// 84, 128x128 23.7 / 40 / 76, 128x256 38 / 67 / 125 / 245.  kStart: a tiles launch
// takes 2 us longer to start and end, whatever K is.  What a tile costs whatever K is
// does not count, so that at K of one step many small tiles look cheaper than they
// are: (16384,4096,16) takes 241 us in 16384 tiles of 64x64, (16384,4096,64) 41 us in
// tiles of 128x256.
MatmulPlan matmul_plan(int64_t M, int64_t N, int64_t K, int64_t a_stride) {
    struct Kind {
        int bm, bn;
        bool rows;
        int64_t cost;
    };
    static constexpr Kind kinds[] = {
        {16, 16, true, 20},   {16, 32, true, 30},     {16, 64, true, 50},
        {32, 16, true, 30},   {32, 32, true, 40},     {32, 64, true, 60},
        {48, 32, true, 50},   {48, 64, true, 70},     {64, 32, true, 60},
        {64, 64, true, 80},   {64, 128, false, 98},   {128, 128, false, 174},
        {128, 256, false, 295},
    };
    constexpr int64_t kCus = 256, kStart = 20 * 4096;
    // the tiles kernel keeps 32-bit distances from a tile's first row
    const bool near = a_stride < int64_t{1} << 24;
    const Kind *best = nullptr;
    int64_t least = 0;
    for (const Kind &k : kinds) {
        if (!k.rows && !near) continue;
        const int64_t tiles = ceil_div(M, k.bm) * ceil_div(N, k.bn);
        const int64_t cost = ceil_div(tiles, kCus) * k.cost * K + (k.rows ? 0 : kStart);
        if (best == nullptr || cost < least) best = &k, least = cost;
    }
    return MatmulPlan{best->bm, best->bn, best->rows, static_cast<int>(ceil_div(M, best->bm)),
                      static_cast<int>(ceil_div(N, best->bn))};
}

}  // namespace
}  // namespace gnsilu

using namespace gnsilu;

extern "C" {

gn_status gn_int8_packed_bytes(int64_t N, int64_t K, int64_t *bytes_out) {
    if (bytes_out == nullptr) return GN_INVALID_ARGUMENT;
    const gn_status st = check_nk(N, K);
    if (st != GN_OK) return st;
    *bytes_out = n_blocks(N) * k_blocks(K) * kFragment;
    return GN_OK;
}

gn_status gn_int8_pack_weights(const void *codes, int64_t codes_stride, void *packed, int64_t N,
                               int64_t K, void *stream) {
    if (codes == nullptr || packed == nullptr) return GN_INVALID_ARGUMENT;
    gn_status st = check_nk(N, K);
    if (st == GN_INVALID_ARGUMENT || codes_stride < 0 || overflows(N, codes_stride, K))
        return GN_INVALID_ARGUMENT;
    if (st != GN_OK) return st;
    if (misaligned(packed, 16)) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {codes, packed}, &c);
    if (st != GN_OK) return st;
    const int64_t pieces = n_blocks(N) * k_blocks(K) * 64;
    gn_int8_pack<<<static_cast<unsigned>(std::min(ceil_div(pieces, 256), kPackBlocks)), 256, 0,
                   c.stream>>>(
        static_cast<const int8_t *>(codes), codes_stride, static_cast<int8_t *>(packed),
        static_cast<int>(N), static_cast<int>(K), static_cast<int>(k_blocks(K)), pieces);
    return finish_launch();
}

gn_status gn_int8_matmul_plan(int64_t M, int64_t N, int64_t K, int64_t a_stride,
                              int64_t plan_out[4]) {
    if (plan_out == nullptr || M < 0 || a_stride < 0) return GN_INVALID_ARGUMENT;
    const gn_status st = check_nk(N, K);
    if (st != GN_OK) return st;
    if (M > GN_INT8_MAX_M) return GN_UNSUPPORTED;
    const MatmulPlan p = matmul_plan(M, N, K, a_stride);
    const int64_t tiles = int64_t{p.mt} * p.nt;
    if (tiles >= kMaxTiles) return GN_UNSUPPORTED;
    plan_out[0] = p.bm;
    plan_out[1] = p.bn;
    plan_out[2] = p.rows ? 0 : 1;
    plan_out[3] = tiles;
    return GN_OK;
}

gn_status gn_int8_matmul(const void *a, int64_t a_stride, const float *a_scales, const void *packed,
                         const float *w_scales, const void *bias, const void *residual,
                         int64_t residual_stride, void *z, int64_t z_stride, int64_t M, int64_t N,
                         int64_t K, int dtype, void *stream) {
    if (a == nullptr || a_scales == nullptr || packed == nullptr || w_scales == nullptr ||
        z == nullptr)
        return GN_INVALID_ARGUMENT;
    if (!valid_dtype(dtype) || M < 0) return GN_INVALID_ARGUMENT;
    gn_status st = check_nk(N, K);
    if (st == GN_INVALID_ARGUMENT) return st;
    if (a_stride < 0 || residual_stride < 0 || z_stride < 0 || (M > 1 && z_stride < N))
        return GN_INVALID_ARGUMENT;
    if (overflows(M, a_stride, K) || overflows(M, residual_stride, N) || overflows(M, z_stride, N))
        return GN_INVALID_ARGUMENT;
    if (st == GN_OK) st = check_affine(bias, nullptr, dtype);
    if (st != GN_OK) return st;
    if (M > GN_INT8_MAX_M) return GN_UNSUPPORTED;
    const int64_t es = elem_bytes(dtype);
    if (misaligned(a_scales, 4) || misaligned(w_scales, 4) || misaligned(packed, 16) ||
        misaligned(residual, es) || misaligned(z, es))
        return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    const MatmulPlan plan = matmul_plan(M, N, K, a_stride);
    const int64_t tiles = int64_t{plan.mt} * plan.nt;
    if (tiles >= kMaxTiles) return GN_UNSUPPORTED;
    Call c;
    st = begin_call(stream, {a, a_scales, packed, w_scales, bias, residual, z}, &c);
    if (st != GN_OK) return st;
    MatmulArgs p{};
    p.a = static_cast<const int8_t *>(a);
    p.sa = a_scales;
    p.b = static_cast<const int8_t *>(packed);
    p.sb = w_scales;
    p.bias = bias;
    p.res = residual;
    p.z = z;
    p.M = M;
    p.a_stride = a_stride;
    p.res_stride = residual_stride;
    p.z_stride = z_stride;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.kb = static_cast<int>(k_blocks(K));
    p.nb = static_cast<int>(n_blocks(N));
    p.bias_type = affine_type(dtype);
    p.mt = plan.mt;
    p.nt = plan.nt;
    const unsigned grid = static_cast<unsigned>(tiles);
    by_type(dtype, [&](auto d) {
        using D = decltype(d);
        constexpr int kWaves = 8;
        auto rows = [&](auto mt, auto nt) {
            gn_int8_rows<D, decltype(mt)::value, decltype(nt)::value, kWaves>
                <<<grid, kWaves * 64, 0, c.stream>>>(p);
        };
        auto by_n = [&](auto mt) {
            switch (plan.bn) {
                case 16: return rows(mt, IC<1>{});
                case 32: return rows(mt, IC<2>{});
                default: return rows(mt, IC<4>{});
            }
        };
        if (plan.rows) {
            switch (plan.bm) {
                case 16: return by_n(IC<1>{});
                case 32: return by_n(IC<2>{});
                case 48: return by_n(IC<3>{});
                default: return by_n(IC<4>{});
            }
        }
        if (plan.bm == 64)
            gn_int8_tiles<D, 4, 2, 1, 2><<<grid, 256, 0, c.stream>>>(p);
        else if (plan.bn == 128)
            gn_int8_tiles<D, 4, 4, 1, 2><<<grid, 256, 0, c.stream>>>(p);
        else
            gn_int8_tiles<D, 4, 4, 2, 1><<<grid, 256, 0, c.stream>>>(p);
    });
    return finish_launch();
}

}  // extern "C"
