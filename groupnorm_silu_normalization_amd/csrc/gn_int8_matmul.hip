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
// is multiplied by zero.  Fragments of rows are read as they lie: 16 bytes of a
// row for each lane.  The weights are the first operand, so that a lane's four
// results are neighbours in a row of z.
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
    const int8_t *a;      // [M][K], rows a_stride apart, 16-byte aligned rows
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
    int split;            // parts of K, each a workgroup's
    i32x4 *part;          // [split][tiles][...] sums of a part, where split > 1
};

constexpr int kKBlock = 64, kNBlock = 16, kFragment = 1024;

// ---- packing ---------------------------------------------------------------------
// One lane, 16 bytes of a fragment.
__global__ __launch_bounds__(256) void gn_int8_pack(const int8_t *w, int64_t stride, int8_t *packed,
                                                    int N, int K, int kb, int64_t pieces) {
    const int64_t i = int64_t{blockIdx.x} * 256 + threadIdx.x;
    if (i >= pieces) return;
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
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = fmaf(static_cast<float>(acc[j]) * sa, sb[j], b[j]) + r[j];
        store4<D>(z, o);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= a.N) break;
        float b[1];
        load_affine<1>(a.bias, a.bias_type, n + j, 0.0f, b);
        float o = fmaf(static_cast<float>(acc[j]) * sa, a.sb[n + j], b[0]);
        if (a.res != nullptr) o += D::to_f32(res[j]);
        z[j] = D::from_f32(o);
    }
}

// 16 bytes of a row from k on, zero behind K.  last: the block may reach behind K.
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
__device__ __forceinline__ u32x4 load16(const int8_t *row, int k, int K, bool last) {
    if (!last || k + 16 <= K) return *reinterpret_cast<const u32x4_a1 *>(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (k + j < K)
            w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + j])) << (8 * (j & 3));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// ---- few rows ------------------------------------------------------------------------
// A workgroup takes 16*MT rows and 16*NT channels; its waves take the blocks of K
// in turn and join their sums through LDS.
template <class D, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gn_int8_rows(MatmulArgs a) {
    constexpr int kTiles = MT * NT, kUnroll = 2;
    __shared__ i32x4 part[WAVES][kTiles][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t m0 = int64_t{blockIdx.y} * (16 * MT);
    const int nb0 = static_cast<int>(blockIdx.x) * NT;
    const int kg = (lane >> 4) * 16;
    const int8_t *ap[MT], *bp[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + i * 16 + (lane & 15);
        ap[i] = a.a + (m < a.M ? m : a.M - 1) * a.a_stride;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int nb = nb0 + j < a.nb ? nb0 + j : a.nb - 1;
        bp[j] = a.b + int64_t{nb} * a.kb * kFragment + lane * 16;
    }
    i32x4 acc[MT][NT] = {};
    for (int k0 = wave; k0 < a.kb; k0 += kUnroll * WAVES) {
        i32x4 fa[kUnroll][MT], fb[kUnroll][NT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int kb = k0 + u * WAVES;
            if (kb >= a.kb) break;
            const bool last = (kb + 1) * kKBlock > a.K;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fa[u][i] = __builtin_bit_cast(i32x4, load16(ap[i], kb * kKBlock + kg, a.K, last));
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fb[u][j] = *reinterpret_cast<const i32x4 *>(bp[j] + int64_t{kb} * kFragment);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (k0 + u * WAVES >= a.kb) break;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][j], fa[u][i], acc[i][j],
                                                                       0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    for (int tile = wave; tile < kTiles; tile += WAVES) {
        i32x4 s = part[0][tile][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += part[w][tile][lane];
        finish4<D>(a, m0 + tile / NT * 16 + (lane & 15),
                   (nb0 + tile % NT) * kNBlock + (lane >> 4) * 4, s);
    }
}

// ---- tiles -----------------------------------------------------------------------
// Eight neighbouring sums of row m from channel n on, scaled and stored.
template <class D>
__device__ __forceinline__ void finish8(const MatmulArgs &a, int64_t m, int n, const i32x4 &lo,
                                        const i32x4 &hi) {
    using T = typename D::storage;
    if constexpr (sizeof(T) == 2) {
        if (m >= a.M || n >= a.N) return;
        if (n + 8 <= a.N) {
            const float sa = a.sa[m];
            float sb[8], b[8], o[8];
            load_affine<8>(a.sb, Affine::kF32, n, 1.0f, sb);
            load_affine<8>(a.bias, a.bias_type, n, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = fmaf(static_cast<float>(j < 4 ? lo[j & 3] : hi[j & 3]) * sa, sb[j], b[j]);
            if (a.res != nullptr) {
                Piece<D, 8> r;
                r.template load<false>(static_cast<const T *>(a.res) + m * a.res_stride + n);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += r.get(j);
            }
            Piece<D, 8>::template store<false>(static_cast<T *>(a.z) + m * a.z_stride + n, o);
            return;
        }
    }
    finish4<D>(a, m, n, lo);
    finish4<D>(a, m, n + 4, hi);
}

// A 32 x 32 product leaves 4 neighbouring sums of channels 8g + 4*(lane / 32) in
// each lane, of row lane % 32.  Swapped between the halves of the wave, two g's
// become 8 neighbours: channels 16*pair + 8*(lane / 32) and up.
__device__ __forceinline__ void join_halves(i32x4 &g0, i32x4 &g1) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const auto s = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(g0[r]),
                                                        static_cast<uint32_t>(g1[r]), false, false);
        g0[r] = static_cast<int>(s[0]);
        g1[r] = static_cast<int>(s[1]);
    }
}

// The tile of a workgroup: consecutive workgroups go to the eight XCDs in turn,
// each of which takes a run of tiles, in strips of kStrip rows of tiles, so
// that the tiles it works on at one time share rows and weights in its L2.
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

// A workgroup of WM x WN waves takes BM = 32*TM*WM rows and BN = 32*TN*WN
// channels, a wave 32*TM by 32*TN of them, as products of 32 x 32 x 32.  Rows go
// through LDS, 128 input channels at a time: 16-byte pieces, of row r at place
// piece ^ (r / 2 % 8) of its 128 bytes, so that the 16 lanes that read one piece
// of 16 rows find them on different banks.  Weights come straight from memory,
// in the order in which the lanes hold them.
template <class D, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(WM *WN * 64) void gn_int8_tiles(MatmulArgs a) {
    constexpr int kThreads = WM * WN * 64, BM = 32 * TM * WM, BN = 32 * TN * WN;
    constexpr int kStage = BM * 8 / kThreads;  // 16-byte pieces that a lane copies
    constexpr int kStep = kThreads / 8;        // rows from one of them to the next
    static_assert(kStep % 16 == 0, "a lane's pieces have one place");
    __shared__ u32x4 rows[3][BM * 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int tiles = a.mt * a.nt;
    int tm, tn;
    tile_of(blockIdx.x % tiles, tiles, a.mt, a.nt, &tm, &tn);
    const int part = blockIdx.x / tiles;
    const int64_t m0 = int64_t{tm} * BM;
    const int n0 = tn * BN;
    // this part's steps of 128 input channels
    const int all = a.kb / 2, it0 = static_cast<int>(int64_t{all} * part / a.split),
              it1 = static_cast<int>(int64_t{all} * (part + 1) / a.split);

    const int srow = tid >> 3;
    const int piece = (tid & 7) ^ (srow >> 1 & 7);
    const int8_t *ap[kStage];
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
        const int64_t m = m0 + srow + i * kStep;
        ap[i] = a.a + (m < a.M ? m : a.M - 1) * a.a_stride;
    }
    const int8_t *bp[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int nb = n0 / kNBlock + (wn * TN + j) * 2 + (lane >> 4 & 1);
        bp[j] = a.b + (int64_t{nb < a.nb ? nb : a.nb - 1} * a.kb + it0 * 2) * kFragment +
                (lane >> 5) * 256 + (lane & 15) * 16;
    }
    u32x4 sa[kStage];
    i32x4 fb[4][TN];
    // FULL: a step that lies wholly inside K, as all but the last are
    auto load_rows = [&](auto full, int it) {
        const int k = it * 128 + piece * 16;
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            sa[i] = load16(ap[i], k, a.K, !decltype(full)::value && it + 1 == all);
    };
    auto load_weights = [&](int ks) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[ks][j] = *reinterpret_cast<const i32x4 *>(bp[j] + ks * 512);
    };
    auto store_rows = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kStage; ++i) rows[buf][tid + i * kThreads] = sa[i];
    };
    // a lane's piece of row r (of the wave's) at products' step ks
    const int r0 = wm * TM * 32 + (lane & 31);
    auto frag = [&](int buf, int t, int ks) {
        const int r = r0 + t * 32;
        return *reinterpret_cast<const i32x4 *>(
            &rows[buf][r * 8 + ((ks * 2 + (lane >> 5)) ^ (r >> 1 & 7))]);
    };
    typedef int i32x16 __attribute__((ext_vector_type(16)));
    i32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
    // One step.  The next one's rows go from registers to LDS and those of the one
    // after it start on their way (`full`: there are both, wholly inside K); each
    // product's operands are read while the product before it runs, and the next
    // step's weights replace each product's as they are used.  With three buffers
    // one barrier is enough, in the middle, where no wave waits for it long: what
    // is written here was last read two steps ago.  The compiler would move the
    // loads behind the products, next to their use: the scheduling barriers keep
    // them where they are.
    i32x4 fa[2][TM];
    int cur = 0;
    auto step = [&](auto full, int it) {
        constexpr bool kFull = decltype(full)::value != 0;
        const int next = cur == 2 ? 0 : cur + 1;
        if (kFull || it + 1 < it1) {
            store_rows(next);
#pragma unroll
            for (int j = 0; j < TN; ++j) bp[j] += 2 * kFragment;
        }
        if (kFull || it + 2 < it1) load_rows(full, it + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (ks < 3 || kFull || it + 1 < it1) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[(ks + 1) & 1][i] = ks < 3 ? frag(cur, i, ks + 1) : frag(next, i, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks][j], fa[ks & 1][i],
                                                                       acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (kFull || it + 1 < it1) load_weights(ks);
            if (ks == 1) __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
        }
        cur = next;
    };
    typedef std::integral_constant<int, 0> Any;
    typedef std::integral_constant<int, 1> Full;
    load_rows(Any{}, it0);
    store_rows(0);
    // rows before weights, as in a step: a wait for the former is none for the latter
    if (it0 + 1 < it1) load_rows(Any{}, it0 + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) load_weights(ks);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[0][i] = frag(0, i, 0);
    int it = it0;
    for (; it + 3 < it1; ++it) step(Full{}, it);
    for (; it < it1; ++it) step(Any{}, it);
    if (a.split > 1) {
        i32x4 *to = a.part + (int64_t{blockIdx.x} * (kThreads / 64) + wave) * (TM * TN * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    to[((i * TN + j) * 4 + g) * 64] =
                        i32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                              acc[i][j][4 * g + 3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + (wm * TM + i) * 32 + (lane & 31);
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                i32x4 g[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) g[h][r] = acc[i][j][8 * p + 4 * h + r];
                join_halves(g[0], g[1]);
                finish8<D>(a, m, n0 + (wn * TN + j) * 32 + p * 16 + (lane >> 5) * 8, g[0], g[1]);
            }
    }
}

// The parts of K joined: one wave's lanes as they hold a product's sums.
template <class D, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(256) void gn_int8_join(MatmulArgs a) {
    constexpr int kWaves = WM * WN, kEach = TM * TN * 2;  // pairs of groups in a wave
    const int lane = threadIdx.x & 63;
    const int tiles = a.mt * a.nt;
    const int64_t u = int64_t{blockIdx.x} * 4 + (threadIdx.x >> 6);
    if (u >= int64_t{tiles} * kWaves * kEach) return;
    const int b = static_cast<int>(u / (kWaves * kEach)), in = static_cast<int>(u % (kWaves * kEach));
    const int wave = in / kEach, pair = in % kEach;
    const i32x4 *from = a.part + u * 128 + lane;
    const int64_t next = int64_t{tiles} * kWaves * kEach * 128;
    i32x4 g0 = {}, g1 = {};
    for (int s = 0; s < a.split; ++s) {
        g0 += from[s * next];
        g1 += from[s * next + 64];
    }
    join_halves(g0, g1);
    int tm, tn;
    tile_of(b, tiles, a.mt, a.nt, &tm, &tn);
    const int i = pair / 2 / TN, j = pair / 2 % TN;
    finish8<D>(a, int64_t{tm} * (32 * TM * WM) + (wave / WN * TM + i) * 32 + (lane & 31),
               tn * (32 * TN * WN) + (wave % WN * TN + j) * 32 + pair % 2 * 16 + (lane >> 5) * 8, g0,
               g1);
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

// Which kernel takes a product, and in what tiles.
struct MatmulPlan {
    int kind;  // 0: few rows; 1: tiles of 128 x 128; 2: of 256 x 256
    int mt, nt, split;
    size_t workspace;
};

MatmulPlan matmul_plan(int64_t M, int64_t N, int64_t K) {
    MatmulPlan p{};
    p.split = 1;
    if (M <= 64) return p;
    const int64_t big = ceil_div(M, 256) * ceil_div(N, 256);
    p.kind = big >= 192 ? 2 : 1;
    const int64_t side = p.kind == 2 ? 256 : 128;
    p.mt = static_cast<int>(ceil_div(M, side));
    p.nt = static_cast<int>(ceil_div(N, side));
    const int64_t tiles = int64_t{p.mt} * p.nt, steps = k_blocks(K) / 2;
    if (p.kind == 1)
        while (tiles * p.split * 2 <= 512 && steps / (p.split * 2) >= 4) p.split *= 2;
    if (p.split > 1) p.workspace = static_cast<size_t>(tiles * p.split * side * side * 4);
    return p;
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
    gn_int8_pack<<<static_cast<unsigned>(ceil_div(pieces, 256)), 256, 0, c.stream>>>(
        static_cast<const int8_t *>(codes), codes_stride, static_cast<int8_t *>(packed),
        static_cast<int>(N), static_cast<int>(K), static_cast<int>(k_blocks(K)), pieces);
    return finish_launch();
}

gn_status gn_int8_matmul_workspace(int64_t M, int64_t N, int64_t K, int64_t *bytes_out) {
    if (bytes_out == nullptr || M < 0) return GN_INVALID_ARGUMENT;
    const gn_status st = check_nk(N, K);
    if (st != GN_OK) return st;
    if (M > GN_INT8_MAX_M) return GN_UNSUPPORTED;
    *bytes_out = static_cast<int64_t>(matmul_plan(M, N, K).workspace);
    return GN_OK;
}

gn_status gn_int8_matmul(const void *a, int64_t a_stride, const float *a_scales, const void *packed,
                         const float *w_scales, const void *bias, const void *residual,
                         int64_t residual_stride, void *z, int64_t z_stride, int64_t M, int64_t N,
                         int64_t K, int dtype, void *workspace, int64_t workspace_bytes,
                         void *stream) {
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
        misaligned(residual, es) || misaligned(z, es) || misaligned(workspace, 16))
        return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    const MatmulPlan plan = matmul_plan(M, N, K);
    const size_t need = plan.workspace;
    if (need > 0 && workspace == nullptr) return GN_INVALID_ARGUMENT;
    if (need > 0 && (workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < need))
        return GN_SCRATCH_TOO_SMALL;
    Call c;
    st = begin_call(stream,
                    {a, a_scales, packed, w_scales, bias, residual, z,
                     need > 0 ? workspace : nullptr},
                    &c);
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
    p.split = plan.split;
    p.part = static_cast<i32x4 *>(workspace);
    by_type(dtype, [&](auto d) {
        using D = decltype(d);
        auto rows = [&](auto mt, auto nt) {
            constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, WAVES = 8;
            const dim3 grid(static_cast<unsigned>(ceil_div(p.nb, NT)),
                            static_cast<unsigned>(ceil_div(M, 16 * MT)));
            gn_int8_rows<D, MT, NT, WAVES><<<grid, WAVES * 64, 0, c.stream>>>(p);
        };
        auto tiles = [&](auto wm, auto wn, auto tm, auto tn) {
            constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value;
            constexpr int TM = decltype(tm)::value, TN = decltype(tn)::value;
            const unsigned n = static_cast<unsigned>(p.mt) * static_cast<unsigned>(p.nt);
            gn_int8_tiles<D, WM, WN, TM, TN>
                <<<n * static_cast<unsigned>(p.split), WM * WN * 64, 0, c.stream>>>(p);
            if (p.split > 1)
                gn_int8_join<D, WM, WN, TM, TN>
                    <<<static_cast<unsigned>(ceil_div(int64_t{n} * WM * WN * TM * TN * 2, 4)), 256,
                       0, c.stream>>>(p);
        };
        if (plan.kind == 2)
            tiles(IC<2>{}, IC<4>{}, IC<4>{}, IC<2>{});
        else if (plan.kind == 1)
            tiles(IC<2>{}, IC<2>{}, IC<2>{}, IC<2>{});
        else if (M <= 16)
            rows(IC<1>{}, IC<1>{});
        else
            rows(IC<4>{}, IC<2>{});
    });
    return finish_launch();
}

}  // extern "C"
