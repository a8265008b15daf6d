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

// Rows off 16-byte boundaries, copied to rows on them.
__global__ __launch_bounds__(256) void gn_int8_align(const int8_t *a, int64_t stride, int8_t *to,
                                                     int64_t to_stride, int K, int64_t pieces) {
    const int64_t i = int64_t{blockIdx.x} * 256 + threadIdx.x;
    if (i >= pieces) return;
    const int64_t per = to_stride / 16, m = i / per;
    const int k = static_cast<int>(i % per) * 16;
    const int8_t *p = a + m * stride + k;
    u32x4 v;
    if (k + 16 <= K) {
        typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
        v = *reinterpret_cast<const u32x4_a1 *>(p);
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (k + j < K)
                w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[j])) << (8 * (j & 3));
        v = u32x4{w[0], w[1], w[2], w[3]};
    }
    *reinterpret_cast<u32x4 *>(to + m * to_stride + k) = v;
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
            const int k = kb * kKBlock + kg;
            // behind K the weights are zero: any byte of the row will do
            const int at = k < a.K ? k : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i) fa[u][i] = *reinterpret_cast<const i32x4 *>(ap[i] + at);
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

// ---- host -----------------------------------------------------------------------
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

size_t align_workspace(int64_t M, int64_t K) { return static_cast<size_t>(M * ceil_div(K, 16) * 16); }

bool rows_aligned(const void *a, int64_t stride, int64_t M) {
    return !misaligned(a, 16) && (stride % 16 == 0 || M == 1);
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

gn_status gn_int8_matmul_workspace(int64_t M, int64_t N, int64_t K, int aligned,
                                   int64_t *bytes_out) {
    if (bytes_out == nullptr || M < 0 || (aligned != 0 && aligned != 1)) return GN_INVALID_ARGUMENT;
    const gn_status st = check_nk(N, K);
    if (st != GN_OK) return st;
    if (M > GN_INT8_MAX_M) return GN_UNSUPPORTED;
    *bytes_out = aligned ? 0 : static_cast<int64_t>(align_workspace(M, K));
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
    const bool aligned = rows_aligned(a, a_stride, M);
    const size_t need = aligned ? 0 : align_workspace(M, K);
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
    if (!aligned) {
        p.a_stride = ceil_div(K, 16) * 16;
        const int64_t pieces = M * (p.a_stride / 16);
        gn_int8_align<<<static_cast<unsigned>(ceil_div(pieces, 256)), 256, 0, c.stream>>>(
            p.a, a_stride, static_cast<int8_t *>(workspace), p.a_stride, p.K, pieces);
        p.a = static_cast<const int8_t *>(workspace);
    }
    by_type(dtype, [&](auto d) {
        using D = decltype(d);
        auto go = [&](auto mt, auto nt) {
            constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, WAVES = 8;
            const dim3 grid(static_cast<unsigned>(ceil_div(p.nb, NT)),
                            static_cast<unsigned>(ceil_div(M, 16 * MT)));
            gn_int8_rows<D, MT, NT, WAVES><<<grid, WAVES * 64, 0, c.stream>>>(p);
        };
        if (M <= 16)
            go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
        else
            go(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
    });
    return finish_launch();
}

}  // extern "C"
