// gn_rows8.hip -- rows kept in 8 bits with one scale each, and widened again, for
// MI355X (gfx950).
//
//   quantize    top = max|x|, q = rint(127*x/top), scale = top/127
//   dequantize  x = q*scale, rounded once
//
// Both are bound by HBM.  A row is read once and held in registers while its
// lanes agree on the maximum, in the lanes and pieces of the norms' forward
// passes (gn_row_passes.hpp).
//
// Measured on MI355X, bf16: quantize (16384,4096) 38 us (5.3 TB/s), (8192,2560)
// 12.7 us (5.0 TB/s, the VALU 95% busy: 320 pieces on 512 places); dequantize 33 us
// (6.1 TB/s), 10.6 us; quantize of fp32 (5003,1001) 5.2 us, x in the caches,
// (4096,8192) 26 us (6.5 TB/s), (16384,12288) 187 us (5.4 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gn_row_passes.hpp"
#include "gn_rows8.hpp"
#include "gnsilu.h"

namespace gnsilu {
namespace {

struct Rows8Args {
    const void *x;
    void *y;
    int8_t *codes_out;
    const int8_t *codes;
    const float *scales;
    float *scales_out;
    int64_t M, x_stride, y_stride, codes_stride;
    int C, P;
};

template <class D, int W, int NV> struct QuantizeRow {
    Piece<D, W> v[NV];
};

template <class D, int W, bool TAIL, int TPR, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void gn_quantize(Rows8Args a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    constexpr int kRed = TPR > 64 ? THREADS / 64 : 1;
    __shared__ uint32_t red[2 * kRed];
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    const T *x = static_cast<const T *>(a.x);
    int c[NV], lo[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
    using Row = QuantizeRow<D, W, NV>;
    auto fetch = [&](Row &r, int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) r.v[j].template load<false>(x + m * a.x_stride + c[j]);
    };
    RowLoop<Row, kSlots, sizeof(T) == 4 && NV < 4> loop{a.M, slot, gridDim.x};
    loop.begin(fetch);
    int par = 0;
    loop.run(fetch, [&](Row &r, int64_t m, bool live) {
        // channels counted twice (a last piece's, those of a lane beyond the
        // row) change no maximum; magnitudes of every type order like their bits
        uint32_t top = 0;
        if constexpr (W == 8) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) m = max2_u16(m, r.v[j].w[k] & 0x7fff7fffu);
            top = max(m >> 16, m & 0xffffu);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    top = max(top, __float_as_uint(r.v[j].get(i)) & 0x7fffffffu);
        }
        top = lane_max<(TPR < 64 ? TPR : 64)>(top);
        if constexpr (TPR > 64) {
            constexpr int kWaves = TPR / 64;
            uint32_t *mine = red + par * kRed + (threadIdx.x / TPR) * kWaves;
            if ((threadIdx.x & 63) == 0) mine[(threadIdx.x % TPR) >> 6] = top;
            __syncthreads();
            top = lane_max<kWaves>(mine[threadIdx.x % kWaves]);
            par ^= 1;
        }
        if (!live) return;  // no barrier from here on
        if constexpr (W == 8) top = __float_as_uint(D::to_f32(static_cast<uint16_t>(top)));
        const Rows8Scale sc(top);
        if (t == 0) a.scales_out[m] = Rows8Scale::step(top);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (lo[j] >= W) continue;
            float o[W];
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = r.v[j].get(i);
            rows8_encode<W>(o, sc).template store<false>(a.codes_out + m * a.codes_stride + c[j]);
        }
    });
}

template <int W, int NV> struct DequantizeRow {
    Codes<W> q[NV];
    float scale;
};

template <class D, int W, bool TAIL, int TPR, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void gn_dequantize(Rows8Args a) {
    using T = typename D::storage;
    constexpr int kSlots = THREADS / TPR;
    const int t = threadIdx.x % TPR, slot = row_slot<TPR>();
    T *y = static_cast<T *>(a.y);
    int c[NV], lo[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) piece_at<W, TAIL>(a, t + j * TPR, &c[j], &lo[j]);
    using Row = DequantizeRow<W, NV>;
    auto fetch = [&](Row &r, int64_t m) {
#pragma unroll
        for (int j = 0; j < NV; ++j) r.q[j].load(a.codes + m * a.codes_stride + c[j]);
        r.scale = a.scales[m];
    };
    RowLoop<Row, kSlots, sizeof(T) == 4> loop{a.M, slot, gridDim.x};
    loop.begin(fetch);
    loop.run(fetch, [&](Row &r, int64_t m, bool live) {
        if (!live) return;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (lo[j] >= W) continue;
            float o[W];
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = static_cast<float>(r.q[j].get(i)) * r.scale;
            Piece<D, W>::template store<false>(y + m * a.y_stride + c[j], o);
        }
    });
}

template <class F> void launch_rows(int64_t M, int64_t C, int dtype, F &&go) {
    const LnShape s = ln_shape(C, dtype, true);
    by_type(dtype, [&](auto d) {
        with_ln_shape<decltype(d), true>(s, [&](auto w, auto tail, auto tpr, auto nv) {
            constexpr int TPR = decltype(tpr)::value, NT = forward_threads(TPR);
            int64_t blocks = one_each_blocks(M, NT / TPR);
            if (sizeof(typename decltype(d)::storage) == 4)  // one_each_blocks' comment
                blocks = std::min(blocks, kForwardLanes / NT);
            go(d, w, tail, tpr, nv, IC<NT>{}, static_cast<unsigned>(blocks), s.P);
        });
    });
}

}  // namespace
}  // namespace gnsilu

using namespace gnsilu;

extern "C" {

gn_status gn_quantize_rows(const void *x, int64_t x_stride, void *codes, int64_t codes_stride,
                           float *scales, int64_t M, int64_t C, int dtype, void *stream) {
    if (x == nullptr || codes == nullptr || scales == nullptr) return GN_INVALID_ARGUMENT;
    gn_status st = check_rows(M, C, dtype, &x_stride, 1, &codes_stride, 1);
    if (st != GN_OK) return st;
    if (misaligned(x, elem_bytes(dtype)) || misaligned(scales, 4)) return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    Rows8Args a{};
    a.x = x;
    a.codes_out = static_cast<int8_t *>(codes);
    a.scales_out = scales;
    a.M = M;
    a.x_stride = x_stride;
    a.codes_stride = codes_stride;
    a.C = static_cast<int>(C);
    launch_rows(M, C, dtype, [&](auto d, auto w, auto tail, auto tpr, auto nv, auto nt,
                                 unsigned grid, int P) {
        a.P = P;
        gn_quantize<decltype(d), decltype(w)::value, decltype(tail)::value != 0,
                    decltype(tpr)::value, decltype(nv)::value, decltype(nt)::value>
            <<<grid, decltype(nt)::value, 0, c.stream>>>(a);
    });
    return finish_launch();
}

gn_status gn_dequantize_rows(const void *codes, int64_t codes_stride, const float *scales, void *x,
                             int64_t x_stride, int64_t M, int64_t C, int dtype, void *stream) {
    if (x == nullptr || codes == nullptr || scales == nullptr) return GN_INVALID_ARGUMENT;
    gn_status st = check_rows(M, C, dtype, &codes_stride, 1, &x_stride, 1);
    if (st != GN_OK) return st;
    if (misaligned(x, elem_bytes(dtype)) || misaligned(scales, 4)) return GN_UNSUPPORTED;
    if (M == 0) return GN_OK;
    Call c;
    st = begin_call(stream, {x, codes, scales}, &c);
    if (st != GN_OK) return st;
    Rows8Args a{};
    a.codes = static_cast<const int8_t *>(codes);
    a.scales = scales;
    a.y = x;
    a.M = M;
    a.codes_stride = codes_stride;
    a.y_stride = x_stride;
    a.C = static_cast<int>(C);
    launch_rows(M, C, dtype, [&](auto d, auto w, auto tail, auto tpr, auto nv, auto nt,
                                 unsigned grid, int P) {
        a.P = P;
        gn_dequantize<decltype(d), decltype(w)::value, decltype(tail)::value != 0,
                      decltype(tpr)::value, decltype(nv)::value, decltype(nt)::value>
            <<<grid, decltype(nt)::value, 0, c.stream>>>(a);
    });
    return finish_launch();
}

}  // extern "C"
