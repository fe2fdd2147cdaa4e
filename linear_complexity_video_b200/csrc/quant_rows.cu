// 8-bit row quantisation: the codes and the scale of each token's activations (or
// of each output channel's weights) for mate_linear_i8_fwd,
//     s_m = max_k |x_mk| / 127,   q_mk = rint(127 x_mk / max_k |x_mk|).
//
// HBM-bound: 2 bytes read and 1 written per element. A row stays in its threads'
// registers as packed bf16 pairs between the maximum and the codes, so that it is
// read once, with all of a thread's loads in flight at once.
#include "common.cuh"
#include "i8.cuh"
#include "kernels.h"
#include "tc.cuh"

#include <cuda_bf16.h>

namespace mate {

namespace {

constexpr int kQThreads = 256;

// largest magnitude of the two bf16 halves over `w`'s words, NaN kept (as bf16 pair bits)
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w)
{
    const uint32_t a = w & 0x7fff7fffu;
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&m),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&a));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// TPR threads per row, up to VPL 16-byte vectors (eight channels) per thread
template <int TPR, int VPL>
__global__ void __launch_bounds__(kQThreads) quant_rows_kernel(QuantArgs a)
{
    constexpr int kRows = kQThreads / TPR, kWarps = TPR / 32;
    __shared__ uint32_t part[kQThreads / 32];
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + slot;
    const bool live = row < a.M;
    const int nv = live ? a.K / 8 : 0;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.x) + row * a.K);
    tc::stream_release();  // a product behind it may set itself up
    uint4 v[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j] = t + j * TPR < nv ? __ldcs(x + t + j * TPR) : make_uint4(0, 0, 0, 0);
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) m2 = abs_max2(abs_max2(abs_max2(abs_max2(m2, v[j].x), v[j].y), v[j].z), v[j].w);
    // magnitudes order as their bits do, NaN last
    uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) m = max(m, part[slot * kWarps + i]);
    }
    const i8::RowScale rs = i8::row_scale<true>(__uint_as_float(m << 16));
    if (!live) return;
    uint2 *q = reinterpret_cast<uint2 *>(a.q + row * a.K);
    if (rs.pre != 1.f) {  // zero, tiny or not finite (where 0 * v would be NaN)
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = tc::unpack_bf16(w[e]);
                w[e] = rs.pre == 0.f ? 0u : tc::pack_bf16(f.x * rs.pre, f.y * rs.pre);
            }
            v[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        if (t + j * TPR < nv) {
            const float2 f0 = tc::unpack_bf16(v[j].x), f1 = tc::unpack_bf16(v[j].y), f2 = tc::unpack_bf16(v[j].z),
                         f3 = tc::unpack_bf16(v[j].w);
            q[t + j * TPR] = make_uint2(i8::codes4(f0, f1, rs.mul), i8::codes4(f2, f3, rs.mul));
        }
    }
    if (t == 0) a.scale[row] = rs.scale;
}

template <int TPR, int VPL> void launch(const QuantArgs &a, cudaStream_t s)
{
    constexpr int kRows = kQThreads / TPR;
    quant_rows_kernel<TPR, VPL><<<(unsigned)((a.M + (int64_t)kRows - 1) / kRows), kQThreads, 0, s>>>(a);
}

constexpr int kQMaxK = 8 * 256 * 10;

}  // namespace

bool quant_rows_supported(const QuantArgs &a) { return a.M > 0 && a.K > 0 && a.K % 8 == 0 && a.K <= kQMaxK; }

cudaError_t launch_quant_rows(const QuantArgs &a, cudaStream_t s)
{
    Phase ph(MATE_PHASE_QUANT_ROWS, s);
    const int nv = a.K / 8;
    if (nv <= 32 * 5)
        launch<32, 5>(a, s);
    else if (nv <= 32 * 10)
        launch<32, 10>(a, s);
    else if (nv <= 128 * 5)
        launch<128, 5>(a, s);
    else if (nv <= 128 * 10)
        launch<128, 10>(a, s);
    else
        launch<256, 10>(a, s);
    return cudaGetLastError();
}

}  // namespace mate
