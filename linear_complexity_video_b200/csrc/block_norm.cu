// The norms before and after a block, with its modulation, gate and residual scale
// (adaLN form: gate, scale and shift are vectors per batch element):
//     r = alpha x + gate_b * (N(y) w_post)       the residual stream after the block
//     h = N(r) w_pre (1 + scale_b) + shift_b     the next block's input
// N(v) = v / sqrt(mean v^2 + eps) (RMS) or (v - mean v) / sqrt(var v + eps) (layer),
// or N(y) = y. Either half may be left out; h is bf16 or 8-bit codes with a scale per
// row (i8.cuh). h follows the fp32 r, not r as rounded for storage: one rounding per
// output.
//
// HBM-bound: x and y read once, r and h written once. A row stays in the registers of
// its threads (a warp's, where it fits: the sums are then shuffles and no barrier)
// from its loads to its stores. Both statistics of a layer norm are taken from the
// registers in turn (mean, then the squares about it), so nothing cancels. Rows of
// one batch element share three vectors, gate w_post, w_pre (1 + scale) and shift;
// a CTA forms them once in shared memory and walks a contiguous range of the
// element's rows. They are kept as two planes of float4 (a thread's eight channels are
// two of them), so that a warp's reads touch every bank once.
#include "common.cuh"
#include "i8.cuh"
#include "kernels.h"
#include "tc.cuh"

#include <algorithm>

namespace mate {

namespace {

constexpr int kBnThreads = 256;
constexpr int kBnMaxC = 8192;

// sums over the TPR threads of a row; `turn` counts the calls of the kernel (the
// partial sums alternate between two buffers, so one barrier per call is enough)
template <int TPR> struct RowReduce {
    float *part;  // [2][kBnThreads / 32]
    int slot, turn = 0;

    __device__ __forceinline__ float sum(float v)
    {
        v = warp_sum(v);
        if (TPR > 32) {
            float *p = buffer(v);
            v = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) v += p[i];
        }
        return v;
    }
    // largest of non-negative values (or NaN, whose bits order last)
    __device__ __forceinline__ float max(float v)
    {
        v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
        if (TPR > 32) {
            float *p = buffer(v);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) m = ::max(m, __float_as_uint(p[i]));
            v = __uint_as_float(m);
        }
        return v;
    }
    __device__ __forceinline__ float *buffer(float v)
    {
        float *p = part + (turn & 1) * (kBnThreads / 32) + slot * (TPR / 32);
        ++turn;
        if ((threadIdx.x & 31) == 0) p[(threadIdx.x % TPR) / 32] = v;
        tc::named_sync(1 + slot, TPR);
        return p;
    }
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const float2 a = tc::unpack_bf16(u.x), b = tc::unpack_bf16(u.y), c = tc::unpack_bf16(u.z), d = tc::unpack_bf16(u.w);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}

__device__ __forceinline__ void load8(const float4 *plane, int nv, int v, float (&f)[8])
{
    const float4 a = plane[v], b = plane[nv + v];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// TPR threads per row, up to VPL vectors of eight channels per thread
template <int TPR, int VPL, bool XF32>
__global__ void __launch_bounds__(kBnThreads, 2) block_norm_kernel(BlockNormArgs a, int blocks_per_item, int rows_per_block)
{
    constexpr int kRows = kBnThreads / TPR;
    extern __shared__ float4 coef[];
    __shared__ float part[2 * (kBnThreads / 32)];
    const int nv = a.C / 8;
    float4 *cg = coef, *ca = coef + 2 * nv, *cs = coef + 4 * nv;
    const int b = blockIdx.x / blocks_per_item, r0 = (blockIdx.x - b * blocks_per_item) * rows_per_block;
    const int r1 = min(a.n, r0 + rows_per_block);
    {
        const int64_t m = (int64_t)b * a.mod_stride;
        float *g = reinterpret_cast<float *>(cg), *w = reinterpret_cast<float *>(ca), *s = reinterpret_cast<float *>(cs);
        for (int c = threadIdx.x; c < a.C; c += kBnThreads) {
            const int at = ((c >> 2 & 1) * nv + (c >> 3)) * 4 + (c & 3);
            if (a.y) g[at] = (a.gate ? a.gate[m + c] : 1.f) * (a.w_post ? a.w_post[c] : 1.f);
            if (a.h) {
                w[at] = (a.w_pre ? a.w_pre[c] : 1.f) * (a.scale ? 1.f + a.scale[m + c] : 1.f);
                s[at] = a.shift ? a.shift[m + c] : 0.f;
            }
        }
    }
    __syncthreads();
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    RowReduce<TPR> red{part, slot};
    const float inv_c = 1.f / (float)a.C;

    uint4 yv[VPL], xv[XF32 ? 2 * VPL : VPL];
    auto load = [&](int i) {
        const int64_t at = ((int64_t)b * a.n + i) * a.C;
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) + at * (XF32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * TPR;
            if (XF32) {
                xv[2 * j] = v < nv ? __ldcs(x + 2 * v) : make_uint4(0, 0, 0, 0);
                xv[XF32 ? 2 * j + 1 : 0] = v < nv ? __ldcs(x + 2 * v + 1) : make_uint4(0, 0, 0, 0);
            } else {
                xv[j] = v < nv ? __ldcs(x + v) : make_uint4(0, 0, 0, 0);
            }
        }
        if (a.y) {
            const uint4 *y = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.y) + at);
#pragma unroll
            for (int j = 0; j < VPL; ++j) yv[j] = t + j * TPR < nv ? __ldcs(y + t + j * TPR) : make_uint4(0, 0, 0, 0);
        }
    };
    auto unpack_x = [&](int j, float (&f)[8]) {
        if (XF32) {
            const uint4 p = xv[2 * j], q = xv[XF32 ? 2 * j + 1 : 0];
            f[0] = __uint_as_float(p.x), f[1] = __uint_as_float(p.y), f[2] = __uint_as_float(p.z);
            f[3] = __uint_as_float(p.w), f[4] = __uint_as_float(q.x), f[5] = __uint_as_float(q.y);
            f[6] = __uint_as_float(q.z), f[7] = __uint_as_float(q.w);
        } else {
            unpack8(xv[j], f);
        }
    };
    if (r0 + slot < r1) load(r0 + slot);
    for (int i = r0 + slot; i < r1; i += kRows) {
        const int64_t row = (int64_t)b * a.n + i, at = row * a.C;
        float r[VPL][8];
        if (a.y) {
            float mu = 0.f, rs = 1.f;
            if (a.post == MATE_NORM_LAYER) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    float f[8];
                    unpack8(yv[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s += f[e];
                }
                mu = red.sum(s) * inv_c;
            }
            if (a.post != MATE_NORM_NONE) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    float f[8];
                    unpack8(yv[j], f);
                    if (t + j * TPR < nv) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) s = fmaf(f[e] - mu, f[e] - mu, s);
                    }
                }
                rs = rsqrtf(red.sum(s) * inv_c + a.eps);
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = t + j * TPR;
                if (v < nv) {
                    float f[8], g[8];
                    unpack8(yv[j], f);
                    load8(cg, nv, v, g);
                    unpack_x(j, r[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[j][e] = fmaf((f[e] - mu) * rs, g[e], a.alpha * r[j][e]);
                    if (XF32) {
                        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.x_out) + at) + 2 * v;
                        o[0] = make_float4(r[j][0], r[j][1], r[j][2], r[j][3]);
                        o[1] = make_float4(r[j][4], r[j][5], r[j][6], r[j][7]);
                    } else {
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.x_out) + at)[v] =
                            make_uint4(tc::pack_bf16(r[j][0], r[j][1]), tc::pack_bf16(r[j][2], r[j][3]),
                                       tc::pack_bf16(r[j][4], r[j][5]), tc::pack_bf16(r[j][6], r[j][7]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[j][e] = 0.f;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) unpack_x(j, r[j]);
        }
        // the packed row is used up: the next one's loads run under the rest of this one
        if (i + kRows < r1) load(i + kRows);
        if (!a.h) continue;
        float mu = 0.f;
        if (a.pre == MATE_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += r[j][e];
            mu = red.sum(s) * inv_c;
        }
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (t + j * TPR < nv) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(r[j][e] - mu, r[j][e] - mu, s);
            }
        const float rs = rsqrtf(red.sum(s) * inv_c + a.eps);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * TPR;
            if (v < nv) {
                float w[8], sh[8];
                load8(ca, nv, v, w);
                load8(cs, nv, v, sh);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[j][e] = fmaf((r[j][e] - mu) * rs, w[e], sh[e]);
                    m = i8::amax_nan(m, r[j][e]);
                }
                if (a.h_type == MATE_BF16)
                    reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.h) + at)[v] =
                        make_uint4(tc::pack_bf16(r[j][0], r[j][1]), tc::pack_bf16(r[j][2], r[j][3]),
                                   tc::pack_bf16(r[j][4], r[j][5]), tc::pack_bf16(r[j][6], r[j][7]));
            }
        }
        if (a.h_type != MATE_I8) continue;
        const i8::RowScale q = i8::row_scale(red.max(m));
        uint2 *o = reinterpret_cast<uint2 *>(static_cast<int8_t *>(a.h) + at);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * TPR;
            if (v < nv) {
                if (q.pre != 1.f) {  // zero, tiny or not finite (where 0 * v would be NaN)
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[j][e] = q.pre == 0.f ? 0.f : r[j][e] * q.pre;
                }
                o[v] = make_uint2(i8::codes4(r[j][0], r[j][1], r[j][2], r[j][3], q.mul),
                                  i8::codes4(r[j][4], r[j][5], r[j][6], r[j][7], q.mul));
            }
        }
        if (t == 0) a.h_scale[row] = q.scale;
    }
}

template <int TPR, int VPL, bool XF32> cudaError_t launch(const BlockNormArgs &a, cudaStream_t s)
{
    constexpr int kRows = kBnThreads / TPR;
    const size_t smem = (size_t)a.C * 12;
    cudaError_t e = cudaFuncSetAttribute(block_norm_kernel<TPR, VPL, XF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBnMaxC * 12);
    if (e != cudaSuccess) return e;
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    // one wave of two CTAs per SM, each with its share of one batch element's rows
    int per_item = std::max(1, std::min((a.n + kRows - 1) / kRows, 2 * nsm / a.batch));
    const int rows = (a.n + per_item - 1) / per_item;
    per_item = (a.n + rows - 1) / rows;
    block_norm_kernel<TPR, VPL, XF32><<<(unsigned)(per_item * (int64_t)a.batch), kBnThreads, smem, s>>>(a, per_item, rows);
    return cudaGetLastError();
}

template <bool XF32> cudaError_t dispatch(const BlockNormArgs &a, cudaStream_t s)
{
    const int nv = a.C / 8;
    constexpr int kV = XF32 ? 3 : 5;  // fp32 rows take twice the registers
    if (nv <= 32 * kV) return launch<32, kV, XF32>(a, s);
    if (nv <= 64 * kV) return launch<64, kV, XF32>(a, s);
    if (nv <= 128 * kV) return launch<128, kV, XF32>(a, s);
    return launch<256, 4, XF32>(a, s);
}

}  // namespace

bool block_norm_supported(const BlockNormArgs &a)
{
    return a.batch > 0 && a.n > 0 && a.C > 0 && a.C % 8 == 0 && a.C <= kBnMaxC &&
           (int64_t)a.batch * a.n <= ((int64_t)1 << 30);  // row counters stay in 32 bits
}

cudaError_t launch_block_norm(const BlockNormArgs &a, cudaStream_t s)
{
    Phase ph(MATE_PHASE_BLOCK_NORM, s);
    return a.x_f32 ? dispatch<true>(a, s) : dispatch<false>(a, s);
}

}  // namespace mate
