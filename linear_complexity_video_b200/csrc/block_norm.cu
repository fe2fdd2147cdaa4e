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

constexpr int kBnMaxC = 8192;

// sums over the TPR threads of a row; `turn` counts the calls of the kernel (the
// partial sums alternate between two buffers, so one barrier per call is enough)
template <int TPR, int ROWS> struct RowReduce {
    float *part;  // [2][ROWS * TPR / 32]
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
        float *p = part + (turn & 1) * (ROWS * TPR / 32) + slot * (TPR / 32);
        ++turn;
        if ((threadIdx.x & 31) == 0) p[(threadIdx.x % TPR) / 32] = v;
        tc::named_sync(1 + slot, TPR);
        return p;
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void unpack8(const uint4 &u, float2 (&f)[4])
{
    f[0] = tc::unpack_bf16(u.x), f[1] = tc::unpack_bf16(u.y), f[2] = tc::unpack_bf16(u.z), f[3] = tc::unpack_bf16(u.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4])
{
    return make_uint4(tc::pack_bf16(f[0].x, f[0].y), tc::pack_bf16(f[1].x, f[1].y), tc::pack_bf16(f[2].x, f[2].y),
                      tc::pack_bf16(f[3].x, f[3].y));
}

__device__ __forceinline__ void load8(const float4 *plane, int nv, int v, float2 (&f)[4])
{
    const float4 a = plane[v], b = plane[nv + v];
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ float4 all4(float v) { return make_float4(v, v, v, v); }

__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }

// four floats of a vector that may start at any of them
__device__ __forceinline__ float4 load4(const float *p)
{
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) return *reinterpret_cast<const float4 *>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}

// TPR threads per row, up to VPL vectors of eight channels per thread. LAYER: one of the
// norms is a layer norm (without, no mean is taken or subtracted). The arithmetic runs on
// packed fp32 pairs: unpacked, the kernel was bound by its issue slots (66% issued, with
// two CTAs of 128 registers per thread on an SM).
template <int TPR, int ROWS, int VPL, int CTAS, bool XF32, bool LAYER>
__global__ void __launch_bounds__(TPR *ROWS, CTAS) block_norm_kernel(BlockNormArgs a, int blocks_per_item, int rows_per_block)
{
    extern __shared__ float4 coef[];
    __shared__ float part[2 * (ROWS * TPR / 32)];
    const int nv = a.C / 8;
    float4 *cg = coef, *ca = coef + 2 * nv, *cs = coef + 4 * nv;
    const int b = blockIdx.x / blocks_per_item, r0 = (blockIdx.x - b * blocks_per_item) * rows_per_block;
    const int r1 = min(a.n, r0 + rows_per_block);
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;

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
    auto unpack_x = [&](int j, float2 (&f)[4]) {
        if (XF32) {
            const uint4 p = xv[2 * j], q = xv[XF32 ? 2 * j + 1 : 0];
            f[0] = make_float2(__uint_as_float(p.x), __uint_as_float(p.y));
            f[1] = make_float2(__uint_as_float(p.z), __uint_as_float(p.w));
            f[2] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
            f[3] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
        } else {
            unpack8(xv[j], f);
        }
    };
    tc::stream_release();  // a product behind it may set itself up
    if (r0 + slot < r1) load(r0 + slot);
    {
        const float *gate = a.gate + (int64_t)b * a.gate_stride, *scale = a.scale + (int64_t)b * a.scale_stride,
                    *shift = a.shift + (int64_t)b * a.shift_stride;  // used where given
        // four channels at a time: half of a thread's eight, in one plane
        for (int q = threadIdx.x; q < 2 * nv; q += TPR * ROWS) {
            const int at = (q & 1) * nv + (q >> 1);
            if (a.y) cg[at] = mul4(a.gate ? load4(gate + 4 * q) : all4(1.f), a.w_post ? load4(a.w_post + 4 * q) : all4(1.f));
            if (a.h) {
                const float4 s = a.scale ? load4(scale + 4 * q) : all4(0.f);
                ca[at] = mul4(a.w_pre ? load4(a.w_pre + 4 * q) : all4(1.f),
                              make_float4(1.f + s.x, 1.f + s.y, 1.f + s.z, 1.f + s.w));
                cs[at] = a.shift ? load4(shift + 4 * q) : all4(0.f);
            }
        }
    }
    __syncthreads();
    RowReduce<TPR, ROWS> red{part, slot};
    const float inv_c = 1.f / (float)a.C;

    for (int i = r0 + slot; i < r1; i += ROWS) {
        const int64_t row = (int64_t)b * a.n + i, at = row * a.C;
        float2 r[VPL][4];
        if (a.y) {
            float mu = 0.f, rs = 1.f;
            if (LAYER && a.post == MATE_NORM_LAYER) {
                float2 s = both(0.f);
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    float2 f[4];
                    unpack8(yv[j], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s = tc::add_f32x2(s, f[e]);
                }
                mu = red.sum(s.x + s.y) * inv_c;
            }
            if (a.post != MATE_NORM_NONE) {
                float2 s = both(0.f);
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    float2 f[4];
                    unpack8(yv[j], f);
                    if (!LAYER || t + j * TPR < nv) {  // channels past the row are zeros
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (LAYER) f[e] = tc::add_f32x2(f[e], both(-mu));
                            s = tc::fma_f32x2(f[e], f[e], s);
                        }
                    }
                }
                rs = rsqrtf(red.sum(s.x + s.y) * inv_c + a.eps);
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = t + j * TPR;
                if (v < nv) {
                    float2 f[4], g[4];
                    unpack8(yv[j], f);
                    load8(cg, nv, v, g);
                    unpack_x(j, r[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (LAYER) f[e] = tc::add_f32x2(f[e], both(-mu));
                        r[j][e] = tc::fma_f32x2(tc::mul_f32x2(f[e], both(rs)), g[e], tc::mul_f32x2(r[j][e], both(a.alpha)));
                    }
                    if (XF32) {
                        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.x_out) + at) + 2 * v;
                        o[0] = make_float4(r[j][0].x, r[j][0].y, r[j][1].x, r[j][1].y);
                        o[1] = make_float4(r[j][2].x, r[j][2].y, r[j][3].x, r[j][3].y);
                    } else {
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.x_out) + at)[v] = pack8(r[j]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[j][e] = both(0.f);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) unpack_x(j, r[j]);
        }
        // the packed row is used up: the next one's loads run under the rest of this one
        if (i + ROWS < r1) load(i + ROWS);
        if (!a.h) continue;
        float mu = 0.f;
        if (LAYER && a.pre == MATE_NORM_LAYER) {
            float2 s = both(0.f);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = tc::add_f32x2(s, r[j][e]);
            mu = red.sum(s.x + s.y) * inv_c;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (t + j * TPR < nv) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[j][e] = tc::add_f32x2(r[j][e], both(-mu));
                }
        }
        float2 s = both(0.f);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = tc::fma_f32x2(r[j][e], r[j][e], s);
        const float rs = rsqrtf(red.sum(s.x + s.y) * inv_c + a.eps);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * TPR;
            if (v < nv) {
                float2 w[4], sh[4];
                load8(ca, nv, v, w);
                load8(cs, nv, v, sh);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[j][e] = tc::fma_f32x2(tc::mul_f32x2(r[j][e], both(rs)), w[e], sh[e]);
                if (a.h_type == MATE_BF16) {
                    reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.h) + at)[v] = pack8(r[j]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = i8::amax_nan(m, r[j][e]);
                }
            }
        }
        if (a.h_type != MATE_I8) continue;
        const i8::RowScale q = i8::row_scale<false>(red.max(m));
        uint2 *o = reinterpret_cast<uint2 *>(static_cast<int8_t *>(a.h) + at);
        if (q.pre != 1.f) {  // zero, tiny or not finite (where 0 * v would be NaN)
#pragma unroll
            for (int j = 0; j < VPL; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) r[j][e] = q.pre == 0.f ? both(0.f) : tc::mul_f32x2(r[j][e], both(q.pre));
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * TPR;
            if (v < nv) o[v] = make_uint2(i8::codes4(r[j][0], r[j][1], q.mul), i8::codes4(r[j][2], r[j][3], q.mul));
        }
        if (t == 0) a.h_scale[row] = q.scale;
    }
}

template <int TPR, int ROWS, int VPL, int CTAS, bool XF32, bool LAYER>
cudaError_t launch(const BlockNormArgs &a, cudaStream_t s)
{
    auto kernel = block_norm_kernel<TPR, ROWS, VPL, CTAS, XF32, LAYER>;
    const size_t smem = (size_t)a.C * 12;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBnMaxC * 12);
    if (e != cudaSuccess) return e;
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    // one wave of CTAs, each with its share of one batch element's rows
    int per_item = std::max(1, std::min((a.n + ROWS - 1) / ROWS, CTAS * nsm / a.batch));
    const int rows = (a.n + per_item - 1) / per_item;
    per_item = (a.n + rows - 1) / rows;
    kernel<<<(unsigned)(per_item * (int64_t)a.batch), TPR * ROWS, smem, s>>>(a, per_item, rows);
    return cudaGetLastError();
}

template <bool XF32, bool LAYER> cudaError_t dispatch(const BlockNormArgs &a, cudaStream_t s)
{
    const int nv = a.C / 8;
    // Measured at 131,072 x 2,560 (after + before, 8-bit h; layer norm with bf16 h): two rows per CTA,
    // five vectors per thread and three CTAs per SM 383 and 438 us; four rows and two CTAs (128
    // registers, spills) 418 and 549; five warps per row and two vectors 437 and 549; a warp per
    // row and ten vectors 411 and 474. fp32 rows take twice the registers: four warps per row and
    // three vectors 654 us against 680 of two warps and five.
    if constexpr (XF32) {
        if (nv <= 32 * 3) return launch<32, 8, 3, 2, XF32, LAYER>(a, s);
        if (nv <= 64 * 3) return launch<64, 4, 3, 2, XF32, LAYER>(a, s);
        if (nv <= 128 * 3) return launch<128, 2, 3, 2, XF32, LAYER>(a, s);
    } else {
        if (nv <= 32 * 5) return launch<32, 4, 5, 3, XF32, LAYER>(a, s);
        if (nv <= 64 * 5) return launch<64, 2, 5, 3, XF32, LAYER>(a, s);
        if (nv <= 128 * 5) return launch<128, 1, 5, 3, XF32, LAYER>(a, s);
    }
    return launch<256, 1, 4, 2, XF32, LAYER>(a, s);
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
    const bool layer = (a.y && a.post == MATE_NORM_LAYER) || (a.h && a.pre == MATE_NORM_LAYER);
    if (layer) return a.x_f32 ? dispatch<true, true>(a, s) : dispatch<false, true>(a, s);
    return a.x_f32 ? dispatch<true, false>(a, s) : dispatch<false, false>(a, s);
}

}  // namespace mate
