// MA-branch output side: the bi-SSD output y gated by the front-end's z and
// RMS-normalised per group of channels (paper review "LinGen ...", section 三,
// MA-Branch item 1: the branch is a bidirectional Mamba2 block; the pages name
// the block and no more of it, so this is the standard Mamba2 gated norm, gate
// first):
//     v_k   = y_k SiLU(z_k)
//     out_k = v_k w_k / sqrt(mean_{k in group} v_k^2 + eps)
// Its output is the MA-branch's input to the MATE composition.
//
// HBM-bound (y and z read once, out written once: 6 bytes per channel in bf16).
// One CTA of 128 threads per token row: thread t holds the 16-byte vectors
// t, t + 128, ... of the row (eight channels each, all loads in flight at once),
// so that every load and store instruction of a warp covers 512 contiguous bytes.
// The sums of squares go per vector to shared memory, warp w reduces groups
// w, w + 4, ... there, and each thread scales its vectors by its groups' factors.
#include "common.cuh"
#include "i8.cuh"
#include "kernels.h"
#include "tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace mate {

namespace {

constexpr int kGnThreads = 128;
constexpr int kGnMaxVec = 8;  // vectors per thread: rows of up to 8 x 8 x 128 = 8192 channels

// SiLU(v) = v / (1 + e^-v) with the fast exponential and divide (relative error
// far below the bf16 rounding of the result, for either sign of v)
__device__ __forceinline__ float silu_fast(float v) { return __fdividef(v, 1.f + __expf(-v)); }

__global__ void __launch_bounds__(kGnThreads) gate_norm_kernel(GateNormArgs a)
{
    __shared__ float ss_vec[kGnMaxVec * kGnThreads];  // sum of squares of each vector of the row
    __shared__ float scale[kGnMaxVec * kGnThreads];   // 1 / rms of each group (at most one per vector)
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int nv = a.C / 8, gv = a.group / 8, ng = a.C / a.group;  // vectors per row, per group; groups
    const size_t row = (size_t)blockIdx.x * a.C;
    const uint4 *y = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.y) + row);
    const uint4 *z = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.z) + row);
    uint4 yv[kGnMaxVec], zv[kGnMaxVec];
#pragma unroll
    for (int j = 0; j < kGnMaxVec; ++j) {
        const int v = t + j * kGnThreads;
        if (v < nv) {
            yv[j] = y[v];
            zv[j] = z[v];
        }
    }
    float g[kGnMaxVec][8];  // the gated values
#pragma unroll
    for (int j = 0; j < kGnMaxVec; ++j) {
        const int v = t + j * kGnThreads;
        if (v < nv) {
            const uint32_t yw[4] = {yv[j].x, yv[j].y, yv[j].z, yv[j].w};
            const uint32_t zw[4] = {zv[j].x, zv[j].y, zv[j].z, zv[j].w};
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 yf = tc::unpack_bf16(yw[e]), zf = tc::unpack_bf16(zw[e]);
                g[j][2 * e] = yf.x * silu_fast(zf.x);
                g[j][2 * e + 1] = yf.y * silu_fast(zf.y);
                s = fmaf(g[j][2 * e], g[j][2 * e], s);
                s = fmaf(g[j][2 * e + 1], g[j][2 * e + 1], s);
            }
            ss_vec[v] = s;
        }
    }
    __syncthreads();
    for (int gi = warp; gi < ng; gi += kGnThreads / 32) {
        float s = 0.f;
        for (int v = gi * gv + lane; v < (gi + 1) * gv; v += 32) s += ss_vec[v];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) scale[gi] = rsqrtf(s / (float)a.group + a.eps);
    }
    __syncthreads();
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row);
    const float4 *w4 = reinterpret_cast<const float4 *>(a.w);
#pragma unroll
    for (int j = 0; j < kGnMaxVec; ++j) {
        const int v = t + j * kGnThreads;
        if (v < nv) {
            const float f = scale[v / gv];
            const float4 wa = w4[2 * v], wb = w4[2 * v + 1];
            const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = tc::pack_bf16(g[j][2 * e] * f * wv[2 * e], g[j][2 * e + 1] * f * wv[2 * e + 1]);
            out[v] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// The same values as 8-bit codes and one scale per row (i8.cuh). The row's largest magnitude
// is a second reduction between the loads and the stores of a row, so a CTA keeps the next
// row's loads in flight meanwhile: persistent CTAs, and the packed vectors of a row are used
// up before its sums are.

// y SiLU(z) on pairs: y (z / (1 + 2^(-z log2 e))), each exponential and reciprocal one
// hardware approximation (2 and 1 fp32 steps). In this order a large y meets a gate that has
// gone to zero, not the infinity of y z.
__device__ __forceinline__ float2 gated(float2 y, float2 z)
{
    const float2 x = tc::mul_f32x2(z, make_float2(-1.44269504f, -1.44269504f));
    const float2 d = tc::add_f32x2(make_float2(tc::ex2_approx(x.x), tc::ex2_approx(x.y)), make_float2(1.f, 1.f));
    return tc::mul_f32x2(y, tc::mul_f32x2(z, make_float2(tc::rcp_approx(d.x), tc::rcp_approx(d.y))));
}

// ONE: the row is one group, whose sum needs one barrier instead of two.
template <int VPL, bool ONE>
__global__ void __launch_bounds__(kGnThreads, VPL <= 2 ? 6 : VPL <= 5 ? 4 : 2) gate_norm_i8_kernel(GateNormArgs a)
{
    __shared__ float ss_vec[ONE ? kGnThreads / 32 : VPL * kGnThreads];  // of each vector, or of each warp
    __shared__ float scale[ONE ? 1 : VPL * kGnThreads];
    __shared__ uint32_t amax[kGnThreads / 32];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int nv = a.C / 8, gv = a.group / 8, ng = a.C / a.group;
    uint4 yv[VPL], zv[VPL];
    auto load = [&](int64_t r) {
        const uint4 *y = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.y) + r * a.C);
        const uint4 *z = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.z) + r * a.C);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * kGnThreads;
            yv[j] = v < nv ? __ldcs(y + v) : make_uint4(0, 0, 0, 0);
            zv[j] = v < nv ? __ldcs(z + v) : make_uint4(0, 0, 0, 0);
        }
    };
    tc::stream_release();  // a product behind it may set itself up
    load(blockIdx.x);
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        float2 g[VPL][4];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const uint32_t yw[4] = {yv[j].x, yv[j].y, yv[j].z, yv[j].w};
            const uint32_t zw[4] = {zv[j].x, zv[j].y, zv[j].z, zv[j].w};
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[j][e] = gated(tc::unpack_bf16(yw[e]), tc::unpack_bf16(zw[e]));
                s = tc::fma_f32x2(g[j][e], g[j][e], s);
            }
            if (ONE)
                ss += s.x + s.y;  // vectors past the row are zeros
            else if (t + j * kGnThreads < nv)
                ss_vec[t + j * kGnThreads] = s.x + s.y;
        }
        if (r + gridDim.x < a.M) load(r + gridDim.x);
        float one = 0.f;
        if (ONE) {
            ss = warp_sum(ss);
            if (lane == 0) ss_vec[warp] = ss;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kGnThreads / 32; ++i) one += ss_vec[i];
            one = rsqrtf(one / (float)a.C + a.eps);
        } else {
            __syncthreads();
            for (int gi = warp; gi < ng; gi += kGnThreads / 32) {
                float s = 0.f;
                for (int v = gi * gv + lane; v < (gi + 1) * gv; v += 32) s += ss_vec[v];
                s = warp_sum(s);
                if (lane == 0) scale[gi] = rsqrtf(s / (float)a.group + a.eps);
            }
            __syncthreads();
        }
        const float4 *w4 = reinterpret_cast<const float4 *>(a.w);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * kGnThreads;
            if (v < nv) {
                const float f = ONE ? one : scale[v / gv];
                const float4 wa = w4[2 * v], wb = w4[2 * v + 1];
                const float2 wv[4] = {make_float2(wa.x, wa.y), make_float2(wa.z, wa.w), make_float2(wb.x, wb.y),
                                      make_float2(wb.z, wb.w)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[j][e] = tc::mul_f32x2(tc::mul_f32x2(g[j][e], make_float2(f, f)), wv[e]);
                    m = i8::amax_nan(m, g[j][e]);
                }
            }
        }
        uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) amax[warp] = mb;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kGnThreads / 32; ++i) mb = max(mb, amax[i]);
        const i8::RowScale rs = i8::row_scale<false>(__uint_as_float(mb));
        uint2 *q = reinterpret_cast<uint2 *>(a.q + r * a.C);
        if (rs.pre != 1.f) {  // zero, tiny or not finite (where 0 * v would be NaN)
#pragma unroll
            for (int j = 0; j < VPL; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    g[j][e] = rs.pre == 0.f ? make_float2(0.f, 0.f) : tc::mul_f32x2(g[j][e], make_float2(rs.pre, rs.pre));
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int v = t + j * kGnThreads;
            if (v < nv) q[v] = make_uint2(i8::codes4(g[j][0], g[j][1], rs.mul), i8::codes4(g[j][2], g[j][3], rs.mul));
        }
        if (t == 0) a.scale[r] = rs.scale;
    }
}

template <int VPL> cudaError_t launch_i8(const GateNormArgs &a, cudaStream_t s)
{
    auto kernel = a.group == a.C ? gate_norm_i8_kernel<VPL, true> : gate_norm_i8_kernel<VPL, false>;
    int dev = 0, nsm = 148, per_sm = 4;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kGnThreads, 0);
    kernel<<<std::min(a.M, std::max(1, nsm * per_sm)), kGnThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

bool gate_norm_supported(const GateNormArgs &a)
{
    return a.M > 0 && a.C > 0 && a.group > 0 && a.C % a.group == 0 && a.group % 8 == 0 &&
           a.C <= 8 * kGnMaxVec * kGnThreads;
}

cudaError_t launch_gate_norm(const GateNormArgs &a, cudaStream_t s)
{
    Phase ph(MATE_PHASE_GATE_NORM, s);
    if (a.q) {
        const int nv = a.C / 8;
        return nv <= 2 * kGnThreads ? launch_i8<2>(a, s) : nv <= 5 * kGnThreads ? launch_i8<5>(a, s) : launch_i8<kGnMaxVec>(a, s);
    }
    gate_norm_kernel<<<a.M, kGnThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mate
