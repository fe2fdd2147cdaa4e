// 8-bit linear layer on the 5th-generation tensor cores: a product of signed 8-bit
// codes with a scale per token and a scale per output channel,
//     out_mn = s_m t_n sum_k x_mk w_nk (+ bias_n) (+ addend_mn).
// The sum is exact: kind::i8 accumulates in int32, and K <= 131,072 keeps
// 127 * 127 * K below 2^31. The two scales, the bias and the addend are applied to it
// in fp32 in the epilogue, and the result is rounded once to the output type.
//
// Persistent, one CTA per SM, 192 threads, in the manner of the bf16 composition GEMM
// with rows of 128 codes in place of 64 bf16 values:
//   warp 0    TMA loads of 128 x 128 x-tiles and 256 x 128 w-tiles into a 4-stage
//             ring (48 KB per stage, 128-byte swizzle, K-major; codes past K, M or N
//             load as zeros);
//   warp 1    TMEM allocation and tcgen05.mma issue: per output tile of 128 x 256,
//             four M = 128, N = 256, K = 32 MMAs per stage into one of two TMEM
//             accumulators, so that a tile's epilogue runs while the next accumulates;
//   warps 2-5 the epilogue: TMEM -> registers -> scales, bias, addend -> a staging tile
//             of 128 rows x 128 bytes in the 128-byte swizzle (two, alternating) -> TMA
//             store.
//
// Every wait is bounded (2 s); a wait that gives up records MATE_ERR_TIMEOUT and
// raises a CTA abort flag that makes every role leave its loop; the CTA then
// waits (bounded) for its copies and MMAs in flight and frees its TMEM.
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tmap.h"

#include <algorithm>

namespace mate {

namespace {

constexpr int kBM = 128, kBN = 256, kBK = 128;  // a K step is 128 codes = one swizzled row
constexpr int kStages = 4;
constexpr uint32_t kATile = kBM * kBK;               // 16 KB
constexpr uint32_t kBTile = kBN * kBK;               // 32 KB
constexpr uint32_t kStage = kATile + kBTile;         // 48 KB
constexpr uint32_t kOutTile = kBM * 128;             // 16 KB: 128 rows x 128 bytes
constexpr uint32_t kOffStages = 0;
constexpr uint32_t kOffOut = kStages * kStage;       // 2 staging tiles
constexpr uint32_t kOffBar = kOffOut + 2 * kOutTile;
// full[4], empty[4], acc_full[2], acc_empty[2], drain; then the TMEM slot and the abort flag
constexpr int kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccEmpty = 2 * kStages + 2,
              kBarDrain = 2 * kStages + 4, kNumBars = 2 * kStages + 5;
constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "linear_i8: shared memory");
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxK = 131072;

struct Geo {
    int M, N, nk;        // rows, columns, 128-wide K steps
    int tiles_n, tiles;  // output tiles along N, in total
    const float *x_scale, *w_scale, *bias;
    const void *addend;
};

// eight (bf16) or four (fp32) outputs of one 16-byte chunk: columns n .. of row m
template <bool F32>
__device__ __forceinline__ uint4 finish(const uint32_t *acc, float xs, int m, int n, bool live, const Geo &geo)
{
    constexpr int kCols = F32 ? 4 : 8;
    float v[kCols];
#pragma unroll
    for (int q = 0; q < kCols / 4; ++q) {
        const float4 ws = *reinterpret_cast<const float4 *>(geo.w_scale + n + 4 * q);
        v[4 * q] = (float)(int)acc[4 * q] * xs * ws.x;
        v[4 * q + 1] = (float)(int)acc[4 * q + 1] * xs * ws.y;
        v[4 * q + 2] = (float)(int)acc[4 * q + 2] * xs * ws.z;
        v[4 * q + 3] = (float)(int)acc[4 * q + 3] * xs * ws.w;
        if (geo.bias) {
            const float4 b = *reinterpret_cast<const float4 *>(geo.bias + n + 4 * q);
            v[4 * q] += b.x, v[4 * q + 1] += b.y, v[4 * q + 2] += b.z, v[4 * q + 3] += b.w;
        }
    }
    if (geo.addend && live) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const char *>(geo.addend) +
                                                         ((int64_t)m * geo.N + n) * (F32 ? 4 : 2));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (F32) {
                v[e] += __uint_as_float(w[e]);
            } else {
                const float2 f = tc::unpack_bf16(w[e]);
                v[2 * e % kCols] += f.x, v[(2 * e + 1) % kCols] += f.y;
            }
        }
    }
    if (F32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    return make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4 % kCols], v[5 % kCols]),
                      tc::pack_bf16(v[6 % kCols], v[7 % kCols]));
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    linear_i8_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                     const __grid_constant__ CUtensorMap mo, const __grid_constant__ Geo geo, int *err)
{
    constexpr int kOutCols = F32 ? 32 : 64;  // columns of a staging tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t *base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + kOffMisc + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bars[kBarFull + i], 1);
            tc::mbar_init(&bars[kBarEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[kBarAccFull + i], 1);
            tc::mbar_init(&bars[kBarAccEmpty + i], 128);
        }
        tc::mbar_init(&bars[kBarDrain], 1);
        tc::fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            uint32_t it = 0;  // stage fills issued
            for (int t = blockIdx.x; t < geo.tiles && !*abort_flag; t += gridDim.x) {
                const int m0 = (t / geo.tiles_n) * kBM, n0 = (t % geo.tiles_n) * kBN;
                for (int ks = 0; ks < geo.nk; ++ks, ++it) {
                    const int s = it % kStages;
                    const uint32_t round = it / kStages;
                    if (round > 0 && !tc::mbar_wait_or_abort(&bars[kBarEmpty + s], (round - 1) & 1u, err, abort_flag))
                        break;
                    uint8_t *sa = base + kOffStages + s * kStage, *sb = sa + kATile;
                    tc::mbar_expect_tx(&bars[kBarFull + s], kStage);
                    tc::tma_load_2d(sa, &ma, &bars[kBarFull + s], ks * kBK, m0);
                    tc::tma_load_2d(sb, &mb, &bars[kBarFull + s], ks * kBK, n0);
                }
            }
            // every load issued has landed before the CTA may leave (bounded)
            if (it > 0) {
                const uint32_t last = it - 1;
                tc::mbar_wait(&bars[kBarFull + last % kStages], (last / kStages) & 1u, nullptr);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issue ----------------
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_i8(kBM, kBN);
            uint32_t it = 0, tl = 0, committed = 0;
            for (int t = blockIdx.x; t < geo.tiles && !*abort_flag; t += gridDim.x, ++tl) {
                const uint32_t acc = tl & 1, use = tl >> 1;
                if (use > 0 && !tc::mbar_wait_or_abort(&bars[kBarAccEmpty + acc], (use - 1) & 1u, err, abort_flag))
                    break;
                tc::tc_fence_after();
                const uint32_t d = tmem + acc * kBN;
                bool ok = true;
                for (int ks = 0; ks < geo.nk; ++ks, ++it) {
                    const int s = it % kStages;
                    if (!tc::mbar_wait_or_abort(&bars[kBarFull + s], (it / kStages) & 1u, err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t a0 = tc::smem_u32(base + kOffStages + s * kStage), b0 = a0 + kATile;
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        tc::mma_i8(d, tc::sdesc_sw128(a0 + kk * 32, 16, 1024), tc::sdesc_sw128(b0 + kk * 32, 16, 1024),
                                   idesc, ks > 0 || kk > 0);
                    tc::mma_commit(&bars[kBarEmpty + s]);  // the stage is free once these MMAs are done
                    ++committed;
                }
                if (!ok) break;
                tc::mma_commit(&bars[kBarAccFull + acc]);
            }
            // every MMA issued has completed before TMEM may be freed (bounded)
            if (committed > 0) {
                tc::mma_commit(&bars[kBarDrain]);
                tc::mbar_wait(&bars[kBarDrain], 0, nullptr);
            }
        }
    } else {
        // ---------------- epilogue: warps 2-5, TMEM lanes 32 (warp % 4) .. ----------------
        const int et = tid - 64;                        // 0..127
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
        const int row = (int)lane_base + lane;          // output row of the tile
        uint32_t tl = 0, chunks = 0;                    // tiles and staging tiles stored
        for (int t = blockIdx.x; t < geo.tiles; t += gridDim.x, ++tl) {
            const uint32_t acc = tl & 1, use = tl >> 1;
            if (!tc::mbar_wait_sleep(&bars[kBarAccFull + acc], use & 1u, err, abort_flag)) break;
            tc::tc_fence_after();
            const int m0 = (t / geo.tiles_n) * kBM, n0 = (t % geo.tiles_n) * kBN;
            const bool live = m0 + row < geo.M;
            const float xs = live ? geo.x_scale[m0 + row] : 0.f;
            for (int c = 0; c < kBN / kOutCols && n0 + kOutCols * c < geo.N; ++c, ++chunks) {
                uint32_t v[kOutCols / 32][32];
#pragma unroll
                for (int q = 0; q < kOutCols / 32; ++q)
                    tc::tmem_ld32u(tc::tmem_addr(tmem + acc * kBN, lane_base, kOutCols * c + 32 * q), v[q]);
                tc::tmem_wait_ld();
                // the store that read this staging tile two chunks ago is done with it
                if (et == 0) tc::bulk_wait_read<1>();
                tc::named_sync(1, 128);
                uint8_t *stg = base + kOffOut + (chunks & 1) * kOutTile;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int n = n0 + kOutCols * c + q * (kOutCols / 8);
                    // N is a multiple of 8: a 16-byte chunk is inside or outside as a whole
                    if (n < geo.N)
                        *reinterpret_cast<uint4 *>(stg + tc::sw128(row, q)) =
                            finish<F32>(&v[q * (kOutCols / 8) / 32][q * (kOutCols / 8) % 32], xs, m0 + row, n, live, geo);
                }
                tc::fence_proxy_async_smem();
                tc::named_sync(1, 128);
                if (et == 0) {
                    // rows past M and columns past N fall outside the tensor and are not written
                    tc::tma_store_2d(&mo, stg, n0 + kOutCols * c, m0);
                    tc::bulk_commit();
                }
            }
            // this accumulator may be overwritten by the tile after next
            tc::tc_fence_before();
            tc::mbar_arrive(&bars[kBarAccEmpty + acc]);
        }
        if (et == 0) tc::bulk_wait_all();
    }

    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

// Rows of codes are 16-byte aligned (K a multiple of 16) and so are rows of outputs;
// output tiles fit 32-bit counters.
bool linear_i8_supported(const LinearI8Args &a)
{
    return a.M > 0 && a.N > 0 && a.K > 0 && a.K % 16 == 0 && a.K <= kMaxK && a.N % 8 == 0 &&
           ((int64_t)a.M + kBM) * ((int64_t)a.N + kBN) / (kBM * kBN) < ((int64_t)1 << 30);
}

cudaError_t launch_linear_i8(const LinearI8Args &a, cudaStream_t s)
{
    auto kernel = a.out_f32 ? linear_i8_kernel<true> : linear_i8_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    if (!tmap_available()) return cudaErrorNotSupported;
    CUtensorMap ma, mb, mo;
    if (!tmap_2d(&ma, TmapType::u8, a.x, a.K, a.M, kBK, kBM) || !tmap_2d(&mb, TmapType::u8, a.w, a.K, a.N, kBK, kBN) ||
        !tmap_2d(&mo, a.out_f32 ? TmapType::f32 : TmapType::bf16, a.out, a.N, a.M, a.out_f32 ? 32 : 64, kBM))
        return cudaErrorInvalidValue;
    Geo geo;
    geo.M = a.M;
    geo.N = a.N;
    geo.nk = (a.K + kBK - 1) / kBK;
    geo.tiles_n = (a.N + kBN - 1) / kBN;
    geo.tiles = (int)(((int64_t)a.M + kBM - 1) / kBM) * geo.tiles_n;
    geo.x_scale = a.x_scale;
    geo.w_scale = a.w_scale;
    geo.bias = a.bias;
    geo.addend = a.addend;
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    const int grid = std::min(geo.tiles, std::max(nsm, 1));
    Phase ph(a.phase ? a.phase : MATE_PHASE_LINEAR_I8, s);
    kernel<<<grid, kThreads, kSmemBytes, s>>>(ma, mb, mo, geo, a.err);
    return cudaGetLastError();
}

}  // namespace mate
