// 8-bit linear layer on the 5th-generation tensor cores: a product of signed 8-bit
// codes with a scale per token and a scale per output channel,
//     out_mn = s_m t_n sum_k x_mk w_nk (+ bias_n) (+ addend_mn).
// The sum is exact: kind::i8 accumulates in int32, and K <= 131,072 keeps
// 127 * 127 * K below 2^31. The two scales, the bias and the addend are applied to it
// in fp32 in the epilogue, and the result is rounded once to the output type.
//
// Persistent CTA pairs (clusters of two, cta_group::2), 192 threads per CTA; a pair
// computes output tiles of 256 x 256, CTA r the rows 128 r ..:
//   warp 0    TMA loads of the CTA's 128 x 128 codes of x and its half, 128 x 128, of
//             the w tile into a 5-stage ring (32 KB per stage and CTA, 128-byte
//             swizzle, K-major; codes past K, M or N load as zeros), all completing on
//             the barriers of rank 0;
//   warp 1    TMEM allocation and, in rank 0, tcgen05.mma issue: four M = 256, N = 256,
//             K = 32 MMAs per stage into one of two TMEM accumulators (2 x 256 columns
//             in each CTA), so that a tile's epilogue runs while the next accumulates;
//   warps 2-5 the epilogue: TMEM -> registers -> scales, bias, addend -> a staging tile
//             of 128 rows x 128 bytes in the 128-byte swizzle (three in turn) -> TMA
//             store. The addend arrives in the staging tile by TMA, two tiles ahead; the
//             columns' scales and bias wait in shared memory, fetched a tile ahead.
// A pair reads 64 KB for the work that two single CTAs would read 96 KB for: the pair
// halves each CTA's share of w. Tiles are walked in groups of eight tile rows, so that the
// 74 pairs at work read about eight rows' x and nine columns' w.
//
// Every wait is bounded (2 s); a wait that gives up records MATE_ERR_TIMEOUT and
// raises a CTA abort flag that makes every role leave its loop; the CTA then
// waits (bounded) for its copies and MMAs in flight, meets its peer (which leaves its
// own waits by the same limit) and frees its TMEM.
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tmap.h"

#include <algorithm>

namespace mate {

namespace {

constexpr int kBM = 256, kBN = 256, kBK = 128;       // tile of a pair; a K step is 128 codes = one swizzled row
constexpr int kStages = 5, kSlots = 3;
constexpr int kGroup = 8;                            // tile rows walked together
constexpr uint32_t kTile = 128 * kBK;                // 16 KB: one CTA's part of x or w
constexpr uint32_t kStage = 2 * kTile;
constexpr uint32_t kOutTile = 128 * 128;             // 16 KB: 128 rows x 128 bytes
constexpr uint32_t kOffStages = 0;
constexpr uint32_t kOffOut = kStages * kStage;
constexpr uint32_t kOffVec = kOffOut + kSlots * kOutTile;  // w_scale and bias of the tile's columns
constexpr uint32_t kOffBar = kOffVec + 2 * kBN * 4;
// full, empty (per stage), acc_full[2], acc_empty[2], addend (per slot), drain; then the TMEM slot and the abort flag
constexpr int kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccEmpty = 2 * kStages + 2,
              kBarAdd = 2 * kStages + 4, kBarDrain = kBarAdd + kSlots, kNumBars = kBarDrain + 1;
constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "linear_i8: shared memory");
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxK = 131072;

struct Geo {
    int M, N, nk;        // rows, columns, 128-wide K steps
    int tiles_m, tiles_n, tiles;  // output tiles along M, along N, in total
    const float *x_scale, *w_scale, *bias;
    int has_addend;
};

// Tile t of the walk: groups of kGroup tile rows, columns in turn inside a group, the
// group's rows fastest.
struct Tile {
    int m, n;
};
__device__ __forceinline__ Tile tile_at(int t, const Geo &geo)
{
    const int g = t / (kGroup * geo.tiles_n), r = t - g * kGroup * geo.tiles_n;
    const int rows = min(kGroup, geo.tiles_m - g * kGroup);
    return {(g * kGroup + r % rows) * kBM, (r / rows) * kBN};
}

// eight (bf16) or four (fp32) outputs, one 16-byte chunk of a staging tile: `acc` scaled, plus
// the bias (`vec`: the columns' w_scale, their bias kBN floats on) and the addend that `stg` holds
template <bool F32>
__device__ __forceinline__ uint4 finish(const uint32_t *acc, float xs, const float *vec, const Geo &geo, const uint4 *stg)
{
    constexpr int kCols = F32 ? 4 : 8;
    float v[kCols];
#pragma unroll
    for (int q = 0; q < kCols / 4; ++q) {
        const float4 ws = *reinterpret_cast<const float4 *>(vec + 4 * q);
        v[4 * q] = (float)(int)acc[4 * q] * xs * ws.x;
        v[4 * q + 1] = (float)(int)acc[4 * q + 1] * xs * ws.y;
        v[4 * q + 2] = (float)(int)acc[4 * q + 2] * xs * ws.z;
        v[4 * q + 3] = (float)(int)acc[4 * q + 3] * xs * ws.w;
        if (geo.bias) {
            const float4 b = *reinterpret_cast<const float4 *>(vec + kBN + 4 * q);
            v[4 * q] += b.x, v[4 * q + 1] += b.y, v[4 * q + 2] += b.z, v[4 * q + 3] += b.w;
        }
    }
    if (geo.has_addend) {
        const uint4 u = *stg;
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

// The staging tiles of a pair's CTA in the order it fills them: column chunks of its tiles.
template <int OUT_COLS> struct Chunks {
    int t, c;  // tile, column chunk
    __device__ __forceinline__ void next(const Geo &geo, int step)
    {
        const int n0 = tile_at(t, geo).n;
        if (++c == kBN / OUT_COLS || n0 + OUT_COLS * c >= geo.N) c = 0, t += step;
    }
};

template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_i8_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                     const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap md,
                     const __grid_constant__ Geo geo, int *err)
{
    constexpr int kOutCols = F32 ? 32 : 64;  // columns of a staging tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t *base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + kOffMisc + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)tc::cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bars[kBarFull + i], 1);
            tc::mbar_init(&bars[kBarEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[kBarAccFull + i], 1);
            tc::mbar_init(&bars[kBarAccEmpty + i], 8);  // the epilogue warps of both CTAs
        }
        for (int i = 0; i < kSlots; ++i) tc::mbar_init(&bars[kBarAdd + i], 1);
        tc::mbar_init(&bars[kBarDrain], 1);
        tc::fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) tc::tmem_alloc_pair(tmem_slot, kTmemCols);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            uint32_t it = 0;  // stage fills issued
            for (int t = pair; t < geo.tiles && !*abort_flag; t += pairs) {
                const Tile at = tile_at(t, geo);
                const int m0 = at.m + rank * 128, n0 = at.n + rank * 128;
                for (int ks = 0; ks < geo.nk; ++ks, ++it) {
                    const int s = it % kStages;
                    const uint32_t round = it / kStages;
                    if (round > 0 && !tc::mbar_wait_or_abort(&bars[kBarEmpty + s], (round - 1) & 1u, err, abort_flag))
                        break;
                    uint8_t *sa = base + kOffStages + s * kStage, *sb = sa + kTile;
                    // both CTAs' four copies complete on rank 0's barrier
                    const uint32_t full = tc::cluster_addr(&bars[kBarFull + s], 0);
                    if (rank == 0) tc::mbar_expect_tx(&bars[kBarFull + s], 2 * kStage);
                    tc::tma_load_2d_pair(sa, &ma, full, ks * kBK, m0);
                    tc::tma_load_2d_pair(sb, &mb, full, ks * kBK, n0);
                }
            }
            // every load issued has landed before the CTA may leave (bounded; rank 0 sees both CTAs')
            if (rank == 0 && it > 0) {
                const uint32_t last = it - 1;
                tc::mbar_wait(&bars[kBarFull + last % kStages], (last / kStages) & 1u, nullptr);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issue ----------------
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = tc::idesc_i8(kBM, kBN);
            uint32_t it = 0, tl = 0, committed = 0;
            for (int t = pair; t < geo.tiles && !*abort_flag; t += pairs, ++tl) {
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
                    const uint32_t a0 = tc::smem_u32(base + kOffStages + s * kStage), b0 = a0 + kTile;
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        tc::mma_i8_pair(d, tc::sdesc_sw128(a0 + kk * 32, 16, 1024),
                                        tc::sdesc_sw128(b0 + kk * 32, 16, 1024), idesc, ks > 0 || kk > 0);
                    tc::mma_commit_pair(&bars[kBarEmpty + s]);  // the stage is free in both CTAs once these MMAs are done
                    ++committed;
                }
                if (!ok) break;
                tc::mma_commit_pair(&bars[kBarAccFull + acc]);
            }
            // every MMA issued has completed before TMEM may be freed (bounded)
            if (committed > 0) {
                tc::mma_commit_pair(&bars[kBarDrain]);
                tc::mbar_wait(&bars[kBarDrain], 0, nullptr);
            }
        }
    } else {
        // ---------------- epilogue: warps 2-5, TMEM lanes 32 (warp % 4) .. ----------------
        const int et = tid - 64;                        // 0..127
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
        const int row = (int)lane_base + lane;          // output row of the CTA's half tile
        uint32_t tl = 0, chunks = 0;                    // tiles and staging tiles done
        Chunks<kOutCols> ahead{pair, 0};                // the next addend chunk to ask for
        uint32_t asked = 0;
        auto ask = [&] {  // one thread: the addend of the next chunk into its slot
            if (ahead.t >= geo.tiles) return;
            const uint32_t slot = asked % kSlots;
            tc::mbar_expect_tx(&bars[kBarAdd + slot], kOutTile);
            const Tile at = tile_at(ahead.t, geo);
            tc::tma_load_2d(base + kOffOut + slot * kOutTile, &md, &bars[kBarAdd + slot], at.n + kOutCols * ahead.c,
                            at.m + rank * 128);
            ++asked;
            ahead.next(geo, pairs);
        };
        if (geo.has_addend && et == 0) ask(), ask();
        // the scales and biases of a tile's columns et and et + 128
        float *vec = reinterpret_cast<float *>(base + kOffVec);
        float ws[2], bs[2];
        auto fetch = [&](int t) {
            const int n = t < geo.tiles ? tile_at(t, geo).n + et : geo.N;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ws[h] = n + 128 * h < geo.N ? geo.w_scale[n + 128 * h] : 0.f;
                bs[h] = geo.bias && n + 128 * h < geo.N ? geo.bias[n + 128 * h] : 0.f;
            }
        };
        fetch(pair);
        bool ok = true;
        for (int t = pair; t < geo.tiles && ok; t += pairs, ++tl) {
            const uint32_t acc = tl & 1, use = tl >> 1;
            // the last tile's readers passed the barrier of its last chunk
#pragma unroll
            for (int h = 0; h < 2; ++h) vec[et + 128 * h] = ws[h], vec[kBN + et + 128 * h] = bs[h];
            fetch(t + pairs);
            if (!tc::named_all(1, 128, tc::mbar_wait_sleep(&bars[kBarAccFull + acc], use & 1u, err, abort_flag))) break;
            tc::tc_fence_after();
            const Tile at = tile_at(t, geo);
            const int m0 = at.m + rank * 128, n0 = at.n;
            const float xs = m0 + row < geo.M ? geo.x_scale[m0 + row] : 0.f;
            for (int c = 0; c < kBN / kOutCols && n0 + kOutCols * c < geo.N; ++c, ++chunks) {
                const uint32_t slot = chunks % kSlots;
                uint32_t v[kOutCols / 32][32];
#pragma unroll
                for (int q = 0; q < kOutCols / 32; ++q)
                    tc::tmem_ld32u(tc::tmem_addr(tmem + acc * kBN, lane_base, kOutCols * c + 32 * q), v[q]);
                tc::tmem_wait_ld();
                if (geo.has_addend) {
                    // asked for after the store that read this slot was done with it
                    ok = tc::named_all(1, 128, tc::mbar_wait_or_abort(&bars[kBarAdd + slot], (chunks / kSlots) & 1u, err,
                                                                      abort_flag));
                    if (!ok) break;
                } else {
                    if (et == 0) tc::bulk_wait_read<kSlots - 1>();
                    tc::named_sync(1, 128);
                }
                uint8_t *stg = base + kOffOut + slot * kOutTile;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int n = n0 + kOutCols * c + q * (kOutCols / 8);
                    uint4 *at = reinterpret_cast<uint4 *>(stg + tc::sw128(row, q));
                    // N is a multiple of 8: a 16-byte chunk is inside or outside as a whole
                    if (n < geo.N)
                        *at = finish<F32>(&v[q * (kOutCols / 8) / 32][q * (kOutCols / 8) % 32], xs, vec + (n - n0), geo, at);
                }
                tc::fence_proxy_async_smem();
                tc::named_sync(1, 128);
                if (et == 0) {
                    // rows past M and columns past N fall outside the tensor and are not written
                    if (m0 < geo.M) tc::tma_store_2d(&mo, stg, n0 + kOutCols * c, m0);
                    tc::bulk_commit();
                    if (geo.has_addend) {
                        tc::bulk_wait_read<kSlots - 2>();  // the slot two chunks on is free again
                        ask();
                    }
                }
            }
            // this accumulator may be overwritten by the tile after next
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::cluster_addr(&bars[kBarAccEmpty + acc], 0));
        }
        if (et == 0) {
            // the addends asked for have landed (bounded), the stores have completed
            for (uint32_t i = chunks; i < asked; ++i)
                tc::mbar_wait(&bars[kBarAdd + i % kSlots], (i / kSlots) & 1u, nullptr);
            tc::bulk_wait_all();
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();  // the peer's loads, commits and arrivals reach this CTA's shared memory until here
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, kTmemCols);
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
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (!tmap_available()) return cudaErrorNotSupported;
    if (linear_i8_few_wanted(a, nsm)) return launch_linear_i8_few(a, nsm, s);
    auto kernel = a.out_f32 ? linear_i8_kernel<true> : linear_i8_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const TmapType ot = a.out_f32 ? TmapType::f32 : TmapType::bf16;
    const int oc = a.out_f32 ? 32 : 64;
    CUtensorMap ma, mb, mo, md;
    if (!tmap_2d(&ma, TmapType::u8, a.x, a.K, a.M, kBK, 128) || !tmap_2d(&mb, TmapType::u8, a.w, a.K, a.N, kBK, 128) ||
        !tmap_2d(&mo, ot, a.out, a.N, a.M, oc, 128) || !tmap_2d(&md, ot, a.addend ? a.addend : a.out, a.N, a.M, oc, 128))
        return cudaErrorInvalidValue;
    Geo geo;
    geo.M = a.M;
    geo.N = a.N;
    geo.nk = (a.K + kBK - 1) / kBK;
    geo.tiles_n = (a.N + kBN - 1) / kBN;
    geo.tiles_m = (int)(((int64_t)a.M + kBM - 1) / kBM);
    geo.tiles = geo.tiles_m * geo.tiles_n;
    geo.x_scale = a.x_scale;
    geo.w_scale = a.w_scale;
    geo.bias = a.bias;
    geo.has_addend = a.addend != nullptr;
    const int grid = 2 * std::min(geo.tiles, std::max(nsm / 2, 1));
    Phase ph(a.phase ? a.phase : MATE_PHASE_LINEAR_I8, s);
    kernel<<<grid, kThreads, kSmemBytes, s>>>(ma, mb, mo, md, geo, a.err);
    return cudaGetLastError();
}

}  // namespace mate
