// 8-bit linear layer on the 5th-generation tensor cores: a product of signed 8-bit
// codes with a scale per token and a scale per output channel,
//     out_mn = s_m t_n sum_k x_mk w_nk (+ bias_n) (+ addend_mn).
// The sum is exact: kind::i8 accumulates in int32, and for K <= 131,072 only the sum of
// 131,072 products of -128 and -128 reaches 2^31 (tc::i8_sum). The two scales, the bias
// and the addend are applied to it in fp32 in the epilogue, and the result is rounded once
// to the output type.
//
// Persistent CTA pairs (clusters of two, cta_group::2), 320 threads per CTA; a pair
// computes output tiles of 256 x 256, CTA r the rows 128 r ..:
//   warp 0    TMA loads of the CTA's 128 x 128 codes of x and its half, 128 x 128, of
//             the w tile into a 5-stage ring (32 KB per stage and CTA, 128-byte
//             swizzle, K-major; codes past K, M or N load as zeros), all completing on
//             the barriers of rank 0;
//   warp 1    TMEM allocation and, in rank 0, tcgen05.mma issue: four M = 256, N = 256,
//             K = 32 MMAs per stage into one of two TMEM accumulators (2 x 256 columns
//             in each CTA), so that a tile's epilogue runs while the next accumulates;
//   warps 2-9 the epilogue, two groups of four warps that take the tile's column chunks
//             alternately: TMEM -> registers -> scales, bias, addend -> a staging tile
//             of 128 rows x 128 bytes in the 128-byte swizzle (two per group) -> TMA
//             store. The addend arrives in the staging tile by TMA, a chunk ahead; the
//             columns' scales and bias wait in shared memory, fetched a tile ahead
//             (read from global memory chunk by chunk they cost in_proj of 131,072
//             tokens 3.20 ms instead of 2.48). One group instead of two: 15.4 us
//             instead of 12.8 for 1,155 tokens, 2,560 -> 2,560.
// What bounds it: the MMAs, at the clock that the board's power limit leaves. The four of a K
// step are 512 cycles nominal and 584 with their operands in place. At 1,965 MHz a K step takes
// 0.33 us = 648 cycles (1,155 tokens -> 2,560 in a graph: 13.3 us at K = 2,560, 7.0 at K = 128).
// In loops of seconds, by the time of a call over the K steps that a pair takes one after another
// and the clock sampled meanwhile: 0.43 us = 596 cycles of 1,387 MHz (32,768 tokens, 7,680 ->
// 2,560: 2,780 TOP/s), 0.48 us = 648 cycles of 1,357 MHz (in_proj of 131,072 tokens: 2,590 TOP/s,
// 0.94 of twice the sustained bf16 rate), 0.48 us = 682 cycles of 1,425 MHz (32,768 tokens,
// 2,560 -> 2,560: 2,490, the unfilled last round of tiles counted in). Single launches after a
// pause, at a higher clock: 3,210, 2,940 and 2,610 TOP/s. Tiles of 192 and 128 columns lost as
// whole kernels (4,096 tokens, 2,560 -> 2,560: 39 us in 128 columns, 30 in 256); what share of
// that is the MMAs' and what the loads' was not told apart. Tried and left: a ring of six stages (no
// change); tiles of 256 x 512 with x loaded once for both halves (a quarter less to load: 476 us
// against 492 for 32,768 tokens, 7,680 -> 2,560, but 181 against 175 at K = 2,560, since one tile
// fills TMEM and its epilogue is exposed).
// Tiles are walked in groups of four tile rows, so that the 74 pairs at work read about
// four rows' x and 19 columns' w from L2 (65,536 tokens, 2,560 -> 10,448, in a graph: 1,370 us
// in groups of 4, 1,399 of 8, 1,390 of 16, 1,378 of 32; 32,768 tokens, 7,680 -> 2,560: 484, 483,
// 493, 540. Row by row, on an earlier form, in_proj of 131,072 tokens took 3.30 ms where groups of
// 8 took 3.20).
//
// Every wait is bounded (2 s); a wait that gives up records MATE_ERR_TIMEOUT and
// raises a CTA abort flag that makes every role leave its loop; the CTA then
// waits (bounded) for its copies and MMAs in flight, meets its peer (which leaves its
// own waits by the same limit), waits (bounded) for the arrivals that the MMA thread's
// commits still owe its own barriers, and frees its TMEM.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

#include <algorithm>

namespace mate {

namespace {

constexpr int kBM = 256, kBK = 128;                  // rows of a pair's tile; a K step is 128 codes = one swizzled row
constexpr int kBN = 256;                             // columns of a tile
constexpr int kStages = 5, kGroups = 2, kSlots = 2;  // staging tiles per epilogue group
constexpr int kGroup = 4;                            // tile rows walked together
constexpr uint32_t kTile = 128 * kBK;                // 16 KB: one CTA's part of x or w
constexpr uint32_t kStage = 2 * kTile;
constexpr uint32_t kOutTile = 128 * 128;             // 16 KB: 128 rows x 128 bytes
constexpr uint32_t kOffStages = 0;
constexpr uint32_t kOffOut = kStages * kStage;
constexpr uint32_t kOffVec = kOffOut + kGroups * kSlots * kOutTile;  // per group: w_scale and bias of its columns
constexpr uint32_t kOffBar = kOffVec + 2 * kBN * 4;
// full, empty (per stage), acc_full[2], acc_empty[2], addend (per slot), drain
constexpr int kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccEmpty = 2 * kStages + 2,
              kBarAdd = 2 * kStages + 4, kBarDrain = kBarAdd + kGroups * kSlots, kNumBars = kBarDrain + 1;
// the TMEM slot, the abort flag, and what rank 0's MMA thread committed: stages, accumulators
constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
constexpr uint32_t kSmemBytes = kOffMisc + 16;
static_assert(kSmemBytes <= 227 * 1024, "linear_i8: shared memory");
constexpr int kThreads = 64 + 128 * kGroups;
constexpr uint32_t kTmemCols = 512;
static_assert(kOffBar % 8 == 0 && kOffVec % 16 == 0, "linear_i8: alignment");

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
// the bias (`vec`: the columns' w_scale, their bias 128 floats on) and the addend that `stg` holds
template <bool F32, bool TOP>
__device__ __forceinline__ uint4 finish(const uint32_t *acc, float xs, const float *vec, const Geo &geo, const uint4 *stg)
{
    constexpr int kCols = F32 ? 4 : 8;
    float v[kCols];
#pragma unroll
    for (int q = 0; q < kCols / 4; ++q) {
        const float4 ws = *reinterpret_cast<const float4 *>(vec + 4 * q);
        v[4 * q] = tc::i8_sum<TOP>(acc[4 * q]) * xs * ws.x;
        v[4 * q + 1] = tc::i8_sum<TOP>(acc[4 * q + 1]) * xs * ws.y;
        v[4 * q + 2] = tc::i8_sum<TOP>(acc[4 * q + 2]) * xs * ws.z;
        v[4 * q + 3] = tc::i8_sum<TOP>(acc[4 * q + 3]) * xs * ws.w;
        if (geo.bias) {
            const float4 b = *reinterpret_cast<const float4 *>(vec + 128 + 4 * q);
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

// Column chunks (staging tiles) of tile t
template <int OUT_COLS> __device__ __forceinline__ int chunks_of(int t, const Geo &geo)
{
    return (min(kBN, geo.N - tile_at(t, geo).n) + OUT_COLS - 1) / OUT_COLS;
}

// The chunks that one epilogue group of a pair's CTA takes, in order: g, g + 2, .. of each tile.
template <int OUT_COLS> struct Chunks {
    int t, c;  // tile, column chunk
    __device__ __forceinline__ void settle(const Geo &geo, int g, int step)
    {
        while (t < geo.tiles && c >= chunks_of<OUT_COLS>(t, geo)) c = g, t += step;
    }
};

// TOP: K == tc::kI8MaxK
template <bool F32, bool TOP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_i8_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                     const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap md,
                     const __grid_constant__ Geo geo, int *err)
{
    constexpr int kOutCols = F32 ? 32 : 64;  // columns of a staging tile
    extern __shared__ __align__(1024) uint8_t base[];
    if (tc::smem_u32(base) & 1023u) {  // the swizzled tiles need it; the same for every thread of both CTAs
        tc::stream_wait();
        if (threadIdx.x == 0) atomicExch(err, MATE_ERR_INVALID_ARG);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + kOffMisc + 4);
    uint32_t *commits = reinterpret_cast<uint32_t *>(base + kOffMisc + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)tc::cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 64) {
        tc::tma_prefetch_map(&mo);
        if (geo.has_addend) tc::tma_prefetch_map(&md);
    }
    if (tid == 0) {
        tc::tma_prefetch_map(&ma);
        tc::tma_prefetch_map(&mb);
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bars[kBarFull + i], 1);
            tc::mbar_init(&bars[kBarEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[kBarAccFull + i], 1);
            tc::mbar_init(&bars[kBarAccEmpty + i], 2 * 4 * kGroups);  // the epilogue warps of both CTAs
        }
        for (int i = 0; i < kGroups * kSlots; ++i) tc::mbar_init(&bars[kBarAdd + i], 1);
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
    tc::stream_wait();
    tc::stream_release();

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
            uint32_t it = 0, tl = 0, committed = 0, filled = 0;
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
                ++filled;
            }
            // every MMA issued has completed before TMEM may be freed (bounded)
            if (committed > 0) {
                tc::mma_commit_pair(&bars[kBarDrain]);
                tc::mbar_wait(&bars[kBarDrain], 0, nullptr);
            }
            for (uint32_t r = 0; r < 2; ++r) {
                tc::st_cluster(tc::cluster_addr(&commits[0], r), committed);
                tc::st_cluster(tc::cluster_addr(&commits[1], r), filled);
            }
        }
    } else {
        // ---------------- epilogue: warps 2-9 in two groups, TMEM lanes 32 (warp % 4) .. ----------------
        const int g = (tid - 64) / 128, et = (tid - 64) % 128;  // group, thread of it
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
        const int row = (int)lane_base + lane;                  // output row of the CTA's half tile
        uint8_t *slots = base + kOffOut + g * kSlots * kOutTile;
        uint64_t *add = bars + kBarAdd + g * kSlots;
        uint32_t tl = 0, done = 0;                              // tiles and staging tiles done
        Chunks<kOutCols> ahead{pair, g};                        // the next addend chunk to ask for
        uint32_t asked = 0;
        auto ask = [&] {  // one thread: the addend of the next chunk into its slot
            ahead.settle(geo, g, pairs);
            if (ahead.t >= geo.tiles) return;
            const uint32_t slot = asked % kSlots;
            const Tile at = tile_at(ahead.t, geo);
            tc::mbar_expect_tx(&add[slot], kOutTile);
            tc::tma_load_2d(slots + slot * kOutTile, &md, &add[slot], at.n + kOutCols * ahead.c, at.m + rank * 128);
            ++asked;
            ahead.c += kGroups;
        };
        if (geo.has_addend && et == 0) ask();
        // the scale and bias of the group's column et of a tile: column et % kOutCols of its chunk et / kOutCols
        float *vec = reinterpret_cast<float *>(base + kOffVec) + g * 256;
        const int own = (et / kOutCols * kGroups + g) * kOutCols + et % kOutCols;
        float ws, bs;
        auto fetch = [&](int t) {
            const int n = t < geo.tiles ? tile_at(t, geo).n + own : geo.N;
            ws = n < geo.N ? geo.w_scale[n] : 0.f;
            bs = geo.bias && n < geo.N ? geo.bias[n] : 0.f;
        };
        fetch(pair);
        bool ok = true;
        for (int t = pair; t < geo.tiles && ok; t += pairs, ++tl) {
            const uint32_t acc = tl & 1, use = tl >> 1;
            // the last tile's readers passed the barrier of its last chunk
            vec[et] = ws, vec[128 + et] = bs;
            fetch(t + pairs);
            const Tile at = tile_at(t, geo);
            const int m0 = at.m + rank * 128, chunks = chunks_of<kOutCols>(t, geo);
            const float xs = m0 + row < geo.M ? geo.x_scale[m0 + row] : 0.f;
            if (!tc::named_all(1 + g, 128, tc::mbar_wait_sleep(&bars[kBarAccFull + acc], use & 1u, err, abort_flag))) break;
            tc::tc_fence_after();
            // the group's columns, all at once, and the accumulator goes back to the MMAs (of the
            // tile after next)
            constexpr int kOwn = 128 / kOutCols;  // chunks of a full tile that are the group's
            uint32_t v[kOwn][kOutCols / 32][32];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const int c = kGroups * i + g;
                if (c < chunks) {
#pragma unroll
                    for (int q = 0; q < kOutCols / 32; ++q)
                        tc::tmem_ld32u(tc::tmem_addr(tmem + acc * kBN, lane_base, kOutCols * c + 32 * q), v[i][q]);
                }
            }
            tc::tmem_wait_ld();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::cluster_addr(&bars[kBarAccEmpty + acc], 0));
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const int c = kGroups * i + g;
                if (c >= chunks) break;
                const uint32_t slot = done % kSlots;
                const int n0 = at.n + kOutCols * c;
                if (geo.has_addend) {
                    if (et == 0) {
                        tc::bulk_wait_read<0>();  // the other slot is free again: the next chunk's addend
                        ask();
                    }
                    ok = tc::named_all(1 + g, 128, tc::mbar_wait_or_abort(&add[slot], (done / kSlots) & 1u, err, abort_flag));
                    if (!ok) break;
                } else {
                    if (et == 0) tc::bulk_wait_read<kSlots - 1>();
                    tc::named_sync(1 + g, 128);
                }
                uint8_t *stg = slots + slot * kOutTile;
                const float *cv = vec + i * kOutCols;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint4 *to = reinterpret_cast<uint4 *>(stg + tc::sw128(row, q));
                    // columns past N hold zeros and are not written
                    *to = finish<F32, TOP>(&v[i][q * (kOutCols / 8) / 32][q * (kOutCols / 8) % 32], xs, cv + q * (kOutCols / 8), geo, to);
                }
                tc::fence_proxy_async_smem();
                tc::named_sync(1 + g, 128);
                if (et == 0) {
                    // rows past M and columns past N fall outside the tensor and are not written
                    if (m0 < geo.M) tc::tma_store_2d(&mo, stg, n0, m0);
                    tc::bulk_commit();
                }
                ++done;
            }
        }
        if (et == 0) {
            // the addends asked for have landed (bounded), the stores have left shared memory
            for (uint32_t i = done; i < asked; ++i) tc::mbar_wait(&add[i % kSlots], (i / kSlots) & 1u, nullptr);
            tc::bulk_wait_read_all();
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    // the peer's loads have landed and its threads' stores and arrivals are done; the arrivals of
    // commits are not part of it: they come by themselves, at each CTA in its own time
    tc::cluster_sync();
    if (warp == 0) {
        // Every commit has arrived on this CTA's barriers before its shared memory may go to
        // another CTA. Commit j of a stage or an accumulator is issued only after commit j - 1
        // was seen in both CTAs, so at most the last phase of each barrier is outstanding.
        const uint32_t first = lane < kStages ? lane : lane - kStages, of = lane < kStages ? kStages : 2;
        const uint32_t issued = lane < kStages ? commits[0] : lane < kStages + 2 ? commits[1] : 0;
        if (issued > first)
            tc::mbar_wait(&bars[lane < kStages ? kBarEmpty + lane : kBarAccFull + first], ((issued - 1 - first) / of) & 1u, err);
        if (lane == kStages + 2 && commits[0] > 0) tc::mbar_wait(&bars[kBarDrain], 0, err);
    } else if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

}  // namespace

// Rows of codes are 16-byte aligned (K a multiple of 16) and so are rows of outputs;
// output tiles fit 32-bit counters.
bool linear_i8_supported(const LinearI8Args &a)
{
    constexpr int kMost = 0x7fffffff - 1023;  // a tile may reach past the last row or column
    return a.M > 0 && a.N > 0 && a.M <= kMost && a.N <= kMost && a.K > 0 && a.K % 16 == 0 && a.K <= tc::kI8MaxK && a.N % 8 == 0 &&
           ((int64_t)a.M + kBM) * ((int64_t)a.N + kBN) / (kBM * kBN) < ((int64_t)1 << 30);
}

cudaError_t launch_linear_i8(const LinearI8Args &a, cudaStream_t s)
{
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (!tmap_available()) return cudaErrorNotSupported;
    if (linear_i8_few_wanted(a, nsm)) return launch_linear_i8_few(a, nsm, s);
    auto kernel = a.K < tc::kI8MaxK ? (a.out_f32 ? linear_i8_kernel<true, false> : linear_i8_kernel<false, false>)
                                    : (a.out_f32 ? linear_i8_kernel<true, true> : linear_i8_kernel<false, true>);
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
    return launch_in_stream(kernel, dim3(grid), kThreads, kSmemBytes, 0, s, ma, mb, mo, md, geo, a.err);
}

}  // namespace mate
