// The 8-bit linear layer (linear_i8.cu) for few tokens, where the pairs' 256 x 256 tiles
// leave most SMs idle and the time is that of reading w once (HBM: K N bytes), or of one
// tile's walk along K.
//
// The product is taken the other way round, out^T = w x^T: output channels are the MMA's
// M = 128 rows and tokens its N = NT columns (16, 32 or 64), so that few tokens waste no
// tensor time and w streams through at the rate of memory. The walk along K is split over
// the CTAs of a cluster (1, 2 or 4), each of which holds an exact int32 partial tile:
// they meet in shared memory, every CTA adding up its share of the tokens from the others'
// (distributed shared memory; integer sums, so the split changes no bit of the result),
// and finishing them (scales, bias, addend, one rounding) as it stores them.
//
// 128 threads, two CTAs per SM: thread 0 requests the CTA's K steps by TMA into a ring of
// 100 KB or so, thread 32 issues the MMAs, then all warps move the accumulator to shared
// memory (TMEM lane = channel), where the ring was, and finish 16-byte pieces of output rows.
//
// Waits are bounded as in linear_i8.cu; the MMA thread always signals the accumulator, so
// that every CTA of a cluster reaches the cluster's barriers.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

namespace mate {

namespace {

constexpr int kThreads = 128;
constexpr int kBC = 128, kBK = 128;  // channels of a tile; a K step is 128 codes = one swizzled row
constexpr uint32_t kWTile = kBC * kBK;

struct FewGeo {
    int M, N, nk;  // tokens, channels, 128-wide K steps
    int tiles_n;   // channel tiles
    const float *x_scale, *w_scale, *bias;
    const void *addend;
    void *out;
};

template <int NT> struct Few {
    static constexpr uint32_t kStage = kWTile + NT * kBK;
    static constexpr int kStages = NT == 16 ? 6 : NT == 32 ? 5 : 4;
    static constexpr uint32_t kOffBar = kStages * kStage;  // full, empty (per stage), acc; TMEM slot, abort flag
    static constexpr uint32_t kOffMisc = kOffBar + 8 * (2 * kStages + 1);
    static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;  // + alignment slack
    static constexpr uint32_t kTmemCols = NT < 32 ? 32 : NT;
    static_assert(NT * kBC * 4 <= kStages * kStage, "the partial tile takes the ring's place");
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

// TOP: K == tc::kI8MaxK
template <int NT, bool F32, bool TOP>
__global__ void __launch_bounds__(kThreads, 2)
    linear_i8_few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                         const __grid_constant__ FewGeo geo, int splits, int *err)
{
    using L = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t *base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(base + L::kOffBar), *empty = full + L::kStages;
    uint64_t *acc = empty + L::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + L::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + L::kOffMisc + 4);

    const int tid = threadIdx.x, warp = tid >> 5;
    const int rank = splits > 1 ? (int)tc::cluster_rank() : 0, tile = blockIdx.x / splits;
    const int c0 = (tile % geo.tiles_n) * kBC, m0 = (tile / geo.tiles_n) * NT;
    // this CTA's K steps; splits <= nk, so at least one
    const int k0 = (int)((int64_t)rank * geo.nk / splits), k1 = (int)((int64_t)(rank + 1) * geo.nk / splits);

    if (tid == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(acc, 1);
        tc::fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, L::kTmemCols);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    tc::stream_wait();
    tc::stream_release();

    if (tid == 0) {
        int it = 0;
        for (int k = k0; k < k1; ++k, ++it) {
            const int s = it % L::kStages, round = it / L::kStages;
            if (round > 0 && !tc::mbar_wait_or_abort(&empty[s], (round - 1) & 1, err, abort_flag)) break;
            uint8_t *sw = base + s * L::kStage, *sx = sw + kWTile;
            tc::mbar_expect_tx(&full[s], L::kStage);
            tc::tma_load_2d(sw, &mw, &full[s], k * kBK, c0);
            tc::tma_load_2d(sx, &mx, &full[s], k * kBK, m0);
        }
        // every load issued has landed before the ring gives way (bounded)
        tc::mbar_wait(&full[(it - 1) % L::kStages], ((it - 1) / L::kStages) & 1, nullptr);
        // and the last commit of each stage has arrived before the CTA may leave (the loads above
        // waited for the earlier ones)
        for (int s = 0; s < L::kStages && s < it; ++s)
            if (!tc::mbar_wait_or_abort(&empty[s], ((it - 1 - s) / L::kStages) & 1, err, abort_flag)) break;
    } else if (tid == 32) {
        const uint32_t idesc = tc::idesc_i8(kBC, NT);
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % L::kStages;
            if (!tc::mbar_wait_or_abort(&full[s], (it / L::kStages) & 1, err, abort_flag)) break;
            tc::tc_fence_after();
            const uint32_t w = tc::smem_u32(base + s * L::kStage), x = w + kWTile;
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)
                tc::mma_i8(tmem, tc::sdesc_sw128(w + kk * 32, 16, 1024), tc::sdesc_sw128(x + kk * 32, 16, 1024), idesc,
                           it > 0 || kk > 0);
            tc::mma_commit(&empty[s]);
        }
        tc::mma_commit(acc);  // also after a wait that gave up: nobody is left waiting
    }
    __syncwarp();
    tc::mbar_wait(acc, 0, err);
    tc::tc_fence_after();
    // channel 32 warp + lane of the partial tile, token by token: [token][channel]
    uint32_t *part = reinterpret_cast<uint32_t *>(base);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
        uint32_t v[16];
        __syncwarp();
        tc::tmem_ld16(tc::tmem_addr(tmem, 32 * warp, c), v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kBC + tid] = v[i];
    }
    tc::tc_fence_before();
    __syncthreads();
    if (splits > 1) tc::cluster_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, L::kTmemCols);

    // pieces of eight channels: this CTA's share of the tile's tokens
    const int pieces = NT * (kBC / 8) / splits;
    for (int p = rank * pieces + tid; p < (rank + 1) * pieces; p += kThreads) {
        const int token = p / (kBC / 8), n = c0 + p % (kBC / 8) * 8, m = m0 + token;
        if (m >= geo.M || n >= geo.N) continue;  // N is a multiple of 8
        const uint32_t *at = part + token * kBC + p % (kBC / 8) * 8;
        uint4 a = *reinterpret_cast<const uint4 *>(at), b = *reinterpret_cast<const uint4 *>(at + 4);
        // the other CTAs' partial tiles, their loads all in flight at once
        uint4 u[3], w[3];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i < splits) {
                const uint32_t addr = tc::cluster_addr(at, (rank + i) % splits);
                u[i - 1] = tc::ld_cluster(addr), w[i - 1] = tc::ld_cluster(addr + 16);
            }
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i < splits) {
                a.x += u[i - 1].x, a.y += u[i - 1].y, a.z += u[i - 1].z, a.w += u[i - 1].w;
                b.x += w[i - 1].x, b.y += w[i - 1].y, b.z += w[i - 1].z, b.w += w[i - 1].w;
            }
        const float xs = geo.x_scale[m];
        const float4 wa = *reinterpret_cast<const float4 *>(geo.w_scale + n);
        const float4 wb = *reinterpret_cast<const float4 *>(geo.w_scale + n + 4);
        auto sum = [](uint32_t acc) { return tc::i8_sum<TOP>(acc); };
        float v[8] = {sum(a.x) * xs * wa.x, sum(a.y) * xs * wa.y, sum(a.z) * xs * wa.z, sum(a.w) * xs * wa.w,
                      sum(b.x) * xs * wb.x, sum(b.y) * xs * wb.y, sum(b.z) * xs * wb.z, sum(b.w) * xs * wb.w};
        if (geo.bias) {
            const float4 ba = *reinterpret_cast<const float4 *>(geo.bias + n);
            const float4 bb = *reinterpret_cast<const float4 *>(geo.bias + n + 4);
            v[0] += ba.x, v[1] += ba.y, v[2] += ba.z, v[3] += ba.w;
            v[4] += bb.x, v[5] += bb.y, v[6] += bb.z, v[7] += bb.w;
        }
        const int64_t o = (int64_t)m * geo.N + n;
        if (F32) {
            float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(geo.out) + o);
            if (geo.addend) {
                const float4 *d = reinterpret_cast<const float4 *>(static_cast<const float *>(geo.addend) + o);
                const float4 da = d[0], db = d[1];
                v[0] += da.x, v[1] += da.y, v[2] += da.z, v[3] += da.w;
                v[4] += db.x, v[5] += db.y, v[6] += db.z, v[7] += db.w;
            }
            out[0] = make_float4(v[0], v[1], v[2], v[3]);
            out[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(geo.out) + o);
            if (geo.addend) {
                const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(geo.addend) + o);
                const float2 d0 = tc::unpack_bf16(u.x), d1 = tc::unpack_bf16(u.y), d2 = tc::unpack_bf16(u.z),
                             d3 = tc::unpack_bf16(u.w);
                v[0] += d0.x, v[1] += d0.y, v[2] += d1.x, v[3] += d1.y;
                v[4] += d2.x, v[5] += d2.y, v[6] += d3.x, v[7] += d3.y;
            }
            *out = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4], v[5]),
                              tc::pack_bf16(v[6], v[7]));
        }
    }
    if (splits > 1) {
        __syncthreads();
        tc::cluster_sync();  // the others read this CTA's partial tile until here
    }
}

template <int NT> cudaError_t launch(const LinearI8Args &a, int nsm, cudaStream_t s)
{
    auto kernel = a.K < tc::kI8MaxK ? (a.out_f32 ? linear_i8_few_kernel<NT, true, false> : linear_i8_few_kernel<NT, false, false>)
                                    : (a.out_f32 ? linear_i8_few_kernel<NT, true, true> : linear_i8_few_kernel<NT, false, true>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Few<NT>::kSmem);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mw;
    if (!tmap_2d(&mx, TmapType::u8, a.x, a.K, a.M, kBK, NT) || !tmap_2d(&mw, TmapType::u8, a.w, a.K, a.N, kBK, kBC))
        return cudaErrorInvalidValue;
    FewGeo geo;
    geo.M = a.M;
    geo.N = a.N;
    geo.nk = (a.K + kBK - 1) / kBK;
    geo.tiles_n = (a.N + kBC - 1) / kBC;
    geo.x_scale = a.x_scale;
    geo.w_scale = a.w_scale;
    geo.bias = a.bias;
    geo.addend = a.addend;
    geo.out = a.out;
    const int64_t tiles = (int64_t)geo.tiles_n * ((a.M + NT - 1) / NT);
    // as many CTAs as fit the GPU at two per SM, four to a tile at most: more spend longer on
    // joining than they save (2,560 -> 2,560 in a graph, 1, 2, 4, 8 CTAs: 16 tokens 8.5, 6.7, 5.6,
    // 6.1 us; 64 tokens 10.4, 8.5, 7.3, 9.0; 7,680 -> 2,560, 64 tokens 21, 14, 10, 11)
    int splits = 1;
    while (splits < 4 && 2 * splits <= geo.nk && 2 * splits * tiles <= 2 * nsm) splits *= 2;
    Phase ph(a.phase ? a.phase : MATE_PHASE_LINEAR_I8, s);
    return launch_in_stream(kernel, dim3((unsigned)(tiles * splits)), kThreads, Few<NT>::kSmem, splits, s, mx, mw, geo, splits,
                            a.err);
}

}  // namespace

// One wave of tiles of 64 tokens, two CTAs per SM, is where the pairs' kernel overtakes this one.
// Measured (2,560 -> 2,560; with a 64 MB read between calls, event overhead of about 5 us
// included): 1 token 12 us against 19, 64 tokens 14 against 19, 512 tokens (160 tiles) 16
// against 18, 1,024 tokens (320 tiles) 27 against 21. 2,560 -> 10,448: 192 tokens (246 tiles)
// 18 against 21, 256 tokens (328 tiles) 27 against 21. Tiles of 128 tokens lost to those of 64
// at every such size (128 tokens: 18 to 22 us against 14 to 16).
bool linear_i8_few_wanted(const LinearI8Args &a, int nsm)
{
    return ((int64_t)a.M + 63) / 64 * (((int64_t)a.N + kBC - 1) / kBC) <= 2 * nsm;
}

cudaError_t launch_linear_i8_few(const LinearI8Args &a, int nsm, cudaStream_t s)
{
    if (a.M <= 16) return launch<16>(a, nsm, s);
    if (a.M <= 32) return launch<32>(a, nsm, s);
    return launch<64>(a, nsm, s);
}

}  // namespace mate
