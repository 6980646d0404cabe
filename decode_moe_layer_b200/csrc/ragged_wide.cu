// ragged_wide.cu -- the ragged products (ragged_gemm.cu) for groups of many rows.
//
// ragged_wide_kernel: persistent, one cluster of two CTAs per pair of SMs.  A tile is 256 weight rows x up to
// 256 tokens of one group; the pair runs it as one tcgen05.mma.cta_group::2 of M = 256, N = the tile's tokens
// rounded up to 32.  Each CTA holds its 128 weight rows and half of the tokens in shared memory (the pair's MMA
// reads both halves), so a stage brings 32 KB into each SM instead of the 48 KB of a 128 x 256 tile, and the
// accumulator of its 128 rows in its own tensor memory, twice (256 columns each), so that one tile's
// epilogue overlaps the next tile's products.
//   * warp 0 (both CTAs): TMA copies of its weight rows and, without the gather, its token rows; they
//     report to the even CTA's barrier.
//   * warp 1 (even CTA): the MMAs; its commits release the stage in both CTAs.
//   * warps 4..7: the epilogue of the CTA's 128 rows.
//   * warps 8..15 (gather): token rows by the routing's indices, four rows an instruction.  A warp issues such
//     an instruction every 50 cycles or so (its operands differ by lane), so eight warps share a stage's 32; one
//     warp took 1500 cycles over them against the MMAs' 512.  (cp.async in the swizzled layout was slower,
//     830 cycles a stage: too few copies in flight.)
// Tiles go round-robin over the clusters: experts in order, for each its blocks of weight rows, for each its
// token tiles, so the tiles that run together share operands in L2.
#include <atomic>

#include "ragged.cuh"

namespace moe {

namespace rwide {
using namespace ragged;
constexpr int kPipe = 6;
constexpr int kNt = 256;                                  // tokens per tile
constexpr int kBBytes = kNt / 2 * kStageKBytes;           // a CTA's half of them
constexpr int kPipeBytes = kABytes + kBBytes;
constexpr int kOffBars = kPipe * kPipeBytes;
constexpr int kOffScales = kOffBars + 256;                // [2][kNt] fp32 row scales (int8)
constexpr int kOffGroups = kOffScales + 8192;             // or, swiglu, what gate and up warps exchange: 8 KB
constexpr int kTmemCols = 512;
constexpr int kEpi0 = 4, kGather0 = 8, kGatherWarps = 8;
static_assert(2 * kNt * 4 <= 8192 && 2 * 4 * 8 * 32 * 4 <= 8192, "either fits");
}  // namespace rwide

// Copies that complete on a barrier of either CTA of the pair (bar: cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_gather4_pair(void *dst, const CUtensorMap *map, int c0, const int (&r)[4],
                                                 uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}
// One arrival on the barrier at the same place in both CTAs once the MMAs issued before are complete.
__device__ __forceinline__ void umma_commit_pair(uint32_t mbar_smem)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(mbar_smem), "h"(static_cast<uint16_t>(3)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait for a barrier that the other CTA arrives on too.
__device__ __forceinline__ void mbar_wait_cluster(uint64_t *bar, uint32_t parity, bool &aborted, const StatusPtrs &st)
{
    if (aborted) return;
    if (mbar_try_wait_cluster(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_cluster(bar, parity)) {
        if (clock64() - t0 > kWaitLimitCycles) {
            aborted = true;
            record_timeout(st);
            return;
        }
    }
}

// The tiles of one cluster, in order: t = cluster, cluster + clusters, ...
struct TileWalk {
    const int *lo, *first;
    int pair_blocks, total, step, t, e;
    int rb, p0, count;   // of the current tile
    __device__ __forceinline__ TileWalk(const int *lo_, const int *first_, int E, int pair_blocks_, int start, int step_)
        : lo(lo_), first(first_), pair_blocks(pair_blocks_), total(first_[E] * pair_blocks_), step(step_), t(start), e(0)
    {
    }
    __device__ __forceinline__ bool locate()
    {
        if (t >= total) return false;
        while (t >= first[e + 1] * pair_blocks) ++e;
        const int tiles = first[e + 1] - first[e], local = t - first[e] * pair_blocks;
        rb = local / tiles;
        const int rows = tile_rows<32>(lo[e + 1] - lo[e], rwide::kNt);
        p0 = lo[e] + (local - rb * tiles) * rows;
        count = min(rows, lo[e + 1] - p0);
        return true;
    }
    __device__ __forceinline__ void next() { t += step; }
};

template <bool kInt8, bool kGather, bool kSwiglu>
__global__ void __launch_bounds__(kGather ? 32 * (rwide::kGather0 + rwide::kGatherWarps) : 256, 1)
ragged_wide_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ BoxMaps xmaps,
                   const __grid_constant__ RaggedArgs a)
{
    using namespace rwide;
    constexpr int kStageK = kInt8 ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBars);   // used in the even CTA
    uint64_t *empty = full + kPipe;
    uint64_t *acc_full = empty + kPipe;
    uint64_t *acc_empty = acc_full + 2;                               // used in the even CTA
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    float *scales = reinterpret_cast<float *>(smem + kOffScales), *exchange = scales;
    int *lo = reinterpret_cast<int *>(smem + kOffGroups), *first = lo + a.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const StatusPtrs status{nullptr, a.status_out};
    const uint32_t rank = cluster_rank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const int pair_blocks = (a.row_blocks + 1) >> 1;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&wmap);
        for (int i = 0; i < (kGather ? 1 : 4); ++i) prefetch_tensormap(&xmaps.m[i]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 64) {
        for (int s = 0; s < kPipe; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);   // four epilogue warps of both CTAs
        }
        fence_barrier_init();
    }
    pdl_wait();
    build_groups<32>(a.offsets, a.R, a.E, kNt, lo, first);
    tc_fence_before();
    __syncwarp();
    cluster_sync();   // barriers, tensor memory and tables of both CTAs are ready
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    bool aborted = false;
    TileWalk w(lo, first, a.E, pair_blocks, cluster, clusters);

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        int it = 0;
        for (; w.locate(); w.next()) {
            // one box of 16, 32, 64 or 128 token rows
            const int half = ((w.count + 31) & ~31) >> 1, box = half <= 16 ? 0 : (half <= 32 ? 1 : (half <= 64 ? 2 : 3));
            const int row0 = w.p0 + static_cast<int>(rank) * half;
            const int block = 2 * w.rb + static_cast<int>(rank);
            // weight rows past the expert's last come from the next one, or are zeros: nobody stores their products
            const int wrow = kSwiglu ? w.e * 2 * a.N + block * 64 : w.e * a.N + block * kRows;
            const uint32_t bytes = 2 * (kABytes + (kGather ? half : 16 << box) * kStageKBytes);   // of both CTAs
            for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
                const int s = it % kPipe;
                mbar_wait(&empty[s], ((it / kPipe) & 1) ^ 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                uint8_t *sa = smem + s * kPipeBytes;
                const uint32_t bar = map_cluster(smem_u32(&full[s]), 0);
                if (lane == 0) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    if (kSwiglu) {   // 64 gate rows, then their 64 up rows
                        tma_load_2d_pair(sa, &wmap, kb * kStageK, wrow, bar);
                        tma_load_2d_pair(sa + kABytes / 2, &wmap, kb * kStageK, wrow + a.N, bar);
                    } else {
                        tma_load_2d_pair(sa, &wmap, kb * kStageK, wrow, bar);
                    }
                    if (!kGather) tma_load_2d_pair(sa + kABytes, &xmaps.m[box], kb * kStageK, row0, bar);
                }
                __syncwarp();
            }
            if (aborted) break;
        }
        // after a timeout the even CTA waits for both CTAs' copies in flight
        if (aborted && rank == 0)
            for (int i = 0; i < kPipe && i < it; ++i) {
                const int j = it - 1 - i;
                mbar_wait_drain(&full[j % kPipe], (j / kPipe) & 1, status);
            }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer
        int it = 0;
        for (int i = 0; w.locate(); w.next(), ++i) {
            const int b = i & 1, n32 = (w.count + 31) & ~31;
            const uint32_t idesc = kInt8 ? umma_idesc_i8(256, n32) : umma_idesc_bf16(256, n32);
            const uint32_t acc = tmem + b * kNt;
            mbar_wait_cluster(&acc_empty[b], ((i >> 1) & 1) ^ 1, aborted, status);
            for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
                const int s = it % kPipe;
                mbar_wait_cluster(&full[s], (it / kPipe) & 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * kPipeBytes);
                const uint64_t ad = umma_sdesc_sw128(sa), bd = umma_sdesc_sw128(sa + kABytes);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_ss<kInt8, 2>(acc, ad + 2 * j, bd + 2 * j, idesc, kb > 0 || j > 0);
                    umma_commit_pair(smem_u32(&empty[s]));
                }
                __syncwarp();
            }
            if (aborted) break;
            if (elect_one()) umma_commit_pair(smem_u32(&acc_full[b]));
            __syncwarp();
        }
    } else if (warp >= kEpi0 && warp < kEpi0 + 4) {
        // ------------------------------------------------------------ epilogue
        const int q = warp - kEpi0;
        for (int i = 0; w.locate(); w.next(), ++i) {
            const int b = i & 1;
            const int block = 2 * w.rb + static_cast<int>(rank);
            const int n = block * kRows + 32 * q + lane;
            float cs = 1.0f;
            float *rs = scales + b * kNt;
            if (kInt8) {
                if (n < a.N) cs = a.col_scale[n];
                for (int j = threadIdx.x - 32 * kEpi0; j < kNt; j += 128) rs[j] = j < w.count ? a.row_scale[w.p0 + j] : 0.f;
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            mbar_wait_cluster(&acc_full[b], (i >> 1) & 1, aborted, status);
            tc_fence_after();
            // (after a timeout the rest runs on whatever is there: the warps keep meeting at their barriers)
            const uint32_t acc = tmem + b * kNt + (static_cast<uint32_t>(32 * q) << 16);
            if (kSwiglu) {
                // Gate rows are lanes 0..63 (warps q = 0, 1), their up rows lanes 64..127 (q = 2, 3).  Warps q and
                // q ^ 2 exchange halves of 16 columns: the gate warp finishes the first 8, the up warp the others.
                const int up = q >> 1, ns = block * 64 + 32 * (q & 1) + lane;
                for (int c = 0; c < w.count; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(acc + c, v);
                    float *ex = exchange + ((c >> 4) & 1) * 1024;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ex[q * 256 + j * 32 + lane] = __uint_as_float(up ? v[j] : v[8 + j]);
                    asm volatile("bar.sync %0, 64;" ::"r"(2 + (q & 1)) : "memory");
                    float h[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float other = ex[(q ^ 2) * 256 + j * 32 + lane];
                        const float own = __uint_as_float(up ? v[8 + j] : v[j]);
                        h[j] = ragged_swiglu(up ? other : own, up ? own : other);
                    }
                    uint32_t hb[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) hb[j] = __float_as_uint(h[j]);
                    const int c0 = c + 8 * up;
                    finish_columns<false, 8>(a, hb, nullptr, 1.0f, static_cast<size_t>(w.p0) + c0, w.count - c0, ns);
                }
            } else {
                for (int c = 0; c < w.count; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(acc + c, v);
                    finish_columns<kInt8, 16>(a, v, rs + c, cs, static_cast<size_t>(w.p0) + c, w.count - c, n);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_cluster(smem_u32(&acc_empty[b]), 0));
        }
    } else if (kGather && warp >= kGather0) {
        // ------------------------------------------------------------ gather
        // Runs of four rows go round the warps, lane i of warp g taking run g + 8 i.
        const int g = warp - kGather0;
        int it = 0;
        for (; w.locate(); w.next()) {
            const int half = ((w.count + 31) & ~31) >> 1;
            const int run = g + kGatherWarps * lane;
            const bool mine = 4 * run < half;
            int idx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(static_cast<int>(rank) * half + 4 * run + i, w.count - 1);
                const uint32_t f = mine ? static_cast<uint32_t>(__ldcg(a.sorted_ids + w.p0 + r)) : 0u;
                idx[i] = static_cast<int>(min(f / static_cast<uint32_t>(a.k), static_cast<uint32_t>(a.M - 1)));
            }
            for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
                const int s = it % kPipe;
                mbar_wait(&empty[s], ((it / kPipe) & 1) ^ 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                if (mine)
                    tma_gather4_pair(smem + s * kPipeBytes + kABytes + run * 4 * kStageKBytes, &xmaps.m[0], kb * kStageK,
                                     idx, map_cluster(smem_u32(&full[s]), 0));
                __syncwarp();
            }
            if (aborted) break;
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();   // neither CTA ends while the other's MMAs read it or its arrivals are on their way
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ launch

void wide_plan(RaggedPlan &p, int E, bool gather)
{
    p.stages = rwide::kPipe;
    p.smem = 1024 + rwide::kOffGroups + 2 * (E + 1) * 4;
    p.threads = gather ? 32 * (rwide::kGather0 + rwide::kGatherWarps) : 256;
}

template <bool kInt8, bool kGather, bool kSwiglu>
static cudaError_t launch_wide_t(const CUtensorMap &wmap, const BoxMaps &xmaps, const RaggedArgs &a,
                                 const RaggedPlan &p, cudaStream_t s)
{
    auto kernel = ragged_wide_kernel<kInt8, kGather, kSwiglu>;
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms() & ~1));
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, wmap, xmaps, a);
}

cudaError_t launch_ragged_wide(bool int8, bool swiglu, const CUtensorMap &wmap, const BoxMaps &xmaps,
                               const RaggedArgs &a, const RaggedPlan &p, cudaStream_t s)
{
    const bool gather = a.sorted_ids != nullptr;
    if (int8) return launch_wide_t<true, false, false>(wmap, xmaps, a, p, s);
    if (gather)
        return swiglu ? launch_wide_t<false, true, true>(wmap, xmaps, a, p, s)
                      : launch_wide_t<false, true, false>(wmap, xmaps, a, p, s);
    return swiglu ? launch_wide_t<false, false, true>(wmap, xmaps, a, p, s)
                  : launch_wide_t<false, false, false>(wmap, xmaps, a, p, s);
}

}  // namespace moe
