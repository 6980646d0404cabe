// ragged_wide.cu -- the ragged products (ragged.cuh) in tiles on tcgen05, from a few rows per group up.
//
// kind::f16 (bf16 products, fp32 sums) or kind::i8 (int8 products, int32 sums, exact), the accumulator in tensor
// memory.  128 bytes of K, 64 bf16 or 128 int8 values, are one pipeline stage and four MMAs in either type, so
// one kernel serves both.  The weight rows are the MMA's M side and the tokens its N side, whose width follows the
// group: a group of one row costs little more than its weights' way in, and rows beyond a group reach only
// accumulator columns that nobody stores.
//
// ragged_wide_kernel: one cluster of two CTAs per pair of SMs, persistent.  A tile is 256 weight rows x up to
// 256 tokens of one group; the pair runs it as one tcgen05.mma.cta_group::2 of M = 256, N = the tile's tokens
// rounded up to 32.  Each CTA holds its 128 weight rows and half of the tokens in shared memory (the pair's MMA
// reads both halves), so a stage brings 32 KB into each SM instead of the 48 KB of a 128 x 256 tile, and the
// accumulator of its 128 rows in its own tensor memory, twice (256 columns each), so that one tile's
// epilogue overlaps the next tile's products.
//   * warps 0 and 2 (both CTAs): TMA copies of its weight rows and, without the gather, its token rows; they
//     report to the even CTA's barrier.  (Issued by one warp they took 400 cycles a stage.)
//   * warp 1 (even CTA): the MMAs; its commits release the stage in both CTAs.
//   * warps 4..7: the epilogue of the CTA's 128 rows.
//   * warps 8..15 (gather): token rows by the routing's indices, four rows an instruction.  A warp issues such
//     an instruction every 50 cycles or so (its operands differ by lane), so eight warps share a stage's 32; one
//     warp took 1500 cycles over them against the MMAs' 512.  (cp.async in the swizzled layout was slower,
//     830 cycles a stage: too few copies in flight.)
// With few tiles, clusters of up to eight CTAs take one each, every pair of them a range of K; they join their sums
// through distributed shared memory in a fixed order.
// The tensor maps have two dimensions: boxes of a map with three or more came in at 10.6 TB/s from L2 over the whole
// chip, those of a flat one at 16.9, and a TMA instruction costs about 100 cycles whatever its size, so boxes are as
// high as the tile allows.
// Tiles go round-robin over the clusters: experts in order, for each its token tiles by eight, with them the blocks of
// weight rows, so the tiles that run together are as many in either direction and share operands in L2 (one group of
// 16384 rows x 4096 x 7168 took 935 us in long runs with all 64 token tiles inside, against HBM and the power limit).
#include <atomic>

#include "ragged.cuh"
#include "ragged_plan.h"

namespace moe {

// Copies that complete on a barrier of either CTA of the pair (dst: shared-memory, bar: cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap *map, int c0, const int (&r)[4],
                                                 uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}
// One arrival on the barrier at the same place in both CTAs of the pair once the MMAs issued before are complete.
__device__ __forceinline__ void umma_commit_pair(uint32_t mbar_smem, uint32_t leader)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(mbar_smem), "h"(static_cast<uint16_t>(3u << leader)) : "memory");
}
// Arrival without ordering memory: of an epilogue warp that is done with an accumulator, whose loads from tensor memory
// have completed (tcgen05.wait::ld), and of a CTA whose MMAs have.  The releasing form would wait until the warp's
// stores to y have arrived, some 1300 cycles a tile.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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
__device__ __forceinline__ void mbar_wait_cluster(uint64_t *bar, uint32_t parity, bool &aborted, const StatusPtrs &st,
                                                  long long limit)
{
    if (aborted) return;
    if (mbar_try_wait_cluster(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_cluster(bar, parity)) {
        if (clock64() - t0 > limit) {
            aborted = true;
            record_timeout(st);
            return;
        }
    }
}

// A whole warp's wait for copies, or MMAs, with one answer for all its lanes (bar: shared-memory address).
__device__ __forceinline__ bool warp_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "vote.sync.all.pred q, p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, bool &aborted, const StatusPtrs &st,
                                          long long limit)
{
    if (warp_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!warp_try_wait(bar, parity)) {
        if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
            aborted = true;
            record_timeout(st);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Token rows of the box for a CTA's half of a tile: just those, or with one group, whose tiles are all but one alike,
// those of a full tile or of half a one.
__device__ __forceinline__ int box_rows(const RaggedArgs &a, int half, bool halved)
{
    return a.offsets != nullptr ? half : (halved ? rwide::kNt / 4 : a.nt / 2);
}

// Where a warp is in the ring of stages: bytes to the stage and to its barriers.  The loops over stages keep to few
// instructions: with 64 tokens a stage's MMAs take 128 cycles and the issuing warp 300 (it was 380).
struct Ring {
    uint32_t stage_bytes, bars, at = 0, bar = 0, parity = 0;
    __device__ __forceinline__ explicit Ring(const RaggedArgs &a) : stage_bytes(a.stage_bytes), bars(8 * a.stages) {}
    __device__ __forceinline__ void next()
    {
        at += stage_bytes;
        bar += 8;
        if (bar == bars) {
            at = bar = 0;
            parity ^= 1;
        }
    }
};

// The tiles of one cluster, in order: t = cluster, cluster + clusters, ...
struct TileWalk {
    const int *lo, *first;
    int nt, pair_blocks, whole, end, step, t, e;   // from t = whole on, halves of tiles
    int rb, p0, count;   // of the current tile
    bool halved;
    __device__ __forceinline__ TileWalk(const int *lo_, const int *first_, const RaggedArgs &a, int start, int step_)
        : lo(lo_), first(first_), nt(a.nt), pair_blocks((a.row_blocks + 1) >> 1), whole(first_[a.E] * pair_blocks),
          end(whole), step(step_), t(start), e(0), halved(false)
    {
        if (rwide::halve_last_wave(whole, step, nt)) {
            const int last = whole % step;
            whole -= last;
            end += last;
        }
    }
    __device__ __forceinline__ bool locate()
    {
        if (t >= end) return false;
        const int tail = t - whole, tile = tail < 0 ? t : whole + (tail >> 1);
        while (tile >= first[e + 1] * pair_blocks) ++e;
        // a group's token tiles in runs of up to kRun; for each run the blocks of weight rows, for each its tiles
        const int tiles = first[e + 1] - first[e], local = tile - first[e] * pair_blocks;
        const int run = local / (rwide::kRun * pair_blocks), in_run = local - run * rwide::kRun * pair_blocks;
        const int width = min(rwide::kRun, tiles - run * rwide::kRun);
        rb = in_run / width;
        const int rows = tile_rows(lo[e + 1] - lo[e], nt);
        p0 = lo[e] + (run * rwide::kRun + in_run - rb * width) * rows;
        count = min(rows, lo[e + 1] - p0);
        if (tail >= 0) {
            halved = count > rwide::kNt / 2;
            if (!halved) return (tail & 1) == 0;   // (no cluster has another tile behind it)
            const int part = (((count + 1) >> 1) + 31) & ~31;
            if (tail & 1) {
                p0 += part;
                count -= part;
            } else {
                count = part;
            }
        }
        return true;
    }
    __device__ __forceinline__ void next() { t += step; }
};

template <bool kInt8, bool kGather, bool kSwiglu>
__global__ void __launch_bounds__(rwide::threads_of(kGather), 2)
ragged_wide_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ BoxMaps xmaps,
                   const __grid_constant__ RaggedArgs a)
{
    using namespace rwide;
    constexpr int kStageK = kInt8 ? 128 : 64, kThreads = threads_of(kGather);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t *tail = smem + a.ring_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(tail);   // used in the pair's even CTA
    uint64_t *empty = full + kMaxPipe;
    uint64_t *acc_full = empty + kMaxPipe;
    uint64_t *acc_empty = acc_full + 2;                    // used in the pair's even CTA
    uint64_t *free_all = acc_empty + 2;                    // split: every pair is done with its stages
    uint64_t *landed = free_all + 1;                       // split: all parts of this CTA's runs are here
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(landed + 1);
    int *part = reinterpret_cast<int *>(tail + 256);
    float *scales = reinterpret_cast<float *>(tail + kOffScales), *exchange = scales;
    int *lo = reinterpret_cast<int *>(tail + kOffGroups), *first = lo + a.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const StatusPtrs status{nullptr, a.status_out};
    const int split = a.split;                             // pairs of the cluster: consecutive ranges of K
    const uint32_t crank = cluster_rank(), leader = crank & ~1u;
    const int half_id = static_cast<int>(crank & 1), slice = static_cast<int>(crank >> 1);
    const int cluster = blockIdx.x / (2 * split), clusters = gridDim.x / (2 * split);
    const int kb0 = a.kblocks * slice / split, kb1 = a.kblocks * (slice + 1) / split;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&xmaps.m[kGather ? 0 : a.nt / 32 - 1]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(a.accs * a.acc_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 64) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);   // four epilogue warps of both CTAs
        }
        mbar_init(free_all, split);
        mbar_init(landed, 1);
        fence_barrier_init();
    }
    if (a.offsets == nullptr && threadIdx.x == 96) {   // one group
        lo[0] = first[0] = 0;
        lo[1] = a.R;
        first[1] = tile_count(a.R, a.nt);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();   // barriers and tensor memory of all CTAs are ready
    tc_fence_after();
    if (a.offsets != nullptr) {
        pdl_wait();
        if (a.E < 32)
            build_few_groups(a.offsets, a.R, a.E, a.nt, lo, first);
        else
            build_groups<kThreads>(a.offsets, a.R, a.E, a.nt, lo, first, part);
    }
    const uint32_t tmem = *tmem_slot;
    bool aborted = false;
    TileWalk w(lo, first, a, cluster, clusters);
    bool more = w.locate();
    const TileWalk tile0 = w;
    const bool any = more;
    const bool elected = elect_one();
    const uint32_t ring0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const uint32_t full_pair = map_cluster(full0, leader);
    if (a.offsets == nullptr) pdl_wait();   // (one group: all of the above is ready by then)
    pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------ weights
        Ring ring(a);
        int issued = 0;
        const uint32_t lost = blockIdx.x == 0 ? a.waits.lost : 0;
        for (; more && !aborted; w.next(), more = w.locate()) {
            const int half = ((w.count + 31) & ~31) >> 1, block = 2 * w.rb + half_id;
            // weight rows past the expert's last come from the next one, or are zeros: nobody stores their products
            const int wrow = kSwiglu ? w.e * 2 * a.N + block * 64 : w.e * a.N + block * kRows;
            // of both CTAs, weights and tokens
            const uint32_t bytes = 2 * (kABytes + (kGather ? max(half, 4 * kGatherWarps) : box_rows(a, half, w.halved)) * kStageKBytes);
            for (int kb = kb0; kb < kb1; ++kb, ring.next(), ++issued) {
                if (!warp_wait(empty0 + ring.bar, ring.parity ^ 1, aborted, status, a.waits.limit)) break;
                const uint32_t sa = ring0 + ring.at, bar = full_pair + ring.bar;
                if (elected) {
                    if (half_id == 0) expect_tx(full0 + ring.bar, bytes + lost);
                    tma_load_2d_pair(sa, &wmap, kb * kStageK, wrow, bar);   // swiglu: 64 gate rows, then their up rows
                    if (kSwiglu) tma_load_2d_pair(sa + kABytes / 2, &wmap, kb * kStageK, wrow + a.N, bar);
                }
            }
        }
        // the MMA warp's releases of the last stages arrive while this CTA lives
        __syncwarp();
        const int filled = min(issued, a.stages);
        for (int i = issued - filled; i < issued && !aborted; ++i)
            warp_wait(empty0 + 8 * (i % a.stages), (i / a.stages) & 1, aborted, status, a.waits.limit);
        // after a timeout the even CTA waits for both CTAs' copies in flight: the stages before the one it gave up on
        if (aborted && half_id == 0)
            for (int i = 0; i < a.stages && i < issued; ++i) {
                const int back = issued - 1 - i;
                mbar_wait_drain(&full[back % a.stages], (back / a.stages) & 1, status, a.waits.limit);
            }
    } else if (!kGather && warp == 2) {
        // ------------------------------------------------------------ tokens: one box
        Ring ring(a);
        for (; more && !aborted; w.next(), more = w.locate()) {
            const int half = ((w.count + 31) & ~31) >> 1, map = box_rows(a, half, w.halved) / 16 - 1, row0 = w.p0 + half_id * half;
            for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
                if (!warp_wait(empty0 + ring.bar, ring.parity ^ 1, aborted, status, a.waits.limit)) break;
                if (elected)
                    tma_load_2d_pair(ring0 + ring.at + kABytes, &xmaps.m[map], kb * kStageK, row0, full_pair + ring.bar);
            }
        }
    } else if (warp == 1 && half_id == 0) {
        // ------------------------------------------------------------ MMA issuer
        Ring ring(a);
        const uint64_t desc = umma_sdesc_sw128(ring0);
        const uint32_t desc_lo = static_cast<uint32_t>(desc), desc_hi = static_cast<uint32_t>(desc >> 32);
        int i = 0;
        for (; more && !aborted; w.next(), more = w.locate(), ++i) {
            const int b = a.accs > 1 ? i & 1 : 0, n32 = (w.count + 31) & ~31;
            const uint32_t idesc = kInt8 ? umma_idesc_i8(256, n32) : umma_idesc_bf16(256, n32);
            const uint32_t acc = tmem + b * a.acc_cols;
            if (!warp_wait(smem_u32(&acc_empty[b]), ((i >> 1) & 1) ^ 1, aborted, status, a.waits.limit)) break;
            for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
                if (!warp_wait(full0 + ring.bar, ring.parity, aborted, status, a.waits.limit)) break;
                tc_fence_after();
                const uint32_t ad = desc_lo + (ring.at >> 4), bd = ad + (kABytes >> 4);
                if (elected) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_pair<kInt8>(acc, ad + 2 * j, bd + 2 * j, desc_hi, idesc, kb > kb0 || j > 0);
                    umma_commit_pair(empty0 + ring.bar, leader);
                }
            }
            if (aborted) break;
            if (elected) umma_commit_pair(smem_u32(&acc_full[b]), leader);
        }
        __syncwarp();
        // the epilogues' last arrivals, of the other CTA too, land while this CTA lives
        if (split == 1)
            for (int j = i > 1 ? i - 2 : 0; j < i; ++j)
                mbar_wait_cluster(&acc_empty[a.accs > 1 ? j & 1 : 0], (j >> 1) & 1, aborted, status, a.waits.limit);
    } else if (warp >= kEpi0 && warp < kEpi0 + 4 && split == 1) {
        // ------------------------------------------------------------ epilogue
        const int q = warp - kEpi0;
        int turn = 0;   // of the exchange buffers, over all tiles
        for (int i = 0; more; w.next(), more = w.locate(), ++i) {
            const int b = a.accs > 1 ? i & 1 : 0;
            const int block = 2 * w.rb + half_id;
            const int n = block * kRows + 32 * q + lane;
            float cs = 1.0f;
            float *rs = scales + b * kNt;
            if (kInt8) {
                if (n < a.N) cs = a.col_scale[n];
                for (int j = threadIdx.x - 32 * kEpi0; j < kNt; j += 128) rs[j] = j < w.count ? a.row_scale[w.p0 + j] : 0.f;
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            mbar_wait_for(&acc_full[b], (i >> 1) & 1, aborted, status, a.waits.limit);
            tc_fence_after();
            // (after a timeout the rest runs on whatever is there, so that the warps keep meeting at their barriers, and
            // NaN goes over it at the end)
            const uint32_t acc = tmem + b * a.acc_cols + (static_cast<uint32_t>(32 * q) << 16);
            if (kSwiglu) {
                // Gate rows are lanes 0..63 (warps q = 0, 1), their up rows lanes 64..127 (q = 2, 3).  Warps q and
                // q ^ 2 exchange halves of 16 columns: the gate warp finishes the first 8, the up warp the others.
                const int up = q >> 1, ns = block * 64 + 32 * (q & 1) + lane;
                for (int c = 0; c < w.count; c += 16, turn ^= 1) {
                    uint32_t v[16];
                    tmem_ld16(acc + c, v);
                    float *ex = exchange + turn * 1024;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ex[q * 256 + j * 32 + lane] = __uint_as_float(up ? v[j] : v[8 + j]);
                    asm volatile("bar.sync %0, 64;" ::"r"(2 + (q & 1)) : "memory");
                    uint32_t h[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float other = ex[(q ^ 2) * 256 + j * 32 + lane];
                        const float own = __uint_as_float(up ? v[8 + j] : v[j]);
                        h[j] = __float_as_uint(ragged_swiglu(up ? other : own, up ? own : other));
                    }
                    const int c0 = c + 8 * up;
                    finish_columns<false, 8>(a, h, nullptr, 1.0f, nullptr, static_cast<size_t>(w.p0) + c0, w.count - c0, ns);
                }
            } else {
                for (int c = 0; c < w.count; c += kEpiCols) {
                    const size_t row = static_cast<size_t>(w.p0) + c;
                    __nv_bfloat16 add[kEpiCols];
                    load_add<kInt8>(a, row, w.count - c, n, add);
                    uint32_t v[kEpiCols];
                    tmem_ld16(acc + c, v);
                    finish_columns<kInt8, kEpiCols>(a, v, rs + c, cs, add, row, w.count - c, n);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(map_cluster(smem_u32(&acc_empty[b]), leader));
        }
    } else if (kGather && warp >= kGather0) {
        // ------------------------------------------------------------ gather
        // Runs of four rows go round the warps, lane i of warp g taking run g + 8 i.  With 16 rows, four runs, the last
        // four warps copy them once more: every warp has a part in every stage, since one that only watched could fall
        // behind by a whole turn of the ring, whose barriers tell two turns apart and no more.
        const int g = warp - kGather0;
        Ring ring(a);
        for (; more; w.next(), more = w.locate()) {
            const int half = ((w.count + 31) & ~31) >> 1;
            const int first_run = 4 * g < half ? g : g - half / 4;
            const int run = first_run + kGatherWarps * lane;
            const bool mine = 4 * run < half && (lane == 0 || first_run == g);
            int idx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(half_id * half + 4 * run + i, w.count - 1);
                const uint32_t f = mine ? static_cast<uint32_t>(a.sorted_ids[w.p0 + r]) : 0u;
                idx[i] = static_cast<int>(min(f / static_cast<uint32_t>(a.k), static_cast<uint32_t>(a.M - 1)));
            }
            for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
                if (!warp_wait(empty0 + ring.bar, ring.parity ^ 1, aborted, status, a.waits.limit)) break;
                if (mine)
                    tma_gather4_pair(ring0 + ring.at + kABytes + run * 4 * kStageKBytes, &xmaps.m[0], kb * kStageK, idx,
                                     full_pair + ring.bar);
                __syncwarp();
            }
            if (aborted) break;
        }
    }
    if (split > 1) {
        // ------------------------------------------------------------ joining the slices of K
        // The cluster has one tile at most.  Runs of 8 columns go round the pairs: run u is summed and stored by the
        // pair u % split, whose CTAs get all slices' parts of it in shared memory, over the stages:
        // [slice][run / split][column half][row][4].  All sums in slice order.  The CTAs tell each other that their
        // stages are free, and the parts report themselves as they land (with two cluster barriers instead, of all threads
        // and with their memory ordered, 8 tokens x 2048 x 4096 took 7.6 us and not 7.1).
        const TileWalk &t = tile0;
        const bool found = warp < 8 && any;
        __syncwarp();
        aborted = __any_sync(0xffffffffu, aborted);
        const int runs = found ? (t.count + 7) >> 3 : 0, own = (runs + split - 1) / split;
        const int group = warp >> 2, row = 32 * (warp & 3) + lane;
        if (found) {
            const int block = 2 * t.rb + half_id;
            const int n = block * kRows + row;
            float cs = 1.0f;
            __nv_bfloat16 add[8];
            if (kInt8) {   // all that the end needs from memory
                if (n < a.N) cs = a.col_scale[n];
                if (threadIdx.x < kNt) scales[threadIdx.x] = threadIdx.x < t.count ? a.row_scale[t.p0 + threadIdx.x] : 0.f;
                const int c = 8 * (group * split + slice);
                load_add<kInt8>(a, static_cast<size_t>(t.p0) + c, t.count - c, n, add);
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
            mbar_wait_for(&acc_full[0], 0, aborted, status, a.waits.limit);
            tc_fence_after();
            // (who gave up tells nobody that it is done and sends nothing: its peers' waits give up too)
            if (warp == 0 && lane < split && !aborted)
                mbar_arrive_cluster_relaxed(map_cluster(smem_u32(free_all), static_cast<uint32_t>(2 * lane + half_id)));
            if (warp == 1 && lane == 0)
                mbar_arrive_expect_tx(landed, static_cast<uint32_t>((runs - slice + split - 1) / split * split * kRunBytes));
            __syncwarp();
            mbar_wait_for(free_all, 0, aborted, status, a.waits.limit);
            aborted = __any_sync(0xffffffffu, aborted);
            const uint32_t acc = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
            for (int u = group; u < runs && !aborted; u += 2) {
                uint32_t v[8];
                tmem_ld8(acc + 8 * u, v);
                const uint32_t to = static_cast<uint32_t>(2 * (u % split) + half_id), bar = map_cluster(smem_u32(landed), to);
                const uint32_t at = map_cluster(smem_u32(smem) + (slice * own + u / split) * kRunBytes + row * 16, to);
                st_async4(at, v, bar);
                st_async4(at + kRunBytes / 2, v + 4, bar);
            }
            mbar_wait_cluster(landed, 0, aborted, status, a.waits.limit);
            // part of slice s for run i, column half h, accumulator row r
            auto part = [&](int s, int i, int h, int r) {
                return *reinterpret_cast<const uint4 *>(smem + (s * own + i) * kRunBytes + h * (kRunBytes / 2) + r * 16);
            };
            auto sum = [&](int i, int h, int r, uint32_t *out) {
                uint4 p = part(0, i, h, r);
                for (int s = 1; s < split; ++s) {
                    const uint4 q = part(s, i, h, r);
                    p.x = ragged_add<kInt8>(p.x, q.x);
                    p.y = ragged_add<kInt8>(p.y, q.y);
                    p.z = ragged_add<kInt8>(p.z, q.z);
                    p.w = ragged_add<kInt8>(p.w, q.w);
                }
                out[0] = p.x;
                out[1] = p.y;
                out[2] = p.z;
                out[3] = p.w;
            };
            for (int i = group; i * split + slice < runs && !aborted; i += 2) {
                const int c = 8 * (i * split + slice), live = t.count - c;
                const size_t row0 = static_cast<size_t>(t.p0) + c;
                if (kSwiglu) {   // two threads per output row, four columns each
                    const int r = row & 63, h = row >> 6;
                    uint32_t g[4], up[4], v[4];
                    sum(i, h, r, g);
                    sum(i, h, 64 + r, up);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = __float_as_uint(ragged_swiglu(__uint_as_float(g[j]), __uint_as_float(up[j])));
                    finish_columns<false, 4>(a, v, nullptr, 1.0f, nullptr, row0 + 4 * h, live - 4 * h, block * 64 + r);
                } else {
                    uint32_t v[8];
                    sum(i, 0, row, v);
                    sum(i, 1, row, v + 4);
                    finish_columns<kInt8, 8>(a, v, scales + c, cs, add, row0, live, n);
                    load_add<kInt8>(a, row0 + 16 * split, live - 16 * split, n, add);   // of run i + 2
                }
            }
        }
    }
    __syncwarp();
    aborted = __any_sync(0xffffffffu, aborted);
    tc_fence_before();
    // Neither CTA ends while the other's MMAs read it.  What a CTA sent to another has been waited for there, so nothing
    // needs ordering; a warp that gave up on a wait cannot know, and orders everything.
    if (aborted) {
        cluster_sync();
        __nanosleep(100000);   // parts that others have sent land while this CTA lives
        // What this warp has stored of the cluster's tiles, or would have, becomes NaN: the sums behind it may lack parts.
        if (split == 1 ? warp >= kEpi0 && warp < kEpi0 + 4 : warp < 8) {
            const int q = warp & 3, row = 32 * q + lane;
            for (TileWalk t(lo, first, a, cluster, clusters); t.locate(); t.next()) {
                const int block = 2 * t.rb + half_id;
                if (split == 1 && !kSwiglu) {
                    store_nan(a, t.p0, t.count, block * kRows + row);
                } else if (split == 1) {
                    const int up = 8 * (q >> 1);
                    for (int c = up; c < t.count; c += 16)
                        store_nan(a, t.p0 + c, min(8, t.count - c), block * 64 + 32 * (q & 1) + lane);
                } else {
                    for (int c = 8 * ((warp >> 2) * split + slice); c < t.count; c += 16 * split) {
                        const int h = 4 * (row >> 6);
                        if (kSwiglu)
                            store_nan(a, t.p0 + c + h, min(4, t.count - c - h), block * 64 + (row & 63));
                        else
                            store_nan(a, t.p0 + c, min(8, t.count - c), block * kRows + row);
                    }
                }
            }
        }
    } else {
        cluster_sync_relaxed();
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.accs * a.acc_cols) : "memory");
}

// ------------------------------------------------------------------ launch

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
    cfg.gridDim = dim3(static_cast<unsigned>(2 * p.split * p.clusters));
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * p.split;
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
