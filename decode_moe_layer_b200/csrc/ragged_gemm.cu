// ragged_gemm.cu -- matrix products whose rows come in groups of any size: bf16 expert weights with
// ragged groups of tokens (moe_grouped_gemm) and int8 weights with one group (moe_int8_gemm).
//
//   y[p][n] = epilogue( sum_c w[e(p)][n][c] * x[row(p)][c] )
//
// Both run on tcgen05 with the accumulator in tensor memory, kind::f16 (bf16 products, fp32 sums) or
// kind::i8 (int8 products, int32 sums, exact).  128 bytes of K, 64 bf16 or 128 int8 values, are one
// pipeline stage and four MMAs in either type, so one kernel serves both.
//
// The weight rows are the MMA's M side (128 per tile) and the tokens its N side, whose width follows
// the group: a tile of `count` tokens runs MMAs of N = count rounded up to 16, so a group of one row
// costs what one row costs, and rows beyond a group reach only accumulator columns that nobody stores.
//
// This file has the kernel for few rows per group and the choice between it and the one for many
// (ragged_wide.cu).  ragged_gemm_kernel: one tile (128 weight rows x up to `nt` tokens) per cluster of
// `split` CTAs.  The CTAs of a cluster take consecutive ranges of K; each holds a partial accumulator,
// sends the columns that another CTA owns into that CTA's shared memory and sums its own in rank order, so
// the result does not depend on timing and no workspace is needed.  Warp 0 issues the TMA copies (weights
// as one box, tokens as 16-row boxes or, by the routing's indices, four rows at a time), warp 1 the MMAs; all
// four warps store.  The tensor maps have two dimensions: boxes of a map with three or more came in at 10.6 TB/s
// from L2 over the whole chip, those of a flat one at 16.9, and a TMA instruction costs about 100 cycles whatever its
// size, so boxes are as high as the tile allows.  The tile of a cluster is found from the group offsets on the device.
//
// Every wait is bounded: one that runs out reports MOE_ERR_TIMEOUT, the copies in flight are waited
// for, and the tensor memory is freed.
#include <atomic>

#include "ragged.cuh"

namespace moe {

namespace ragged {
constexpr int kMaxStages = 8;
constexpr int kThreads = 128;
constexpr int kTailBytes = 256;  // barriers, tile description
}  // namespace ragged

// A gather of four rows of a 2-D map (box one row high).
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int c0, const int (&r)[4], uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_u32(bar))
        : "memory");
}

// The tt-th token tile of the groups, found by one warp: lanes take ceil(E / 32) consecutive groups each.  A
// group of c rows is cut as in build_groups.  Offsets are clamped to [0, R], so wrong ones cannot lead out of
// the tensors.
__device__ __forceinline__ bool find_tile(const int32_t *off, int R, int E, int nt, int tt, int &expert, int &p0,
                                          int &count)
{
    const int lane = threadIdx.x & 31;
    const int per = (E + 31) >> 5, e0 = lane * per, e1 = min(E, e0 + per);
    auto at = [&](int e) { return off != nullptr ? min(max(__ldcg(off + e), 0), R) : (e == 0 ? 0 : R); };
    int mine = 0;
    const int lo0 = e0 < E ? at(e0) : 0;
    int lo = lo0;
#pragma unroll 8
    for (int e = e0; e < e1; ++e) {
        const int hi = max(at(e + 1), lo);
        mine += tile_count<16>(hi - lo, nt);
        lo = hi;
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    const bool here = tt >= incl - mine && tt < incl;
    const uint32_t who = __ballot_sync(0xffffffffu, here);
    if (who == 0) return false;
    int fe = 0, fp = 0, fc = 0;
    if (here) {
        int t = tt - (incl - mine);
        lo = lo0;
        for (int e = e0; e < e1; ++e) {
            const int hi = max(at(e + 1), lo), n = tile_count<16>(hi - lo, nt);
            if (t < n) {
                const int rows = tile_rows<16>(hi - lo, nt);
                fe = e;
                fp = lo + t * rows;
                fc = min(rows, hi - fp);
                break;
            }
            t -= n;
            lo = hi;
        }
    }
    const int src = __ffs(who) - 1;
    expert = __shfl_sync(0xffffffffu, fe, src);
    p0 = __shfl_sync(0xffffffffu, fp, src);
    count = __shfl_sync(0xffffffffu, fc, src);
    return true;
}

template <bool kInt8, bool kGather, bool kSwiglu>
__global__ void __launch_bounds__(ragged::kThreads)
ragged_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const __grid_constant__ RaggedArgs a)
{
    using namespace ragged;
    constexpr int kStageK = kInt8 ? 128 : 64;   // elements of K per stage
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int stage_bytes = kABytes + a.nt * kStageKBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + a.stages * stage_bytes);
    uint64_t *empty = full + kMaxStages;
    uint64_t *done = empty + kMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *tile = reinterpret_cast<volatile int *>(tmem_slot + 2);   // found, expert, p0, count
    float *rs = reinterpret_cast<float *>(smem + a.stages * stage_bytes + kTailBytes);   // [nt], int8

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const StatusPtrs status{nullptr, a.status_out};
    const int split = a.split;
    const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / split;
    const int rb = unit % a.row_blocks, tt = unit / a.row_blocks;
    const int tmem_cols = max(32, a.nt);   // nt is a power of two

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&xmap);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    if (threadIdx.x == 64) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_barrier_init();
    }
    pdl_wait();
    if (warp == 0) {
        int e = 0, p = 0, c = 0;
        const bool ok = find_tile(a.offsets, a.R, a.E, a.nt, tt, e, p, c);
        if (lane == 0) {
            tile[0] = ok;
            tile[1] = e;
            tile[2] = p;
            tile[3] = c;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const bool found = tile[0];   // the same for every CTA of the cluster
    const int expert = tile[1], p0 = tile[2], count = tile[3];
    const int n16 = (count + 15) & ~15;
    const int kb0 = a.kblocks * rank / split, kb1 = a.kblocks * (rank + 1) / split;
    bool aborted = false;

    if (found) {
        if (warp == 0) {
            // ------------------------------------------------------------ TMA producer
            int idx[2][4];
            const int groups = (count + 3) >> 2;
            if (kGather) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = min(4 * (lane + 32 * h) + i, count - 1);
                        const uint32_t f = static_cast<uint32_t>(__ldcg(a.sorted_ids + p0 + p));
                        idx[h][i] = static_cast<int>(min(f / static_cast<uint32_t>(a.k), static_cast<uint32_t>(a.M - 1)));
                    }
            }
            const int boxes = (n16 + a.box_rows - 1) / a.box_rows;
            const uint32_t bytes = kABytes + (kGather ? groups * 4 : boxes * a.box_rows) * kStageKBytes;
            // rows past the expert's last come from the next one, or are zeros: nobody stores their products
            const int wrow = kSwiglu ? expert * 2 * a.N + rb * 64 : expert * a.N + rb * kRows;
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % a.stages;
                mbar_wait(&empty[s], ((it / a.stages) & 1) ^ 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                uint8_t *sa = smem + s * stage_bytes, *sb = sa + kABytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], bytes);
                    if (kSwiglu) {   // 64 gate rows, then their 64 up rows
                        tma_load_2d(sa, &wmap, kb * kStageK, wrow, &full[s]);
                        tma_load_2d(sa + kABytes / 2, &wmap, kb * kStageK, wrow + a.N, &full[s]);
                    } else {
                        tma_load_2d(sa, &wmap, kb * kStageK, wrow, &full[s]);
                    }
                }
                __syncwarp();
                if (kGather) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (lane + 32 * h < groups)
                            tma_gather4(sb + (lane + 32 * h) * 4 * kStageKBytes, &xmap, kb * kStageK, idx[h], &full[s]);
                } else if (lane < boxes) {
                    tma_load_2d(sb + lane * a.box_rows * kStageKBytes, &xmap, kb * kStageK, p0 + lane * a.box_rows,
                                &full[s]);
                }
                __syncwarp();
            }
            // copies in flight land before the CTA can end (on the usual path the MMAs have waited for them)
            if (aborted)
                for (int i = 0; i < a.stages && i < it; ++i) {
                    const int j = it - 1 - i;
                    mbar_wait_drain(&full[j % a.stages], (j / a.stages) & 1, status);
                }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            const uint32_t idesc = kInt8 ? umma_idesc_i8(kRows, n16) : umma_idesc_bf16(kRows, n16);
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % a.stages;
                mbar_wait(&full[s], (it / a.stages) & 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * stage_bytes);
                const uint64_t ad = umma_sdesc_sw128(sa), bd = umma_sdesc_sw128(sa + kABytes);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)   // 32 bytes of K each
                        umma_ss<kInt8, 1>(tmem, ad + 2 * j, bd + 2 * j, idesc, it > 0 || j > 0);
                    umma_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit(smem_u32(done));
            __syncwarp();
        } else if (kInt8) {
            for (int i = threadIdx.x - 64; i < n16; i += 64) rs[i] = i < count ? a.row_scale[p0 + i] : 0.f;
        }
        __syncwarp();
        // every MMA of this CTA has completed: the accumulator is whole, the stages are free
        mbar_wait_drain(done, 0, status);
        if (kInt8) __syncthreads();   // rs
        tc_fence_after();

        // ------------------------------------------------------------ epilogue
        // this thread's accumulator row is TMEM lane 32 * warp + lane
        const uint32_t acc = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const int n = rb * kRows + 32 * warp + lane;
        const float cs = kInt8 && n < a.N ? a.col_scale[n] : 1.0f;
        if (!kSwiglu && split == 1) {
            for (int c = 0; c < n16; c += 16) {
                uint32_t v[16];
                tmem_ld16(acc + c, v);
                finish_columns<kInt8, 16>(a, v, rs + c, cs, static_cast<size_t>(p0) + c, count - c, n);
            }
        } else {
            // The accumulators go through shared memory, over the stages: [split][own][128] words in the CTA that
            // owns the columns (rank r: r * own ..).  With one CTA, for the sake of SwiGLU alone, whose gate rows
            // are lanes 0..63 and up rows lanes 64..127.
            const int own = ((n16 + 2 * split - 1) / (2 * split)) * 2;
            const uint32_t buf = smem_u32(smem);
            if (split > 1)
                cluster_sync();   // every CTA's MMAs are done with its stages
            else
                __syncthreads();
            for (int c = 0; c < n16; c += 16) {
                uint32_t v[16];
                tmem_ld16(acc + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int to = split > 1 ? (c + j) / own : 0, lc = (c + j) - to * own;
                    const uint32_t at = buf + ((rank * own + lc) * kRows + 32 * warp + lane) * 4;
                    if (split > 1)
                        st_cluster(map_cluster(at, to), v[j]);
                    else
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v[j]) : "memory");
                }
            }
            if (split > 1)
                cluster_sync();
            else
                __syncthreads();
            const uint32_t *part = reinterpret_cast<const uint32_t *>(smem);
            auto sum = [&](int lc, int r128) -> uint32_t {   // of the CTAs' parts, in rank order
                const uint32_t *q = part + lc * kRows + r128;
                if (kInt8) {
                    int32_t t = 0;
                    for (int r = 0; r < split; ++r) t += static_cast<int32_t>(q[r * own * kRows]);
                    return static_cast<uint32_t>(t);
                }
                float t = 0.f;
                for (int r = 0; r < split; ++r) t += __uint_as_float(q[r * own * kRows]);
                return __float_as_uint(t);
            };
            const int mine = min(own, count - rank * own);   // of this CTA's columns, those of the tile
            const size_t row0 = static_cast<size_t>(p0) + rank * own;
            if (kSwiglu) {
                const int r64 = threadIdx.x & 63, ns = rb * 64 + r64;
                if (ns < a.N)
                    for (int lc = threadIdx.x >> 6; lc < mine; lc += 2)
                        store_pair(a, __uint_as_float(sum(lc, r64)), __uint_as_float(sum(lc, 64 + r64)), row0 + lc, ns);
            } else {
                for (int lc = 0; lc < mine; lc += 2) {
                    const uint32_t v[2] = {sum(lc, 32 * warp + lane), sum(lc + 1, 32 * warp + lane)};
                    finish_columns<kInt8, 2>(a, v, rs + rank * own + lc, cs, row0 + lc, mine - lc, n);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, tmem_cols);
}

// ------------------------------------------------------------------ launch

RaggedPlan ragged_plan(int R, int N, int K, int E, bool int8, bool swiglu, bool gather)
{
    RaggedPlan p = {};
    const int avg = (R + E - 1) / E;
    p.row_blocks = swiglu ? (N + 63) / 64 : (N + ragged::kRows - 1) / ragged::kRows;
    p.kblocks = (K * (int8 ? 1 : 2) + ragged::kStageKBytes - 1) / ragged::kStageKBytes;
    const long long pair_tiles = static_cast<long long>(E == 1 ? (R + 255) / 256 : (R < E ? R : E) + R / 256) *
                                 ((p.row_blocks + 1) / 2);
    p.wide = avg >= (E == 1 ? 128 : 32) && pair_tiles >= kPlanSMs / 2;
    if (p.wide) {
        p.nt = 256;
        p.split = 1;
        wide_plan(p, E, gather);
        return p;
    }
    // widest token tile; MMAs and copies follow the group's own size, so this only sets the stage size
    if (E == 1)
        p.nt = avg <= 32 ? 32 : (avg <= 64 ? 64 : (avg <= 128 ? 128 : 256));
    else
        p.nt = avg <= 8 ? 32 : (avg <= 32 ? 64 : (avg <= 96 ? 128 : 256));
    p.box_rows = p.nt / 2;
    p.stages = p.nt == 32 ? 5 : (p.nt == 128 ? 6 : 4);
    p.smem = 1024 + p.stages * (ragged::kABytes + p.nt * ragged::kStageKBytes) + ragged::kTailBytes + p.nt * 4;
    p.max_tiles = E == 1 ? (R + p.nt - 1) / p.nt : (R < E ? R : E) + R / p.nt;
    const long long units = static_cast<long long>(p.max_tiles) * p.row_blocks;
    const int want = 2 * kPlanSMs;
    p.split = 1;
    while (p.split < 8 && units * p.split * 2 <= want && p.split * 4 <= p.kblocks) p.split *= 2;
    return p;
}

template <bool kInt8, bool kGather, bool kSwiglu>
static cudaError_t launch_ragged_t(const CUtensorMap &wmap, const CUtensorMap &xmap, const RaggedArgs &a,
                                   const RaggedPlan &p, cudaStream_t s)
{
    auto kernel = ragged_gemm_kernel<kInt8, kGather, kSwiglu>;
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
    cfg.gridDim = dim3(static_cast<unsigned>(p.max_tiles) * p.row_blocks * p.split);
    cfg.blockDim = dim3(ragged::kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, a);
}

cudaError_t launch_ragged(bool int8, bool swiglu, const CUtensorMap &wmap, const CUtensorMap &xmap, const RaggedArgs &a,
                          const RaggedPlan &p, cudaStream_t s)
{
    const bool gather = a.sorted_ids != nullptr;
    if (int8) return launch_ragged_t<true, false, false>(wmap, xmap, a, p, s);
    if (gather)
        return swiglu ? launch_ragged_t<false, true, true>(wmap, xmap, a, p, s)
                      : launch_ragged_t<false, true, false>(wmap, xmap, a, p, s);
    return swiglu ? launch_ragged_t<false, false, true>(wmap, xmap, a, p, s)
                  : launch_ragged_t<false, false, false>(wmap, xmap, a, p, s);
}

}  // namespace moe
