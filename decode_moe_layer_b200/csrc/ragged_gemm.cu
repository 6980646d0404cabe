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
// ragged_gemm_kernel: one tile (128 weight rows x up to `nt` tokens) per cluster of `split` CTAs.  The
// CTAs of a cluster take consecutive ranges of K; each holds a partial accumulator, sends the columns
// that another CTA owns into that CTA's shared memory and sums its own in rank order, so the result
// does not depend on timing and no workspace is needed.  Warp 0 issues the TMA copies (weights as one
// box, tokens as 16-row boxes or, by the routing's indices, four rows at a time), warp 1 the MMAs; all
// four warps store.  The tile of a cluster is found from the group offsets on the device.
//
// Every wait is bounded: one that runs out reports MOE_ERR_TIMEOUT, the copies in flight are waited
// for, and the tensor memory is freed.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace moe {

namespace ragged {
constexpr int kRows = 128;       // weight rows per tile (MMA M)
constexpr int kStageKBytes = 128;   // bytes of K per stage: one 128-byte swizzle row
constexpr int kABytes = kRows * kStageKBytes;
constexpr int kBoxRows = 16;     // token rows per TMA box
constexpr int kMaxStages = 8;
constexpr int kThreads = 128;
constexpr int kTailBytes = 256;  // barriers, tile description
}  // namespace ragged

// D (+)= A * B^T, both operands in shared memory (K-major, 128-byte swizzle).
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Instruction descriptor of kind::i8: s32 accumulator (bits 4-5 = 2), signed A and B (bits 7-9 and
// 10-12 = 1), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ uint32_t umma_idesc_i8(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// 5-D tiled copy of a weight box, and a gather of four rows of a 2-D map (box one row high).
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int c0, const int (&r)[4], uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t smem_addr, uint32_t rank, uint32_t v)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

// clamp-SwiGLU that lets a NaN through (a comparison with NaN is false).
__device__ __forceinline__ float ragged_swiglu(float g, float u)
{
    const float a = g > 7.0f ? 7.0f : g;
    const float c = u > 7.0f ? 7.0f : (u < -7.0f ? -7.0f : u);
    return a / (1.0f + expf(-a)) * c;
}

// One value of the product, final: scaled (int8), rounded to the output's type and stored.
template <bool kInt8>
__device__ __forceinline__ void ragged_store(const RaggedArgs &a, float v, size_t row, int n)
{
    const size_t at = row * static_cast<size_t>(a.N) + n;
    if (kInt8 && a.add != nullptr) v += __bfloat162float(a.add[at]);
    if (a.y_f32)
        static_cast<float *>(a.y)[at] = v;
    else
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
}

// The tt-th token tile of the groups, found by one warp: lanes take E / 32 consecutive groups each.
// Offsets are clamped to [0, R] and to ascending order, so wrong ones cannot lead out of the tensors.
__device__ __forceinline__ bool find_tile(const int32_t *off, int R, int E, int nt, int tt, int &expert, int &p0,
                                          int &count)
{
    const int lane = threadIdx.x & 31;
    if (off == nullptr) {
        expert = 0;
        p0 = tt * nt;
        count = min(nt, R - p0);
        return count > 0;
    }
    const int per = (E + 31) >> 5, e0 = lane * per, e1 = min(E, e0 + per);
    int mine = 0;
    int lo = e0 < E ? min(max(__ldcg(off + e0), 0), R) : 0;
    const int lo0 = lo;
#pragma unroll 8
    for (int e = e0; e < e1; ++e) {
        const int hi = min(max(__ldcg(off + e + 1), lo), R);
        mine += (hi - lo + nt - 1) / nt;
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
            const int hi = min(max(__ldcg(off + e + 1), lo), R);
            const int n = (hi - lo + nt - 1) / nt;
            if (t < n) {
                fe = e;
                fp = lo + t * nt;
                fc = min(nt, hi - fp);
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
        const bool found = find_tile(a.offsets, a.R, a.E, a.nt, tt, e, p, c);
        if (lane == 0) {
            tile[0] = found;
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
            const uint32_t bytes = kABytes + (kGather ? groups * 4 : n16) * kStageKBytes;
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % a.stages;
                mbar_wait(&empty[s], ((it / a.stages) & 1) ^ 1, aborted, status);
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                uint8_t *sa = smem + s * stage_bytes, *sb = sa + kABytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], bytes);
                    tma_load_5d(sa, &wmap, kb * kStageK, kSwiglu ? 0 : rb * kRows, 0, kSwiglu ? rb * 4 : 0, expert,
                                &full[s]);
                }
                __syncwarp();
                if (kGather) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (lane + 32 * h < groups)
                            tma_gather4(sb + (lane + 32 * h) * 4 * kStageKBytes, &xmap, kb * kStageK, idx[h], &full[s]);
                } else if (lane < n16 / kBoxRows) {
                    tma_load_2d(sb + lane * kBoxRows * kStageKBytes, &xmap, kb * kStageK, p0 + lane * kBoxRows,
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
                    for (int j = 0; j < 4; ++j) {   // 32 bytes of K each
                        if (kInt8)
                            umma_i8_ss(tmem, ad + 2 * j, bd + 2 * j, idesc, it > 0 || j > 0);
                        else
                            umma_f16_ss(tmem, ad + 2 * j, bd + 2 * j, idesc, it > 0 || j > 0);
                    }
                    umma_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit(smem_u32(done));
            __syncwarp();
        }
        __syncwarp();
        // every MMA of this CTA has completed: the accumulator is whole, the stages are free
        mbar_wait_drain(done, 0, status);
        tc_fence_after();

        // ------------------------------------------------------------ epilogue
        // this thread's weight row is TMEM lane 32 * warp + lane
        const uint32_t acc = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const int n = kSwiglu ? rb * 64 + 16 * warp + (lane & 15) : rb * kRows + 32 * warp + lane;
        const bool n_ok = n < a.N;
        const float cs = kInt8 && n_ok ? a.col_scale[n] : 1.0f;
        // the value of column c (of the two columns c, c + 1 when kSwiglu: gate rows sit in lanes 0..15,
        // their up rows in lanes 16..31; the lower half finishes column c, the upper half c + 1)
        auto finish = [&](uint32_t b0, uint32_t b1, int c, int cols) {
            if (kSwiglu) {
                const float v0 = __uint_as_float(b0), v1 = __uint_as_float(b1);
                const bool up = lane >= 16;
                const float other = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 16);
                const float h = up ? ragged_swiglu(other, v1) : ragged_swiglu(v0, other);
                const int col = c + (up ? 1 : 0);
                if (n_ok && col < cols) ragged_store<false>(a, h, static_cast<size_t>(p0) + col, n);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = c + q;
                    if (!n_ok || col >= cols) continue;
                    const uint32_t b = q == 0 ? b0 : b1;
                    const size_t row = static_cast<size_t>(p0) + col;
                    float v;
                    if (kInt8)
                        v = static_cast<float>(static_cast<int32_t>(b)) * a.row_scale[row] * cs;
                    else
                        v = __uint_as_float(b);
                    ragged_store<kInt8>(a, v, row, n);
                }
            }
        };
        if (split == 1) {
            for (int c = 0; c < n16; c += 16) {
                uint32_t v[16];
                tmem_ld16(acc + c, v);
#pragma unroll
                for (int j = 0; j < 16; j += 2) finish(v[j], v[j + 1], c + j, count);
            }
        } else {
            // rank r owns columns [r * own, (r + 1) * own); `own` is even, for the column pairs
            const int own = ((n16 + 2 * split - 1) / (2 * split)) * 2;
            const uint32_t buf = smem_u32(smem);   // [split][own][128] words over the stages
            cluster_sync();                        // every CTA's MMAs are done with its stages
            for (int c = 0; c < n16; c += 16) {
                uint32_t v[16];
                tmem_ld16(acc + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int to = (c + j) / own, lc = (c + j) - to * own;
                    st_cluster(buf + ((rank * own + lc) * kRows + 32 * warp + lane) * 4, to, v[j]);
                }
            }
            cluster_sync();
            const uint32_t *part = reinterpret_cast<const uint32_t *>(smem) + 32 * warp + lane;
            for (int lc = 0; lc < own; lc += 2) {
                const int c = rank * own + lc;
                if (c >= count) break;   // warp-uniform
                uint32_t s[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (kInt8) {
                        int32_t t = 0;
                        for (int r = 0; r < split; ++r) t += static_cast<int32_t>(part[(r * own + lc + q) * kRows]);
                        s[q] = static_cast<uint32_t>(t);
                    } else {
                        float t = 0.f;
                        for (int r = 0; r < split; ++r) t += __uint_as_float(part[(r * own + lc + q) * kRows]);
                        s[q] = __float_as_uint(t);
                    }
                }
                finish(s[0], s[1], c, count);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, tmem_cols);
}

// ------------------------------------------------------------------ launch

RaggedPlan ragged_plan(int R, int N, int K, int E, bool int8, bool swiglu)
{
    RaggedPlan p;
    const int avg = (R + E - 1) / E;
    // widest token tile; MMAs and copies follow the group's own size, so this only sets the stage size
    if (E == 1)
        p.nt = avg <= 32 ? 32 : (avg <= 64 ? 64 : (avg <= 128 ? 128 : 256));
    else
        p.nt = avg <= 8 ? 32 : (avg <= 32 ? 64 : (avg <= 96 ? 128 : 256));
    p.stages = p.nt == 32 ? 5 : (p.nt == 128 ? 6 : 4);
    p.smem = 1024 + p.stages * (ragged::kABytes + p.nt * ragged::kStageKBytes) + ragged::kTailBytes;
    p.row_blocks = swiglu ? (N + 63) / 64 : (N + ragged::kRows - 1) / ragged::kRows;
    p.kblocks = (K * (int8 ? 1 : 2) + ragged::kStageKBytes - 1) / ragged::kStageKBytes;
    p.max_tiles = (R < E ? R : E) + R / p.nt;
    if (E == 1) p.max_tiles = (R + p.nt - 1) / p.nt;
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
