// ragged.cuh -- what the kernels of the ragged products share: matrix products whose rows come in groups of any
// size, bf16 expert weights with ragged groups of tokens (moe_grouped_gemm) and int8 weights with one group
// (moe_int8_gemm):
//
//   y[p][n] = epilogue( sum_c w[e(p)][n][c] * x[row(p)][c] )
//
// For a token or a few, weight rows are streamed by warps (ragged_rows.cu); all else runs in tiles on tcgen05 by
// pairs of CTAs (ragged_wide.cu), whose width follows the groups' sizes.  Here: tcgen05 and cluster forms, the
// table of token tiles, the epilogue.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ops.h"
#include "ragged_plan.h"
#include "tcgen05.cuh"

namespace moe {

// ------------------------------------------------------------------ tcgen05, both operands in shared memory

// Instruction descriptor of kind::i8: s32 accumulator (bits 4-5 = 2), signed A and B (bits 7-9 and
// 10-12 = 1), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ uint32_t umma_idesc_i8(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// D (+)= A * B^T over 32 bytes of K by the CTA pair: kind::f16 (16 bf16 elements) or kind::i8 (32 int8 elements).
// Issued by the pair's even CTA; each CTA holds half of A's rows and half of B's.  a, b: the low words of the
// operands' descriptors (umma_sdesc_sw128), which hold the address; hi: the high word of both.
template <bool kInt8>
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate)
{
    if (kInt8)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                     "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
                     "tcgen05.mma.cta_group::2.kind::i8 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
                     "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                     "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
                     "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// 8 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Without ordering memory: for the end of a kernel, where it only keeps CTAs alive (the ordering form waits until
// the stores before it have arrived, 1000 cycles and more).
__device__ __forceinline__ void cluster_sync_relaxed()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared-memory address of CTA `rank` of the cluster that corresponds to this CTA's smem_addr.
__device__ __forceinline__ uint32_t map_cluster(uint32_t smem_addr, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr), "r"(rank));
    return remote;
}
// Stores 16 bytes in another CTA's shared memory and reports them to that CTA's barrier as they land.
__device__ __forceinline__ void st_async4(uint32_t cluster_addr, const uint32_t *v, uint32_t cluster_bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.u32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(cluster_addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(cluster_bar)
                 : "memory");
}

// Sum of two accumulator words.
template <bool kInt8>
__device__ __forceinline__ uint32_t ragged_add(uint32_t a, uint32_t b)
{
    return kInt8 ? a + b : __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// ------------------------------------------------------------------ token tiles

// The groups of the rows, in shared memory: lo[e] is where group e starts (lo[E] where the last ends) and
// first[e] the number of token tiles before it.  A group of c rows is cut into ceil(c / nt) tiles of equal
// size rounded up to 32 rows (the MMA's N step), so that no tile is left with a few rows and a full price.
// Offsets are clamped to [0, R] and to ascending order, so wrong ones cannot lead out of the tensors.
__device__ __forceinline__ int tile_rows(int c, int nt)
{
    if (c <= nt) return nt;
    const int t = (c + nt - 1) / nt;
    return ((c + t - 1) / t + 31) & ~31;
}
__device__ __forceinline__ int tile_count(int c, int nt)
{
    if (c <= nt) return c > 0;
    const int rows = tile_rows(c, nt);
    return (c + rows - 1) / rows;
}
// A scan over the CTA's kThreads threads, inclusive: op is addition or maximum.  `part` holds one value per warp;
// the caller puts a barrier between two scans.
template <int kThreads, typename Op>
__device__ __forceinline__ int block_scan(int v, int *part, Op op)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = op(v, o);
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32 - 1; ++w)
        if (w < warp) v = op(v, part[w]);
    return v;
}
// The table for up to 31 groups by every warp for itself, the same values in the same places: without a barrier, which
// would cost a small call 0.4 us.
__device__ __forceinline__ void build_few_groups(const int32_t *off, int R, int E, int nt, int *lo, int *first)
{
    const int e = threadIdx.x & 31;
    int start = e <= E ? min(max(off[e], 0), R) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, start, d);
        if (e >= d) start = max(start, v);
    }
    const int before = __shfl_up_sync(0xffffffffu, start, 1);
    int tiles = e > 0 && e <= E ? tile_count(start - before, nt) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, tiles, d);
        if (e >= d) tiles += v;
    }
    if (e <= E) {
        lo[e] = start;
        first[e] = tiles;
    }
    __syncwarp();
}

// The table by a whole CTA of kThreads threads; `lo` and `first` hold E + 1 ints each, `part` 64.  Ends with a barrier.
template <int kThreads>
__device__ __forceinline__ void build_groups(const int32_t *off, int R, int E, int nt, int *lo, int *first, int *part)
{
    int high = 0, tiles = 0;   // of the groups before this round's
    for (int base = 0; base <= E; base += kThreads) {
        const int e = base + static_cast<int>(threadIdx.x);
        // where the group starts, not before any earlier one
        const int at = e <= E ? min(max(off[e], 0), R) : 0;
        const int start = max(high, block_scan<kThreads>(at, part, [](int a, int b) { return max(a, b); }));
        if (e <= E) lo[e] = start;
        __syncthreads();
        // the group before e is whole now (entry base - 1 comes from the round before)
        const int mine = e > 0 && e <= E ? tile_count(lo[e] - lo[e - 1], nt) : 0;
        const int sum = tiles + block_scan<kThreads>(mine, part + 32, [](int a, int b) { return a + b; });
        if (e <= E) first[e] = sum;
        __syncthreads();
        if (base + kThreads <= E) {
            high = lo[base + kThreads - 1];
            tiles = first[base + kThreads - 1];
        }
    }
}

// ------------------------------------------------------------------ epilogue

// clamp-SwiGLU that lets a NaN through (a comparison with NaN is false).
__device__ __forceinline__ float ragged_swiglu(float g, float u)
{
    const float a = g > 7.0f ? 7.0f : g;
    const float c = u > 7.0f ? 7.0f : (u < -7.0f ? -7.0f : u);
    return a / (1.0f + expf(-a)) * c;
}

// One pair of gate and up, finished and stored at y[row][n].
__device__ __forceinline__ void store_pair(const RaggedArgs &a, float g, float u, size_t row, int n)
{
    const size_t at = row * static_cast<size_t>(a.N) + n;
    const float h = ragged_swiglu(g, u);
    if (a.y_f32)
        static_cast<float *>(a.y)[at] = h;
    else
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(h);
}

// NaN in column n of `count` rows of y from `row` on.
__device__ __forceinline__ void store_nan(const RaggedArgs &a, int row, int count, int n)
{
    if (n >= a.N) return;
    const size_t ld = static_cast<size_t>(a.N), at = row * ld + n;
    for (int j = 0; j < count; ++j) {
        if (a.y_f32)
            static_cast<float *>(a.y)[at + j * ld] = __int_as_float(0x7FFFFFFF);
        else
            static_cast<__nv_bfloat16 *>(a.y)[at + j * ld] = __ushort_as_bfloat16(0x7FFF);
    }
}

// The addend of kCols columns as finish_columns takes it.  The loads are unconditional, the last live column's again
// past it: behind branches they go out one after the other.
template <bool kInt8, int kCols>
__device__ __forceinline__ void load_add(const RaggedArgs &a, size_t row, int live, int n, __nv_bfloat16 (&t)[kCols])
{
    if (!kInt8 || a.add == nullptr || n >= a.N || live <= 0) return;
    const size_t ld = static_cast<size_t>(a.N);
    const __nv_bfloat16 *add = a.add + row * ld + n;
#pragma unroll
    for (int j = 0; j < kCols; ++j) t[j] = add[min(j, live - 1) * ld];
}

// Finishes kCols accumulator columns (consecutive rows of y from `row`, of which `live` are the tile's) of
// the weight row n: scales and adds (int8: rs[] the rows' scales, cs the channel's, t[] the addend), rounds once and
// stores.
// For a column a warp writes 64 consecutive bytes (bf16), whole sectors.  The common case, all columns live,
// has no branch between columns: a thread's chain of address, conversion and store took about 120 cycles a
// column when each column branched, and a fifth of that without.
template <bool kInt8, int kCols>
__device__ __forceinline__ void finish_columns(const RaggedArgs &a, const uint32_t (&v)[kCols], const float *rs, float cs,
                                               const __nv_bfloat16 *t, size_t row, int live, int n)
{
    if (n >= a.N) return;
    const size_t ld = static_cast<size_t>(a.N);
    const size_t at = row * ld + n;
    float f[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        f[j] = kInt8 ? static_cast<float>(static_cast<int32_t>(v[j])) * rs[j] * cs : __uint_as_float(v[j]);
    if (kInt8 && a.add != nullptr) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) f[j] += __bfloat162float(t[j]);
    }
    if (a.y_f32) {
        float *y = static_cast<float *>(a.y) + at;
        if (live >= kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) y[j * ld] = f[j];
        } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                if (j < live) y[j * ld] = f[j];
        }
    } else {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + at;
        if (live >= kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) y[j * ld] = __float2bfloat16_rn(f[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                if (j < live) y[j * ld] = __float2bfloat16_rn(f[j]);
        }
    }
}

}  // namespace moe
