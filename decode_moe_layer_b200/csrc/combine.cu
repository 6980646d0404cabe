// combine.cu -- the weighted sum of a token's k expert rows, taken straight from the expert-grouped
// order (moe_combine):
//
//   out[t] = bf16( sum_j w[t,j] * y[inv_pos[t*k+j]] + add[t] )
//
// Bound by memory: each row of y is read once.  A thread owns one vector of 8 columns of a token and has eight
// (then four, two, one) of its k pieces in flight before it adds them, in slot order, in fp32, with one rounding.
// The loads are unconditional, a dropped slot reading row 0 and adding nothing: behind branches they went out one
// after the other (2048 tokens x 8 x 7168 with an addend: 100 us; now 51, 5.7 TB/s).
#include <cuda_bf16.h>

#include "common.cuh"
#include "ops.h"

namespace moe {

// acc[v] += w[j] * y[pos[j]] for kBatch slots and kVecs vectors of columns (c, c + step, ..).
template <bool kF32, int kBatch, int kVecs>
__device__ __forceinline__ void add_rows(const uint4 *y, const float *w, const int32_t *pos, int R, int nvec, int c,
                                         int step, float (&acc)[kVecs][8])
{
    constexpr int kWords = kF32 ? 2 : 1;
    uint4 p[kBatch][kVecs][kWords];
    float wj[kBatch];
    bool live[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int at = __ldcg(pos + i);
        live[i] = at >= 0 && at < R;   // any other position: a dropped assignment
        wj[i] = __ldcg(w + i);
        const uint4 *src = y + static_cast<size_t>(live[i] ? at : 0) * nvec * kWords;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int h = 0; h < kWords; ++h) p[i][v][h] = __ldcs(src + min(c + v * step, nvec - 1) * kWords + h);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float f[8];
#pragma unroll
            for (int h = 0; h < kWords; ++h) {
                const uint32_t u[4] = {p[i][v][h].x, p[i][v][h].y, p[i][v][h].z, p[i][v][h].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (kF32) {
                        f[4 * h + q] = __uint_as_float(u[q]);
                    } else {
                        f[2 * q] = __uint_as_float(u[q] << 16);
                        f[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[v][q] = live[i] ? fmaf(wj[i], f[q], acc[v][q]) : acc[v][q];
        }
}

template <bool kF32, int kBatch, int kVecs>
__global__ void __launch_bounds__(256, 3)
combine_rows_kernel(const void *y, const float *topk_w, const int32_t *inv_pos, const __nv_bfloat16 *add,
                    __nv_bfloat16 *out, int M, int nvec, int k)
{
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, step = blockDim.x, c = blockIdx.y * (step * kVecs) + threadIdx.x;
    if (c >= nvec) return;
    const size_t id = static_cast<size_t>(t) * nvec + c;
    const int R = M * k;
    const uint4 *rows = static_cast<const uint4 *>(y);
    const float *w = topk_w + t * k;
    const int32_t *pos = inv_pos + t * k;
    uint4 sum[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
        sum[v] = add != nullptr && c + v * step < nvec ? __ldcg(reinterpret_cast<const uint4 *>(add) + id + v * step)
                                                       : make_uint4(0u, 0u, 0u, 0u);
    float acc[kVecs][8] = {};
    int j = 0;
    for (; j + kBatch <= k; j += kBatch) add_rows<kF32, kBatch, kVecs>(rows, w + j, pos + j, R, nvec, c, step, acc);
    if (kBatch > 4 && j + 4 <= k) {
        add_rows<kF32, 4, kVecs>(rows, w + j, pos + j, R, nvec, c, step, acc);
        j += 4;
    }
    if (kBatch > 2 && j + 2 <= k) {
        add_rows<kF32, 2, kVecs>(rows, w + j, pos + j, R, nvec, c, step, acc);
        j += 2;
    }
    if (kBatch > 1 && j < k) add_rows<kF32, 1, kVecs>(rows, w + j, pos + j, R, nvec, c, step, acc);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        if (c + v * step >= nvec) continue;
        const uint32_t u[4] = {sum[v].x, sum[v].y, sum[v].z, sum[v].w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 b =
                __floats2bfloat162_rn(acc[v][2 * q] + __uint_as_float(u[q] << 16),
                                      acc[v][2 * q + 1] + __uint_as_float(u[q] & 0xFFFF0000u));
            o[q] = *reinterpret_cast<const uint32_t *>(&b);
        }
        reinterpret_cast<uint4 *>(out)[id + v * step] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <bool kF32, int kBatch, int kVecs>
static cudaError_t launch_combine_t(const void *y, const float *topk_w, const int32_t *inv_pos,
                                    const __nv_bfloat16 *add, __nv_bfloat16 *out, int M, int nvec, int k, cudaStream_t s)
{
    const int chunks = (nvec + 256 * kVecs - 1) / (256 * kVecs);   // of a token's columns
    const int threads = ((nvec + chunks * kVecs - 1) / (chunks * kVecs) + 31) / 32 * 32;
    return launch_ex(combine_rows_kernel<kF32, kBatch, kVecs>, dim3(M, chunks), dim3(threads), 0, s, true, y, topk_w,
                     inv_pos, add, out, M, nvec, k);
}

cudaError_t launch_combine_rows(const void *y, bool y_f32, const float *topk_w, const int32_t *inv_pos,
                                const __nv_bfloat16 *add, __nv_bfloat16 *out, int M, int H, int k, cudaStream_t s)
{
    const int nvec = H / 8;
    if (y_f32) return launch_combine_t<true, 4, 1>(y, topk_w, inv_pos, add, out, M, nvec, k, s);
    // few slots: more columns a thread, for the sake of loads in flight
    if (k < 8) return launch_combine_t<false, 4, 2>(y, topk_w, inv_pos, add, out, M, nvec, k, s);
    return launch_combine_t<false, 8, 1>(y, topk_w, inv_pos, add, out, M, nvec, k, s);
}

}  // namespace moe
