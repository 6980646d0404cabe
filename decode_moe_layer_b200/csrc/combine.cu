// combine.cu -- the weighted sum of a token's k expert rows, taken straight from the expert-grouped
// order (moe_combine):
//
//   out[t] = bf16( sum_j w[t,j] * y[inv_pos[t*k+j]] + add[t] )
//
// Bound by memory: each row of y is read once.  A thread owns one vector of 8 columns of a token, loads
// its k pieces before it adds them (slot order, fp32) and rounds once.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ops.h"

namespace moe {

template <bool kF32>
__global__ void __launch_bounds__(256)
combine_rows_kernel(const void *y, const float *topk_w, const int32_t *inv_pos, const __nv_bfloat16 *add,
                    __nv_bfloat16 *out, int M, int nvec, int k)
{
    pdl_wait();
    pdl_trigger();
    const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int t = static_cast<int>(id / nvec), c = static_cast<int>(id - static_cast<long long>(t) * nvec);
    if (t >= M) return;
    const int R = M * k;
    float acc[8] = {};
    constexpr int kBatch = kF32 ? 4 : 8;
    for (int j0 = 0; j0 < k; j0 += kBatch) {
        uint4 p[kBatch][kF32 ? 2 : 1];
        float w[kBatch];
        bool live[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + i;
            const int pos = j < k ? __ldcg(inv_pos + t * k + j) : -1;
            live[i] = pos >= 0 && pos < R;   // any other position: a dropped assignment
            if (!live[i]) continue;
            w[i] = __ldcg(topk_w + t * k + j);
            const uint4 *src = static_cast<const uint4 *>(y) + (static_cast<size_t>(pos) * nvec + c) * (kF32 ? 2 : 1);
            p[i][0] = __ldcg(src);
            if (kF32) p[i][kF32 ? 1 : 0] = __ldcg(src + 1);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!live[i]) continue;
            const uint32_t u[4] = {p[i][0].x, p[i][0].y, p[i][0].z, p[i][0].w};
            if (kF32) {
                const uint4 p1 = p[i][kF32 ? 1 : 0];
                const uint32_t u1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[q] = fmaf(w[i], __uint_as_float(u[q]), acc[q]);
                    acc[4 + q] = fmaf(w[i], __uint_as_float(u1[q]), acc[4 + q]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[2 * q] = fmaf(w[i], __uint_as_float(u[q] << 16), acc[2 * q]);
                    acc[2 * q + 1] = fmaf(w[i], __uint_as_float(u[q] & 0xFFFF0000u), acc[2 * q + 1]);
                }
            }
        }
    }
    if (add != nullptr) {
        const uint4 p = reinterpret_cast<const uint4 *>(add)[id];
        const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            acc[2 * q] += __uint_as_float(u[q] << 16);
            acc[2 * q + 1] += __uint_as_float(u[q] & 0xFFFF0000u);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
        o[q] = *reinterpret_cast<const uint32_t *>(&b);
    }
    reinterpret_cast<uint4 *>(out)[id] = make_uint4(o[0], o[1], o[2], o[3]);
}

cudaError_t launch_combine_rows(const void *y, bool y_f32, const float *topk_w, const int32_t *inv_pos,
                                const __nv_bfloat16 *add, __nv_bfloat16 *out, int M, int H, int k, cudaStream_t s)
{
    const int nvec = H / 8;
    const long long n = static_cast<long long>(M) * nvec;
    const int threads = 256;
    const dim3 grid(static_cast<unsigned>((n + threads - 1) / threads));
    return y_f32 ? launch_ex(combine_rows_kernel<true>, grid, dim3(threads), 0, s, true, y, topk_w, inv_pos, add, out,
                             M, nvec, k)
                 : launch_ex(combine_rows_kernel<false>, grid, dim3(threads), 0, s, true, y, topk_w, inv_pos, add, out,
                             M, nvec, k);
}

}  // namespace moe
