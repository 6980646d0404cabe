// block_norm.cu -- the norms before and after a block with the block's gate and the residual scale in
// one pass over the rows (moe_block_norm), and the int8 codes of rows (moe_int8_quantize).
//
//   z  = x * rsqrt(mean(x^2) + eps) * (w_post + o)      (z = x without w_post)
//   r' = block_scale * gate * z + residual_scale * r     (stored as bf16)
//   h  = r' * rsqrt(mean(r'^2) + eps) * (w_pre + o)      (stored as bf16 and / or int8 codes)
//   q  = rne(h / s), s = max|h| / 127 per row
//
// A row stays in the registers of one CTA, so x, r, r' and h each cross HBM once.  All arithmetic is in
// fp32; r' and h are rounded once, as they are stored, and h is computed from the unrounded r'.  The
// codes need no reduction of their own: max|h| = rsqrt(..) * max|r' (w_pre + o)| comes with the second sum.
#include <cuda_bf16.h>

#include "common.cuh"
#include "moe.h"
#include "ops.h"

namespace moe {

namespace norm {
constexpr int kVec = 8;             // elements per 16-byte vector
constexpr int kMaxThreads = 1024;
}  // namespace norm

__device__ __forceinline__ void unpack8(uint4 p, float (&f)[8])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The code of v for the row scale s = max / 127: rne(v / s), |code| <= 127; a row of zeros has s = 0 and codes 0.
__device__ __forceinline__ uint32_t int8_code(float v, float s)
{
    const int c = s > 0.f ? __float2int_rn(v / s) : 0;
    return static_cast<uint32_t>(max(-127, min(127, c))) & 0xFFu;
}
__device__ __forceinline__ uint2 int8_codes8(const float (&f)[8], float s)
{
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo |= int8_code(f[i], s) << (8 * i);
        hi |= int8_code(f[4 + i], s) << (8 * i);
    }
    return make_uint2(lo, hi);
}

// Sum and maximum of a pair over the CTA; every thread gets both.  `buf` holds one pair per warp and is
// free again after the next call's barrier on the other buffer (callers alternate two).
__device__ __forceinline__ float2 block_sum_max(float sum, float mx, float2 *buf)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(sum, mx);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float2 v = lane < static_cast<int>(blockDim.x >> 5) ? buf[lane] : make_float2(0.f, 0.f);
    sum = v.x;
    mx = v.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    }
    return make_float2(sum, mx);
}

template <int V>
__global__ void __launch_bounds__(norm::kMaxThreads) block_norm_kernel(const __grid_constant__ NormArgs a)
{
    using norm::kVec;
    __shared__ float2 red[2][32];
    const int nvec = a.H / kVec;
    const float inv_h = 1.0f / static_cast<float>(a.H);
    pdl_wait();
    pdl_trigger();
    for (int row = blockIdx.x; row < a.M; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * nvec;
        float v[V][8], r[V][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nvec) {
                unpack8(reinterpret_cast<const uint4 *>(a.x)[base + c], v[i]);
                if (a.residual != nullptr) unpack8(reinterpret_cast<const uint4 *>(a.residual)[base + c], r[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
            }
        }
        float scale = a.block_scale;
        if (a.gate_kind == MOE_GATE_TOKEN) scale *= static_cast<const float *>(a.gate)[row];
        if (a.w_post != nullptr) scale *= rsqrtf(block_sum_max(ss, 0.f, red[0]).x * inv_h + a.eps);
        const size_t gbase = a.gate_kind == MOE_GATE_FULL ? base : 0;
        float ss2 = 0.f, mx = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float t[8];
            if (a.w_post != nullptr) {
                unpack8(reinterpret_cast<const uint4 *>(a.w_post)[c], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] *= t[j] + a.w_offset;
            }
            if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL) {
                unpack8(reinterpret_cast<const uint4 *>(a.gate)[gbase + c], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] *= t[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= scale;
                if (a.residual != nullptr) v[i][j] = fmaf(a.residual_scale, r[i][j], v[i][j]);
                ss2 = fmaf(v[i][j], v[i][j], ss2);
            }
            if (a.res_out != nullptr) reinterpret_cast<uint4 *>(a.res_out)[base + c] = pack8(v[i]);
            if (a.w_pre != nullptr) {
                unpack8(reinterpret_cast<const uint4 *>(a.w_pre)[c], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] *= t[j] + a.w_offset;
                    mx = fmaxf(mx, fabsf(v[i][j]));
                }
            }
        }
        if (a.w_pre == nullptr) {
            __syncthreads();   // red[0] is free for the next row
            continue;
        }
        const float2 st = block_sum_max(ss2, mx, red[1]);
        const float inv = rsqrtf(st.x * inv_h + a.eps);
        const float qs = st.y * inv / 127.0f;
        if (a.q_out != nullptr && threadIdx.x == 0) a.q_s[row] = qs;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= inv;
            if (a.h_out != nullptr) reinterpret_cast<uint4 *>(a.h_out)[base + c] = pack8(v[i]);
            if (a.q_out != nullptr) reinterpret_cast<uint2 *>(a.q_out)[base + c] = int8_codes8(v[i], qs);
        }
    }
}

// Codes of the rows of x [M, K], or of clamp-SwiGLU of the rows' halves [gate | up] ([M, 2K], kSwiglu;
// the activation stays in fp32).
template <int V, bool kSwiglu>
__global__ void __launch_bounds__(norm::kMaxThreads)
int8_quantize_kernel(const __nv_bfloat16 *x, int8_t *q, float *q_s, int M, int K)
{
    using norm::kVec;
    __shared__ float2 red[2][32];
    const int nvec = K / kVec;
    pdl_wait();
    pdl_trigger();
    int turn = 0;
    for (int row = blockIdx.x; row < M; row += gridDim.x, turn ^= 1) {
        const uint4 *src = reinterpret_cast<const uint4 *>(x) + static_cast<size_t>(row) * nvec * (kSwiglu ? 2 : 1);
        float v[V][8];
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            unpack8(src[c], v[i]);
            if (kSwiglu) {
                float u[8];
                unpack8(src[nvec + c], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float g = fminf(v[i][j], 7.0f);
                    v[i][j] = g / (1.0f + expf(-g)) * fminf(fmaxf(u[j], -7.0f), 7.0f);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[i][j]));
        }
        const float s = block_sum_max(0.f, mx, red[turn]).y / 127.0f;
        if (threadIdx.x == 0) q_s[row] = s;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nvec) reinterpret_cast<uint2 *>(q)[static_cast<size_t>(row) * nvec + c] = int8_codes8(v[i], s);
        }
    }
}

// ------------------------------------------------------------------ launch

// Rows of up to 1024 vectors: a vector per thread; longer ones two.
static int row_threads(int nvec, int v)
{
    const int t = (nvec + v - 1) / v;
    return (t + 31) / 32 * 32;
}

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s)
{
    const int nvec = a.H / norm::kVec;
    const int v = nvec <= norm::kMaxThreads ? 1 : 2;
    const int threads = row_threads(nvec, v);
    const int grid = a.M;
    return v == 1 ? launch_ex(block_norm_kernel<1>, dim3(grid), dim3(threads), 0, s, true, a)
                  : launch_ex(block_norm_kernel<2>, dim3(grid), dim3(threads), 0, s, true, a);
}

cudaError_t launch_int8_quantize(const __nv_bfloat16 *x, bool swiglu, int8_t *q, float *q_s, int M, int K,
                                 cudaStream_t s)
{
    const int nvec = K / norm::kVec;
    const int v = nvec <= norm::kMaxThreads ? 1 : 2;
    const dim3 threads(row_threads(nvec, v)), grid(M);
    if (swiglu)
        return v == 1 ? launch_ex(int8_quantize_kernel<1, true>, grid, threads, 0, s, true, x, q, q_s, M, K)
                      : launch_ex(int8_quantize_kernel<2, true>, grid, threads, 0, s, true, x, q, q_s, M, K);
    return v == 1 ? launch_ex(int8_quantize_kernel<1, false>, grid, threads, 0, s, true, x, q, q_s, M, K)
                  : launch_ex(int8_quantize_kernel<2, false>, grid, threads, 0, s, true, x, q, q_s, M, K);
}

}  // namespace moe
