// block_norm.cu -- the norms before and after a block with the block's gate and the residual scale in
// one pass over the rows (moe_block_norm), and the int8 codes of rows (moe_int8_quantize).
//
//   z  = x * rsqrt(mean(x^2) + eps) * (w_post + o)      (z = x without w_post)
//   r' = block_scale * gate * z + residual_scale * r     (stored as bf16)
//   h  = r' * rsqrt(mean(r'^2) + eps) * (w_pre + o)      (stored as bf16 and / or int8 codes)
//   q  = rne(127 h / max|h|), s = max|h| / 127 per row
//
// A row stays in the registers of one CTA, so x, r, r' and h each cross HBM once.  All arithmetic is in
// fp32; r' and h are rounded once, as they are stored, and h is computed from the unrounded r'.  The
// codes need no reduction of their own: max|h| = rsqrt(..) * max|r' (w_pre + o)| comes with the second sum.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "moe.h"
#include "ops.h"

namespace moe {

namespace norm {
constexpr int kVec = 8;             // elements per 16-byte vector
constexpr int kMaxThreads = 1024;
constexpr int kRingThreads = 512;   // ring kernel: up to 4 vectors a thread
constexpr int kMaxStages = 4;
constexpr int kRingBytes = 200 * 1024;   // of an SM's shared memory, over its CTAs
constexpr int kRingRows = 4 * kPlanSMs;  // rows from which on the ring kernel runs
constexpr int kWideVecs = 512;           // wider rows: from the second row of an SM on
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

// The codes rne(127 v / max) of eight values and the row scale s = max / 127; a row of zeros has s = 0 and codes 0, one
// with NaN or Inf a scale that is not finite and codes 0.
// `inv` is 1 / s.  v * inv is off from the quotient by less than 127 * 2^-22, so the two round to the same integer
// unless it lies that near to a half (one value in five thousand).  Only then the side of the half is decided, by
// comparing 254 v with (2 n + 1) max, whose products an FMA completes to all their bits: the rounded s would decide ties
// at random, and ties are common (bf16 rows hold max / 2, whose code is 63.5).  Rounded with a division each, the codes
// took 2.5 times as long as their memory traffic.  Rows whose scale is below 2^-100, where 1 / s may overflow and the
// products' last bits fall below fp32's smallest number, are decided one by one after a multiplication by 2^100 (their
// inv has a minus sign); their scale, as it is stored, may be denormal or 0.
struct CodeScale {
    float s, inv, top;   // inv 0: a row of zeros, with NaN or with Inf
    __device__ __forceinline__ explicit CodeScale(float max_abs) : s(max_abs / 127.0f), inv(0.f), top(max_abs)
    {
        if (s > 0x1p-100f)
            inv = 1.0f / s;
        else if (top > 0.f)
            inv = -127.0f / (top * 0x1p100f);
    }
};
// One such code (not inlined: 32 copies of it cost the quantiser a quarter of its speed).
__device__ __noinline__ uint32_t int8_code_exact(float v, float inv, float max_abs)
{
    if (inv == 0.f) return 0;
    if (inv < 0.f) {
        v *= 0x1p100f;
        max_abs *= 0x1p100f;
        inv = -inv;
    }
    const float t = v * inv, r = rintf(t), n2 = 2.f * r + (t >= r ? 1.f : -1.f);   // n2 / 2: the half next to t
    const float a = 254.f * 0x1p-8f, top = max_abs * 0x1p-8f;   // (no overflow for the largest rows)
    const float p = n2 * top, w = a * v;
    const float d = (w - p) + (fmaf(a, v, -w) - fmaf(n2, top, -p));
    const float c = d > 0.f ? 0.5f * (n2 + 1.f) : (d < 0.f ? 0.5f * (n2 - 1.f) : rintf(0.5f * n2));
    return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(c))));
}
__device__ __forceinline__ uint2 int8_codes8(const float (&f)[8], const CodeScale &k)
{
    constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, held in the low bits
    uint32_t c[8];
    float far = 0.f;                        // largest distance from the integer taken
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = f[i] * k.inv, m = t + kMagic;
        c[i] = __float_as_uint(m);
        far = fmaxf(far, fabsf(t - (m - kMagic)));
    }
    if (!(far < 0.4999f) || !(k.inv > 0.f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = f[i] * k.inv;
            if (!(fabsf(t - rintf(t)) < 0.4999f) || !(k.inv > 0.f)) c[i] = int8_code_exact(f[i], k.inv, k.top);
        }
    }
    return make_uint2(prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u),
                      prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u));
}

// The larger of two values, NaN if either is (fmaxf would drop it): a row that holds NaN has to have a NaN scale.
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum and maximum (NaN if there is one) of a pair over the CTA; every thread gets both.  `buf` holds one pair per
// warp and is free again after the next call's barrier on the other buffer (callers alternate two).
__device__ __forceinline__ float2 block_sum_max(float sum, float mx, float2 *buf)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        mx = max_or_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
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
        mx = max_or_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    }
    return make_float2(sum, mx);
}

// Few rows: a CTA per row, every piece loaded before the first reduction, so that a row costs one trip to memory.
template <int V>
__global__ void __launch_bounds__(norm::kMaxThreads) block_norm_kernel(const __grid_constant__ NormArgs a)
{
    using norm::kVec;
    __shared__ float2 red[2][32];
    const int nvec = a.H / kVec, row = blockIdx.x;
    const size_t base = static_cast<size_t>(row) * nvec;
    pdl_wait();
    pdl_trigger();
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 x[V], p[4][V];   // residual, gate, w_post, w_pre
    const uint4 *src[4] = {reinterpret_cast<const uint4 *>(a.residual), nullptr,
                           reinterpret_cast<const uint4 *>(a.w_post), reinterpret_cast<const uint4 *>(a.w_pre)};
    if (a.residual != nullptr) src[0] += base;
    if (a.gate_kind == MOE_GATE_FULL) src[1] = static_cast<const uint4 *>(a.gate) + base;
    if (a.gate_kind == MOE_GATE_CHANNEL) src[1] = static_cast<const uint4 *>(a.gate);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        x[i] = c < nvec ? reinterpret_cast<const uint4 *>(a.x)[base + c] : zero;
#pragma unroll
        for (int q = 0; q < 4; ++q) p[q][i] = src[q] != nullptr && c < nvec ? src[q][c] : zero;
    }
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) unpack8(x[i], v[i]);
    const float inv_h = 1.0f / static_cast<float>(a.H);
    float scale = a.block_scale;
    if (a.gate_kind == MOE_GATE_TOKEN) scale *= static_cast<const float *>(a.gate)[row];
    if (a.w_post != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        scale *= rsqrtf(block_sum_max(ss, 0.f, red[0]).x * inv_h + a.eps);
    }
    float ss2 = 0.f, mx = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float t[8];
        if (a.w_post != nullptr) {
            unpack8(p[2][i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= t[j] + a.w_offset;
        }
        if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL) {
            unpack8(p[1][i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= t[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= scale;
        if (a.residual != nullptr) {
            unpack8(p[0][i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(a.residual_scale, t[j], v[i][j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss2 = fmaf(v[i][j], v[i][j], ss2);
        if (a.res_out != nullptr) reinterpret_cast<uint4 *>(a.res_out)[base + c] = pack8(v[i]);
        if (a.w_pre != nullptr) {
            unpack8(p[3][i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= t[j] + a.w_offset;
                mx = max_or_nan(mx, fabsf(v[i][j]));
            }
        }
    }
    if (a.w_pre == nullptr) return;
    const float2 st = block_sum_max(ss2, mx, red[1]);
    const float inv = rsqrtf(st.x * inv_h + a.eps);
    const CodeScale qs(st.y * inv);
    if (a.q_out != nullptr && threadIdx.x == 0) a.q_s[row] = qs.s;
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

// Two fp32 values in one register pair: sm_100's packed fp32 arithmetic, each half rounded as the scalar
// instruction rounds it.
struct f2 {
    float x, y;
};
__device__ __forceinline__ uint64_t f2_bits(f2 v)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ f2 f2_of(uint64_t r)
{
    f2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return f2_of(r);
}
__device__ __forceinline__ void unpack8(uint4 p, f2 (&f)[4])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
}
__device__ __forceinline__ uint4 pack8(const f2 (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// bulk_load of rows that nobody reads again: first to leave L2 (1 to 8% off the ring kernel's time).
__device__ __forceinline__ void bulk_load_once(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// NaN in every output of the CTA's rows from `row` on (codes 0).
__device__ __noinline__ void nan_rows(const NormArgs &a, long long row)
{
    const int nvec = a.H / norm::kVec;
    const uint4 bad = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    for (; row < a.M; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * nvec;
        for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
            if (a.res_out != nullptr) reinterpret_cast<uint4 *>(a.res_out)[base + c] = bad;
            if (a.h_out != nullptr) reinterpret_cast<uint4 *>(a.h_out)[base + c] = bad;
            if (a.q_out != nullptr) reinterpret_cast<uint2 *>(a.q_out)[base + c] = make_uint2(0u, 0u);
        }
        if (a.q_out != nullptr && threadIdx.x == 0) a.q_s[row] = __int_as_float(0x7FFFFFFF);
    }
}

// Many rows: a few CTAs per SM, each with its rows (blockIdx.x, + gridDim.x, ..) on their way through a ring of
// shared-memory stages (bulk copies of x, residual and a per-element gate), so that loads never wait for a
// reduction.  What is the same for every row stays in registers in fp32: f_post = block_scale * (w_post + o) *
// channel gate and f_pre = w_pre + o.  With a CTA per row 16384 x 7168 took 340 us; with this ring and
// packed weights taken apart for every row 175 us and 30 instructions an element, most of the issue slots; now 146 to
// 150, 96% of the memory's rate.
// A row whose copies have not come within the wait's limit is NaN in every output, and so are the CTA's rows behind it:
// there is no status word, and what the stage held would pass for values.
template <int V, bool kQuant, bool kFullGate>
__global__ void __launch_bounds__(norm::kRingThreads)
block_norm_ring_kernel(const __grid_constant__ NormArgs a, int stages)
{
    using norm::kVec;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float2 red[2][32];
    __shared__ uint64_t full[norm::kMaxStages];
    const int nvec = a.H / kVec;
    const float inv_h = 1.0f / static_cast<float>(a.H);
    const uint32_t row_bytes = static_cast<uint32_t>(a.H) * 2;
    const bool has_res = a.residual != nullptr, has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr;
    const uint32_t inputs = 1 + has_res + kFullGate;
    const uint32_t gate_at = (inputs - 1) * row_bytes;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint32_t lost = blockIdx.x == 0 ? a.waits.lost : 0;
    auto issue = [&](int s, int row) {   // thread 0
        uint8_t *dst = ring + s * inputs * row_bytes;
        const size_t at = static_cast<size_t>(row) * a.H;
        mbar_arrive_expect_tx(&full[s], inputs * row_bytes + lost);
        bulk_load_once(dst, a.x + at, row_bytes, &full[s]);
        if (has_res) bulk_load_once(dst + row_bytes, a.residual + at, row_bytes, &full[s]);
        if (kFullGate) bulk_load_once(dst + gate_at, static_cast<const __nv_bfloat16 *>(a.gate) + at, row_bytes, &full[s]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages; ++s) {
            const long long row = blockIdx.x + static_cast<long long>(s) * gridDim.x;
            if (row < a.M) issue(s, static_cast<int>(row));
        }
    f2 f_post[V][4], f_pre[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool in = c < nvec;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f_post[i][j] = {a.block_scale, a.block_scale};
            f_pre[i][j] = {1.f, 1.f};
        }
        f2 t[4];
        if (in && has_post) {
            unpack8(reinterpret_cast<const uint4 *>(a.w_post)[c], t);
#pragma unroll
            for (int j = 0; j < 4; ++j) f_post[i][j] = mul2(f_post[i][j], {t[j].x + a.w_offset, t[j].y + a.w_offset});
        }
        if (in && a.gate_kind == MOE_GATE_CHANNEL) {
            unpack8(static_cast<const uint4 *>(a.gate)[c], t);
#pragma unroll
            for (int j = 0; j < 4; ++j) f_post[i][j] = mul2(f_post[i][j], t[j]);
        }
        if (in && has_pre) {
            unpack8(reinterpret_cast<const uint4 *>(a.w_pre)[c], t);
#pragma unroll
            for (int j = 0; j < 4; ++j) f_pre[i][j] = {t[j].x + a.w_offset, t[j].y + a.w_offset};
        }
    }
    const StatusPtrs status{nullptr, nullptr};
    const f2 rs2 = {a.residual_scale, a.residual_scale};
    int s = 0, parity = 0;
    for (long long row = blockIdx.x; row < a.M; row += gridDim.x) {
        float tg = a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float *>(a.gate)[row] : 1.0f;
        bool late = false;
        mbar_wait_for(&full[s], parity, late, status, a.waits.limit);
        const uint8_t *st = ring + s * inputs * row_bytes;
        const size_t base = static_cast<size_t>(row) * nvec;
        f2 v[V][4];
        f2 ss = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            unpack8(c < nvec ? reinterpret_cast<const uint4 *>(st)[c] : make_uint4(0u, 0u, 0u, 0u), v[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma2(v[i][j], v[i][j], ss);
        }
        // No result hangs on this, since nan_rows below overwrites the row; with it the compiler orders the loop better:
        // 16384 x 7168 with a gate per token 146 us instead of 159.  With codes it would cost: 191 us instead of 183.
        if (!kQuant && late) tg = ss.x = __int_as_float(0x7FFFFFFF);
        float scale = tg;
        if (has_post) scale *= rsqrtf(block_sum_max(ss.x + ss.y, 0.f, red[0]).x * inv_h + a.eps);
        const f2 scale2 = {scale, scale};
        ss = {0.f, 0.f};
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            f2 t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(v[i][j], f_post[i][j]), scale2);
            if (kFullGate) {
                unpack8(reinterpret_cast<const uint4 *>(st + gate_at)[c], t);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], t[j]);
            }
            if (has_res) {
                unpack8(reinterpret_cast<const uint4 *>(st + row_bytes)[c], t);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = fma2(rs2, t[j], v[i][j]);
            }
            if (a.res_out != nullptr) reinterpret_cast<uint4 *>(a.res_out)[base + c] = pack8(v[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ss = fma2(v[i][j], v[i][j], ss);
                v[i][j] = mul2(v[i][j], f_pre[i][j]);
                if (kQuant) mx = max_or_nan(mx, max_or_nan(fabsf(v[i][j].x), fabsf(v[i][j].y)));
            }
        }
        if (has_pre) {
            const float2 sum = block_sum_max(ss.x + ss.y, mx, red[1]);
            const float inv = rsqrtf(sum.x * inv_h + a.eps);
            const f2 inv2 = {inv, inv};
            const CodeScale qs(sum.y * inv);
            if (kQuant && threadIdx.x == 0) a.q_s[row] = qs.s;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= nvec) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], inv2);
                if (a.h_out != nullptr) reinterpret_cast<uint4 *>(a.h_out)[base + c] = pack8(v[i]);
                if (kQuant) {
                    const float f[8] = {v[i][0].x, v[i][0].y, v[i][1].x, v[i][1].y,
                                        v[i][2].x, v[i][2].y, v[i][3].x, v[i][3].y};
                    reinterpret_cast<uint2 *>(a.q_out)[base + c] = int8_codes8(f, qs);
                }
            }
        }
        if (__syncthreads_or(late)) {   // (the stage has been read, the sums too)
            // not the row alone: whatever made its copies late, the ones behind it are no better
            nan_rows(a, row);
            if (threadIdx.x == 0)   // the copies in flight land while the CTA lives
                for (int left = stages; row < a.M && left > 0; row += gridDim.x, --left) {
                    mbar_wait_drain(&full[s], parity, status, a.waits.limit);
                    if (++s == stages) {
                        s = 0;
                        parity ^= 1;
                    }
                }
            return;
        }
        const long long next = row + static_cast<long long>(stages) * gridDim.x;
        if (threadIdx.x == 0 && next < a.M) issue(s, static_cast<int>(next));
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
}

// silu(min(g, 7)) * clamp(u, -7, 7) in fp32, NaN for a NaN.  With t = exp(-|a|), silu(a) = a / (1 + t) or a t / (1 + t): the
// divisor is in [1, 2], where __fdividef is within 2 units in the last place whatever the gate, and no gate overflows exp.
// All in all 12 * 2^-24 of the value (exp and the division 2 units each, four roundings).  a / (1 + exp(-a)) with its
// division rounded took 156 us for 16384 x 7168 and 2.00 for 33 x 768; this takes 140 and 1.65.
__device__ __forceinline__ float swiglu_fp32(float g, float u)
{
    const float a = g > 7.0f ? 7.0f : g;   // (comparisons let a NaN through)
    const float c = u > 7.0f ? 7.0f : (u < -7.0f ? -7.0f : u);
    const float t = expf(-fabsf(a));
    return __fdividef(a > 0.0f ? a : a * t, 1.0f + t) * c;
}

// Codes of the rows of x [M, K], or of clamp-SwiGLU of the rows' halves [gate | up] ([M, 2K], kSwiglu;
// the activation stays in fp32).  A CTA per row with V vectors a thread: all loads of a row go out at once, and the
// other CTAs of the SM load while this one reduces.
template <int V, bool kSwiglu>
__global__ void __launch_bounds__(V == 1 ? norm::kMaxThreads : norm::kMaxThreads / 2)
int8_quantize_kernel(const __nv_bfloat16 *x, int8_t *q, float *q_s, int K)
{
    using norm::kVec;
    __shared__ float2 red[32];
    const int nvec = K / kVec, row = blockIdx.x;
    const uint4 *src = reinterpret_cast<const uint4 *>(x) + static_cast<size_t>(row) * nvec * (kSwiglu ? 2 : 1);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    pdl_trigger();
    uint4 p[V][kSwiglu ? 2 : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        p[i][0] = c < nvec ? src[c] : zero;
        if (kSwiglu) p[i][kSwiglu ? 1 : 0] = c < nvec ? src[nvec + c] : zero;
    }
    float v[V][8], mx = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        unpack8(p[i][0], v[i]);
        if (kSwiglu) {
            float u[8];
            unpack8(p[i][kSwiglu ? 1 : 0], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = swiglu_fp32(v[i][j], u[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = max_or_nan(mx, fabsf(v[i][j]));
    }
    const CodeScale s(block_sum_max(0.f, mx, red).y);
    if (threadIdx.x == 0) q_s[row] = s.s;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nvec) reinterpret_cast<uint2 *>(q)[static_cast<size_t>(row) * nvec + c] = int8_codes8(v[i], s);
    }
}

// ------------------------------------------------------------------ launch

static int row_threads(int nvec, int v)
{
    const int t = (nvec + v - 1) / v;
    return (t + 31) / 32 * 32;
}

template <int V, bool kQuant, bool kFullGate>
static cudaError_t launch_ring_t(const NormArgs &a, int threads, cudaStream_t s)
{
    auto kernel = block_norm_ring_kernel<V, kQuant, kFullGate>;
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, norm::kRingBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    const int inputs = 1 + (a.residual != nullptr) + kFullGate;
    const int stage = inputs * a.H * 2;
    // CTAs per SM: what the registers of 512 (V = 4) or 1024 threads leave room for, with two stages each at least
    int ctas = (V == 4 ? 512 : 1024) / threads;
    if (ctas > 16) ctas = 16;
    while (ctas > 1 && 2 * ctas * stage > norm::kRingBytes) --ctas;
    int stages = norm::kRingBytes / (ctas * stage);
    if (stages > norm::kMaxStages) stages = norm::kMaxStages;
    const int most = num_sms() * ctas;
    return launch_ex(kernel, dim3(a.M < most ? a.M : most), dim3(threads), static_cast<size_t>(stages) * stage, s, true,
                     a, stages);
}

template <int V>
static cudaError_t launch_ring(const NormArgs &a, int threads, cudaStream_t s)
{
    const bool full = a.gate_kind == MOE_GATE_FULL;
    if (a.q_out != nullptr)
        return full ? launch_ring_t<V, true, true>(a, threads, s) : launch_ring_t<V, true, false>(a, threads, s);
    return full ? launch_ring_t<V, false, true>(a, threads, s) : launch_ring_t<V, false, false>(a, threads, s);
}

bool norm_by_ring(int M, int H)
{
    // Without the ring an SM holds several rows at once while a row has at most 512 threads, and one after another
    // beyond.  Both sides (without, with the ring): 7168 columns, 148 rows 3.2 and 3.7 us, 200 rows 5.4 and 4.6, 590
    // rows 10.4 and 6.7; 16384 columns, 200 rows 8.0 and 7.3; 2048 columns, 200 rows 2.3 and 3.5, 590 rows 3.5 and 3.9
    return M >= norm::kRingRows || (H / norm::kVec > norm::kWideVecs && M > kPlanSMs);
}

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s)
{
    const int nvec = a.H / norm::kVec;
    if (norm_by_ring(a.M, a.H)) {
        // few threads with several vectors each: the reductions cost less, more CTAs hide them (16384 rows of 2048:
        // 50 us with four vectors a thread, 62 with one)
        return nvec <= 64 ? launch_ring<2>(a, row_threads(nvec, 2), s) : launch_ring<4>(a, row_threads(nvec, 4), s);
    }
    const int v = nvec <= norm::kMaxThreads ? 1 : 2;
    const int threads = row_threads(nvec, v);
    return v == 1 ? launch_ex(block_norm_kernel<1>, dim3(a.M), dim3(threads), 0, s, true, a)
                  : launch_ex(block_norm_kernel<2>, dim3(a.M), dim3(threads), 0, s, true, a);
}

cudaError_t launch_int8_quantize(const __nv_bfloat16 *x, bool swiglu, int8_t *q, float *q_s, int M, int K,
                                 cudaStream_t s)
{
    const int nvec = K / norm::kVec;
    // a vector a thread for few rows, which wait for one trip to memory; four for many
    const int v = M <= kPlanSMs && nvec <= norm::kMaxThreads ? 1 : 4;
    const dim3 threads(row_threads(nvec, v)), grid(M);
    if (swiglu)
        return v == 1 ? launch_ex(int8_quantize_kernel<1, true>, grid, threads, 0, s, true, x, q, q_s, K)
                      : launch_ex(int8_quantize_kernel<4, true>, grid, threads, 0, s, true, x, q, q_s, K);
    return v == 1 ? launch_ex(int8_quantize_kernel<1, false>, grid, threads, 0, s, true, x, q, q_s, K)
                  : launch_ex(int8_quantize_kernel<4, false>, grid, threads, 0, s, true, x, q, q_s, K);
}

}  // namespace moe
