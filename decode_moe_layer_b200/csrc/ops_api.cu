// ops_api.cu -- C entry points of the operators around the routed layer (declared in include/moe.h):
// argument checks and TMA maps, and the self-tests that run them with waits that give up.  None of them needs a workspace, waits for the device or allocates.
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "moe.h"
#include "ops.h"
#include "ragged_plan.h"

#define OPS_TRY(expr)                                \
    do {                                             \
        cudaError_t _e = (expr);                     \
        if (_e != cudaSuccess) return cuda_fail(_e); \
    } while (0)

namespace moe {

static bool is_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

static bool ranges_meet(const void *a, size_t an, const void *b, size_t bn)
{
    if (!a || !b) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + bn && pb < pa + an;
}

// An output may not meet an input, except exactly (the same start) where `in_place` says so.
static bool bad_overlap(const void *out, size_t on, const void *in, size_t n, bool in_place)
{
    if (in_place && out == in) return false;
    return ranges_meet(out, on, in, n);
}

static bool finite_f(float v) { return v - v == 0.0f; }

// Maps and launch of a ragged product whose arguments have been checked: w [w_rows][K], x [a.M][K].
static int run_ragged(bool int8, bool swiglu, const void *w, uint64_t w_rows, RaggedArgs &a, cudaStream_t stream)
{
    auto clear_status = [&]() {   // last before the launch: a call that fails has enqueued nothing
        return a.status_out ? cudaMemsetAsync(a.status_out, 0, sizeof(int32_t), stream) : cudaSuccess;
    };
    if (ragged_by_rows(a.R, a.E, int8)) {
        if (a.waits.lost) return MOE_ERR_UNSUPPORTED_SHAPE;   // (the self-test: this kernel waits for nothing)
        cudaError_t e = clear_status();
        if (e == cudaSuccess) e = launch_ragged_rows(int8, swiglu, w, a, stream);
        return e == cudaSuccess ? MOE_OK : cuda_fail(e);
    }
    const bool gather = a.sorted_ids != nullptr;
    const RaggedPlan p = wide_plan(a.R, a.N, a.K, a.E, int8, swiglu, gather);
    a.nt = p.nt;
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.accs = p.accs;
    a.acc_cols = p.acc_cols;
    a.row_blocks = p.row_blocks;
    a.kblocks = p.kblocks;
    a.split = p.split;
    a.ring_bytes = p.ring_bytes;
    // weight boxes of 128 rows, or (swiglu) of 64 gate rows and of 64 up rows; token boxes of the heights that tiles
    // can have
    CUtensorMap wmap;
    BoxMaps maps = {};
    const uint64_t rows = static_cast<uint64_t>(a.M), K = static_cast<uint64_t>(a.K);
    int rc = encode_rows_map(&wmap, int8, w, w_rows, K, swiglu ? 64 : 128);
    const int top = gather ? 0 : p.nt / 32 - 1;
    if (a.offsets == nullptr && rc == MOE_OK &&
        rwide::halve_last_wave((a.R + p.nt - 1) / p.nt * ((p.row_blocks + 1) / 2), p.clusters, p.nt))
        rc = encode_rows_map(&maps.m[3], int8, a.x, rows, K, rwide::kNt / 4);
    for (int i = a.offsets != nullptr ? 0 : top; i <= top && rc == MOE_OK; ++i)
        rc = encode_rows_map(&maps.m[i], int8, a.x, rows, K, gather ? 1u : 16u * (i + 1));
    if (rc != MOE_OK) return rc;
    cudaError_t e = clear_status();
    if (e == cudaSuccess) e = launch_ragged_wide(int8, swiglu, wmap, maps, a, p, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

static int block_norm(const void *x, const void *residual, const void *w_post, const void *gate, int gate_kind,
                      const void *w_pre, float block_scale, float residual_scale, float eps, float w_offset,
                      void *res_out, void *h_out, int8_t *q_out, float *q_s, int M, int H, const WaitRules &waits,
                      cudaStream_t stream)
{
    if (M < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !finite_f(eps) || !finite_f(block_scale) || !finite_f(residual_scale) || !finite_f(w_offset))
        return MOE_ERR_INVALID_ARG;
    if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > kMaxRowElems) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M > kMaxProductRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (!x || (gate_kind != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!res_out && !h_out && !q_out) return MOE_ERR_INVALID_ARG;
    if ((q_out != nullptr) != (q_s != nullptr)) return MOE_ERR_INVALID_ARG;
    if ((h_out != nullptr || q_out != nullptr) != (w_pre != nullptr)) return MOE_ERR_INVALID_ARG;
    const void *al[] = {x, residual, w_post, w_pre, res_out, h_out};
    for (const void *p : al)
        if (!is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(q_out, 16) || !is_aligned(q_s, 4) || !is_aligned(gate, gate_kind == MOE_GATE_TOKEN ? 4 : 16))
        return MOE_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(M) * H, row = static_cast<size_t>(H) * 2;
    const size_t gn = gate_kind == MOE_GATE_TOKEN ? static_cast<size_t>(M) * 4 : (gate_kind == MOE_GATE_FULL ? n * 2 : row);
    const void *outs[] = {res_out, h_out, q_out, q_s};
    const size_t outn[] = {n * 2, n * 2, n, static_cast<size_t>(M) * 4};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i]) continue;
        const bool rows = i < 2;   // the bf16 outputs may take the place of x or the residual
        if (bad_overlap(outs[i], outn[i], x, n * 2, rows) || bad_overlap(outs[i], outn[i], residual, n * 2, rows) ||
            bad_overlap(outs[i], outn[i], gate, gn, false) || bad_overlap(outs[i], outn[i], w_post, row, false) ||
            bad_overlap(outs[i], outn[i], w_pre, row, false))
            return MOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (ranges_meet(outs[i], outn[i], outs[j], outn[j])) return MOE_ERR_INVALID_ARG;
    }
    NormArgs a;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.residual = static_cast<const __nv_bfloat16 *>(residual);
    a.w_post = static_cast<const __nv_bfloat16 *>(w_post);
    a.w_pre = static_cast<const __nv_bfloat16 *>(w_pre);
    a.gate = gate;
    a.res_out = static_cast<__nv_bfloat16 *>(res_out);
    a.h_out = static_cast<__nv_bfloat16 *>(h_out);
    a.q_out = q_out;
    a.q_s = q_s;
    a.block_scale = block_scale;
    a.residual_scale = residual_scale;
    a.eps = eps;
    a.w_offset = w_offset;
    a.gate_kind = gate_kind;
    a.M = M;
    a.H = H;
    a.waits = waits;
    OPS_TRY(launch_block_norm(a, stream));
    return MOE_OK;
}

static int int8_gemm(const int8_t *q, const float *q_s, const int8_t *w_q, const float *w_s, const void *add_bf16,
                     void *out, int out_f32, int M, int N, int K, int32_t *status_out, const WaitRules &waits,
                     cudaStream_t stream)
{
    if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > kMaxProductDim || N > kMaxProductDim || M > kMaxProductRows)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (!q || !q_s || !w_q || !w_s || !out) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(q, 16) || !is_aligned(w_q, 16) || !is_aligned(out, 16) || !is_aligned(add_bf16, 16) ||
        !is_aligned(q_s, 4) || !is_aligned(w_s, 4) || !is_aligned(status_out, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t mn = static_cast<size_t>(M) * N, on = mn * (out_f32 ? 4 : 2);
    if (ranges_meet(out, on, q, static_cast<size_t>(M) * K) || ranges_meet(out, on, w_q, static_cast<size_t>(N) * K) ||
        ranges_meet(out, on, q_s, static_cast<size_t>(M) * 4) || ranges_meet(out, on, w_s, static_cast<size_t>(N) * 4) ||
        bad_overlap(out, on, add_bf16, mn * 2, out_f32 == 0))
        return MOE_ERR_INVALID_ARG;
    if (ranges_meet(status_out, 4, out, on) || ranges_meet(status_out, 4, q, static_cast<size_t>(M) * K) ||
        ranges_meet(status_out, 4, w_q, static_cast<size_t>(N) * K) ||
        ranges_meet(status_out, 4, q_s, static_cast<size_t>(M) * 4) ||
        ranges_meet(status_out, 4, w_s, static_cast<size_t>(N) * 4) || ranges_meet(status_out, 4, add_bf16, mn * 2))
        return MOE_ERR_INVALID_ARG;
    RaggedArgs a = {};
    a.waits = waits;
    a.x = q;
    a.K = K;
    a.row_scale = q_s;
    a.col_scale = w_s;
    a.add = static_cast<const __nv_bfloat16 *>(add_bf16);
    a.y = out;
    a.y_f32 = out_f32 != 0;
    a.status_out = status_out;
    a.R = M;
    a.M = M;
    a.N = N;
    a.E = 1;
    a.k = 1;
    return run_ragged(true, false, w_q, static_cast<uint64_t>(N), a, stream);
}

static int grouped_gemm(const void *x_bf16, const void *w_bf16, const int32_t *expert_offsets,
                        const int32_t *sorted_ids, void *y, int y_f32, int swiglu, int M, int N, int K, int E, int k,
                        int32_t *status_out, const WaitRules &waits, cudaStream_t stream)
{
    if (M < 0 || N <= 0 || K <= 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > kMaxProductDim || N > kMaxProductDim || E > kMaxE || k > kMaxK ||
        static_cast<long long>(M) * k > kMaxProductRows)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (!x_bf16 || !w_bf16 || !expert_offsets || !y) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(x_bf16, 16) || !is_aligned(w_bf16, 16) || !is_aligned(y, 16) || !is_aligned(expert_offsets, 4) ||
        !is_aligned(sorted_ids, 4) || !is_aligned(status_out, 4))
        return MOE_ERR_INVALID_ARG;
    const int R = M * k;
    const int x_rows = sorted_ids ? M : R;
    const size_t yn = static_cast<size_t>(R) * N * (y_f32 ? 4 : 2);
    const uint64_t uK = static_cast<uint64_t>(K), uN = static_cast<uint64_t>(N), uE = static_cast<uint64_t>(E);
    const size_t wn = uE * uN * uK * (swiglu ? 4 : 2);
    if (ranges_meet(y, yn, x_bf16, static_cast<size_t>(x_rows) * K * 2) || ranges_meet(y, yn, w_bf16, wn) ||
        ranges_meet(y, yn, expert_offsets, (uE + 1) * 4) || ranges_meet(y, yn, sorted_ids, static_cast<size_t>(R) * 4))
        return MOE_ERR_INVALID_ARG;
    if (ranges_meet(status_out, 4, y, yn) || ranges_meet(status_out, 4, x_bf16, static_cast<size_t>(x_rows) * K * 2) ||
        ranges_meet(status_out, 4, w_bf16, wn) || ranges_meet(status_out, 4, expert_offsets, (uE + 1) * 4) ||
        ranges_meet(status_out, 4, sorted_ids, static_cast<size_t>(R) * 4))
        return MOE_ERR_INVALID_ARG;
    RaggedArgs a = {};
    a.waits = waits;
    a.offsets = expert_offsets;
    a.sorted_ids = sorted_ids;
    a.x = x_bf16;
    a.K = K;
    a.y = y;
    a.y_f32 = y_f32 != 0;
    a.status_out = status_out;
    a.R = R;
    a.M = x_rows;
    a.N = N;
    a.E = E;
    a.k = k;
    return run_ragged(false, swiglu != 0, w_bf16, uE * uN * (swiglu ? 2 : 1), a, stream);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm(const void *x, const void *residual, const void *w_post, const void *gate, int gate_kind,
                   const void *w_pre, float block_scale, float residual_scale, float eps, float w_offset, void *res_out,
                   void *h_out, int8_t *q_out, float *q_s, int M, int H, cudaStream_t stream)
{
    return block_norm(x, residual, w_post, gate, gate_kind, w_pre, block_scale, residual_scale, eps, w_offset, res_out,
                      h_out, q_out, q_s, M, H, kWaits, stream);
}

int moe_selftest_norm_timeout(const void *x, const void *residual, const void *w_post, const void *w_pre, void *res_out,
                              void *h_out, int8_t *q_out, float *q_s, int M, int H, cudaStream_t stream)
{
    if (M <= 0 || H <= 0) return MOE_ERR_INVALID_ARG;
    if (!norm_by_ring(M, H)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return block_norm(x, residual, w_post, nullptr, MOE_GATE_NONE, w_pre, 1.0f, 1.0f, 1e-6f, 0.0f, res_out, h_out, q_out,
                      q_s, M, H, kSelfTestWaits, stream);
}

int moe_int8_quantize(const void *x_bf16, int swiglu, int8_t *q, float *q_s, int M, int K, cudaStream_t stream)
{
    if (M < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > kMaxRowElems || M > kMaxProductRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (!x_bf16 || !q || !q_s) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(x_bf16, 16) || !is_aligned(q, 16) || !is_aligned(q_s, 4)) return MOE_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(M) * K, xn = n * (swiglu ? 4 : 2), sn = static_cast<size_t>(M) * 4;
    if (ranges_meet(q, n, x_bf16, xn) || ranges_meet(q_s, sn, x_bf16, xn) || ranges_meet(q, n, q_s, sn))
        return MOE_ERR_INVALID_ARG;
    OPS_TRY(launch_int8_quantize(static_cast<const __nv_bfloat16 *>(x_bf16), swiglu != 0, q, q_s, M, K, stream));
    return MOE_OK;
}

int moe_int8_gemm(const int8_t *q, const float *q_s, const int8_t *w_q, const float *w_s, const void *add_bf16,
                  void *out, int out_f32, int M, int N, int K, int32_t *status_out, cudaStream_t stream)
{
    return int8_gemm(q, q_s, w_q, w_s, add_bf16, out, out_f32, M, N, K, status_out, kWaits, stream);
}

int moe_grouped_gemm(const void *x_bf16, const void *w_bf16, const int32_t *expert_offsets, const int32_t *sorted_ids,
                     void *y, int y_f32, int swiglu, int M, int N, int K, int E, int k, int32_t *status_out,
                     cudaStream_t stream)
{
    return grouped_gemm(x_bf16, w_bf16, expert_offsets, sorted_ids, y, y_f32, swiglu, M, N, K, E, k, status_out, kWaits,
                        stream);
}

int moe_selftest_product_timeout(int int8, const void *x, const float *q_s, const void *w, const float *w_s,
                                 const int32_t *expert_offsets, const int32_t *sorted_ids, void *y, int y_f32,
                                 int swiglu, int M, int N, int K, int E, int k, int32_t *status_out,
                                 cudaStream_t stream)
{
    if (M <= 0 || !status_out) return MOE_ERR_INVALID_ARG;
    if (int8)
        return int8_gemm(static_cast<const int8_t *>(x), q_s, static_cast<const int8_t *>(w), w_s, nullptr, y, y_f32, M,
                         N, K, status_out, kSelfTestWaits, stream);
    return grouped_gemm(x, w, expert_offsets, sorted_ids, y, y_f32, swiglu, M, N, K, E, k, status_out, kSelfTestWaits,
                        stream);
}

int moe_combine(const void *y, int y_f32, const float *topk_w, const int32_t *inv_pos, const void *add_bf16,
                void *out_bf16, int M, int H, int k, cudaStream_t stream)
{
    if (M < 0 || H <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > kMaxProductDim || k > kMaxK || static_cast<long long>(M) * k > kMaxProductRows)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (!y || !topk_w || !inv_pos || !out_bf16) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(y, 16) || !is_aligned(out_bf16, 16) || !is_aligned(add_bf16, 16) || !is_aligned(topk_w, 4) ||
        !is_aligned(inv_pos, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t R = static_cast<size_t>(M) * k, on = static_cast<size_t>(M) * H * 2;
    if (ranges_meet(out_bf16, on, y, R * H * (y_f32 ? 4 : 2)) || ranges_meet(out_bf16, on, topk_w, R * 4) ||
        ranges_meet(out_bf16, on, inv_pos, R * 4) || bad_overlap(out_bf16, on, add_bf16, on, true))
        return MOE_ERR_INVALID_ARG;
    OPS_TRY(launch_combine_rows(y, y_f32 != 0, topk_w, inv_pos, static_cast<const __nv_bfloat16 *>(add_bf16),
                                static_cast<__nv_bfloat16 *>(out_bf16), M, H, k, stream));
    return MOE_OK;
}

}  // extern "C"
