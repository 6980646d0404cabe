// ops.h -- declarations of the operators around the routed layer: block norms and int8 codes
// (block_norm.cu), ragged products (ragged_wide.cu, ragged_rows.cu), the weighted combine of expert rows
// (combine.cu).  Their C entry points are in ops_api.cu.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {

constexpr int kMaxRowElems = 16384;      // longest row of block_norm and of the quantiser
constexpr int kMaxProductDim = 65536;    // N and K of the products
constexpr int kMaxProductRows = 1 << 22;

// How long a kernel waits for its copies; and, for the self-tests, bytes that its first CTA expects and never gets.
struct WaitRules {
    long long limit;
    uint32_t lost;
};
constexpr WaitRules kWaits = {kWaitLimitCycles, 0}, kSelfTestWaits = {kSelfTestWaitCycles, 16};

struct NormArgs {
    const __nv_bfloat16 *x, *residual, *w_post, *w_pre;
    const void *gate;
    __nv_bfloat16 *res_out, *h_out;
    int8_t *q_out;
    float *q_s;
    float block_scale, residual_scale, eps, w_offset;
    int gate_kind;
    int M, H;
    WaitRules waits;
};
bool norm_by_ring(int M, int H);   // whether the rows take the kernel that waits for copies
cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s);
cudaError_t launch_int8_quantize(const __nv_bfloat16 *x, bool swiglu, int8_t *q, float *q_s, int M, int K,
                                 cudaStream_t s);
cudaError_t launch_combine_rows(const void *y, bool y_f32, const float *topk_w, const int32_t *inv_pos,
                                const __nv_bfloat16 *add, __nv_bfloat16 *out, int M, int H, int k, cudaStream_t s);

struct RaggedPlan;   // ragged_plan.h

struct RaggedArgs {
    const int32_t *offsets;      // [E+1]; nullptr: one group of all R rows
    const int32_t *sorted_ids;   // nullptr: the rows of x are the rows of y
    const void *x;
    const float *row_scale, *col_scale;   // int8
    const __nv_bfloat16 *add;             // int8, nullable
    void *y;
    int32_t *status_out;
    int y_f32;
    int R, M, N, K, E, k;
    int nt, stages, stage_bytes, row_blocks, kblocks, split, ring_bytes, accs, acc_cols;   // ragged_wide.cu
    WaitRules waits;
};
// Maps of the same rows with boxes of 16, 32, .. 128 of them; the first alone, one row high, for the gather.
struct BoxMaps {
    CUtensorMap m[8];
};
cudaError_t launch_ragged_wide(bool int8, bool swiglu, const CUtensorMap &wmap, const BoxMaps &xmaps,
                               const RaggedArgs &a, const RaggedPlan &p, cudaStream_t s);

cudaError_t launch_ragged_rows(bool int8, bool swiglu, const void *w, const RaggedArgs &a, cudaStream_t s);

// Map of a row-major [rows][K] matrix of 8-bit or bf16 elements: boxes of 128 bytes x box_rows, 128-byte
// swizzle, zeros outside; MOE_OK or MOE_ERR_CUDA (api.cu).
int encode_rows_map(CUtensorMap *map, bool bytes, const void *base, uint64_t rows, uint64_t K, uint32_t box_rows);

}  // namespace moe
