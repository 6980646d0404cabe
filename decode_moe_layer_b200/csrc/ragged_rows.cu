// ragged_rows.cu -- the ragged products (ragged.cuh) for the smallest calls: a token or a few.
//
// ragged_rows_kernel: a warp streams weight rows with plain 16-byte loads against up to kT tokens of one group,
// kW rows at a time (swiglu: a gate row and its up row), the next eight loads of a lane always on their way while it
// works on the last; products and sums on the ordinary pipes (fp32 FMA; dp4a into int32), a warp reduction at the
// end of a row.  No tensor map, barrier, cluster or tensor memory: what a call of this size waits for is the launch,
// one trip to memory and the stream of the weights; the tensor-core kernel's set-up costs it 2 to 3 us more (int8, one
// token, weights out of L2: 1536 x 2048 1.9 against 4.8 us, 4096 x 7168 7.1 against 8.8; the weights alone 0.5 and
// 4.5).  8 of 128 experts of 1536 x 2048 with a row each: 10.4 us, 50 MB.
// With several groups a tile is one position of the grouped order, whose group a warp finds among the offsets; rows
// of the same group then read its weights from L2 again, which is why groups of more than a row or so go to the tiles
// (ragged_by_rows, ragged_plan.h).
// The order of the sums is fixed: lane, then the reduction tree.
#include "ragged.cuh"

namespace moe {

namespace rrows {
constexpr int kWarps = 4;
// rows at a time and 512-byte runs of each in flight: tokens share the weights' registers
constexpr int rows_of(bool int8, int t) { return int8 && t > 1 ? 4 : 2; }
constexpr int runs_of(bool int8, int t) { return int8 && t > 1 ? 2 : 4; }
constexpr int kWarpsPerSm = 64;   // aimed at: more than an SM holds, so that SMs that are done early find work
// weights up to here are asked for whole ahead of the call's dependency; several tokens, which take longer, gain from
// that only with small ones (4 tokens and their codes, 7168 x 2048: whole 7.8 us, first loads 7.4, none 7.8; 512 x 7168:
// 9.7, 10.1, 10.1)
constexpr uint32_t ahead_bytes(int t) { return (t == 1 ? 32u : 8u) << 20; }
}  // namespace rrows

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// acc += dot product of 16 bytes of weights and of a token.
__device__ __forceinline__ void dot16(float &acc, uint4 w, uint4 x)
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = fmaf(bf16_lo(a[i]), bf16_lo(b[i]), acc);
        acc = fmaf(bf16_hi(a[i]), bf16_hi(b[i]), acc);
    }
}
__device__ __forceinline__ void dot16(int &acc, uint4 w, uint4 x)
{
    acc = __dp4a(static_cast<int>(w.x), static_cast<int>(x.x), acc);
    acc = __dp4a(static_cast<int>(w.y), static_cast<int>(x.y), acc);
    acc = __dp4a(static_cast<int>(w.z), static_cast<int>(x.z), acc);
    acc = __dp4a(static_cast<int>(w.w), static_cast<int>(x.w), acc);
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <bool kInt8>
struct RowAcc {
    typedef float type;
};
template <>
struct RowAcc<true> {
    typedef int type;
};

// steps: kW-row steps per warp.
template <bool kInt8, bool kSwiglu, int kT>
__global__ void __launch_bounds__(32 * rrows::kWarps)
ragged_rows_kernel(const void *wbase, const __grid_constant__ RaggedArgs a, int row_blocks, int steps)
{
    using namespace rrows;
    typedef typename RowAcc<kInt8>::type Acc;
    constexpr int kW = rows_of(kInt8, kT), kRuns = runs_of(kInt8, kT), kCols = kSwiglu ? 1 : kW;
    static_assert(!kSwiglu || (kW == 2 && kT == 1), "a gate row and its up row");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rb = blockIdx.x % row_blocks, tt = blockIdx.x / row_blocks;
    // the warp's steps: columns n_first, + n_next, .. below a.N
    const int n_first = (rb * steps * kWarps + warp) * kCols, n_next = kWarps * kCols;
    if (n_first >= a.N) return;
    if (a.offsets == nullptr) {
        // What the warp reads first, into L2 while the kernel before (that makes the codes, say) still runs: its rows, or
        // of larger weights what its first loads bring.  Codes and product of one token in a run of calls, 4096 x 7168,
        // 8.4 against 7.5 us, 16384 x 7168 20.1 against 18.3 (with whole rows 22.1).  Into L2 only: that kernel may still
        // write the weights.
        const uint32_t row_bytes = static_cast<uint32_t>(a.K) * (kInt8 ? 1 : 2), rows = min(kW, a.N - n_first);
        const char *w = static_cast<const char *>(wbase) + static_cast<size_t>(n_first) * row_bytes;
        if (static_cast<uint64_t>(gridDim.x) * kWarps * kW * row_bytes <= ahead_bytes(kT)) {
            for (uint32_t b = lane * 128u; b < rows * row_bytes; b += 4096u) prefetch_l2(w + b);
        } else {
            constexpr uint32_t kLines = 4 * kRuns;   // of 128 bytes, in each row
            const uint32_t r = lane / kLines, b = lane % kLines * 128u;
            if (r < rows && b < row_bytes) prefetch_l2(w + static_cast<size_t>(r) * row_bytes + b);
        }
    }
    pdl_wait();
    pdl_trigger();
    int expert = 0, p0 = tt * kT, count = min(kT, a.R - p0);
    if (a.offsets != nullptr) {
        // position tt is in the group that is the first to end behind it (if offsets descend, as the tiles have it: a
        // group starts where the ones before it end)
        int end = a.E;
        for (int e = a.E - 1 - lane; e >= 0; e -= 32) end = a.offsets[e + 1] > tt ? e : end;
        expert = static_cast<int>(__reduce_min_sync(0xffffffffu, end));
        if (expert >= a.E || a.offsets[0] > tt) return;
    }

    const int pieces = a.K * (kInt8 ? 1 : 2) / 16;   // 16-byte pieces of a row
    const uint4 *w0 = static_cast<const uint4 *>(wbase) +
                      static_cast<size_t>(expert) * a.N * (kSwiglu ? 2 : 1) * pieces;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 v[kRuns][kW];
    auto load = [&](int n, int c0) {   // rows n.. (the last one again past a.N), pieces c0 + 32 u
#pragma unroll
        for (int r = 0; r < kW; ++r) {
            const size_t row = kSwiglu ? static_cast<size_t>(n) + (r ? a.N : 0) : min(n + r, a.N - 1);
            const uint4 *src = w0 + row * pieces;
#pragma unroll
            for (int u = 0; u < kRuns; ++u) v[u][r] = c0 + 32 * u < pieces ? __ldcs(src + c0 + 32 * u) : zero;
        }
    };
    load(n_first, lane);
    const uint4 *x[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
        const int p = p0 + min(t, count - 1);
        size_t row = static_cast<size_t>(p);
        if (a.sorted_ids != nullptr) {
            const uint32_t f = static_cast<uint32_t>(a.sorted_ids[p]);
            row = min(f / static_cast<uint32_t>(a.k), static_cast<uint32_t>(a.M - 1));
        }
        x[t] = static_cast<const uint4 *>(a.x) + row * pieces;
    }
    Acc acc[kW][kT] = {};
    int n = n_first, c0 = lane, left = steps;
    while (true) {
        uint4 now[kRuns][kW];
#pragma unroll
        for (int u = 0; u < kRuns; ++u)
#pragma unroll
            for (int r = 0; r < kW; ++r) now[u][r] = v[u][r];
        const int c = c0, at = n;
        // (by the row's first piece, so that all lanes go on together)
        c0 += 32 * kRuns;
        const bool row_done = c0 - lane >= pieces;
        if (row_done) {
            c0 = lane;
            n += n_next;
            --left;
        }
        const bool more = left > 0 && n < a.N;
        if (more) load(n, c0);
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                // (zeros for both past the end: a token's NaN times a weight that is not there adds nothing)
                const uint4 xv = c + 32 * u < pieces ? x[t][c + 32 * u] : zero;
#pragma unroll
                for (int r = 0; r < kW; ++r) dot16(acc[r][t], now[u][r], xv);
            }
        }
        if (row_done) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int r = 0; r < kW; ++r)
#pragma unroll
                    for (int t = 0; t < kT; ++t) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], d);
            // every lane has every sum: lane kW * t + r (swiglu: 0) stores its own
            if (kSwiglu) {
                if (lane == 0)
                    store_pair(a, static_cast<float>(acc[0][0]), static_cast<float>(acc[1][0]), static_cast<size_t>(p0), at);
            } else {
#pragma unroll
                for (int t = 0; t < kT; ++t)
#pragma unroll
                    for (int r = 0; r < kW; ++r)
                        if (lane == kW * t + r && t < count && at + r < a.N) {
                            const size_t row = static_cast<size_t>(p0) + t, to = row * a.N + at + r;
                            float f = static_cast<float>(acc[r][t]);
                            if (kInt8) {
                                f = f * a.row_scale[row] * a.col_scale[at + r];
                                if (a.add != nullptr) f += __bfloat162float(a.add[to]);
                            }
                            if (a.y_f32)
                                static_cast<float *>(a.y)[to] = f;
                            else
                                static_cast<__nv_bfloat16 *>(a.y)[to] = __float2bfloat16_rn(f);
                        }
            }
#pragma unroll
            for (int r = 0; r < kW; ++r)
#pragma unroll
                for (int t = 0; t < kT; ++t) acc[r][t] = 0;
        }
        if (!more) break;
    }
}

// ------------------------------------------------------------------ launch

template <bool kInt8, bool kSwiglu, int kT>
static cudaError_t launch_rows_t(const void *w, const RaggedArgs &a, cudaStream_t s)
{
    using namespace rrows;
    const int tiles = a.offsets != nullptr ? a.R : (a.R + kT - 1) / kT;
    const int cols = kSwiglu ? 1 : rows_of(kInt8, kT), units = (a.N + cols - 1) / cols;   // steps of a tile
    const long long target = static_cast<long long>(kWarpsPerSm) * kPlanSMs;
    long long steps = static_cast<long long>(tiles) * units / target;
    steps = steps < 1 ? 1 : (steps > 8 ? 8 : steps);
    const int row_blocks = static_cast<int>((units + kWarps * steps - 1) / (kWarps * steps));
    return launch_ex(ragged_rows_kernel<kInt8, kSwiglu, kT>, dim3(static_cast<unsigned>(tiles) * row_blocks),
                     dim3(32 * kWarps), 0, s, true, w, a, row_blocks, static_cast<int>(steps));
}

cudaError_t launch_ragged_rows(bool int8, bool swiglu, const void *w, const RaggedArgs &a, cudaStream_t s)
{
    if (int8) {
        if (a.R == 1) return launch_rows_t<true, false, 1>(w, a, s);
        return a.R == 2 ? launch_rows_t<true, false, 2>(w, a, s) : launch_rows_t<true, false, 4>(w, a, s);
    }
    return swiglu ? launch_rows_t<false, true, 1>(w, a, s) : launch_rows_t<false, false, 1>(w, a, s);
}

}  // namespace moe
