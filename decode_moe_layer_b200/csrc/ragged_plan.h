// ragged_plan.h -- how the ragged products (ragged.cuh) are cut, decided on the host from the sizes alone.  No device
// code: a host program can check it.
#pragma once

#include "moe_internal.h"

namespace moe {

// ------------------------------------------------------------------ by weight rows or by tiles

// Measured on this part (times on the GPU, weights out of L2), by rows against tiles:
//  * int8, codes and product: 4 tokens 4096 x 7168 11.7 us against 11.8, 16384 x 7168 25.3 against 24.4, 1536 x 2048 5.3
//    against 7.0, 7168 x 2048 7.2 against 9.1, so within 4% for large weights and ahead for small ones; with 8 tokens the
//    rows take about twice their time with 4, the tiles no longer.
//  * grouped, 128 experts of 1536 x 2048, top-8: 4, 8, 12 tokens 28, 52, 69 us against 35, 53, 67; 256 experts of 7168 x
//    2048: 8, 16, 20, 32 tokens 235, 414, 495, 727 us against 237, 416, 505, 681.  From about 0.7 rows a group on, groups
//    of two and more rows pay for a tile.
//    That is of routing that spreads.  The host knows only R and E: by rows an expert's weights are read once a row, in
//    tiles once, so where few experts get the rows this rule is wrong, by up to seven times: 128 experts of 1536 x 2048, 40
//    rows over 35, 15, 1 of them 35, 25, 21 us against 36, 23, 10, 80 rows over 63, 22, 1 of them 64, 44, 40 against 62, 28,
//    11; 256 of 2048 x 2048, 160 rows over 116, 35, 1 of them 141, 108, 106 against 143, 52, 15; 1024 of 512 x 1024, 680 rows
//    over 502, 96, 1 of them 80, 63, 61 against 103, 49, 25, and 80 rows over 78, 23, 1 of them 15, 12, 11 against 47, 39, 24
//    (a CTA goes through all the groups to find its tile's).
//  * with 16 rows at most the call is so short that the tiles' set-up decides: 4 tokens x 4 of 16 experts of 1024 x 1024
//    7.1 us against 8.4, 1 token 3.7 against 7.4.
constexpr int kRowsMaxTokens = 4;    // int8
constexpr int kRowsMaxShort = 16;    // grouped
inline bool ragged_by_rows(int R, int E, bool int8)
{
    if (int8) return R <= kRowsMaxTokens;
    return 3LL * R <= 2LL * E || (R <= kRowsMaxShort && R <= E);
}

// ------------------------------------------------------------------ tiles (ragged_wide.cu)

namespace ragged {
constexpr int kRows = 128;          // weight rows per CTA and tile: the lanes of tensor memory
constexpr int kStageKBytes = 128;   // bytes of K per stage: one 128-byte swizzle row
constexpr int kABytes = kRows * kStageKBytes;
}  // namespace ragged

namespace rwide {
using namespace ragged;
constexpr int kMaxPipe = 8;
constexpr int kNt = 256;                                  // most tokens per tile
constexpr int kMaxRingBytes = 6 * (kABytes + kNt / 2 * kStageKBytes);
constexpr int kSmBytes = 228 * 1024, kReservedBytes = 1024;   // shared memory of an SM; what a CTA takes besides its own
constexpr int kHalfSmBytes = 102 * 1024;                  // ring of a CTA that leaves room for another on its SM
// behind the stages
constexpr int kOffScales = 512;                           // [2][kNt] fp32 row scales (int8)
constexpr int kOffGroups = kOffScales + 8192;             // or, swiglu, what gate and up warps exchange: 8 KB
static_assert(2 * kNt * 4 <= 8192 && 2 * 4 * 8 * 32 * 4 <= 8192, "either fits");
constexpr int kEpi0 = 4, kGather0 = 8, kGatherWarps = 8;
constexpr int threads_of(bool gather) { return 32 * (gather ? kGather0 + kGatherWarps : kGather0); }
constexpr int kEpiCols = 16;                              // columns of an accumulator that a thread finishes together
constexpr int kRun = 8;                                   // token tiles of a group that run beside each other
// split: partial sums in runs of 8 columns x 128 rows
constexpr int kRunBytes = 8 * kRows * 4;
constexpr int kMaxSplit = 4;                              // pairs per cluster

// Whether the tiles of the last, partial wave run as two halves of their tokens each, since there are clusters enough:
// half a tile has half the MMAs and 3/4 of the copies.  In short runs, halves against whole tiles (int8): 4096 tokens x
// 4096 x 7168, 3.46 waves, 76.5 against 79.0 us; 2500 x 4096 x 7168, 2.16 waves, 53.0 against 56.0; 2560 x 4096 x 2048
// 21.2 against 22.8.
constexpr bool halve_last_wave(int tiles, int clusters, int nt)
{
    return nt == kNt && tiles > clusters && tiles % clusters > 0 && 2 * (tiles % clusters) <= clusters;
}
}  // namespace rwide

// How the tiles of 256 weight rows x up to nt tokens are run: `clusters` clusters of `split` CTA pairs, each pair
// with its range of K.
struct RaggedPlan {
    int nt, split, clusters, stages, stage_bytes, ring_bytes, smem, threads;
    int accs, acc_cols;        // accumulators and their columns of tensor memory
    int row_blocks, kblocks;   // of 128 weight rows (swiglu: 64 output columns), of 128 bytes of K
};
inline RaggedPlan wide_plan(int R, int N, int K, int E, bool int8, bool swiglu, bool gather)
{
    using namespace rwide;
    RaggedPlan p = {};
    p.row_blocks = swiglu ? (N + 63) / 64 : (N + kRows - 1) / kRows;
    p.kblocks = (K * (int8 ? 1 : 2) + kStageKBytes - 1) / kStageKBytes;
    const int pair_blocks = (p.row_blocks + 1) / 2;
    const int least = E == 1 ? (R + kNt - 1) / kNt : (R < E ? R : E) + (R - 1) / kNt;   // token tiles of up to 256
    const int widest = R < kNt ? (R + 31) / 32 * 32 : kNt;
    // Token tiles and pairs per cluster by the estimated cycles of the longest cluster: waves x stages x a stage (its
    // bytes at 60 a cycle, half as many where two CTAs share an SM, or its MMAs), the last tile's columns (20 cycles each)
    // and, if pairs share a tile, the joining (1200 and 42 a column).  More, narrower tiles than `least` only for a single group, whose size the host
    // knows.  Where two CTAs fit an SM, 33 clusters of eight or 71 of four run at once, else 15 or 33.
    // Measured (int8): 33 tokens x 1536 x 2048 by four pairs a tile 5.5 us, by one 6.0, 128 tokens 6.7 and 5.9; 8 x 7168 x
    // 2048 by four pairs (two CTAs an SM) 7.3, by one 6.7; 256 tokens x 4096 x 7168 as four tiles of 64 by two pairs 15.
    long long best = -1;
    for (int tokens = least; tokens == least || (E == 1 && tokens * pair_blocks <= kPlanSMs && tokens * 32 <= R + 31); ++tokens) {
        const int nt = tokens == least ? widest : ((R + tokens - 1) / tokens + 31) / 32 * 32;
        const int stage = kABytes + nt / 2 * kStageKBytes;
        const long long tiles = static_cast<long long>(tokens) * pair_blocks;
        for (int split = 1; split <= kMaxSplit; split *= 2) {
            const int need = split > 1 ? split * ((nt / 8 + split - 1) / split) * kRunBytes : 0;   // partial sums
            const bool twice = need <= kHalfSmBytes;
            const int fit = split == 4 ? (twice ? 33 : 15) : (split == 2 ? (twice ? 71 : 33) : kPlanSMs / 2);
            if (split > 1 && (tiles > fit || p.kblocks < 2 * split)) continue;
            const int copies = stage / 60 * (tiles * split > kPlanSMs / 2 && split > 1 ? 2 : 1);
            const int cycles = copies > 2 * nt ? copies : 2 * nt;
            const int slice = (p.kblocks + split - 1) / split;
            const bool halves = E == 1 && halve_last_wave(static_cast<int>(tiles), fit, nt);
            const long long cost = (tiles + fit - 1) / fit * slice * cycles - (halves ? slice * (cycles / 4) : 0) + 20 * nt +
                                   (split > 1 ? 1200 + 42 * nt : 0);
            if (best >= 0 && cost >= best) continue;
            best = cost;
            // a cluster with one tile at most: one accumulator, no more stages than it can use, and (narrow tiles) half an
            // SM, so that the next kernel's CTAs get ready beside it
            const bool once = tiles <= fit;
            int stages = (once && twice && (split > 1 || nt <= 64) ? kHalfSmBytes : kMaxRingBytes) / stage;
            if (stages > kMaxPipe) stages = kMaxPipe;
            if (once && stages > slice) stages = slice;
            p.split = split;
            p.nt = nt;
            p.stages = stages;
            p.stage_bytes = stage;
            p.ring_bytes = stages * stage > need ? stages * stage : need;
            p.clusters = static_cast<int>(tiles < fit ? tiles : fit);
            p.accs = once ? 1 : 2;
            p.acc_cols = nt <= 32 ? 32 : (nt <= 64 ? 64 : (nt <= 128 ? 128 : 256));
        }
    }
    p.smem = 1024 + p.ring_bytes + kOffGroups + 2 * (E + 1) * 4;
    // An SM's CTAs, of whatever calls, must not ask for more tensor memory than there is: a CTA that waits for some while
    // its pair holds some could wait on one that waits on it.  So a CTA takes at least its columns' share of an SM's
    // shared memory.
    const int share = p.accs * p.acc_cols * (kSmBytes / 512) - kReservedBytes;
    if (p.smem < share) p.smem = share;
    p.threads = threads_of(gather);
    return p;
}

}  // namespace moe
