// Host check of csrc/ragged_plan.h over a grid of shapes: what the tile kernel relies on.
#include <cstdio>

#include "ragged_plan.h"

using namespace moe;

static int bad = 0;

#define CHECK(c)                                                                                                     \
    do {                                                                                                             \
        if (!(c) && bad++ < 20)                                                                                      \
            printf("%s: R %d N %d K %d E %d int8 %d swiglu %d gather %d: nt %d split %d clusters %d stages %d x %d " \
                   "ring %d smem %d accs %d x %d\n", #c, R, N, K, E, int8, swiglu, gather, p.nt, p.split, p.clusters, \
                   p.stages, p.stage_bytes, p.ring_bytes, p.smem, p.accs, p.acc_cols);                               \
    } while (0)

int main()
{
    long long n = 0;
    const int Es[] = {1, 2, 3, 8, 60, 128, 256, 1024}, Ns[] = {1, 16, 77, 128, 129, 300, 1536, 4096, 7168, 65536};
    const int Ks[] = {8, 16, 64, 136, 512, 1024, 2048, 7168, 65536};
    for (int E : Es)
        for (int R = 1; R <= (1 << 22); R += 1 + R / 6)
            for (int N : Ns)
                for (int K : Ks)
                    for (int f = 0; f < 8; ++f) {
                        const bool int8 = (f & 1) && E == 1, swiglu = (f & 2) && !int8, gather = (f & 4) && !int8;
                        const RaggedPlan p = wide_plan(R, N, K, E, int8, swiglu, gather);
                        ++n;
                        CHECK(p.nt >= 32 && p.nt <= 256 && p.nt % 32 == 0);
                        CHECK(p.stages >= 1 && p.stages <= rwide::kMaxPipe && p.stages * p.stage_bytes <= p.ring_bytes);
                        CHECK(p.stage_bytes % 1024 == 0 && p.ring_bytes % 1024 == 0 && p.smem <= 227 * 1024);
                        // a stage holds the box of half a tile
                        CHECK(p.stage_bytes == rwide::kABytes + p.nt / 2 * rwide::kStageKBytes);
                        // tensor memory: a power of two of columns, and no more of it than of shared memory
                        const long long cols = static_cast<long long>(p.accs) * p.acc_cols;
                        CHECK(p.acc_cols >= p.nt && (p.acc_cols & (p.acc_cols - 1)) == 0 && cols <= 512);
                        CHECK((p.smem + 1024LL) * 512 >= cols * 228 * 1024);
                        // several groups: only the widest tile is sure to cut each as counted
                        CHECK(E == 1 || p.nt == 256 || p.nt >= R);
                        // token tiles at most: one per group that has rows, and one more for each nt rows above it
                        const long long tokens = E == 1 ? (R + p.nt - 1) / p.nt : (R < E ? R : E) + (R - 1) / p.nt;
                        const long long tiles = tokens * ((p.row_blocks + 1) / 2);
                        CHECK(tiles < (1LL << 31));
                        CHECK(p.clusters >= 1 && p.clusters <= tiles && 2 * p.split * p.clusters <= 2 * kPlanSMs);
                        CHECK(p.accs == 2 || tiles <= p.clusters);   // one accumulator: one tile at most
                        CHECK(p.split == 1 || (p.accs == 1 && p.kblocks >= p.split));
                        if (p.split > 1) {   // partial sums fit the ring
                            const int rows = p.nt < (R + 31) / 32 * 32 ? p.nt : (R + 31) / 32 * 32, runs = rows / 8;
                            CHECK(p.split * ((runs + p.split - 1) / p.split) * rwide::kRunBytes <= p.ring_bytes);
                        }
                    }
    if (bad) {
        printf("%d of %lld plans wrong\n", bad, n);
        return 1;
    }
    printf("ok %lld plans\n", n);
    return 0;
}
