// What the experts' product kernels share: the arguments of a launch, the
// experts' segments and the search for a tile's expert.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace fp8 {

constexpr int kMoeBlock = 128;    // rows of a tile, and contraction elements a scale
constexpr int kMoeFewRows = 64;   // tokens of a tile where an expert has few

struct MoeArgs {
    const int32_t *offsets;
    int experts;
    int capacity;
    int rows_out, cols_out;  // wgrad: rows of an expert's dw; columns of the output
    int depth;               // contraction blocks (fprop, dgrad)
    int by, bx;              // per expert: where its rows and its columns of B begin
    const float *sa, *sb;
    int64_t sa_row, sa_k;  // scale of A's row i, block kb: sa[i sa_row + kb sa_k]
    int64_t sb_expert, sb_col, sb_k;  // of B's 128 rows j: sb[e sb_expert + j sb_col + kb sb_k]
    uint16_t *d;
    uint64_t wait_limit_ns;
    unsigned int *status;
    int lose;  // (tests) a CTA's third hand-off of copies is waited for but not copied
};

// One output tile.
struct __align__(16) MoeTile {
    int expert, n;   // n: first output column
    int row0, rows;  // A's first row (fprop, dgrad: in the sorted order), rows to store
    int kb0, nk;     // contraction blocks (kb0: the first, wgrad); nk < 0: no tile is left
    int bad, unused;  // bad (wgrad): a segment that does not lie on 128-row blocks
};
static_assert(sizeof(MoeTile) == 32, "two 16-byte loads");

// The experts' segments and the row tiles before each, in shared memory: a
// tile is found without a load from global memory.
struct MoeSegments {
    int32_t *first, *lo, *hi;  // [experts + 1], [experts], [experts]
    __device__ __forceinline__ MoeSegments(int32_t *at, int experts)
        : first(at), lo(at + experts + 1), hi(at + 2 * experts + 1) {}
};
constexpr size_t kMoeSegmentBytes = (3 * kMoeMaxExperts + 1) * sizeof(int32_t);

// For tiles of ROWS rows, by one warp.
template <int ROWS>
__device__ __forceinline__ void moe_count_tiles(const MoeArgs &p, const MoeSegments &g, int lane) {
    int before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
        int lo = 0, hi = 0;
        const int e = e0 + lane;
        if (e < p.experts) {
            // whatever the offsets hold, a segment lies in the rows that exist
            lo = min(max(p.offsets[e], 0), p.capacity);
            hi = min(max(p.offsets[e + 1], lo), p.capacity);
        }
        int sum = (hi - lo + ROWS - 1) / ROWS;
        const int own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        if (e < p.experts) {
            g.first[e] = before + sum - own;
            g.lo[e] = lo;
            g.hi[e] = hi;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) g.first[p.experts] = before;
}

// The expert that the at-th row tile of all belongs to.
__device__ __forceinline__ int moe_expert_of(const MoeSegments &g, int experts, int at) {
    int a = 0, b = experts;  // first[a] <= at < first[b]
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (g.first[mid] <= at) a = mid;
        else b = mid;
    }
    return a;
}

// What the search for tiles allows a tile of `blocks` contraction blocks beside
// the limit of a wait, at 10 us a block (they take 0.3 to 1).
__device__ __forceinline__ uint64_t moe_tile_ns(int blocks) { return 10000ull * (uint64_t)blocks; }

// fprop and dgrad of few rows an expert (gemm_moe_few.cu); a, b as in MoeGemm.
cudaError_t launch_moe_few(const MoeArgs &p, const uint8_t *a, int64_t a_cols, const uint8_t *b,
                           int64_t b_rows, int64_t b_cols, cudaStream_t s, const char **why);

}  // namespace fp8
