// Tokens sorted by expert and back, for a layer whose linears are split over
// experts: every token t has topk assignments (t, j) to an expert, and expert
// e's rows form one segment of the sorted order, padded to a multiple of rows
// so that an FP8 GEMM can take it as it is.
//
//   sort:      row_of[t, j] = offsets[e] + (assignments to e before (t, j)),
//              source[row] = t * topk + j, -1 for padding
//   dispatch:  rows[row_of[t, j]] = x[t] (as stored, or as E4M3 bytes of
//              x * scale_inv with max |x|), padding rows zero
//   combine:   y[t] = sum_j w[t, j] rows[row_of[t, j]]
//   gradients: drows[row_of[t, j]] = w[t, j] dy[t],
//              dw[t, j] = sum_h dy[t, h] rows[row_of[t, j], h],
//              dx[t] = sum_j drows[row_of[t, j]]  (combine with weights of 1)
//
// An id outside 0..experts-1 drops its assignment (row_of = -1): it has no
// row, adds nothing and has a zero weight gradient.  Everything but the sort
// moves rows and is bound by HBM; all kernels go token by token, so x, dy and
// y move once and the sorted rows once (expert by expert the tokens' rows
// would be read topk times: copies of one token lie far apart), and sums over j
// run in a fixed order in fp32.  All of a token's loads are issued before the
// first is used.
//
// Measured (device time; share of the copy bandwidth): combine of 16384 x 2048,
// top 6 of 64, bf16 69 us (1.00); its backward 130 us (0.99), of 16384 x 4096
// top 4 of 32 190 us (0.94); dispatch of 16384 x 4096 to 2 of 8 as E4M3 with the
// sort 50 us (0.81: the sort 5 us, clearing the amax 2); rows of odd width,
// 5003 x 1001 top 6, combine bf16 27 us (0.39), fp32 26 us (0.78), backward 52 us
// (0.37) and 49 us (0.80): a token's setup weighs as much as its words, and a
// bf16 word that lies across two costs two loads.  The sort: 64 assignments 2.7
// us, 32768 4.8 us, 131072 8.3 us.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
// Assignments to a thread that are held in registers from the counting to the
// placing; larger chunks (more than kMoeMaxChunks * 4096 assignments) are read
// twice.
constexpr int kSortFew = 2, kSortMany = 8;
static_assert(kSortFew * kSortThreads == kMoeMinChunk, "the least chunk needs no workspace");

struct SortArgs {
    const void *ids;
    int64_t n, chunk, capacity, multiple;
    int experts, chunks;
    int32_t *row_of, *source, *offsets, *counts, *hist;
};

// Expert of assignment i, or `experts` when it is dropped or i is past `end`.
template <typename ID>
__device__ __forceinline__ int expert_at(const SortArgs &a, int64_t i, int64_t end) {
    if (i >= end) return a.experts;
    const ID id = reinterpret_cast<const ID *>(a.ids)[i];
    return id >= 0 && id < a.experts ? (int)id : a.experts;
}

__device__ __forceinline__ void warp_share(const SortArgs &a, int64_t &lo, int64_t &hi) {
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, per = a.chunk / kSortWarps;
    const int64_t end = min(a.n, begin + a.chunk);
    lo = min(end, begin + (threadIdx.x >> 5) * per);
    hi = min(end, lo + per);
}

// act(i, expert) for each 32 assignments of a warp's share, in order; with
// KEPT > 0 the experts come from `kept`, loaded at once before.
template <typename ID, int KEPT, typename F>
__device__ __forceinline__ void each_32(const SortArgs &a, int64_t lo, int64_t hi,
                                        const int (&kept)[KEPT > 0 ? KEPT : 1], F act) {
    if constexpr (KEPT > 0) {
#pragma unroll
        for (int k = 0; k < KEPT; ++k)
            if (lo + 32 * k < hi) act(lo + 32 * k, kept[k]);
    } else {
        for (int64_t i = lo; i < hi; i += 32)
            act(i, expert_at<ID>(a, i + (threadIdx.x & 31), hi));
    }
}

// Assignments to each expert in each chunk.  The lanes of one expert find each
// other by a match, and the lowest of them adds their number.
template <typename ID, int KEPT>
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const SortArgs a) {
    extern __shared__ int32_t hist[];  // [experts]
    for (int i = threadIdx.x; i < a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    const int lane = threadIdx.x & 31;
    int64_t lo, hi;
    warp_share(a, lo, hi);
    int kept[KEPT > 0 ? KEPT : 1];
#pragma unroll
    for (int k = 0; k < KEPT; ++k) kept[k] = expert_at<ID>(a, lo + 32 * k + lane, hi);
    each_32<ID, KEPT>(a, lo, hi, kept, [&](int64_t, int e) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        if (e < a.experts && lane == __ffs(same) - 1) atomicAdd(&hist[e], __popc(same));
    });
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
        a.hist[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// Places of one chunk's assignments.  Every block forms the segment offsets
// itself from the chunks' counts (a few KB), so no block waits for another.
template <typename ID, int KEPT>
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const SortArgs a) {
    extern __shared__ int32_t smem[];
    int32_t *hist = smem;                            // [kSortWarps][experts]
    int32_t *total = hist + kSortWarps * a.experts;  // [experts]
    int32_t *earlier = total + a.experts;            // [experts] in earlier chunks
    int32_t *first = earlier + a.experts;            // [experts + 1] segment starts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (kSortWarps + 2) * a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    int64_t lo, hi;
    warp_share(a, lo, hi);
    int kept[KEPT > 0 ? KEPT : 1];
#pragma unroll
    for (int k = 0; k < KEPT; ++k) kept[k] = expert_at<ID>(a, lo + 32 * k + lane, hi);
    if (a.chunks > 1) {
        // the chunks' counts: warps side by side over the chunks, lanes over
        // the experts (whole numbers: the order of additions does not matter)
        for (int e = lane; e < a.experts; e += 32) {
            int32_t all = 0, before = 0;
#pragma unroll 8
            for (int c = warp; c < a.chunks; c += kSortWarps) {
                const int32_t v = a.hist[(int64_t)c * a.experts + e];
                all += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&earlier[e], before);
        }
    }
    int32_t *mine = hist + warp * a.experts;
    each_32<ID, KEPT>(a, lo, hi, kept, [&](int64_t, int e) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        if (e < a.experts && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
    __syncthreads();
    // hist[w][e] = assignments to e in earlier warps of this chunk and, with
    // more than one chunk, in earlier chunks
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
        int32_t before = earlier[e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t v = hist[w * a.experts + e];
            hist[w * a.experts + e] = before;
            before += v;
        }
        if (a.chunks == 1) total[e] = before;
    }
    __syncthreads();
    // segment starts: a scan of the padded counts, 32 experts at a time
    if (warp == 0) {
        int32_t base = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            const int32_t n = e < a.experts ? total[e] : 0;
            const int32_t padded = (int32_t)(((int64_t)n + a.multiple - 1) / a.multiple * a.multiple);
            int32_t s = padded;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
                if (lane >= o) s += u;
            }
            if (e < a.experts) first[e] = base + s - padded;
            base += __shfl_sync(0xFFFFFFFFu, s, 31);
        }
        if (lane == 0) first[a.experts] = base;
    }
    __syncthreads();
    each_32<ID, KEPT>(a, lo, hi, kept, [&](int64_t i, int e) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int32_t seen = e < a.experts ? mine[e] : 0;
        __syncwarp();
        if (i + lane < hi) {
            int32_t row = -1;
            if (e < a.experts) {
                row = first[e] + seen + rank;
                a.source[row] = (int32_t)(i + lane);
                if (rank == 0) mine[e] = seen + __popc(same);
            }
            a.row_of[i + lane] = row;
        }
        __syncwarp();
    });
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) {
            a.offsets[e] = first[e];
            if (e < a.experts) a.counts[e] = total[e];
        }
    }
    // padding: each expert's last rows (a warp to an expert), and what lies
    // past the last segment
    for (int e = blockIdx.x * kSortWarps + warp; e < a.experts; e += gridDim.x * kSortWarps)
        for (int64_t r = (int64_t)first[e] + total[e] + lane; r < first[e + 1]; r += 32)
            a.source[r] = -1;
    for (int64_t r = first[a.experts] + (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
         r < a.capacity; r += (int64_t)gridDim.x * kSortThreads)
        a.source[r] = -1;
}

// ------------------------------------------------------------------ rows ---

struct RowArgs {
    MoeRows m;
    const void *x;     // [tokens, hidden]: x or dy
    int64_t ldx;
    const void *rows;  // [capacity, hidden]
    int64_t ldr;
    const float *weights;  // [tokens, topk], nullable
    void *out;             // rows or tokens, contiguous
    uint8_t *outq;
    const float *scale_inv;
    float *amax;
    float *dweights;
    int token_blocks;   // blocks that walk tokens; the others zero padding rows
    int rows_per_block; // rows that one padding block looks at
};

// A block is eight teams of a warp or one larger team; a team takes a token.
constexpr int row_threads(int tpt) { return tpt == 32 ? 256 : tpt; }

// Zeroes the padding rows (source = -1) among this block's share of them: the
// block looks at as many rows as it has threads at once, and lists those.  (One
// stretch of rows to a block left what follows the last segment to few blocks:
// the gradient of 16384 x 1024 top 8 of 128, padded to 128 rows, 109 us, now 98.)
template <typename O>
__device__ __forceinline__ void zero_padding(const RowArgs &a, O *out, int block) {
    __shared__ int32_t list[256];
    __shared__ int count;
    const int64_t H = a.m.hidden;
    // every blocks-th row: the padding past the last segment is spread over all
    const int64_t blocks = gridDim.x - a.token_blocks;
    for (int64_t lo = 0; lo < a.rows_per_block; lo += blockDim.x) {
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        const int64_t mine = (lo + threadIdx.x) * blocks + block;
        if (mine < a.m.capacity && a.m.source[mine] < 0)
            list[atomicAdd(&count, 1)] = (int32_t)mine;
        __syncthreads();
        // a warp to a row, 16 bytes at a time from the first such boundary on
        const int n = count, lane = threadIdx.x & 31;
        for (int k = threadIdx.x >> 5; k < n; k += blockDim.x >> 5) {
            uint8_t *to = reinterpret_cast<uint8_t *>(out + list[k] * H);
            const int64_t bytes = H * (int64_t)sizeof(O);
            const int64_t head = min(bytes, (int64_t)(-reinterpret_cast<uintptr_t>(to) & 15u));
            const int64_t body = head + ((bytes - head) & ~int64_t(15));
            for (int64_t i = head + 16 * lane; i < body; i += 16 * 32)
                *reinterpret_cast<uint4 *>(to + i) = make_uint4(0, 0, 0, 0);
            if (lane < head) to[lane] = 0;
            if (body + lane < bytes) to[body + lane] = 0;
        }
        __syncthreads();
    }
}

// The places of assignments j0 to j0 + KM - 1 of token t, -1 for none (a place
// outside the sorted rows counts as dropped, so a stale index cannot reach out
// of bounds), and their weights, 0 for none.
template <int KM>
__device__ __forceinline__ void places(const RowArgs &a, int64_t t, int j0, int32_t (&r)[KM],
                                       float (&w)[KM]) {
#pragma unroll
    for (int i = 0; i < KM; ++i) {
        const int64_t at = t * a.m.topk + j0 + i;
        r[i] = t < a.m.tokens && j0 + i < a.m.topk ? a.m.row_of[at] : -1;
        if (r[i] >= a.m.capacity) r[i] = -1;
        w[i] = r[i] >= 0 ? (a.weights != nullptr ? a.weights[at] : 1.f) : 0.f;
    }
}

// One load of each group of V columns, topk stores.  U groups at a time, and
// the places of KM assignments, are loaded before anything waits for them.
template <typename T, bool QUANT, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_dispatch_kernel(const RowArgs a) {
    using RV = RowVec<T, true>;
    constexpr int V = RV::V, TPB = row_threads(TPT) / TPT, U = 2;
    pdl_wait_prior();
    pdl_allow_next();
    if ((int)blockIdx.x >= a.token_blocks) {
        if constexpr (QUANT)
            zero_padding<uint8_t>(a, a.outq, blockIdx.x - a.token_blocks);
        else
            zero_padding<T>(a, reinterpret_cast<T *>(a.out), blockIdx.x - a.token_blocks);
        return;
    }
    const float si = QUANT ? *a.scale_inv : 0.f;
    const int64_t H = a.m.hidden;
    const int64_t h0 = (int64_t)(threadIdx.x % TPT) * V;
    float m = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)a.token_blocks * TPB) {
        const T *x = reinterpret_cast<const T *>(a.x) + t * a.ldx;
        int32_t r[KM];
        float w[KM];
        places(a, t, 0, r, w);
        for (int64_t h = h0; h < H; h += TPT * V * U) {
            typename RV::Raw raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                raw[u] = h + u * TPT * V < H ? RV::load(x + h + u * TPT * V) : RV::zero();
            float f[U][V];
            if constexpr (QUANT) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    RV::unpack(raw[u], f[u]);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        m = max_abs_nan(m, f[u][i]);
                        f[u][i] = __fmul_rn(f[u][i], si);
                    }
                }
            }
            for (int j0 = 0; j0 < a.m.topk; j0 += KM) {
                if (j0 > 0) places(a, t, j0, r, w);
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    if (r[i] < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t at = r[i] * H + h + u * TPT * V;
                        if (h + u * TPT * V >= H) continue;
                        if constexpr (QUANT)
                            RV::store_e4m3(a.outq + at, f[u]);
                        else
                            RV::store_raw(reinterpret_cast<T *>(a.out) + at, raw[u]);
                    }
                }
                if (a.m.topk > KM && j0 + KM >= a.m.topk) places(a, t, 0, r, w);
            }
        }
    }
    if constexpr (QUANT) {
        if (a.amax != nullptr) {
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
            if ((threadIdx.x & 31) == 0 && bits != 0)
                atomicMax(reinterpret_cast<unsigned int *>(a.amax), bits);
        }
    }
}

// All KM rows' groups are loaded before they are added, in the order of j.
template <typename T, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_combine_kernel(const RowArgs a) {
    using RV = RowVec<T, true>;
    constexpr int V = RV::V, TPB = row_threads(TPT) / TPT, U = KM > 4 ? 1 : 2;
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t H = a.m.hidden;
    const T *rows = reinterpret_cast<const T *>(a.rows);
    const int64_t h0 = (int64_t)(threadIdx.x % TPT) * V;
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)gridDim.x * TPB) {
        int32_t r[KM];
        float w[KM];
        places(a, t, 0, r, w);
        for (int64_t h = h0; h < H; h += TPT * V * U) {
            float acc[U][V] = {};
            for (int j0 = 0; j0 < a.m.topk; j0 += KM) {
                if (a.m.topk > KM) places(a, t, j0, r, w);
                typename RV::Raw raw[U][KM];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < KM; ++i)
                        raw[u][i] = r[i] >= 0 && h + u * TPT * V < H
                                        ? RV::load(rows + r[i] * a.ldr + h + u * TPT * V)
                                        : RV::zero();
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < KM; ++i) {
                        float f[V];
                        RV::unpack(raw[u][i], f);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[u][v] = fmaf(w[i], f[v], acc[u][v]);
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * TPT * V < H)
                    RV::store(reinterpret_cast<T *>(a.out) + t * H + h + u * TPT * V, acc[u]);
        }
    }
}

// dy's groups are loaded once for KM assignments, whose dot products are
// summed over the team together at the end of the row.
template <typename T, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_combine_bwd_kernel(const RowArgs a) {
    using RV = RowVec<T, true>;
    constexpr int V = RV::V, TPB = row_threads(TPT) / TPT, U = KM > 4 ? 1 : 2;
    __shared__ float red[2][KM * (TPT > 32 ? TPT / 32 : 1)];
    pdl_wait_prior();
    pdl_allow_next();
    if ((int)blockIdx.x >= a.token_blocks) {
        zero_padding<T>(a, reinterpret_cast<T *>(a.out), blockIdx.x - a.token_blocks);
        return;
    }
    const int64_t H = a.m.hidden;
    const T *rows = reinterpret_cast<const T *>(a.rows), *dy = reinterpret_cast<const T *>(a.x);
    const int64_t h0 = (int64_t)(threadIdx.x % TPT) * V;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.m.tokens;
         t0 += (int64_t)a.token_blocks * TPB) {
        const int64_t t = t0 + threadIdx.x / TPT;
        for (int j0 = 0; j0 < a.m.topk; j0 += KM, ++turn) {
            int32_t r[KM];
            float w[KM], s[KM];
            places(a, t, j0, r, w);
#pragma unroll
            for (int i = 0; i < KM; ++i) s[i] = 0.f;
            for (int64_t h = t < a.m.tokens ? h0 : H; h < H; h += TPT * V * U) {
                typename RV::Raw g[U], raw[U][KM];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = h + u * TPT * V < H;
                    g[u] = in ? RV::load(dy + t * a.ldx + h + u * TPT * V) : RV::zero();
#pragma unroll
                    for (int i = 0; i < KM; ++i)
                        raw[u][i] = in && r[i] >= 0 ? RV::load(rows + r[i] * a.ldr + h + u * TPT * V)
                                                    : RV::zero();
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float fg[V];
                    RV::unpack(g[u], fg);
#pragma unroll
                    for (int i = 0; i < KM; ++i) {
                        if (r[i] < 0) continue;
                        float f[V];
                        RV::unpack(raw[u][i], f);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            s[i] = fmaf(fg[v], f[v], s[i]);
                            f[v] = fg[v] * w[i];
                        }
                        if (h + u * TPT * V < H)
                            RV::store(reinterpret_cast<T *>(a.out) + r[i] * H + h + u * TPT * V, f);
                    }
                }
            }
            if (a.dweights == nullptr) continue;
            row_sum<TPT, KM>(s, red[turn & 1]);
            if (t < a.m.tokens && threadIdx.x % TPT == 0) {
#pragma unroll
                for (int i = 0; i < KM; ++i)
                    if (j0 + i < a.m.topk) a.dweights[t * a.m.topk + j0 + i] = s[i];
            }
        }
    }
}

// Rows that 16-byte groups do not fit (an odd width, an unaligned address).  A
// team goes along the row it writes by *that* row's aligned words of WordRow's
// V elements, so that stores stay whole; elements of half a word, at the row's
// ends, go singly.  What it reads is shifted into place, without branches, so
// that many loads are in flight.  A word's loads may take in the element before
// the row or the two after it; where the tensor has none, at its first and last rows, a
// token goes element by element.

// The rows of a [rows, H] tensor of row stride ld that have neighbours for that.
template <typename T>
struct Inner {
    const T *p;
    int64_t ld, first, last;
    __device__ __forceinline__ Inner(const void *base, int64_t rows, int64_t stride) {
        p = reinterpret_cast<const T *>(base);
        ld = stride;
        const int64_t margin = WordRow<T>::V == 1 ? 0 : ld > 1 ? 1 : ld > 0 ? 2 : rows;
        first = margin;
        last = rows - margin;
    }
    __device__ __forceinline__ const T *row(int64_t r) const { return p + r * ld; }
    // (a dropped assignment loads row `first` instead, and drops what it got:
    // loads under a condition of their own would wait for one another)
    __device__ __forceinline__ bool holds(int64_t r) const { return r >= first && r < last; }
};

// Elements of the row at p before its first whole word of V (0 or 1).
template <int V, typename O>
__device__ __forceinline__ int before_words(const O *p) {
    return (int)((reinterpret_cast<uintptr_t>(p) / sizeof(O)) & (V - 1));
}

// Whether a row of H elements, `head` before its first word, leaves an element
// out of its words for this lane: lane 0 the first, lane 1 the last.
template <int V>
__device__ __forceinline__ bool at_end(int lane, int head, int64_t H) {
    return V > 1 && ((lane == 0 && head > 0) || (lane == 1 && ((H - head) & (V - 1)) != 0));
}

template <typename T, bool QUANT, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_dispatch_any_kernel(const RowArgs a) {
    using W = WordRow<T>;
    using O = typename std::conditional<QUANT, uint8_t, T>::type;
    constexpr int V = W::V, TPB = row_threads(TPT) / TPT, U = 4;
    pdl_wait_prior();
    pdl_allow_next();
    O *out = QUANT ? reinterpret_cast<O *>(a.outq) : reinterpret_cast<O *>(a.out);
    if ((int)blockIdx.x >= a.token_blocks) {
        zero_padding<O>(a, out, blockIdx.x - a.token_blocks);
        return;
    }
    const float si = QUANT ? *a.scale_inv : 0.f;
    const int64_t H = a.m.hidden;
    const int lane = threadIdx.x % TPT;
    const Inner<T> in(a.x, a.m.tokens, a.ldx);
    float m = 0.f;
    auto one = [&](O *to, float f) {
        if constexpr (QUANT)
            *to = (uint8_t)(cvt_e4m3x2(__fmul_rn(f, si), 0.f) & 0xFFu);
        else
            float_to_elem(to, f);
    };
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)a.token_blocks * TPB) {
        const T *x = in.row(t);
        const bool whole = in.holds(t);
        for (int j0 = 0; j0 < a.m.topk; j0 += KM) {
            int32_t r[KM];
            float w[KM];
            places(a, t, j0, r, w);
            if (!whole) {
                for (int64_t e = lane; e < H; e += TPT) {
                    const float f = elem_to_float(x[e]);
                    m = max_abs_nan(m, f);
                    for (int i = 0; i < KM; ++i)
                        if (r[i] >= 0) one(out + r[i] * H + e, f);
                }
                continue;
            }
            int head[KM];
#pragma unroll
            for (int i = 0; i < KM; ++i) {
                head[i] = r[i] >= 0 ? before_words<V>(out + r[i] * H) : 0;
                if (r[i] < 0) continue;
                if (at_end<V>(lane, head[i], H)) {
                    const int64_t e = lane > 0 ? H - 1 : 0;
                    one(out + r[i] * H + e, elem_to_float(x[e]));
                }
            }
            // x in words from its first element on and from its second on:
            // each row takes those that its own words hold
            const W even(x), odd(x + (V - 1));
            for (int64_t w0 = lane; w0 * V < H; w0 += U * TPT) {
                typename W::Raw from[V][U];
                uint32_t raw[V][U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = w0 + u * TPT;
                    from[0][u] = even.load(at, at * V < H);
                    if constexpr (V == 2) from[1][u] = odd.load(at, at * V + 1 < H);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[0][u] = even.word(from[0][u]);
                    if constexpr (V == 2) raw[1][u] = odd.word(from[1][u]);
                }
                if constexpr (QUANT) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float f[V], q[2] = {0.f, 0.f};
                            W::unpack(raw[v][u], f);
                            const int64_t e = (w0 + u * TPT) * V + v;
#pragma unroll
                            for (int k = 0; k < V; ++k) {
                                if (v == 0 && e + k < H) m = max_abs_nan(m, f[k]);
                                q[k] = __fmul_rn(f[k], si);
                            }
                            raw[v][u] = cvt_e4m3x2(q[0], q[1]);
                        }
                }
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    if (r[i] < 0) continue;
                    O *to = out + r[i] * H + head[i];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t at = w0 + u * TPT;
                        if (head[i] + at * V + V > H) continue;
                        const uint32_t v = V == 2 && head[i] > 0 ? raw[V - 1][u] : raw[0][u];
                        if constexpr (!QUANT)
                            *reinterpret_cast<uint32_t *>(to + at * V) = v;
                        else if constexpr (V == 2)
                            *reinterpret_cast<uint16_t *>(to + at * V) = (uint16_t)v;
                        else
                            to[at] = (uint8_t)v;
                    }
                }
            }
        }
    }
    if constexpr (QUANT) {
        if (a.amax != nullptr) {
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
            if ((threadIdx.x & 31) == 0 && bits != 0)
                atomicMax(reinterpret_cast<unsigned int *>(a.amax), bits);
        }
    }
}

template <typename T, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_combine_any_kernel(const RowArgs a) {
    using W = WordRow<T>;
    constexpr int V = W::V, TPB = row_threads(TPT) / TPT, U = KM <= 2 ? 4 : 2;
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t H = a.m.hidden;
    const int lane = threadIdx.x % TPT;
    const Inner<T> in(a.rows, a.m.capacity, a.ldr);
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)gridDim.x * TPB) {
        T *to = reinterpret_cast<T *>(a.out) + t * H;
        const int head = before_words<V>(to);
        const int64_t words = (H - head) / V;
        int32_t r[KM];
        float w[KM];
        W src[KM];
        bool whole = in.first < in.last;
        auto take = [&](int j0) {
            places(a, t, j0, r, w);
#pragma unroll
            for (int i = 0; i < KM; ++i) {
                whole = whole && (r[i] < 0 || in.holds(r[i]));
                src[i] = W(in.row(r[i] < 0 ? in.first : r[i]) + head);
            }
        };
        auto single = [&](int64_t e) {
            float acc = 0.f;
            for (int j0 = 0; j0 < a.m.topk; j0 += KM) {
                places(a, t, j0, r, w);
#pragma unroll
                for (int i = 0; i < KM; ++i)
                    acc = fmaf(w[i], r[i] >= 0 ? elem_to_float(in.row(r[i])[e]) : 0.f, acc);
            }
            float_to_elem(to + e, acc);
        };
        for (int j0 = 0; j0 < a.m.topk; j0 += KM) take(j0);
        if (!whole) {
            for (int64_t e = lane; e < H; e += TPT) single(e);
            continue;
        }
        for (int64_t w0 = lane; w0 < words; w0 += U * TPT) {
            float acc[U][V] = {};
            for (int j0 = 0; j0 < a.m.topk; j0 += KM) {
                if (a.m.topk > KM) take(j0);
                typename W::Raw raw[KM][U];
#pragma unroll
                for (int i = 0; i < KM; ++i)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        raw[i][u] = src[i].load(w0 + u * TPT, w0 + u * TPT < words);
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    if (r[i] < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float f[V];
                        W::unpack(src[i].word(raw[i][u]), f);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[u][v] = fmaf(w[i], f[v], acc[u][v]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (w0 + u * TPT < words)
                    *reinterpret_cast<uint32_t *>(to + head + (w0 + u * TPT) * V) = W::pack(acc[u]);
        }
        if (at_end<V>(lane, head, H)) single(lane > 0 ? H - 1 : 0);
    }
}

template <typename T, int TPT, int KM>
__global__ void __launch_bounds__(row_threads(TPT)) moe_combine_bwd_any_kernel(const RowArgs a) {
    using W = WordRow<T>;
    constexpr int V = W::V, TPB = row_threads(TPT) / TPT, U = 4;
    __shared__ float red[2][KM * (TPT > 32 ? TPT / 32 : 1)];
    pdl_wait_prior();
    pdl_allow_next();
    if ((int)blockIdx.x >= a.token_blocks) {
        zero_padding<T>(a, reinterpret_cast<T *>(a.out), blockIdx.x - a.token_blocks);
        return;
    }
    const int64_t H = a.m.hidden;
    const int lane = threadIdx.x % TPT;
    const Inner<T> in(a.rows, a.m.capacity, a.ldr), grad(a.x, a.m.tokens, a.ldx);
    T *out = reinterpret_cast<T *>(a.out);
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.m.tokens;
         t0 += (int64_t)a.token_blocks * TPB) {
        const int64_t t = t0 + threadIdx.x / TPT;
        const T *dy = grad.row(t);
        for (int j0 = 0; j0 < a.m.topk; j0 += KM, ++turn) {
            int32_t r[KM];
            float w[KM], s[KM] = {};
            places(a, t, j0, r, w);
            bool whole = grad.holds(t) && in.first < in.last;
            auto single = [&](int i, int64_t e) {
                const float g = elem_to_float(dy[e]);
                s[i] = fmaf(g, elem_to_float(in.row(r[i])[e]), s[i]);
                float_to_elem(out + r[i] * H + e, g * w[i]);
            };
            int head[KM];
            W src[KM];
#pragma unroll
            for (int i = 0; i < KM; ++i) {
                whole = whole && (r[i] < 0 || in.holds(r[i]));
                head[i] = r[i] >= 0 ? before_words<V>(out + r[i] * H) : 0;
                src[i] = W(in.row(r[i] < 0 ? in.first : r[i]) + head[i]);
            }
            if (whole) {
                const W even(dy), odd(dy + (V - 1));  // as the dispatch's
                for (int64_t w0 = lane; w0 * V < H; w0 += U * TPT) {
                    typename W::Raw raw[KM][U], from[V][U];
                    uint32_t g[V][U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t at = w0 + u * TPT;
                        from[0][u] = even.load(at, at * V < H);
                        if constexpr (V == 2) from[1][u] = odd.load(at, at * V + 1 < H);
                    }
#pragma unroll
                    for (int i = 0; i < KM; ++i)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int64_t at = w0 + u * TPT;
                            raw[i][u] = src[i].load(at, head[i] + at * V + V <= H);
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        g[0][u] = even.word(from[0][u]);
                        if constexpr (V == 2) g[1][u] = odd.word(from[1][u]);
                    }
#pragma unroll
                    for (int i = 0; i < KM; ++i) {
                        if (r[i] < 0) continue;
                        T *to = out + r[i] * H + head[i];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int64_t at = w0 + u * TPT;
                            if (head[i] + at * V + V > H) continue;
                            float f[V], fg[V];
                            W::unpack(src[i].word(raw[i][u]), f);
                            W::unpack(V == 2 && head[i] > 0 ? g[V - 1][u] : g[0][u], fg);
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                s[i] = fmaf(fg[v], f[v], s[i]);
                                f[v] = fg[v] * w[i];
                            }
                            *reinterpret_cast<uint32_t *>(to + at * V) = W::pack(f);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    if (r[i] >= 0 && at_end<V>(lane, head[i], H)) single(i, lane > 0 ? H - 1 : 0);
                }
            } else if (t < a.m.tokens) {
#pragma unroll
                for (int i = 0; i < KM; ++i)
                    if (r[i] >= 0)
                        for (int64_t e = lane; e < H; e += TPT) single(i, e);
            }
            if (a.dweights == nullptr) continue;
            row_sum<TPT, KM>(s, red[turn & 1]);
            if (t < a.m.tokens && lane == 0) {
#pragma unroll
                for (int i = 0; i < KM; ++i)
                    if (j0 + i < a.m.topk) a.dweights[t * a.m.topk + j0 + i] = s[i];
            }
        }
    }
}

// Blocks of a persistent walk over the tokens and, for the kernels that also
// write padding rows, the blocks after them.
template <auto KERNEL, int TPT>
cudaError_t launch_rows(RowArgs a, bool padding, cudaStream_t s) {
    constexpr int THREADS = row_threads(TPT), TPB = THREADS / TPT;
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(THREADS, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)num_sms() * per_sm, units = (a.m.tokens + TPB - 1) / TPB;
    a.token_blocks = (int)(units < most ? units : most);
    int64_t grid = a.token_blocks;
    if (padding && a.m.capacity > 0) {
        const int64_t rpb = (a.m.capacity + 4 * num_sms() - 1) / (4 * num_sms());
        a.rows_per_block = (int)rpb;
        grid += (a.m.capacity + rpb - 1) / rpb;
    }
    if (grid == 0) return cudaSuccess;
    return launch_pdl(KERNEL, (int)grid, THREADS, 0, s, a);
}

// Whether rows of `es`-byte elements at p, `ld` apart, can move 16 bytes at a time.
bool row_vectors(const void *p, int64_t ld, int64_t cols, int es) {
    return aligned_to(p, 16) && ld * es % 16 == 0 && cols * es % 16 == 0;
}

// f(threads to a token, assignments at a time): the fewest threads that have
// at most `per_lane` of `units` each, at most 256; the fewest assignments at a
// time that take them all, at most 8.
template <typename F>
cudaError_t with_team(const MoeRows &m, int64_t units, int per_lane, F f) {
    auto km = [&](auto tpt) -> cudaError_t {
        if (m.topk <= 1) return f(tpt, std::integral_constant<int, 1>{});
        if (m.topk <= 2) return f(tpt, std::integral_constant<int, 2>{});
        if (m.topk <= 4) return f(tpt, std::integral_constant<int, 4>{});
        if (m.topk <= 6) return f(tpt, std::integral_constant<int, 6>{});
        return f(tpt, std::integral_constant<int, 8>{});
    };
    if (units <= 32 * per_lane) return km(std::integral_constant<int, 32>{});
    if (units <= 128 * per_lane) return km(std::integral_constant<int, 128>{});
    return km(std::integral_constant<int, 256>{});
}

// Rows of 16-byte groups, `per_lane` of them to a thread.
template <typename F>
cudaError_t with_groups(const MoeRows &m, int per_lane, F f) {
    return with_team(m, m.hidden / (m.f32 ? 4 : 8), per_lane, f);
}

// Rows of 4-byte words: as few threads as share a row (5003 x 1001 fp32 by 128
// threads: combine 26 us, by 256 29), unless there are too few tokens to fill
// the GPU with (100 x 2047 bf16: 5.5 and 7.6 the other way).  The gradient takes
// two assignments at a time (1000 x 4095 top 8 bf16: 73 us, by four 81).
template <typename F>
cudaError_t with_words(const MoeRows &m, F f) {
    return with_team(m, m.hidden / (m.f32 ? 1 : 2), m.tokens >= 8 * (int64_t)num_sms() ? 8 : 4, f);
}

template <typename T>
cudaError_t dispatch_rows(const RowArgs &a, bool vec, cudaStream_t s) {
    if (vec)
        return with_groups(a.m, 4, [&](auto tpt, auto km) {
            constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value;
            return a.scale_inv != nullptr
                       ? launch_rows<moe_dispatch_kernel<T, true, TPT, KM>, TPT>(a, true, s)
                       : launch_rows<moe_dispatch_kernel<T, false, TPT, KM>, TPT>(a, true, s);
        });
    return with_words(a.m, [&](auto tpt, auto km) {
        constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value;
        return a.scale_inv != nullptr
                   ? launch_rows<moe_dispatch_any_kernel<T, true, TPT, KM>, TPT>(a, true, s)
                   : launch_rows<moe_dispatch_any_kernel<T, false, TPT, KM>, TPT>(a, true, s);
    });
}

template <typename T>
cudaError_t combine_rows(const RowArgs &a, bool vec, cudaStream_t s) {
    if (vec)
        return with_groups(a.m, 2, [&](auto tpt, auto km) {
            constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value;
            return launch_rows<moe_combine_kernel<T, TPT, KM>, TPT>(a, false, s);
        });
    return with_words(a.m, [&](auto tpt, auto km) {
        constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value;
        return launch_rows<moe_combine_any_kernel<T, TPT, KM>, TPT>(a, false, s);
    });
}

template <typename T>
cudaError_t combine_bwd_rows(const RowArgs &a, bool vec, cudaStream_t s) {
    if (vec)
        return with_groups(a.m, 4, [&](auto tpt, auto km) {
            constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value;
            return launch_rows<moe_combine_bwd_kernel<T, TPT, KM>, TPT>(a, true, s);
        });
    return with_words(a.m, [&](auto tpt, auto km) {
        constexpr int TPT = decltype(tpt)::value, KM = decltype(km)::value > 2 ? 2 : decltype(km)::value;
        return launch_rows<moe_combine_bwd_any_kernel<T, TPT, KM>, TPT>(a, true, s);
    });
}

}  // namespace

cudaError_t launch_moe_sort(const void *ids, int ids_64, int64_t n, int experts, int64_t multiple,
                            int64_t capacity, int32_t *row_of, int32_t *source, int32_t *offsets,
                            int32_t *counts, int32_t *workspace, cudaStream_t s) {
    // chunks of a multiple of the block's threads, at most kMoeMaxChunks, as
    // small as that allows so that more SMs share the work
    int64_t chunk = kSortFew * kSortThreads;
    if (n > kMoeMaxChunks * chunk) chunk = kSortMany * kSortThreads;
    if (n > kMoeMaxChunks * chunk)
        chunk = ((n + kMoeMaxChunks - 1) / kMoeMaxChunks + kSortThreads - 1) / kSortThreads *
                kSortThreads;
    SortArgs a = {ids, n, chunk, capacity, multiple, experts, 0, row_of, source, offsets, counts,
                  workspace};
    a.chunks = n > 0 ? (int)((n + chunk - 1) / chunk) : 1;
    const size_t hist = (size_t)kSortWarps * experts * sizeof(int32_t);
    const size_t all = hist + (size_t)(3 * experts + 1) * sizeof(int32_t);
    auto run = [&](auto count, auto place) -> cudaError_t {
        cudaError_t e;
        if (all > 48 * 1024) {
            e = cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)all);
            if (e != cudaSuccess) return e;
        }
        if (a.chunks > 1) {
            e = launch_pdl(count, a.chunks, kSortThreads, experts * sizeof(int32_t), s, a);
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(place, a.chunks, kSortThreads, all, s, a);
    };
    auto pick = [&](auto id) -> cudaError_t {
        using ID = decltype(id);
        if (chunk == kSortFew * kSortThreads)
            return run(moe_count_kernel<ID, kSortFew>, moe_place_kernel<ID, kSortFew>);
        if (chunk == kSortMany * kSortThreads)
            return run(moe_count_kernel<ID, kSortMany>, moe_place_kernel<ID, kSortMany>);
        return run(moe_count_kernel<ID, 0>, moe_place_kernel<ID, 0>);
    };
    return ids_64 ? pick(int64_t{}) : pick(int32_t{});
}

cudaError_t launch_moe_dispatch(const MoeRows &m, const void *x, int64_t ldx, void *out,
                                uint8_t *outq, const float *scale_inv, float *amax,
                                cudaStream_t s) {
    if (amax != nullptr) {
        cudaError_t e = launch_zero_f32(amax, 1, s);
        if (e != cudaSuccess) return e;
    }
    if (m.hidden == 0) return cudaSuccess;
    RowArgs a = {};
    a.m = m;
    a.x = x, a.ldx = ldx;
    a.out = out, a.outq = outq, a.scale_inv = scale_inv, a.amax = amax;
    // (a cast without rows to write still finds the amax)
    const bool quant = scale_inv != nullptr;
    const bool vec = row_vectors(x, ldx, m.hidden, m.f32 ? 4 : 2) &&
                     aligned_to(quant ? outq : out, quant ? (m.f32 ? 4 : 8) : 16);
    return m.f32 ? dispatch_rows<float>(a, vec, s) : dispatch_rows<uint16_t>(a, vec, s);
}

cudaError_t launch_moe_combine(const MoeRows &m, const void *rows, int64_t ldr,
                               const float *weights, void *y, cudaStream_t s) {
    if (m.hidden == 0) return cudaSuccess;
    RowArgs a = {};
    a.m = m;
    a.rows = rows, a.ldr = ldr, a.weights = weights, a.out = y;
    const bool vec = row_vectors(rows, ldr, m.hidden, m.f32 ? 4 : 2) && aligned_to(y, 16);
    return m.f32 ? combine_rows<float>(a, vec, s) : combine_rows<uint16_t>(a, vec, s);
}

cudaError_t launch_moe_combine_backward(const MoeRows &m, const void *dy, int64_t lddy,
                                        const void *rows, int64_t ldr, const float *weights,
                                        void *drows, float *dweights, cudaStream_t s) {
    if (m.hidden == 0)
        return dweights != nullptr ? launch_zero_f32(dweights, m.tokens * m.topk, s) : cudaSuccess;
    RowArgs a = {};
    a.m = m;
    a.x = dy, a.ldx = lddy;
    a.rows = rows, a.ldr = ldr, a.weights = weights, a.out = drows, a.dweights = dweights;
    const int es = m.f32 ? 4 : 2;
    const bool vec = row_vectors(dy, lddy, m.hidden, es) && row_vectors(rows, ldr, m.hidden, es) &&
                     aligned_to(drows, 16);
    return m.f32 ? combine_bwd_rows<float>(a, vec, s) : combine_bwd_rows<uint16_t>(a, vec, s);
}

}  // namespace fp8
