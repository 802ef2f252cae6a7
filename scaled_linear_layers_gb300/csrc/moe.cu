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
// y move once and the sorted rows once, and sums over j run in a fixed order
// in fp32.
#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

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

// Histogram of each warp's share of this block's chunk: hist[warp][expert].
// A warp counts 32 assignments at a time; the lanes of one expert find each
// other by a match, and the lowest of them adds their number, so no atomics.
template <typename ID>
__device__ __forceinline__ void warp_histogram(const SortArgs &a, int64_t lo, int64_t hi,
                                               int32_t *mine) {
    const int lane = threadIdx.x & 31;
    for (int64_t i = lo; i < hi; i += 32) {
        const int e = expert_at<ID>(a, i + lane, hi);
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        if (e < a.experts && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

__device__ __forceinline__ void warp_share(const SortArgs &a, int64_t &lo, int64_t &hi) {
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, per = a.chunk / kSortWarps;
    const int64_t end = min(a.n, begin + a.chunk);
    lo = min(end, begin + (threadIdx.x >> 5) * per);
    hi = min(end, lo + per);
}

// Assignments to each expert in each chunk.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const SortArgs a) {
    extern __shared__ int32_t hist[];  // [kSortWarps][experts]
    for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    int64_t lo, hi;
    warp_share(a, lo, hi);
    warp_histogram<ID>(a, lo, hi, hist + (threadIdx.x >> 5) * a.experts);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
        int32_t v = 0;
        for (int w = 0; w < kSortWarps; ++w) v += hist[w * a.experts + e];
        a.hist[(int64_t)blockIdx.x * a.experts + e] = v;
    }
}

// Places of one chunk's assignments.  Every block forms the segment offsets
// itself from the chunks' counts (a few KB), so no block waits for another.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const SortArgs a) {
    extern __shared__ int32_t smem[];
    int32_t *hist = smem;                          // [kSortWarps][experts]
    int32_t *total = hist + kSortWarps * a.experts;  // [experts]
    int32_t *first = total + a.experts;            // [experts + 1] segment starts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    int64_t lo, hi;
    warp_share(a, lo, hi);
    warp_histogram<ID>(a, lo, hi, hist + warp * a.experts);
    __syncthreads();
    // hist[w][e] = assignments to e in earlier warps of this chunk and, with
    // more than one chunk, in earlier chunks
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
        int32_t before = 0, all = 0;
        if (a.chunks > 1)
            for (int c = 0; c < a.chunks; ++c) {
                const int32_t v = a.hist[(int64_t)c * a.experts + e];
                before += c < (int)blockIdx.x ? v : 0;
                all += v;
            }
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t v = hist[w * a.experts + e];
            hist[w * a.experts + e] = before;
            before += v;
        }
        total[e] = a.chunks > 1 ? all : before;
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
    int32_t *mine = hist + warp * a.experts;
    for (int64_t i = lo; i < hi; i += 32) {
        const int e = expert_at<ID>(a, i + lane, hi);
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
    }
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) {
            a.offsets[e] = first[e];
            if (e < a.experts) a.counts[e] = total[e];
        }
    }
    // padding: each expert's last rows (a warp to an expert), and what lies
    // past the last segment
    for (int e = blockIdx.x * kSortWarps + warp; e < a.experts; e += gridDim.x * kSortWarps)
        for (int32_t r = first[e] + total[e] + lane; r < first[e + 1]; r += 32) a.source[r] = -1;
    for (int64_t r = first[a.experts] + (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
         r < a.capacity; r += (int64_t)gridDim.x * kSortThreads)
        a.source[r] = -1;
}

// ------------------------------------------------------------------ rows ---

constexpr int kRowThreads = 256;

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

// Zeroes the padding rows (source = -1) among this block's share of them.
template <typename O, int V>
__device__ __forceinline__ void zero_padding(const RowArgs &a, O *out, int block) {
    const int64_t lo = (int64_t)block * a.rows_per_block;
    const int64_t hi = min(a.m.capacity, lo + a.rows_per_block);
    struct alignas(sizeof(O) * V) Group {
        O v[V];
    };
    const Group zero = {};
    for (int64_t r = lo; r < hi; ++r) {
        if (a.m.source[r] >= 0) continue;
        O *to = out + r * a.m.hidden;
        for (int64_t h = (int64_t)threadIdx.x * V; h < a.m.hidden; h += kRowThreads * V)
            *reinterpret_cast<Group *>(to + h) = zero;
    }
}

// The place of assignment j of token t, or -1 (a place outside the sorted
// rows counts as dropped, so a stale index cannot write out of bounds).
__device__ __forceinline__ int64_t place_of(const MoeRows &m, int64_t t, int j) {
    const int64_t r = m.row_of[t * m.topk + j];
    return r < m.capacity ? r : -1;
}

// TPT threads to a token, which each carry one group of V columns at a time:
// one load, topk stores.
template <typename T, bool VECTOR, bool QUANT, int TPT>
__global__ void __launch_bounds__(kRowThreads) moe_dispatch_kernel(const RowArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V, TPB = kRowThreads / TPT;
    pdl_wait_prior();
    pdl_allow_next();
    if ((int)blockIdx.x >= a.token_blocks) {
        if constexpr (QUANT)
            zero_padding<uint8_t, V>(a, a.outq, blockIdx.x - a.token_blocks);
        else
            zero_padding<T, V>(a, reinterpret_cast<T *>(a.out), blockIdx.x - a.token_blocks);
        return;
    }
    const float si = QUANT ? *a.scale_inv : 0.f;
    const int64_t H = a.m.hidden;
    uint32_t m = 0;
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)a.token_blocks * TPB) {
        const T *x = reinterpret_cast<const T *>(a.x) + t * a.ldx;
        for (int64_t h = (int64_t)(threadIdx.x % TPT) * V; h < H; h += TPT * V) {
            const typename RV::Raw v = RV::load(x + h);
            float f[V];
            if constexpr (QUANT) {
                RV::unpack(v, f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    m = max(m, abs_bits(f[i]));
                    f[i] = __fmul_rn(f[i], si);
                }
            }
            for (int j = 0; j < a.m.topk; ++j) {
                const int64_t r = place_of(a.m, t, j);
                if (r < 0) continue;
                if constexpr (QUANT)
                    RV::store_e4m3(a.outq + r * H + h, f);
                else
                    RV::store_raw(reinterpret_cast<T *>(a.out) + r * H + h, v);
            }
        }
    }
    if constexpr (QUANT) {
        if (a.amax != nullptr) {
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            if ((threadIdx.x & 31) == 0 && m != 0)
                atomicMax(reinterpret_cast<unsigned int *>(a.amax), m);
        }
    }
}

template <typename T, bool VECTOR, int TPT>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const RowArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V, TPB = kRowThreads / TPT;
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t H = a.m.hidden;
    const T *rows = reinterpret_cast<const T *>(a.rows);
    for (int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / TPT; t < a.m.tokens;
         t += (int64_t)gridDim.x * TPB) {
        for (int64_t h = (int64_t)(threadIdx.x % TPT) * V; h < H; h += TPT * V) {
            float acc[V] = {};
#pragma unroll 4
            for (int j = 0; j < a.m.topk; ++j) {
                const int64_t r = place_of(a.m, t, j);
                if (r < 0) continue;
                const float w = a.weights != nullptr ? a.weights[t * a.m.topk + j] : 1.f;
                float f[V];
                RV::unpack(RV::load(rows + r * a.ldr + h), f);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(w, f[i], acc[i]);
            }
            RV::store(reinterpret_cast<T *>(a.out) + t * H + h, acc);
        }
    }
}

// One assignment at a time: the dot product's terms need every column of the
// row before the next one starts.
template <typename T, bool VECTOR, int TPT>
__global__ void __launch_bounds__(kRowThreads) moe_combine_bwd_kernel(const RowArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V, TPB = kRowThreads / TPT;
    __shared__ float red[2][TPT > 32 ? TPT / 32 : 1];
    pdl_wait_prior();
    pdl_allow_next();
    if ((int)blockIdx.x >= a.token_blocks) {
        zero_padding<T, V>(a, reinterpret_cast<T *>(a.out), blockIdx.x - a.token_blocks);
        return;
    }
    const int64_t H = a.m.hidden;
    const T *rows = reinterpret_cast<const T *>(a.rows), *dy = reinterpret_cast<const T *>(a.x);
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.m.tokens;
         t0 += (int64_t)a.token_blocks * TPB) {
        const int64_t t = t0 + threadIdx.x / TPT;
        for (int j = 0; j < a.m.topk; ++j, ++turn) {
            const int64_t r = t < a.m.tokens ? place_of(a.m, t, j) : -1;
            float s[1] = {0.f};
            if (r >= 0) {
                const float w = a.weights != nullptr ? a.weights[t * a.m.topk + j] : 1.f;
                for (int64_t h = (int64_t)(threadIdx.x % TPT) * V; h < H; h += TPT * V) {
                    float g[V], f[V];
                    RV::unpack(RV::load(dy + t * a.ldx + h), g);
                    RV::unpack(RV::load(rows + r * a.ldr + h), f);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s[0] = fmaf(g[i], f[i], s[0]);
                        g[i] *= w;
                    }
                    RV::store(reinterpret_cast<T *>(a.out) + r * H + h, g);
                }
            }
            row_sum<TPT, 1>(s, red[turn & 1]);
            if (a.dweights != nullptr && t < a.m.tokens && threadIdx.x % TPT == 0)
                a.dweights[t * a.m.topk + j] = s[0];
        }
    }
}

// Blocks of a persistent walk over the tokens and, for the kernels that also
// write padding rows, the blocks after them.
template <auto KERNEL, int TPT>
cudaError_t launch_rows(RowArgs a, bool padding, cudaStream_t s) {
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(kRowThreads, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)num_sms() * per_sm;
    const int64_t units = (a.m.tokens + kRowThreads / TPT - 1) / (kRowThreads / TPT);
    a.token_blocks = (int)(units < most ? units : most);
    int64_t grid = a.token_blocks;
    if (padding && a.m.capacity > 0) {
        int64_t rpb = (a.m.capacity + 4 * num_sms() - 1) / (4 * num_sms());
        a.rows_per_block = (int)rpb;
        grid += (a.m.capacity + rpb - 1) / rpb;
    }
    if (grid == 0) return cudaSuccess;
    return launch_pdl(KERNEL, (int)grid, kRowThreads, 0, s, a);
}

// Whether rows of `es`-byte elements at p, `ld` apart, can move 16 bytes at a time.
bool row_vectors(const void *p, int64_t ld, int64_t cols, int es) {
    return aligned_to(p, 16) && ld * es % 16 == 0 && cols * es % 16 == 0;
}

// A warp to a token of up to 32 16-byte groups, else a block.
bool narrow(const MoeRows &m, bool vec) { return m.hidden <= 32 * (vec ? (m.f32 ? 4 : 8) : 1); }

template <typename T, bool VECTOR>
cudaError_t dispatch_rows(const RowArgs &a, cudaStream_t s) {
    if (a.outq != nullptr)
        return narrow(a.m, VECTOR)
                   ? launch_rows<moe_dispatch_kernel<T, VECTOR, true, 32>, 32>(a, true, s)
                   : launch_rows<moe_dispatch_kernel<T, VECTOR, true, 256>, 256>(a, true, s);
    return narrow(a.m, VECTOR)
               ? launch_rows<moe_dispatch_kernel<T, VECTOR, false, 32>, 32>(a, true, s)
               : launch_rows<moe_dispatch_kernel<T, VECTOR, false, 256>, 256>(a, true, s);
}

template <typename T, bool VECTOR>
cudaError_t combine_rows(const RowArgs &a, cudaStream_t s) {
    return narrow(a.m, VECTOR) ? launch_rows<moe_combine_kernel<T, VECTOR, 32>, 32>(a, false, s)
                               : launch_rows<moe_combine_kernel<T, VECTOR, 256>, 256>(a, false, s);
}

template <typename T, bool VECTOR>
cudaError_t combine_bwd_rows(const RowArgs &a, cudaStream_t s) {
    return narrow(a.m, VECTOR)
               ? launch_rows<moe_combine_bwd_kernel<T, VECTOR, 32>, 32>(a, true, s)
               : launch_rows<moe_combine_bwd_kernel<T, VECTOR, 256>, 256>(a, true, s);
}

}  // namespace

cudaError_t launch_moe_sort(const void *ids, int ids_64, int64_t n, int experts, int64_t multiple,
                            int64_t capacity, int32_t *row_of, int32_t *source, int32_t *offsets,
                            int32_t *counts, int32_t *workspace, cudaStream_t s) {
    // chunks of a multiple of the block's threads, at most kMoeMaxChunks
    int64_t chunk = kMoeMinChunk;
    if ((n + chunk - 1) / chunk > kMoeMaxChunks)
        chunk = ((n + kMoeMaxChunks - 1) / kMoeMaxChunks + kSortThreads - 1) / kSortThreads *
                kSortThreads;
    SortArgs a = {ids, n, chunk, capacity, multiple, experts, 0, row_of, source, offsets, counts,
                  workspace};
    a.chunks = n > 0 ? (int)((n + chunk - 1) / chunk) : 1;
    const size_t hist = (size_t)kSortWarps * experts * sizeof(int32_t);
    const size_t all = hist + (size_t)(2 * experts + 1) * sizeof(int32_t);
    void (*count)(SortArgs) = ids_64 ? moe_count_kernel<int64_t> : moe_count_kernel<int32_t>;
    void (*place)(SortArgs) = ids_64 ? moe_place_kernel<int64_t> : moe_place_kernel<int32_t>;
    cudaError_t e;
    if (all > 48 * 1024) {
        e = cudaFuncSetAttribute(count, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)hist);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)all);
        if (e != cudaSuccess) return e;
    }
    if (a.chunks > 1) {
        e = launch_pdl(count, a.chunks, kSortThreads, hist, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(place, a.chunks, kSortThreads, all, s, a);
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
    const bool vec = row_vectors(x, ldx, m.hidden, m.f32 ? 4 : 2) &&
                     aligned_to(outq != nullptr ? outq : out, outq != nullptr ? (m.f32 ? 4 : 8) : 16);
    if (m.f32) return vec ? dispatch_rows<float, true>(a, s) : dispatch_rows<float, false>(a, s);
    return vec ? dispatch_rows<uint16_t, true>(a, s) : dispatch_rows<uint16_t, false>(a, s);
}

cudaError_t launch_moe_combine(const MoeRows &m, const void *rows, int64_t ldr,
                               const float *weights, void *y, cudaStream_t s) {
    if (m.hidden == 0) return cudaSuccess;
    RowArgs a = {};
    a.m = m;
    a.rows = rows, a.ldr = ldr, a.weights = weights, a.out = y;
    const bool vec = row_vectors(rows, ldr, m.hidden, m.f32 ? 4 : 2) && aligned_to(y, 16);
    if (m.f32) return vec ? combine_rows<float, true>(a, s) : combine_rows<float, false>(a, s);
    return vec ? combine_rows<uint16_t, true>(a, s) : combine_rows<uint16_t, false>(a, s);
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
    if (m.f32)
        return vec ? combine_bwd_rows<float, true>(a, s) : combine_bwd_rows<float, false>(a, s);
    return vec ? combine_bwd_rows<uint16_t, true>(a, s) : combine_bwd_rows<uint16_t, false>(a, s);
}

}  // namespace fp8
