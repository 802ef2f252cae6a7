// The router of a layer whose linears are split over experts, and its gradient.
//
//   p = softmax(l) over the experts of a token's logits l
//   ids = the topk largest logits (ties: the lowest id), weights = p there, or
//         p over their sum; counts[e] = tokens that chose e, live = tokens
//   losses: balance = E / (live^2 topk) sum_e counts[e] sum_t p[t, e],
//           z = 1/live sum_t lse(l_t)^2
//   gradient at l, with c_e = dbalance E counts[e] / (live^2 topk) and dw the
//   weights' gradient (zero elsewhere):
//     p_e (c_e - sum p c) + 2 dz lse p_e / live
//     + p_e (dw_e - sum p dw), or w_e (dw_e - sum w dw) on the chosen ones for
//     weights over their sum
//
// The counts are constants of the balance loss (whole numbers have no
// gradient).  A logit of -inf closes its expert to the token; a token whose
// mask is 0 or whose experts are all closed has ids of -1, and is in no sum.
//
// A warp takes a token and its lanes share the experts.  A logit and its expert become
// one whole number that orders as the logits do, the lowest expert first among
// equal ones; a lane sorts its own, and a round of the top-k is a maximum over
// the lanes' first ones, whose owner moves on to its next.  Of more experts
// most logits are left out first: topk lanes have one that is at least the
// topk-th largest of the lanes' largest, so only logits from there on can be
// chosen.  Up to a topk of 16 or so they are a few more than topk and are dealt out
// to the lanes anew; near 32 that bar is the least of the lanes' largest, most
// tokens have more above it than are dealt out, and all logits go through the
// rounds.  The chosen logits are read back from their numbers.  Sums over tokens
// are formed per warp, per block and over the blocks (by a cluster of eight
// blocks, a share of the experts each), always in the same order; the counts are
// whole numbers, so their atomics are exact in any order.  Few tokens stay in one
// block and one launch.
//
// Not the bytes bound it: 16384 tokens of 256 fp32 logits, top 8, 14.7 us (2.6 for the
// bytes; bf16 15.0).  The second launch, whose blocks find room only as the first's
// leave, is 3.2 of them, and 570 instructions a token are 8 us of issue slots, which
// bound it while all warps have a token; 304 blocks take the tokens in four passes, the
// last for a third of the warps, so that the SMs issue at 54 % of their rate.  Other
// topk, fp32: 16 16.9, 24 24, 28 43, 32 77; 1024 experts 37 at 8, 40 at 16, 258 at 32.
// With each round of the top-k over all logits and a logit a load it was 68 us, with
// the few logits dealt out by a vote a register 15.6, with the sums over the blocks by
// parts instead of by experts 16.2.  Its gradient, 9.3 us (5.1; bf16 7.9), was 16 with
// a logit a load.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSumCtas = 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kClosed = 0x007FFFFFu;  // the order of -inf

// Logits in their order as whole numbers: NaN the largest (an addition makes
// every NaN the same positive one), equal for the two zeros.
__device__ __forceinline__ uint32_t order_of(float l) {
    const uint32_t b = __float_as_uint(__fadd_rn(l, 0.f));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t order) {
    return __uint_as_float((order >> 31) != 0 ? order ^ 0x80000000u : ~order);
}

// -inf, which stands behind the last expert: a closed one.
template <typename T>
__device__ __forceinline__ T closed_logit() {
    if constexpr (std::is_same<T, float>::value) return -INFINITY;
    else return T(0xFF80u);
}

// How a warp shares a token's experts, R to a lane: every 32nd one, or, where a
// row lies on groups of four (VEC), four neighbours of every 128.
template <int R, bool VEC>
__device__ __forceinline__ int expert_of(int r, int lane) {
    return VEC ? (r >> 2) * 128 + lane * 4 + (r & 3) : r * 32 + lane;
}

template <typename T, int R, bool VEC>
__device__ __forceinline__ void load_logits(const T *row, bool there, int experts, int lane,
                                            T (&l)[R]) {
    if constexpr (VEC) {
        using Four = typename std::conditional<sizeof(T) == 4, float4, ushort4>::type;
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            Four v = {closed_logit<T>(), closed_logit<T>(), closed_logit<T>(), closed_logit<T>()};
            if (there && expert_of<R, VEC>(r, lane) < experts)
                v = *reinterpret_cast<const Four *>(row + expert_of<R, VEC>(r, lane));
            l[r] = v.x, l[r + 1] = v.y, l[r + 2] = v.z, l[r + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
            l[r] = there && r * 32 + lane < experts ? row[r * 32 + lane] : closed_logit<T>();
    }
}

template <typename T, int R, bool VEC>
__device__ __forceinline__ void store_logits(T *row, int experts, int lane, const float (&l)[R]) {
    if constexpr (VEC) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            if (expert_of<R, VEC>(r, lane) >= experts) continue;
            T *at = row + expert_of<R, VEC>(r, lane);
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4 *>(at) = make_float4(l[r], l[r + 1], l[r + 2], l[r + 3]);
            else
                *reinterpret_cast<uint2 *>(at) = make_uint2(pack_bf16x2(l[r], l[r + 1]),
                                                            pack_bf16x2(l[r + 2], l[r + 3]));
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r * 32 + lane < experts) float_to_elem(row + r * 32 + lane, l[r]);
    }
}

// 1/x and log x for x >= 1, by the hardware's approximations: two units in the last
// place; 2^-21.4 of an absolute error up to 2, three units above.  With logf and a
// division 15.5 us and 9.8 for the gradient (14.7 and 9.3); errors against 64 bits as
// before: weights 6e-8 in the 2-norm (6e-8), log-sums' gradient 7e-8 (7e-8).
__device__ __forceinline__ float inverse(float x) { return __fdividef(1.f, x); }
__device__ __forceinline__ float logarithm(float x) { return __logf(x); }

// The order of a logit and its expert as one number; 0 orders behind all.
// bf16 logits leave their order in 16 bits.
template <typename T>
struct Choice {  // fp32
    using Key = uint64_t;
    static __device__ __forceinline__ Key make(uint32_t order, int e) {
        return ((uint64_t)order << 32) | (uint32_t)~e;
    }
    static __device__ __forceinline__ uint32_t order(Key k) { return (uint32_t)(k >> 32); }
    static __device__ __forceinline__ int expert(Key k) { return (int)~(uint32_t)k; }
    static __device__ __forceinline__ Key warp_max(Key k) {
        const uint32_t hi = __reduce_max_sync(kAll, order(k));
        const uint32_t lo = __reduce_max_sync(kAll, order(k) == hi ? (uint32_t)k : 0u);
        return ((uint64_t)hi << 32) | lo;
    }
};
template <>
struct Choice<uint16_t> {
    using Key = uint32_t;
    static __device__ __forceinline__ Key make(uint32_t order, int e) {
        return (order & 0xFFFF0000u) | (uint32_t)(0xFFFF - e);
    }
    // (the low half of a negative logit's order is all ones)
    static __device__ __forceinline__ uint32_t order(Key k) {
        return (k >> 31) != 0 ? k & 0xFFFF0000u : k | 0xFFFFu;
    }
    static __device__ __forceinline__ int expert(Key k) { return 0xFFFF - (int)(k & 0xFFFFu); }
    static __device__ __forceinline__ Key warp_max(Key k) { return __reduce_max_sync(kAll, k); }
};

// Falling order, by Batcher's odd-even merge network.
template <typename K, int N>
__device__ __forceinline__ void sort_falling(K (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const K a = k[i + j], b = k[i + j + q];
                        k[i + j] = a > b ? a : b;
                        k[i + j + q] = a > b ? b : a;
                    }
}

// A lane's largest number that is left, and its removal.
template <typename K, int R, bool SORTED = (R <= 4)>
struct Left;
template <typename K, int R>
struct Left<K, R, true> {
    K k[R];
    __device__ __forceinline__ void begin() { sort_falling(k); }
    __device__ __forceinline__ K first() const { return k[0]; }
    __device__ __forceinline__ void remove(K top) {
        const bool mine = k[0] == top;
#pragma unroll
        for (int r = 0; r + 1 < R; ++r) k[r] = mine ? k[r + 1] : k[r];
        k[R - 1] = mine ? 0 : k[R - 1];
    }
};
template <typename K, int R>
struct Left<K, R, false> {
    K k[R];
    __device__ __forceinline__ void begin() {}
    __device__ __forceinline__ K first() const {
        K best = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) best = k[r] > best ? k[r] : best;
        return best;
    }
    __device__ __forceinline__ void remove(K top) {
#pragma unroll
        for (int r = 0; r < R; ++r) k[r] = k[r] == top ? 0 : k[r];
    }
};

// The topk largest in their order: lane j returns the j-th (0: none).
template <typename C, typename K, int R, bool S>
__device__ __forceinline__ K choose(Left<K, R, S> &left, int topk, int lane) {
    K mine = 0;
    for (int j = 0; j < topk; ++j) {
        const K top = C::warp_max(left.first());
        if (C::order(top) <= kClosed) break;
        if (lane == j) mine = top;
        left.remove(top);
    }
    return mine;
}

template <typename C, bool VEC, int R>
__device__ __forceinline__ Left<typename C::Key, R> numbered(const uint32_t (&order)[R], int lane) {
    Left<typename C::Key, R> left;
#pragma unroll
    for (int r = 0; r < R; ++r)
        left.k[r] = C::make(order[r], expert_of<R, VEC>(r, lane));
    left.begin();
    return left;
}

// Whether the topk go by way of the few logits that can be among them: 64-bit
// numbers cost a round more.  Without and with, 16384 tokens, top 8 (more than 16
// gains less: see the fallback), us: fp32 64
// experts 11.1 and 10.5, 128 13.5 and 11.6, 256 25.9 and 14.6; bf16 128 10.7 and 11.4,
// 256 17.0 and 14.8.
template <typename T, int R>
constexpr bool kByFew = R >= (sizeof(T) == 4 ? 2 : 8);

// The same from the logits' orders, by way of the few that can be among them;
// best: the lane's largest, least: the warp's.  A number's place is the count of
// larger ones.
constexpr int kDealt = 64;
template <typename K>
struct __align__(4 * sizeof(K) > 16 ? 16 : 4 * sizeof(K)) Four {
    K a, b, c, d;
};
template <typename C, bool VEC, int R>
__device__ __forceinline__ typename C::Key choose_few(const uint32_t (&order)[R], uint32_t best,
                                                      uint32_t least, int topk, int lane,
                                                      typename C::Key *dealt) {
    using K = typename C::Key;
    for (int j = 1; j < topk && least > kClosed; ++j) {
        best = best == least ? 0u : best;
        least = __reduce_max_sync(kAll, best);
    }
    least = max(least, kClosed + 1);
    int count = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) count += order[r] >= least;
    int at = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, at, o);
        if (lane >= o) at += v;
    }
    const int found = __shfl_sync(kAll, at, 31);
    K mine = 0;
    if (found <= kDealt) {
        at -= count;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (order[r] >= least) dealt[at++] = C::make(order[r], expert_of<R, VEC>(r, lane));
        if (lane < 3) dealt[found + lane] = 0;  // places are counted four numbers at a time
        __syncwarp();
        const K one = lane < found ? dealt[lane] : K(0);
        const K two = lane + 32 < found ? dealt[lane + 32] : K(0);
        auto larger = [&](K than) {
            int n = 0;
            for (int i = 0; i < found; i += 4) {
                const Four<K> f = *reinterpret_cast<const Four<K> *>(dealt + i);
                n += (f.a > than) + (f.b > than) + (f.c > than) + (f.d > than);
            }
            return n;
        };
        const int place = larger(one), place2 = found > 32 ? larger(two) : 0;
        __syncwarp();
        // back by their places
        if (lane < found) dealt[place] = one;
        if (lane + 32 < found) dealt[place2] = two;
        __syncwarp();
        if (lane < min(found, topk)) mine = dealt[lane];
    } else {  // a topk near 32, or many equal logits
        auto left = numbered<C, VEC>(order, lane);
        mine = choose<C>(left, topk, lane);
    }
    __syncwarp();
    return mine;
}

// e^x for x <= 0: the hardware's 2^y, relative error 2^-22 + |x| 2^-23, zero below
// 2^-126.  expf takes 16.4 us where this takes 14.7, and gives the same errors in the
// 2-norm of weights and gradients (6e-8, 8e-8).
__device__ __forceinline__ float exp_falling(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}

// The sum of probabilities (of lse^2) and the count of one expert (of tokens).
using Part = float2;
__device__ __forceinline__ Part part(float sum, int32_t count) {
    return make_float2(sum, __int_as_float(count));
}
__device__ __forceinline__ int32_t count_of(const Part &p) { return __float_as_int(p.y); }

// balance: the sum of counts times probabilities; z: of lse^2.
__device__ __forceinline__ void write_losses(const Route &a, int32_t tokens, float balance, float z) {
    const float n = (float)max(tokens, 1);
    *a.live = tokens;
    if (a.losses != nullptr) {
        a.losses[0] = balance / n / n * ((float)a.experts / (float)a.topk);
        a.losses[1] = z / n;
    }
}

// The counts and losses from the whole sums, parts(e) for e <= experts, by one
// block; red: 2 + kWarps floats.
template <typename F>
__device__ __forceinline__ void finish(const Route &a, float *red, F parts) {
    float balance = 0.f;
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) {
        const Part p = parts(e);
        if (e < a.experts) {
            a.counts[e] = count_of(p);
            balance += (float)count_of(p) * p.x;
        } else {
            red[0] = __int_as_float(count_of(p));
            red[1] = p.x;
        }
    }
    float v[1] = {balance};
    row_sum<kThreads, 1>(v, red + 2);
    if (threadIdx.x == 0) write_losses(a, __float_as_int(red[0]), v[0], red[1]);
}

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(kThreads, R <= 8 ? 2 : 1) moe_route_kernel(const Route a) {
    using C = Choice<T>;
    using K = typename C::Key;
    extern __shared__ float smem[];
    const int width = a.experts + 1;
    float *sums = smem;                                                     // [kWarps / 2][width]
    int32_t *counts = reinterpret_cast<int32_t *>(sums + kWarps / 2 * width);  // [width]
    float *red = reinterpret_cast<float *>(counts + width);                 // [2 + kWarps]
    __shared__ __align__(16) K dealt[kByFew<T, R> ? kWarps * (kDealt + 4) : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < width; e += kThreads) counts[e] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    float psum[R], zsum = 0.f;
    int32_t tokens = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) psum[r] = 0.f;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    constexpr bool kAhead = R <= 8;  // the next token's logits come while one is worked on
    T next[R];
    bool next_masked = false;
    auto fetch = [&](int64_t at) {
        const bool there = at < a.tokens;
        load_logits<T, R, VEC>(reinterpret_cast<const T *>(a.logits) + at * a.ldl, there, a.experts,
                               lane, next);
        next_masked = there && a.mask != nullptr && a.mask[at] == 0;
    };
    if (kAhead) fetch(t);
    for (; t < a.tokens; t += step) {
        if (!kAhead) fetch(t);
        const bool masked = next_masked;
        float l[R];
        uint32_t order[R], best = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] = elem_to_float(next[r]);
            order[r] = order_of(l[r]);
            best = max(best, order[r]);
        }
        if (kAhead) fetch(t + step);
        const uint32_t top = __reduce_max_sync(kAll, best);
        int my_id = -1;
        float my_w = 0.f;
        if (!masked && top > kClosed) {
            const float peak = logit_of(top);
            float total = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                l[r] = exp_falling(l[r] - peak);
                total += l[r];
            }
            total = warp_sum(total);
            const float inv = inverse(total);
            const float lse = peak + logarithm(total);
            zsum += lse * lse;
            ++tokens;
#pragma unroll
            for (int r = 0; r < R; ++r) psum[r] = fmaf(l[r], inv, psum[r]);
            K mine;
            if constexpr (kByFew<T, R>) {
                mine = choose_few<C, VEC>(order, best, top, a.topk, lane, dealt + warp * (kDealt + 4));
            } else {
                auto left = numbered<C, VEC>(order, lane);
                mine = choose<C>(left, a.topk, lane);
            }
            if (mine != 0) {
                my_id = C::expert(mine);
                my_w = exp_falling(logit_of(C::order(mine)) - peak);
                atomicAdd(&counts[my_id], 1);
            }
            const float chosen = a.renormalize ? inverse(warp_sum(my_w)) : inv;
            my_w = my_id >= 0 ? my_w * chosen : 0.f;
        }
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = my_id;
            a.weights[t * a.topk + lane] = my_w;
        }
    }
    // the warps' sums: the upper half's first, the lower half's added to them
    float *own = sums + (warp % (kWarps / 2)) * width;
#pragma unroll
    for (int upper = 1; upper >= 0; --upper) {
        if (warp / (kWarps / 2) == upper) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = expert_of<R, VEC>(r, lane);
                if (e < a.experts) own[e] = upper ? psum[r] : own[e] + psum[r];
            }
            if (lane == 0) {
                own[a.experts] = upper ? zsum : own[a.experts] + zsum;
                atomicAdd(&counts[a.experts], tokens);
            }
        }
        __syncthreads();
    }
    auto block_part = [&](int e) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps / 2; ++w) v += sums[w * width + e];
        return part(v, counts[e]);
    };
    if (gridDim.x == 1) {
        finish(a, red, block_part);
    } else {
        Part *out = reinterpret_cast<Part *>(a.workspace) + (int64_t)blockIdx.x * width;
        for (int e = threadIdx.x; e < width; e += kThreads) out[e] = block_part(e);
    }
}

// The blocks' parts added up by one cluster: a CTA takes 32 of every 256 columns
// of parts (experts, then the tokens), a lane each, and its warps each 16th block;
// the CTAs' shares of the balance meet in the first.
__global__ void __cluster_dims__(kSumCtas, 1, 1) __launch_bounds__(kThreads)
    moe_route_sum_kernel(const Route a, int blocks) {
    __shared__ Part share[kWarps][32];
    __shared__ float balances;
    __shared__ Part all_tokens;
    const int width = a.experts + 1, rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_prior();
    pdl_allow_next();
    const Part *parts = reinterpret_cast<const Part *>(a.workspace);
    float balance = 0.f;
    for (int e0 = 32 * rank; e0 < width; e0 += 32 * kSumCtas) {
        const int e = e0 + lane;
        float sum = 0.f, err = 0.f;
        int32_t n = 0;
        constexpr int kBatch = 20;  // loads in flight
        for (int b0 = warp; b0 < blocks; b0 += kWarps * kBatch) {
            Part p[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int b = b0 + kWarps * i;
                p[i] = b < blocks && e < width ? parts[(int64_t)b * width + e] : part(0.f, 0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                add_exact(sum, err, p[i].x);
                n += count_of(p[i]);
            }
        }
        share[warp][lane] = part(isinf(sum) ? sum : sum + err, n);  // (inf's err is NaN)
        __syncthreads();
        if (warp == 0 && e < width) {
            sum = 0.f;
            n = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                sum += share[w][lane].x;
                n += count_of(share[w][lane]);
            }
            if (e < a.experts) {
                a.counts[e] = n;
                balance += (float)n * sum;
            } else {
                all_tokens = part(sum, n);
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        balance = warp_sum(balance);
        if (lane == 0) balances = balance;
    }
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
        float sum = 0.f, z, tokens;
        float v[kSumCtas];
#pragma unroll
        for (int c = 0; c < kSumCtas; ++c)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v[c])
                         : "r"(mapa_shared(smem_u32(&balances), c)));
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(z), "=f"(tokens)
                     : "r"(mapa_shared(smem_u32(&all_tokens), a.experts / 32 % kSumCtas)));
#pragma unroll
        for (int c = 0; c < kSumCtas; ++c) sum += v[c];
        write_losses(a, __float_as_int(tokens), sum, z);
    }
    cluster_sync_all();  // the others' sums stay until they have been read
}

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(kThreads, R <= 8 ? 2 : 1)
    moe_route_backward_kernel(const RouteBackward a) {
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *chosen = smem + warp * R * 32;  // the weights' path by expert, zero between tokens
#pragma unroll
    for (int r = 0; r < R; ++r) chosen[r * 32 + lane] = 0.f;
    __syncwarp();
    pdl_wait_prior();
    pdl_allow_next();
    const float n = (float)max(*a.live, 1);
    const float db = a.dlosses == nullptr ? 0.f : a.dlosses[0];
    const float dz = a.dlosses == nullptr ? 0.f : 2.f * a.dlosses[1] / n;
    float c[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = expert_of<R, VEC>(r, lane);
        c[r] = e < a.experts
                   ? db * ((float)a.experts / (float)a.topk) * ((float)a.counts[e] / n) / n
                   : 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * kWarps;
    int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    T next[R];
    int next_id = -1;
    float next_dw = 0.f;
    auto fetch = [&](int64_t at) {
        const bool there = at < a.tokens;
        load_logits<T, R, VEC>(reinterpret_cast<const T *>(a.logits) + at * a.ldl, there, a.experts,
                               lane, next);
        next_id = there && lane < a.topk ? a.ids[at * a.topk + lane] : -1;
        next_dw = there && lane < a.topk && a.dweights != nullptr ? a.dweights[at * a.topk + lane] : 0.f;
    };
    constexpr bool kAhead = R <= 8;
    if (kAhead) fetch(t);
    for (; t < a.tokens; t += step) {
        if (!kAhead) fetch(t);
        T *out = reinterpret_cast<T *>(a.dlogits) + t * a.experts;
        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = elem_to_float(next[r]);
        const bool on = __shfl_sync(kAll, next_id, 0) >= 0;
        const int id = next_id < a.experts ? next_id : -1;
        const float dw = id >= 0 ? next_dw : 0.f;
        if (kAhead) fetch(t + step);
        if (on) {
            // (a NaN is no maximum, but makes the total NaN)
            float best = l[0];
#pragma unroll
            for (int r = 1; r < R; ++r) best = fmaxf(best, l[r]);
            const float peak = logit_of(__reduce_max_sync(kAll, order_of(best)));
            float total = 0.f, pc = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                l[r] = exp_falling(l[r] - peak);
                total += l[r];
                pc = fmaf(l[r], c[r], pc);
            }
            const float mine = id >= 0 ? exp_falling(elem_to_float(
                reinterpret_cast<const T *>(a.logits)[t * a.ldl + id]) - peak) : 0.f;
            total = warp_sum(total);
            pc = warp_sum(pc);
            const float inv = inverse(total);
            float common = dz * (peak + logarithm(total)) - pc * inv;
            const float w = mine * (a.renormalize ? inverse(warp_sum(mine)) : inv);
            const float dot = warp_sum(id >= 0 ? w * dw : 0.f);
            if (!a.renormalize) common -= dot;
            if (id >= 0) chosen[id] = a.renormalize ? w * (dw - dot) : w * dw;
            __syncwarp();
            common *= inv;
            if constexpr (VEC) {
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(chosen + expert_of<R, VEC>(r, lane));
                    l[r] = fmaf(l[r], fmaf(c[r], inv, common), v.x);
                    l[r + 1] = fmaf(l[r + 1], fmaf(c[r + 1], inv, common), v.y);
                    l[r + 2] = fmaf(l[r + 2], fmaf(c[r + 2], inv, common), v.z);
                    l[r + 3] = fmaf(l[r + 3], fmaf(c[r + 3], inv, common), v.w);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    l[r] = fmaf(l[r], fmaf(c[r], inv, common), chosen[r * 32 + lane]);
            }
            __syncwarp();
            if (id >= 0) chosen[id] = 0.f;
            __syncwarp();
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] = 0.f;
        }
        store_logits<T, R, VEC>(out, a.experts, lane, l);
    }
}

// Blocks of a warp to a token, as many as stay on the device at once.
template <auto KERNEL>
cudaError_t route_blocks(int64_t tokens, int most, int *blocks) {
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(kThreads, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t want = (tokens + kWarps - 1) / kWarps, room = (int64_t)per_sm * num_sms();
    *blocks = (int)min(min(want, room), (int64_t)most);
    return cudaSuccess;
}

template <typename T, int R, bool VEC>
cudaError_t route(const Route &a, cudaStream_t s) {
    int blocks = 1;  // at least: the counts of no tokens are zeros
    if (a.tokens > kRouteOneBlock) {
        cudaError_t e = route_blocks<moe_route_kernel<T, R, VEC>>(a.tokens, kRouteMaxBlocks, &blocks);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = ((kWarps / 2 + 1) * (a.experts + 1) + 2 + kWarps) * sizeof(float);
    cudaError_t e = launch_pdl(moe_route_kernel<T, R, VEC>, blocks, kThreads, smem, s, a);
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_pdl(moe_route_sum_kernel, kSumCtas, kThreads, 0, s, a, blocks);
}

template <typename T, int R, bool VEC>
cudaError_t route_backward(const RouteBackward &a, cudaStream_t s) {
    int blocks = 0;
    cudaError_t e = route_blocks<moe_route_backward_kernel<T, R, VEC>>(a.tokens, 1 << 20, &blocks);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)kWarps * R * 32 * sizeof(float);
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(moe_route_backward_kernel<T, R, VEC>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(moe_route_backward_kernel<T, R, VEC>, blocks, kThreads, smem, s, a);
}

// f<T, R, VEC>(a, s) with the smallest R that holds the experts, 32 to a
// register; `four` says that rows lie on groups of four logits.
#define FP8_BY_EXPERTS(f, four)                                                   \
    (a.experts <= 32    ? f<T, 1, false>(a, s)                                    \
     : a.experts <= 64  ? f<T, 2, false>(a, s)                                    \
     : a.experts <= 128 ? (four ? f<T, 4, true>(a, s) : f<T, 4, false>(a, s))     \
     : a.experts <= 256 ? (four ? f<T, 8, true>(a, s) : f<T, 8, false>(a, s))     \
     : a.experts <= 512 ? (four ? f<T, 16, true>(a, s) : f<T, 16, false>(a, s))   \
                        : (four ? f<T, 32, true>(a, s) : f<T, 32, false>(a, s)))

template <typename T>
cudaError_t route_by_type(const Route &a, cudaStream_t s) {
    const bool four = a.experts % 4 == 0 && a.ldl % 4 == 0 && aligned_to(a.logits, 4 * sizeof(T));
    return FP8_BY_EXPERTS(route, four);
}

template <typename T>
cudaError_t backward_by_type(const RouteBackward &a, cudaStream_t s) {
    const bool four = a.experts % 4 == 0 && a.ldl % 4 == 0 && aligned_to(a.logits, 4 * sizeof(T)) &&
                      aligned_to(a.dlogits, 4 * sizeof(T));
    return FP8_BY_EXPERTS(route_backward, four);
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t tokens, int64_t experts) {
    const int64_t blocks = (tokens + kWarps - 1) / kWarps;
    return (blocks > kRouteMaxBlocks ? kRouteMaxBlocks : blocks > 0 ? blocks : 1) *
           (experts + 1) * (int64_t)sizeof(Part);
}

cudaError_t launch_moe_route(const Route &a, cudaStream_t s) {
    return a.f32 ? route_by_type<float>(a, s) : route_by_type<uint16_t>(a, s);
}

cudaError_t launch_moe_route_backward(const RouteBackward &a, cudaStream_t s) {
    if (a.tokens == 0) return cudaSuccess;
    return a.f32 ? backward_by_type<float>(a, s) : backward_by_type<uint16_t>(a, s);
}

}  // namespace fp8
