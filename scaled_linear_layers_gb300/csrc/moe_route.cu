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
// A warp takes a token, a lane every 32nd expert.  The order of logits is the
// order of whole numbers made of their bits, so a round of the top-k is a
// maximum over the lane's own, one over the warp, and a minimum over the ids
// that have it.  Sums over tokens are formed per warp, then per block, then
// over the blocks, always in the same order; the counts are whole numbers, so
// their atomics are exact in any order.
#include "common.cuh"
#include "kernels.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Logits in their order as whole numbers: 0 for -inf (closed), the largest for
// NaN, equal ones for the two zeros.
__device__ __forceinline__ uint32_t order_key(float l) {
    if (l != l) return kAll;
    const uint32_t b = __float_as_uint(l + 0.f);
    if (b == 0xFF800000u) return 0u;
    return b ^ ((b >> 31) != 0 ? kAll : 0x80000000u);
}

template <typename T>
__device__ __forceinline__ float logit_at(const T *row, int e, int experts) {
    return e < experts ? elem_to_float(row[e]) : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// A block's part of the sums: probabilities [experts], then the sum of lse^2;
// counts [experts], then the tokens.
struct Parts {
    float *sums;
    int32_t *counts;
};

__device__ __forceinline__ Parts parts_of(const Route &a, int block) {
    float *base = a.workspace + (int64_t)block * 2 * (a.experts + 1);
    return {base, reinterpret_cast<int32_t *>(base + a.experts + 1)};
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const Route a) {
    extern __shared__ float smem[];
    float *sums = smem;                                                   // [kWarps][experts + 1]
    int32_t *counts = reinterpret_cast<int32_t *>(sums + kWarps * (a.experts + 1));  // [experts + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) counts[e] = 0;
    __syncthreads();
    pdl_wait_prior();
    pdl_allow_next();
    float psum[R], zsum = 0.f;
    int32_t tokens = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) psum[r] = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.tokens;
         t += (int64_t)gridDim.x * kWarps) {
        const T *row = reinterpret_cast<const T *>(a.logits) + t * a.ldl;
        const bool masked = a.mask != nullptr && a.mask[t] == 0;
        float l[R];
        uint32_t key[R];
        float peak = -INFINITY;
        bool open = false;
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = logit_at(row, r * 32 + lane, a.experts);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            key[r] = order_key(l[r]);
            open |= key[r] != 0;
            peak = fmaxf(peak, l[r]);
        }
        const bool on = !masked && __any_sync(kAll, open);
        int my_id = -1;
        float my_w = 0.f;
        if (on) {
            peak = warp_max(peak);
            float total = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                l[r] = r * 32 + lane < a.experts ? expf(l[r] - peak) : 0.f;
                total += l[r];
            }
            total = warp_sum(total);
            const float lse = peak + logf(total);
            zsum += lse * lse;
            ++tokens;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                l[r] = __fdiv_rn(l[r], total);
                psum[r] += l[r];
            }
            for (int j = 0; j < a.topk; ++j) {
                uint32_t best = 0;
                int at = 0;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (key[r] > best) best = key[r], at = r;
                const uint32_t top = __reduce_max_sync(kAll, best);
                if (top == 0) break;
                const uint32_t id =
                    __reduce_min_sync(kAll, best == top ? (uint32_t)(at * 32 + lane) : kAll);
                float w = 0.f;
                const bool mine = lane == (int)(id & 31u);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (mine && r == (int)(id >> 5)) {
                        key[r] = 0;
                        w = l[r];
                    }
                w = __shfl_sync(kAll, w, id & 31u);
                if (lane == j) {
                    my_id = (int)id;
                    my_w = w;
                }
            }
            if (a.renormalize) {
                const float chosen = warp_sum(my_w);
                if (my_id >= 0) my_w = __fdiv_rn(my_w, chosen);
            }
            if (my_id >= 0) atomicAdd(&counts[my_id], 1);
        }
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = my_id;
            a.weights[t * a.topk + lane] = my_w;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r * 32 + lane < a.experts) sums[warp * (a.experts + 1) + r * 32 + lane] = psum[r];
    if (lane == 0) {
        sums[warp * (a.experts + 1) + a.experts] = zsum;
        atomicAdd(&counts[a.experts], tokens);
    }
    __syncthreads();
    const Parts out = parts_of(a, blockIdx.x);
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sums[w * (a.experts + 1) + e];
        out.sums[e] = v;
        out.counts[e] = counts[e];
    }
}

// The blocks' parts added in order; one block.
__global__ void __launch_bounds__(1024) moe_route_sum_kernel(const Route a, int blocks) {
    __shared__ float red[64];
    __shared__ int32_t tokens;
    __shared__ float zsum;
    pdl_wait_prior();
    pdl_allow_next();
    float balance = 0.f;
    for (int e = threadIdx.x; e <= a.experts; e += 1024) {
        float sum = 0.f, err = 0.f;
        int32_t n = 0;
        for (int b = 0; b < blocks; ++b) {
            const Parts p = parts_of(a, b);
            add_exact(sum, err, p.sums[e]);
            n += p.counts[e];
        }
        if (e < a.experts) {
            a.counts[e] = n;
            balance += (float)n * (sum + err);
        } else {
            tokens = n;
            zsum = sum + err;
        }
    }
    float v[1] = {balance};
    row_sum<1024, 1>(v, red);
    if (threadIdx.x == 0) {
        const float n = (float)max(tokens, 1);
        *a.live = tokens;
        if (a.losses != nullptr) {
            a.losses[0] = v[0] / n / n * ((float)a.experts / (float)a.topk);
            a.losses[1] = zsum / n;
        }
    }
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(const RouteBackward a) {
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *chosen = smem + warp * R * 32;  // the weights' path, by expert
    pdl_wait_prior();
    pdl_allow_next();
    const float n = (float)max(*a.live, 1);
    const float db = a.dlosses == nullptr ? 0.f : a.dlosses[0];
    const float dz = a.dlosses == nullptr ? 0.f : 2.f * a.dlosses[1] / n;
    float c[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        c[r] = r * 32 + lane < a.experts
                   ? db * ((float)a.experts / (float)a.topk) * ((float)a.counts[r * 32 + lane] / n) / n
                   : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.tokens;
         t += (int64_t)gridDim.x * kWarps) {
        const T *row = reinterpret_cast<const T *>(a.logits) + t * a.ldl;
        T *out = reinterpret_cast<T *>(a.dlogits) + t * a.experts;
        int id = -1;
        float dw = 0.f;
        if (lane < a.topk) {
            id = a.ids[t * a.topk + lane];
            if (id >= a.experts) id = -1;
            if (id >= 0 && a.dweights != nullptr) dw = a.dweights[t * a.topk + lane];
        }
        const bool on = __shfl_sync(kAll, lane < a.topk ? a.ids[t * a.topk + lane] : -1, 0) >= 0;
        float l[R];
        if (on) {
            float peak = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] = logit_at(row, r * 32 + lane, a.experts);
#pragma unroll
            for (int r = 0; r < R; ++r) peak = fmaxf(peak, l[r]);
            peak = warp_max(peak);
            const float mine = id >= 0 ? expf(elem_to_float(row[id]) - peak) : 0.f;
            float total = 0.f, pc = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                l[r] = r * 32 + lane < a.experts ? expf(l[r] - peak) : 0.f;
                total += l[r];
                pc += l[r] * c[r];
            }
            total = warp_sum(total);
            const float inv = __fdiv_rn(1.f, total);
            float common = dz * (peak + logf(total)) - warp_sum(pc) * inv;
            float w, d;
            if (a.renormalize) {
                const float sum = warp_sum(mine);
                w = id >= 0 ? __fdiv_rn(mine, sum) : 0.f;
                d = w * (dw - warp_sum(w * dw));
            } else {
                w = mine * inv;
                common -= warp_sum(w * dw);
                d = w * dw;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) chosen[r * 32 + lane] = 0.f;
            __syncwarp();
            if (id >= 0) atomicAdd(&chosen[id], d);
            __syncwarp();
#pragma unroll
            for (int r = 0; r < R; ++r)
                l[r] = l[r] * inv * (c[r] + common) + chosen[r * 32 + lane];
            __syncwarp();
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r * 32 + lane < a.experts) float_to_elem(out + r * 32 + lane, l[r]);
    }
}

template <typename T, int R>
cudaError_t route(const Route &a, int blocks, cudaStream_t s) {
    const size_t smem = (size_t)(kWarps + 1) * (a.experts + 1) * sizeof(float);
    cudaError_t e = launch_pdl(moe_route_kernel<T, R>, blocks, kThreads, smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_route_sum_kernel, 1, 1024, 0, s, a, blocks);
}

template <typename T, int R>
cudaError_t route_backward(const RouteBackward &a, int blocks, cudaStream_t s) {
    const size_t smem = (size_t)kWarps * R * 32 * sizeof(float);
    return launch_pdl(moe_route_backward_kernel<T, R>, blocks, kThreads, smem, s, a);
}

int route_blocks(int64_t tokens, int per_sm) {
    const int64_t blocks = (tokens + kWarps - 1) / kWarps, most = (int64_t)per_sm * num_sms();
    return (int)(blocks < most ? blocks : most);
}

// f<R>(): the smallest R with 32 R >= experts
#define FP8_BY_EXPERTS(experts, f)                \
    ((experts) <= 32    ? f<T, 1>(a, blocks, s)   \
     : (experts) <= 64  ? f<T, 2>(a, blocks, s)   \
     : (experts) <= 128 ? f<T, 4>(a, blocks, s)   \
     : (experts) <= 256 ? f<T, 8>(a, blocks, s)   \
     : (experts) <= 512 ? f<T, 16>(a, blocks, s)  \
                        : f<T, 32>(a, blocks, s))

template <typename T>
cudaError_t route_by_type(const Route &a, int blocks, cudaStream_t s) {
    return FP8_BY_EXPERTS(a.experts, route);
}

template <typename T>
cudaError_t backward_by_type(const RouteBackward &a, int blocks, cudaStream_t s) {
    return FP8_BY_EXPERTS(a.experts, route_backward);
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t tokens, int64_t experts) {
    const int64_t blocks = (tokens + kWarps - 1) / kWarps;
    return (blocks < kRouteMaxBlocks ? (blocks > 0 ? blocks : 1) : kRouteMaxBlocks) * 2 *
           (experts + 1) * (int64_t)sizeof(float);
}

cudaError_t launch_moe_route(const Route &a, cudaStream_t s) {
    // a block at least: the counts of no tokens are zeros
    int blocks = route_blocks(a.tokens, 2);
    blocks = blocks < 1 ? 1 : blocks < kRouteMaxBlocks ? blocks : kRouteMaxBlocks;
    return a.f32 ? route_by_type<float>(a, blocks, s) : route_by_type<uint16_t>(a, blocks, s);
}

cudaError_t launch_moe_route_backward(const RouteBackward &a, cudaStream_t s) {
    if (a.tokens == 0) return cudaSuccess;
    const int blocks = route_blocks(a.tokens, 8);
    return a.f32 ? backward_by_type<float>(a, blocks, s)
                 : backward_by_type<uint16_t>(a, blocks, s);
}

}  // namespace fp8
