// Orthogonalisation of a weight's update by Newton-Schulz products, for one
// matrix or a batch of equal ones: with s the shorter side (here the rows; a
// tall matrix works on its columns in the same way),
//
//   X = G / (|G|_F + eps),  then `steps` times
//   A = X Xᵀ,  B = b A + c A A,  X <- a X + B X,
//
// which drives the singular values of X towards 1.  A and A·A are symmetric,
// so only the tiles on and below the diagonal are computed and each is stored
// twice: s²l + s³ + 2 s²l multiply-adds' operations a step for an s x l matrix.
//
// Every product is a tcgen05 GEMM on fp16 operands with fp32 accumulation.
// fp16 holds 11 significant bits where bf16 holds 8; its short exponent is
// enough because the values are bounded: X and A are stored times 2^12, which
// leaves room for singular values up to 4 and keeps entries down to 2^-26
// normal, and B times a power of two of the step's own, the largest up to 2^10
// that leaves room for what (a, b, c) make of such singular values (2^7 with the
// usual coefficients).  Rounding X itself to fp16 would cost more than the
// products' roundings do: its error lies in all directions alike, and the first
// steps multiply small singular values by `a` each.  So X is held as the sum of
// two fp16 numbers (22 bits) in the first three steps and until the last two, and
// a X is added from that sum in the epilogue; only the products see the rounded X.  In the other steps the singular values are of
// order 1 and a X goes through the product instead, as (a I + B) X, which rounds
// less and reads nothing in the epilogue.
//
// Accuracy, besides the bf16 output's own rounding (1.66e-3 in the 2-norm):
// 0.5e-3 to 2e-3 for Gaussian matrices and noise of 1 % and more on a low rank,
// 2.9e-3 for noise of 1e-3 and less and after eight steps.  Roundings grow by the
// slopes of the steps' polynomials: coefficients whose intervals end at the largest
// singular value, where their slope is largest, leave a nearly rank-one matrix
// (noise 1e-4) 2.5e-2 off; divided by a safety factor of 1.01 (a / f, b / f^3,
// c / f^5) 2.9e-3.  The PRECISE form holds both operands of every product as sums
// of two fp16 numbers, three products for one: as near the formula as fp32
// products are (0 to 6e-4 from its rounded value, fp32 0 to 8e-4; in that worst
// case 2.9e-3 and 1.3e-3).  bf16 operands: 1e-2 and more.
//
// Neither operand is ever transposed in memory: the tensor core reads X with
// either of its dims as the contraction, straight from its row-major tiles.
//
// Large matrices are bound by the tensor cores at the clock that the power
// limit leaves: 4096 x 4096 in 0.88 to 0.94 ms in short runs (1460 to 1570 TFLOP/s
// of the operations above; the launch of the products 0.83 ms), 0.96 to 1.03 ms
// kept up (1.6 GHz); 4096 x 14336 in 2.64 to 2.83 ms, eight of 4096 x 4096 in 7.4
// ms.  Small ones are bound by the 15 dependent products, about
// 6 us each from tile to tile: 256 x 256 89 to 96 us, 1024 x 1024 150 us.  Eight of
// 1531 x 1000: 267 to 280 us, between the two.  PRECISE: 2.8 ms, 8.1 ms, 138 us,
// 288 us and 553 us.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rowops.cuh"
#include "tmap.h"

namespace fp8 {

extern std::atomic<uint64_t> g_wait_limit_ns;

namespace {

constexpr float kXScale = 4096.f, kAScale = 4096.f;
// Of the low parts: where they are only added, in the epilogue, they keep 11 bits
// however small; as operands they have the high parts' scale.
__host__ __device__ constexpr float lo_scale(bool precise) { return precise ? 1.f : 2048.f; }
constexpr int kBScaleMost = 10;  // log2
// The steps whose a X goes through the product: the last two, but none of the
// first three, before which small singular values have not been raised.
__host__ __device__ constexpr bool folded(int step, int steps) {
    return step >= 3 && step >= steps - 2;
}

// ---------------------------------------------------------------- scaling ---

// The input's sum of squares three times: of x, of x 2^-96 and of x 2^90.  The
// first is used from 2^-60 to 2^100 (|G| from 2^-30 to 2^50); above that the
// second, whose terms are below 2^64 each, and below it the third, whose sum is
// below 2^120 and whose terms are 2^-118 or more.  So the one that is used
// neither overflows nor loses terms that count.
struct SquareSums {
    float mid, big, small;
};
constexpr float kSquareBig = 0x1p-96f, kSquareSmall = 0x1p90f;

struct PrepArgs {
    const void *g;
    int64_t ldg, bsg;  // row and batch strides in elements
    int rows, cols, ldx;
    float eps, lo_scale;
    SquareSums *sums;  // [batch][parts]
    int parts;
    int tx;            // threads along a row (a power of two)
    __half *hi, *lo;   // [batch][rows][ldx]
    uint32_t *flags;   // [batch][flags_per], cleared for the products' launch
    int flags_per;
};

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 4;  // rows whose loads a thread has in flight together

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kPrepThreads) ns_square_kernel(const PrepArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V;
    __shared__ float red[3 * kPrepThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    for (int i = blockIdx.x * kPrepThreads + threadIdx.x; i < a.flags_per; i += gridDim.x * kPrepThreads)
        a.flags[(int64_t)blockIdx.y * a.flags_per + i] = 0;
    const T *g = reinterpret_cast<const T *>(a.g) + blockIdx.y * a.bsg;
    const int ty = kPrepThreads / a.tx;
    float s[3] = {0.f, 0.f, 0.f};
    const int64_t step = (int64_t)a.parts * ty;
    for (int64_t r = (int64_t)blockIdx.x * ty + threadIdx.x / a.tx; r < a.rows;
         r += kPrepRows * step)
        for (int c = (threadIdx.x & (a.tx - 1)) * V; c < a.cols; c += a.tx * V) {
            typename RV::Raw raw[kPrepRows];
#pragma unroll
            for (int u = 0; u < kPrepRows; ++u)
                raw[u] = r + u * step < a.rows ? RV::load(g + (r + u * step) * a.ldg + c) : RV::zero();
#pragma unroll
            for (int u = 0; u < kPrepRows; ++u) {
                float f[V];
                RV::unpack(raw[u], f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float b = f[i] * kSquareBig, l = f[i] * kSquareSmall;
                    s[0] = fmaf(f[i], f[i], s[0]);
                    s[1] = fmaf(b, b, s[1]);
                    s[2] = fmaf(l, l, s[2]);
                }
            }
        }
    row_sum<kPrepThreads, 3>(s, red);
    if (threadIdx.x == 0)
        a.sums[(int64_t)blockIdx.y * a.parts + blockIdx.x] = SquareSums{s[0], s[1], s[2]};
}

// X 2^12 = hi + lo / lo_scale; every block adds the partial sums itself, in the
// same order.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kPrepThreads) ns_scale_kernel(const PrepArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V;
    __shared__ float red[3 * kPrepThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    float s[3] = {0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < a.parts; i += kPrepThreads) {
        const SquareSums p = a.sums[(int64_t)blockIdx.y * a.parts + i];
        s[0] += p.mid;
        s[1] += p.big;
        s[2] += p.small;
    }
    row_sum<kPrepThreads, 3>(s, red);
    // |G| 2^k = sqrt(sum), X = (g 2^k) / (|G| 2^k + eps 2^k)
    float pre = 1.f, sum = s[0];
    if (!(s[0] < 0x1p100f)) pre = kSquareBig, sum = s[1];
    else if (s[0] < 0x1p-60f) pre = kSquareSmall, sum = s[2];
    const float den = sqrtf(sum) + a.eps * pre;
    const float mul = kXScale / den;
    const T *g = reinterpret_cast<const T *>(a.g) + blockIdx.y * a.bsg;
    const int64_t at = (int64_t)blockIdx.y * a.rows;
    const int ty = kPrepThreads / a.tx;
    const int64_t step = (int64_t)a.parts * ty;
    for (int64_t r = (int64_t)blockIdx.x * ty + threadIdx.x / a.tx; r < a.rows;
         r += kPrepRows * step)
        for (int c = (threadIdx.x & (a.tx - 1)) * V; c < a.cols; c += a.tx * V) {
            typename RV::Raw raw[kPrepRows];
#pragma unroll
            for (int u = 0; u < kPrepRows; ++u)
                raw[u] = r + u * step < a.rows ? RV::load(g + (r + u * step) * a.ldg + c) : RV::zero();
#pragma unroll
            for (int u = 0; u < kPrepRows; ++u) {
                if (r + u * step >= a.rows) continue;
                float f[V];
                RV::unpack(raw[u], f);
                struct alignas(2 * V) Halves {
                    __half v[V];
                } hi, lo;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = (f[i] * pre) * mul;
                    hi.v[i] = __float2half_rn(x);
                    lo.v[i] = __float2half_rn((x - __half2float(hi.v[i])) * a.lo_scale);
                }
                const int64_t o = (at + r + u * step) * a.ldx + c;
                *reinterpret_cast<Halves *>(a.hi + o) = hi;
                *reinterpret_cast<Halves *>(a.lo + o) = lo;
            }
        }
}

// ---------------------------------------------------------------- products ---
//
// All steps' products run in one launch whose CTAs (pairs of CTAs on large
// matrices) stay resident and walk one list of output tiles: step by step the
// tiles of A, of B and of the new X.  A tile may start before the ones that it
// reads are all done: tiles announce themselves by counters in memory, and the
// thread that loads a tile's operands waits, 128 or 256 columns of the
// contraction at a time, for just the tiles those columns come from.  The list
// is in the order in which the next product consumes its operand (A and B
// column by column of the lower triangle, X along its longer side), so the
// waits are short, no CTA idles while a product's last tiles finish (a launch
// per product left 2 waves where 1.8 were full), and a product costs no launch.
// Every tile only waits for tiles earlier in the list, all CTAs are resident
// (a cooperative launch), and every wait is bounded.
//
// Reuse of a buffer needs no wait of its own: a tile of the next step's A is
// written only after its operands, all of a row panel of the new X, are there,
// which themselves needed every B tile, and so every read of A, of that panel;
// likewise B, and X, which has two buffers.

enum NsPhase { kGram, kPoly, kUpdate };

constexpr int kMaxSteps = 64;

struct NsPlan {
    // geometry (tiles of BT x BT)
    int rows, cols, batch, steps, tall;
    int T, U;                  // tiles along the shorter and the longer side
    int tri, upd;              // tiles of a symmetric product and of X, per matrix
    int splits;                // parts of A's contraction (128-tiles only)
    int per_step, tiles;       // over the batch; over all steps
    // memory
    uint16_t *direct;          // bf16 output without a tensor map (nullable)
    float *parts;              // [batch][tri][splits][BT][BT] of A, with splits
    uint32_t *flags;           // per matrix: of its A, B and X tiles, and 8 of
                               // each A tile's parts
    int flags_per;
    // arithmetic: step i has coefficients (a, b, c) at 3 i
    float coefficients[3 * kMaxSteps];
    float b_scale[kMaxSteps];  // of B as it is stored
    float scale;
    uint64_t wait_limit_ns;
    unsigned int *status;
};

struct NsMaps {
    // operands: boxes of 64 columns x 128 rows where the columns are
    // contracted; where the rows are (xm), 64 rows x 2 groups of 64 columns
    CUtensorMap x[2], xm[2], a, b;
    CUtensorMap xl[2], xml[2], al, bl;         // PRECISE: of their low parts
    CUtensorMap dx[2], dlo[2], da, db, dout;   // outputs: boxes of 32 x 32
    CUtensorMap dal, dbl;
};

constexpr int NS_EPI_WARPS = 8;                // two to each quarter of the lanes
constexpr int NS_THREADS = 64 + 32 * NS_EPI_WARPS + 32;  // loads, MMAs, output, scout
constexpr int NS_BOX = 2048;                   // a 32 x 32 box of 2-byte outputs
constexpr int NS_STAGING = NS_EPI_WARPS * 4 * NS_BOX;  // two that come in, two that go out
constexpr int NS_OPERAND = 128 * 128;          // 128 rows of 64 fp16
constexpr int NS_STAGE = 2 * NS_OPERAND;
constexpr int NS_STAGES = 5;
constexpr size_t NS_SMEM = 1024 + (size_t)NS_STAGES * NS_STAGE + 1024 + NS_STAGING;
static_assert(NS_SMEM <= 227 * 1024, "shared memory");

// Instruction descriptor, kind::f16: D fp32, A and B fp16; bits 15 / 16 set
// for an operand whose M (N) dim is the contiguous one.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((m >> 4) << 24);
}

// Shared-memory descriptor of an operand whose M (N) dim is contiguous, from
// 64 (M) x 64 (K) boxes with 128-byte swizzling: 8192 bytes from one group of
// 64 rows of M to the next (leading offset), 1024 from 8 values of K to the
// next 8 (stride offset).  16 values of K further on is 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t smem_addr) {
    uint64_t d = smem_desc_sw128(smem_addr) & ~((uint64_t)0x3FFFu << 16);
    return d | ((uint64_t)(8192u >> 4) << 16);
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A box at (x, y) of matrix z into shared memory at dst, completing on the
// leader's barrier.
template <int CG>
__device__ __forceinline__ void ns_load(uint32_t dst, const void *tmap, uint32_t bar, int x, int y,
                                        int z) {
    if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
            "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void ns_store(const void *tmap, uint32_t src, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
}

// Orders this thread's accesses by the usual path with its bulk copies'.
__device__ __forceinline__ void fence_proxy_async_all() {
    asm volatile("fence.proxy.async;" ::: "memory");
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Waits until *p >= target; false (and the status word set) when the limit
// runs out or another thread of the block gave up.
__device__ __forceinline__ bool flag_wait_bounded(const uint32_t *p, uint32_t target,
                                                  volatile int *abort, uint64_t limit_ns,
                                                  unsigned int *status) {
    if (load_acquire(p) >= target) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (load_acquire(p) >= target) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                *abort = 1;
                atomicOr(status, kStatusTimeoutBarrier);
                return false;
            }
        }
    }
}

// The words of the scout to the producer (panels found) and back (its tile),
// in shared memory.
__device__ __forceinline__ void store_release_cta(uint32_t *p, uint32_t v) {
    asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t load_acquire_cta(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
    return v;
}

// Waits until a word of shared memory is at least `least`; *seen: what it is.
__device__ __forceinline__ bool word_wait_bounded(const uint32_t *p, uint32_t least, uint32_t *seen,
                                                  volatile int *abort, uint64_t limit_ns,
                                                  unsigned int *status) {
    if ((*seen = load_acquire_cta(p)) >= least) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if ((*seen = load_acquire_cta(p)) >= least) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                *abort = 1;
                atomicOr(status, kStatusTimeoutBarrier);
                return false;
            }
        }
    }
}

// A tile of the list.  r, c: its place in A or B (r >= c), or in X with c
// along the shorter and r along the longer side.
struct NsTile {
    int step, phase, z, r, c;
    int tm, tn;   // row and column tile of the output
    int split;    // which part of A's contraction
};

__device__ __forceinline__ NsTile ns_locate(const NsPlan &p, int i) {
    NsTile t;
    t.step = i / p.per_step;
    int k = i - t.step * p.per_step;
    const int gram = p.tri * p.splits, gram_all = gram * p.batch, poly_all = p.tri * p.batch;
    t.phase = k < gram_all ? kGram : k < gram_all + poly_all ? kPoly : kUpdate;
    t.split = 0;
    if (t.phase == kUpdate) {
        k -= gram_all + poly_all;
        t.z = k / p.upd;
        k -= t.z * p.upd;
        t.r = k / p.T;
        t.c = k - t.r * p.T;
        t.tm = p.tall ? t.r : t.c;
        t.tn = p.tall ? t.c : t.r;
    } else {
        const int per = t.phase == kGram ? gram : p.tri;
        k -= t.phase == kGram ? 0 : gram_all;
        t.z = k / per;
        k -= t.z * per;
        t.split = k / p.tri;
        // column by column: counted from the end, row by row of the mirrored
        // triangle
        const int u = p.tri - 1 - (k - t.split * p.tri);
        int q = (int)((sqrtf(8.f * (float)u + 1.f) - 1.f) * 0.5f);
        while ((q + 1) * (q + 2) / 2 <= u) ++q;
        while (q * (q + 1) / 2 > u) --q;
        t.c = p.T - 1 - q;
        t.r = p.T - 1 - (u - q * (q + 1) / 2);
        t.tm = t.r;
        t.tn = t.c;
    }
    return t;
}

// The counters: of a tile of A or B at row r and column c (in either order),
// and of a tile of X.
__device__ __forceinline__ uint32_t *sym_flag(const NsPlan &p, int z, int phase, int r, int c) {
    const int hi = max(r, c), lo = min(r, c);
    return p.flags + (int64_t)z * p.flags_per + phase * p.tri + hi * (hi + 1) / 2 + lo;
}
__device__ __forceinline__ uint32_t *x_flag(const NsPlan &p, int z, int r, int c) {
    return p.flags + (int64_t)z * p.flags_per + 2 * p.tri + r * p.T + c;
}
// The part of a tile's A that each epilogue warp keeps count of.
__device__ __forceinline__ uint32_t *part_flag(const NsPlan &p, int z, int r, int c, int warp) {
    return p.flags + (int64_t)z * p.flags_per + 2 * p.tri + p.upd +
           NS_EPI_WARPS * (r * (r + 1) / 2 + c) + warp;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 half2_floats(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// A stage of an operand: 128 rows of M (N) x 64 of K from (row, k) on.
template <int CG, bool MN>
__device__ __forceinline__ void ns_load_operand(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                                int row, int k, int z) {
    if constexpr (!MN)
        ns_load<CG>(dst, map, bar, k, row, z);
    else if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
            "bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k), "r"(row / 64), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k), "r"(row / 64), "r"(z), "r"(bar)
            : "memory");
}

// The ring of operand stages as the thread that fills it or drains it sees it.
struct NsRing {
    uint64_t *full, *empty;
    int stage;
    uint32_t phase;
    __device__ __forceinline__ void next() {
        if (++stage == NS_STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Loads blocks kb to end - 1 of a tile's operands.  One loop for each kind of
// operands: deciding inside it cost the loading thread so long (430 ns a block
// instead of 290) that it, not the tensor cores, set the pace.
template <int CG, bool A_MN, bool B_MN>
__device__ __forceinline__ bool ns_fill(NsRing &ring, uint32_t a0, uint32_t b0,
                                        const CUtensorMap *ma, const CUtensorMap *mb, int arow,
                                        int brow, int z, int kb, int end, uint32_t rank,
                                        volatile int *abort_flag, const NsPlan &p) {
#pragma unroll 1
    for (; kb < end; ++kb) {
        if (!mbar_wait_bounded(&ring.empty[ring.stage], ring.phase ^ 1u, abort_flag,
                               p.wait_limit_ns, kStatusTimeoutTma, p.status))
            return false;
        uint64_t *full = &ring.full[ring.stage];
        if (rank == 0) mbar_arrive_expect_tx(full, CG * NS_STAGE);
        const uint32_t bar = CG == 2 ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
        const uint32_t at = ring.stage * NS_OPERAND;
        ns_load_operand<CG, A_MN>(a0 + at, ma, bar, arow, kb * 64, z);
        ns_load_operand<CG, B_MN>(b0 + at, mb, bar, brow, kb * 64, z);
        ring.next();
    }
    return true;
}

// Issues a tile's MMAs: blocks of 64 of K, two to a round, since this single
// thread's path between two waits paces the tensor pipe.
template <int CG, bool A_MN, bool B_MN>
__device__ __forceinline__ bool ns_mma_tile(NsRing &ring, uint32_t a0, uint32_t b0, uint32_t d_tmem,
                                            int nk, volatile int *abort_flag, const NsPlan &p) {
    constexpr uint32_t IDESC = idesc_f16_f32(128 * CG, 128 * CG, A_MN, B_MN);
    constexpr int A_STEP = (A_MN ? 2048 : 32) >> 4, B_STEP = (B_MN ? 2048 : 32) >> 4;
    const uint64_t a_desc0 = A_MN ? smem_desc_mn128(a0) : smem_desc_sw128(a0);
    const uint64_t b_desc0 = B_MN ? smem_desc_mn128(b0) : smem_desc_sw128(b0);
    int kb = 0;
    auto round = [&](auto count) -> bool {
        constexpr int NB = decltype(count)::value;
        NsRing look = ring;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (!mbar_wait_bounded(&look.full[look.stage], look.phase, abort_flag, p.wait_limit_ns,
                                   kStatusTimeoutMma, p.status))
                return false;
            look.next();
        }
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint64_t off = (uint64_t)((ring.stage * NS_OPERAND) >> 4);
            const uint64_t ad = a_desc0 + off, bd = b_desc0 + off;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_f16<CG>(d_tmem, ad + (uint64_t)(k * A_STEP), bd + (uint64_t)(k * B_STEP), IDESC,
                            ((kb + b) | k) != 0);
            if constexpr (CG == 2) mma_commit_pair(&ring.empty[ring.stage], 0x3);
            else mma_commit(&ring.empty[ring.stage]);
            ring.next();
        }
        kb += NB;
        return true;
    };
    while (kb + 2 <= nk)
        if (!round(std::integral_constant<int, 2>{})) return false;
    if (kb < nk) return round(std::integral_constant<int, 1>{});
    return true;
}

// Warp 0 loads, warp 1 issues the MMAs, the others write the output from the
// other of two accumulators.  PRECISE: every operand is the sum of two fp16
// numbers and a product three of theirs (the low parts' own is below what the
// others round away), one after the other into the same accumulator.
template <int CG, bool PRECISE>
__device__ __forceinline__ void ns_body(const NsMaps &maps, const NsPlan &p) {
    constexpr int BT = 128 * CG;
    constexpr uint32_t TMEM_COLS = 2 * BT;
    constexpr uint32_t ARRIVALS = NS_EPI_WARPS * CG;  // that complete a tile
    constexpr int PRODUCTS = PRECISE ? 3 : 1;
    constexpr float LO_SCALE = lo_scale(PRECISE);
    constexpr int PANEL = BT / 64;                    // blocks of 64 that a tile spans
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + NS_STAGES * NS_OPERAND;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NS_STAGES * NS_STAGE);
    uint64_t *full = bars, *empty = bars + NS_STAGES, *tfull = bars + 2 * NS_STAGES;
    uint64_t *tempty = tfull + 2, *drain = tempty + 2, *ebars = drain + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(ebars + NS_EPI_WARPS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    uint32_t *scouted = tmem_holder + 2, *filling = tmem_holder + 3;
    uint8_t *staging = smem + NS_STAGES * NS_STAGE + 1024;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int worker = blockIdx.x / CG, workers = gridDim.x / CG;
    const int S = p.tall ? p.cols : p.rows, L = p.tall ? p.rows : p.cols;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], NS_EPI_WARPS * CG);
        }
        mbar_init(drain, 1);
        for (int w = 0; w < NS_EPI_WARPS; ++w) mbar_init(&ebars[w], 1);
        *abort_flag = 0;
        *scouted = *filling = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&maps.x[0]);
        tma_prefetch_desc(&maps.x[1]);
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_holder, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_holder, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    // Contraction of a phase, in blocks of 64.  Which operands have M (N), not
    // K, contiguous: A = X Xᵀ contracts X's columns: neither (tall: XᵀX, its
    // rows: both); B X contracts the rows of X: the second (tall, X B: neither);
    // A and B are their own transposes.
    auto blocks = [&](int phase) { return ((phase == kGram ? L : S) + 63) / 64; };
    // the panels (of PANEL blocks) that a tile contracts
    auto panels_of = [&](const NsTile &t, int &first, int &end) {
        const int all = (blocks(t.phase) + PANEL - 1) / PANEL;
        if (t.phase == kGram) {
            const int per = (all + p.splits - 1) / p.splits;
            first = min(all, t.split * per);
            end = min(all, first + per);
        } else {
            first = 0;
            end = all;
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        NsRing ring = {full, empty, 0, 0};
        bool ok = true;
        if (lane == 0) {
            uint32_t want = 0, seen = 0;  // panels of the contraction, over all tiles
            const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
            uint32_t n = 0;
            for (int i = worker; i < p.tiles && ok; i += workers, ++n) {
                store_release_cta(filling, n);
                const NsTile t = ns_locate(p, i);
                const int cur = t.step & 1;
                const CUtensorMap *ma, *mb, *la = nullptr, *lb = nullptr;
                if (t.phase == kGram) {
                    ma = mb = p.tall ? &maps.xm[cur] : &maps.x[cur];
                    if constexpr (PRECISE) la = lb = p.tall ? &maps.xml[cur] : &maps.xl[cur];
                } else if (t.phase == kPoly) {
                    ma = mb = &maps.a;
                    if constexpr (PRECISE) la = lb = &maps.al;
                } else {
                    ma = p.tall ? &maps.x[cur] : &maps.b;
                    mb = p.tall ? &maps.b : &maps.xm[cur];
                    if constexpr (PRECISE) {
                        la = p.tall ? &maps.xl[cur] : &maps.bl;
                        lb = p.tall ? &maps.bl : &maps.xml[cur];
                    }
                }
                const int arow = t.tm * BT + (int)rank * 128, brow = t.tn * BT + (int)rank * 128;
                const int nk = blocks(t.phase);
                int first, panels;
                panels_of(t, first, panels);
                auto fill = [&](const CUtensorMap *a, const CUtensorMap *b, int kb, int end) {
                    if (t.phase == kGram && p.tall)
                        return ns_fill<CG, true, true>(ring, a0, b0, a, b, arow, brow, t.z, kb, end,
                                                       rank, abort_flag, p);
                    if (t.phase == kUpdate && !p.tall)
                        return ns_fill<CG, false, true>(ring, a0, b0, a, b, arow, brow, t.z, kb, end,
                                                        rank, abort_flag, p);
                    return ns_fill<CG, false, false>(ring, a0, b0, a, b, arow, brow, t.z, kb, end,
                                                     rank, abort_flag, p);
                };
                for (int kp = first; kp < panels && ok;) {
                    if (seen == want) {
                        ok = word_wait_bounded(scouted, want + 1, &seen, abort_flag,
                                               p.wait_limit_ns, p.status);
                        fence_proxy_async_all();
                        if (!ok) break;
                    }
                    const int next = min(panels, kp + (int)(seen - want));
                    // (PRECISE: the small products first; then all panels are there)
                    ok = fill(PRECISE ? la : ma, mb, kp * PANEL, min(nk, next * PANEL));
                    want += next - kp;
                    kp = next;
                }
                if constexpr (PRECISE) {
                    const int kb = first * PANEL, end = min(nk, panels * PANEL);
                    ok = ok && fill(ma, lb, kb, end) && fill(ma, mb, kb, end);
                }
            }
        }
        if (!ok && rank == 0 && lane == 0) {
            // wait (bounded) for the copies in flight before teardown
            for (int s = 0; s < NS_STAGES; ++s) {
                ring.stage = ring.stage == 0 ? NS_STAGES - 1 : ring.stage - 1;
                if (ring.stage == NS_STAGES - 1) ring.phase ^= 1u;
                volatile int no_abort = 0;
                mbar_wait_bounded(&full[ring.stage], ring.phase, &no_abort, 10000000ull,
                                  kStatusTimeoutTma, p.status);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ------------------------------------------- MMA issuer (leader)
            NsRing ring = {full, empty, 0, 0};
            int it = 0;
            bool ok = true;
            const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
            for (int i = worker; i < p.tiles && ok; i += workers, ++it) {
                const NsTile t = ns_locate(p, i);
                const int what = t.phase;
                const int acc = it & 1;
                const uint32_t acc_phase = (it >> 1) & 1;
                if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, p.wait_limit_ns,
                                       kStatusTimeoutMma, p.status))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BT);
                int first, panels;
                panels_of(t, first, panels);
                const int nk = PRODUCTS * (min(blocks(what), panels * PANEL) - first * PANEL);
                if (what == kGram && p.tall)
                    ok = ns_mma_tile<CG, true, true>(ring, a0, b0, d_tmem, nk, abort_flag, p);
                else if (what == kUpdate && !p.tall)
                    ok = ns_mma_tile<CG, false, true>(ring, a0, b0, d_tmem, nk, abort_flag, p);
                else
                    ok = ns_mma_tile<CG, false, false>(ring, a0, b0, d_tmem, nk, abort_flag, p);
                if (ok) {
                    if constexpr (CG == 2) mma_commit_pair(&tfull[acc], 0x3);
                    else mma_commit(&tfull[acc]);
                }
            }
            if constexpr (CG == 2) mma_commit_pair(drain, 0x1);
            else mma_commit(drain);
            volatile int no_abort = 0;  // a short limit must not cut this wait short
            mbar_wait_bounded(drain, 0, &no_abort, kDefaultWaitLimitNs, kStatusTimeoutMma, p.status);
        }
    } else if (warp == NS_THREADS / 32 - 1) {
        // ---------------------------------------------------------- scout
        // Looks at the counters ahead of the producer, 32 panels of the
        // contraction at a time, and tells it how many are there: the looking
        // takes longer than the producer has between two tiles.  It stays one
        // tile ahead (further, its waits would last as long as a product).
        uint32_t found = 0, n = 0, at;
        bool ok = true;
        for (int i = worker; i < p.tiles && ok; i += workers, ++n) {
            ok = word_wait_bounded(filling, n > 0 ? n - 1 : 0, &at, abort_flag, p.wait_limit_ns,
                                   p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const NsTile t = ns_locate(p, i);
            // what the operands come from: A from the step's X, B from its A,
            // the new X from its B; the first X is there already
            const uint32_t done = (uint32_t)(t.phase == kGram ? t.step : t.step + 1) * ARRIVALS;
            int first, panels;
            panels_of(t, first, panels);
            for (int kp = first; kp < panels && ok;) {
                const int mine = kp + lane;
                int run = 32;
                if (done > 0) {
                    const uint32_t *f0 = nullptr, *f1 = nullptr;
                    if (mine < panels) {
                        if (t.phase == kGram) {
                            f0 = x_flag(p, t.z, mine, t.tm);
                            f1 = x_flag(p, t.z, mine, t.tn);
                        } else if (t.phase == kPoly) {
                            f0 = sym_flag(p, t.z, kGram, t.tm, mine);
                            f1 = sym_flag(p, t.z, kGram, t.tn, mine);
                        } else {
                            f0 = f1 = sym_flag(p, t.z, kPoly, t.c, mine);
                        }
                    }
                    uint64_t t0 = 0;
                    for (uint32_t turn = 0;; ++turn) {
                        bool have = true;
                        if (f0 != nullptr) {
                            const uint32_t v0 = load_acquire(f0), v1 = load_acquire(f1);
                            have = v0 >= done && v1 >= done;
                        }
                        const uint32_t got = __ballot_sync(0xFFFFFFFFu, have);
                        run = ~got == 0 ? 32 : __ffs(~got) - 1;
                        if (run > 0) break;
                        if ((turn & 63u) == 0) {
                            const uint64_t now = global_timer_ns();
                            if (turn == 0) t0 = now;
                            const bool late = now - t0 > p.wait_limit_ns;
                            if (__any_sync(0xFFFFFFFFu, late || *abort_flag != 0)) {
                                if (lane == 0 && *abort_flag == 0) {
                                    *abort_flag = 1;
                                    atomicOr(p.status, kStatusTimeoutBarrier);
                                }
                                ok = false;
                                break;
                            }
                        }
                    }
                }
                run = min(run, panels - kp);
                kp += run;
                found += run;
                __syncwarp();
                if (lane == 0 && ok) store_release_cta(scouted, found);
            }
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        // Two warps to each quarter of the accumulator's lanes (rows): chunks
        // of 32 columns go to them in turn.
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t *ebox = staging + (warp - 2) * 4 * NS_BOX, *box = ebox + 2 * NS_BOX;
        uint8_t *box2 = box + NS_BOX;
        uint64_t *ebar = &ebars[warp - 2];
        uint32_t ephase = 0;
        bool coming = false;  // (lane 0) a copy into ebox is on its way
        int it = 0;
        for (int i = worker; i < p.tiles; i += workers, ++it) {
            const int acc = it & 1;
            const uint32_t acc_phase = (it >> 1) & 1;
            const NsTile t = ns_locate(p, i);
            const bool update = t.phase == kUpdate;
            const bool fold = !PRECISE && folded(t.step, p.steps), last = t.step == p.steps - 1;
            const int M = update ? p.rows : S, N = update ? p.cols : S;
            const int row0 = t.tm * BT + (int)rank * 128 + quarter * 32, row = row0 + lane;
            const bool mirror = !update && t.tm != t.tn;
            const int width = row0 < M ? min(BT, N - t.tn * BT) : 0;
            const float ca = p.coefficients[3 * t.step], cb = p.coefficients[3 * t.step + 1],
                        cc = p.coefficients[3 * t.step + 2], b_scale = p.b_scale[t.step];
            // output = acc_mul * acc + e_mul * (E + lo / LO_SCALE) + diag on the diagonal
            float acc_mul, e_mul = 0.f, diag = 0.f;
            const CUtensorMap *e = nullptr, *e_lo = nullptr, *out, *out_lo = nullptr;
            const uint32_t *e_flag = nullptr;
            uint32_t e_done = 0;
            if (t.phase == kGram) {
                acc_mul = kAScale / (kXScale * kXScale);
                out = &maps.da;
                if constexpr (PRECISE) out_lo = &maps.dal;
            } else if (t.phase == kPoly) {
                acc_mul = cc * (b_scale / (kAScale * kAScale));
                e_mul = cb * (b_scale / kAScale);
                diag = fold ? ca * b_scale : 0.f;
                e = &maps.da;
                if constexpr (PRECISE) e_lo = &maps.dal, out_lo = &maps.dbl;
                e_flag = sym_flag(p, t.z, kGram, t.tm, t.tn);
                e_done = (uint32_t)(t.step + 1) * ARRIVALS;
                out = &maps.db;
            } else {
                acc_mul = last ? p.scale / (b_scale * kXScale) : 1.f / b_scale;
                if (!fold) {
                    e = &maps.dx[t.step & 1];
                    e_lo = &maps.dlo[t.step & 1];
                    e_mul = last ? ca * (p.scale / kXScale) : ca;
                    e_flag = x_flag(p, t.z, t.r, t.c);
                    e_done = (uint32_t)t.step * ARRIVALS;
                }
                out = last ? &maps.dout : &maps.dx[(t.step + 1) & 1];
                if (!last && (PRECISE || !folded(t.step + 1, p.steps))) out_lo = &maps.dlo[(t.step + 1) & 1];
            }
            // The added matrix's boxes of a chunk come in one chunk ahead of
            // the accumulator, the first before the tile's products are done.
            auto fetch = [&](int c) {
                if (lane == 0 && e != nullptr && c * 32 < width) {
                    const int col = t.tn * BT + c * 32;
                    mbar_arrive_expect_tx(ebar, e_lo != nullptr ? 2 * NS_BOX : NS_BOX);
                    ns_load<1>(smem_u32(ebox), e, smem_u32(ebar), col, row0, t.z);
                    if (e_lo != nullptr)
                        ns_load<1>(smem_u32(ebox + NS_BOX), e_lo, smem_u32(ebar), col, row0, t.z);
                    coming = true;
                }
            };
            bool ok = true;
            if (lane == 0 && e_done > 0) {
                ok = flag_wait_bounded(e_flag, e_done, abort_flag, p.wait_limit_ns, p.status);
                fence_proxy_async_all();
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            fetch(half);
            ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, p.wait_limit_ns,
                                   kStatusTimeoutEpilogue, p.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            // A tile whose contraction is split: each part leaves its sums in
            // fp32, and the warp that comes last to its 32 rows adds the parts,
            // in their order, and goes on as if it had contracted alone.
            const bool split = CG == 1 && t.phase == kGram && p.splits > 1;
            const float *parts = nullptr;
            if (split) {
                const int64_t tile = (int64_t)t.z * p.tri + t.r * (t.r + 1) / 2 + t.c;
                // a chunk's 32 x 32 sums as [8][32 lanes][4]: whole lines
                float *all = p.parts + tile * p.splits * (BT * BT) + quarter * 32 * BT + lane * 4;
                float *mine = all + (int64_t)t.split * (BT * BT);
#pragma unroll 1
                for (int c = half; c * 32 < width; c += 2) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                           (uint32_t)(acc * BT + c * 32),
                                       r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4 *>(mine + c * 1024 + j * 32) =
                            make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                }
                __threadfence();
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0)
                    before = atomicAdd(part_flag(p, t.z, t.r, t.c, warp - 2), 1u);
                before = __shfl_sync(0xFFFFFFFFu, before, 0);
                __threadfence();
                if (before + 1 == (uint32_t)(t.step + 1) * p.splits) parts = all;
            }
#pragma unroll 1
            for (int c = half; c * 32 < width && (!split || parts != nullptr); c += 2) {
                const int col = t.tn * BT + c * 32;
                float v[32];
                if (split) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                    const float *from = parts + c * 1024;
#pragma unroll 1
                    for (int k = 0; k < p.splits; k += 2) {
                        const bool two = k + 1 < p.splits;
                        float4 f[2][8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float *at = from + (int64_t)k * (BT * BT) + j * 128;
                            f[0][j] = __ldcg(reinterpret_cast<const float4 *>(at));
                            f[1][j] = two ? __ldcg(reinterpret_cast<const float4 *>(at + BT * BT))
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                v[4 * j] += f[u][j].x, v[4 * j + 1] += f[u][j].y;
                                v[4 * j + 2] += f[u][j].z, v[4 * j + 3] += f[u][j].w;
                            }
                    }
                } else {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                           (uint32_t)(acc * BT + c * 32),
                                       r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= acc_mul;
                if (e != nullptr) {
                    ok = mbar_wait_bounded(ebar, ephase, abort_flag, p.wait_limit_ns,
                                           kStatusTimeoutTma, p.status);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    ephase ^= 1u;
                    coming = false;
                    uint4 eh[4], el[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint8_t *at = ebox + lane * 64 + 16 * (q ^ ((lane >> 1) & 3));
                        eh[q] = *reinterpret_cast<const uint4 *>(at);
                        el[q] = e_lo != nullptr ? *reinterpret_cast<const uint4 *>(at + NS_BOX)
                                                : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t hw[4] = {eh[q].x, eh[q].y, eh[q].z, eh[q].w};
                        const uint32_t lw[4] = {el[q].x, el[q].y, el[q].z, el[q].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = 8 * q + 2 * k;
                            const float2 h = half2_floats(hw[k]), l = half2_floats(lw[k]);
                            v[j] = fmaf(e_mul, fmaf(l.x, 1.f / LO_SCALE, h.x), v[j]);
                            v[j + 1] = fmaf(e_mul, fmaf(l.y, 1.f / LO_SCALE, h.y), v[j + 1]);
                        }
                    }
                    __syncwarp();  // every lane has read the boxes
                    fetch(c + 2);
                }
                if (diag != 0.f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += row == col + j ? diag : 0.f;
                }
                uint32_t packed[16];
                if (update && last) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = pack_half2(v[2 * j], v[2 * j + 1]);
                }
                // box <- a lane's 32 values to a row; mirrored: box row j holds
                // column j, lane's value at place `lane`
                auto put = [&](uint8_t *to, const uint32_t (&w)[16]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(to + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) =
                            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                };
                auto put_mirrored = [&](uint8_t *to, const uint32_t (&w)[16]) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        *reinterpret_cast<uint16_t *>(to + j * 64 +
                                                      16 * ((lane >> 3) ^ ((j >> 1) & 3)) +
                                                      2 * (lane & 7)) =
                            (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
                };
                auto low_parts = [&](uint32_t (&w)[16]) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 h = half2_floats(packed[j]);
                        w[j] = pack_half2((v[2 * j] - h.x) * LO_SCALE, (v[2 * j + 1] - h.y) * LO_SCALE);
                    }
                };
                if (lane == 0) bulk_wait_group_read<0>();  // the last copies have read the boxes
                __syncwarp();
                if (PRECISE && out_lo != nullptr) {
                    uint32_t plo[16];
                    low_parts(plo);
                    put(box, plo);
                    if (mirror) put_mirrored(box2, plo);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ns_store(out_lo, smem_u32(box), col, row0, t.z);
                        if (mirror) ns_store(out_lo, smem_u32(box2), row0, col, t.z);
                        bulk_commit_group();
                        bulk_wait_group_read<0>();
                    }
                    __syncwarp();
                }
                put(box, packed);
                if (mirror) put_mirrored(box2, packed);
                if (!PRECISE && out_lo != nullptr) {
                    uint32_t plo[16];
                    low_parts(plo);
                    put(box2, plo);
                }
                if (update && last && p.direct != nullptr) {
                    // an output whose rows no tensor map can describe: row by
                    // row, 32 neighbouring values to a store
                    __syncwarp();
                    for (int k = 0; k < 32; ++k)
                        if (row0 + k < M && col + lane < N)
                            p.direct[((int64_t)t.z * M + row0 + k) * N + col + lane] =
                                *reinterpret_cast<const uint16_t *>(
                                    box + k * 64 + 16 * ((lane >> 3) ^ ((k >> 1) & 3)) +
                                    2 * (lane & 7));
                    __syncwarp();
                    continue;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ns_store(out, smem_u32(box), col, row0, t.z);
                    if (mirror) ns_store(out, smem_u32(box2), row0, col, t.z);
                    if (!PRECISE && out_lo != nullptr)
                        ns_store(out_lo, smem_u32(box2), col, row0, t.z);
                    bulk_commit_group();
                }
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
                else mbar_arrive(&tempty[acc]);
                if (!(update && last) && (!split || parts != nullptr)) {
                    // announce this warp's part once it is in memory
                    bulk_wait_group_all();  // its writes are this thread's from here on
                    __threadfence();
                    atomicAdd(update ? x_flag(p, t.z, t.r, t.c)
                                     : sym_flag(p, t.z, t.phase, t.tm, t.tn), 1u);
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            bulk_wait_group_all();
            volatile int no_abort = 0;
            if (coming)  // after a wait that ran out: let the copy land
                mbar_wait_bounded(ebar, ephase, &no_abort, 10000000ull, kStatusTimeoutTma, p.status);
        }
    }

    __syncwarp();
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <bool PRECISE>
__global__ void __launch_bounds__(NS_THREADS, 1)
    ns_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ NsPlan p) {
    ns_body<1, PRECISE>(maps, p);
}

template <bool PRECISE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NS_THREADS, 1)
    ns_pair_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ NsPlan p) {
    ns_body<2, PRECISE>(maps, p);
}

// ------------------------------------------------------------------- host ---

// A batch of row-major 2-byte matrices [rows, cols] in memory, `ld` elements
// from row to row and rows * ld from matrix to matrix.
bool ns_tmap(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols,
             int64_t ld, int box_cols, int box_rows, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promo) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(rows * ld * 2)};
    cuuint32_t boxes[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, boxes,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promo,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The matrices as [batch][groups of 64 columns][rows][64]: one copy brings 64
// rows of two groups, an operand stage whose contraction runs over the rows.
// The columns past the end of a last group that is not full are the rows'
// padding: unwritten memory that only reaches output rows or columns past the
// end, which are not stored.
bool ns_operand_mn(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols,
                   int64_t ld) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)((cols + 63) / 64), (cuuint64_t)batch};
    cuuint64_t strides[3] = {(cuuint64_t)(ld * 2), 128, (cuuint64_t)(rows * ld * 2)};
    cuuint32_t boxes[4] = {64, 64, 2, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), dims, strides, boxes,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ns_operand(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols,
                int64_t ld) {
    return ns_tmap(m, base, batch, rows, cols, ld, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bool ns_output(CUtensorMap *m, const void *base, int64_t batch, int64_t rows, int64_t cols,
               int64_t ld) {
    return ns_tmap(m, base, batch, rows, cols, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// CTAs (CG = 1) or pairs that are resident at once, asked once per device.
template <int CG, bool PRECISE>
cudaError_t ns_resident(int *workers) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < 64;
    int n = cached ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if constexpr (CG == 2) {
            e = cudaFuncSetAttribute(ns_pair_kernel<PRECISE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)NS_SMEM);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = 2 * (num_sms() / 2);
            cfg.blockDim = NS_THREADS;
            cfg.dynamicSmemBytes = NS_SMEM;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, ns_pair_kernel<PRECISE>, &cfg);
        } else {
            e = cudaFuncSetAttribute(ns_kernel<PRECISE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)NS_SMEM);
            if (e != cudaSuccess) return e;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, ns_kernel<PRECISE>, NS_THREADS, NS_SMEM);
            n *= num_sms();
        }
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (cached) known[dev].store(n, std::memory_order_relaxed);
    }
    *workers = n;
    return cudaSuccess;
}

// Cooperative: the CTAs wait for one another's tiles.
cudaError_t ns_launch(void (*kernel)(NsMaps, NsPlan), int grid, cudaStream_t s, const NsMaps &maps,
                      const NsPlan &p) {
    if (tl_fail_launches > 0) {
        --tl_fail_launches;
        return cudaErrorLaunchFailure;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = NS_THREADS;
    cfg.dynamicSmemBytes = NS_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

// Rows of 128-byte lines: a copy's 128-byte row then is one line, not two.
int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }

// The power of two that B = b A + c A A (+ a I) is stored times.  No entry of a
// symmetric matrix is larger than its largest |eigenvalue|, here |a + b t + c t^2|
// for t = s^2 of a singular value s below 4.
float poly_scale(float a, float b, float c) {
    auto value = [&](double t) { return std::fabs((double)a + (double)b * t + (double)c * t * t); };
    double most = std::max(value(0.), value(16.));
    const double turn = c != 0.f ? -(double)b / (2. * (double)c) : 0.;
    if (turn > 0. && turn < 16.) most = std::max(most, value(turn));
    // (65504 is fp16's largest; the rest is for A's rounding)
    const double room = 60000. / most;
    if (!(room < std::exp2(kBScaleMost))) return std::exp2f(kBScaleMost);  // also NaN, and 0 / 0
    return std::exp2f((float)std::max(-100, std::ilogb(room)));
}

// Blocks that share a matrix in the scaling, at most: a large batch fills the
// GPU with few to a matrix, and a block takes a row or more.
int64_t prep_parts(int64_t batch, int64_t rows) {
    return std::min<int64_t>(rows, std::max<int64_t>(16, 2048 / batch));
}

// A's contraction is split where its 128-tiles would leave CTAs idle: up to 16
// tiles to a side, 8 parts of at least 8 blocks of 64, from a contraction of
// 2048 on (us without / with: 128 x 8192 240 / 131, 512 x 4096 196 / 158, 512 x
// 2048 150 / 143; 256 x 1024, not split, 114 / 118; 16 parts of 128 x 8192: 135).
constexpr int64_t kSplitMaxSide = 2048, kSplitMinLength = 2048, kSplitMinBlocks = 8,
                  kSplitMost = 8;

struct NsLayout {
    int64_t ldx, lds, x[2], lo[2], a, b, alo, blo, sums, flags, parts, parts_bytes, bytes;
};

int64_t ns_flags_per(int64_t T, int64_t U) {
    return T * (T + 1) + U * T + NS_EPI_WARPS * T * (T + 1) / 2;
}

NsLayout ns_layout(int64_t batch, int64_t rows, int64_t cols, bool precise) {
    NsLayout w;
    const int64_t s = std::min(rows, cols), l = std::max(rows, cols);
    w.ldx = pad64(cols);
    w.lds = pad64(s);
    const int64_t x = pad256(batch * rows * w.ldx * 2), q = pad256(batch * s * w.lds * 2);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += bytes;
        return here;
    };
    w.x[0] = take(x);
    w.x[1] = take(x);
    w.lo[0] = take(x);
    w.lo[1] = take(x);
    w.a = take(q);
    w.b = take(q);
    w.alo = take(precise ? q : 0);
    w.blo = take(precise ? q : 0);
    w.sums = take(pad256(batch * prep_parts(batch, rows) * (int64_t)sizeof(SquareSums)));
    w.flags = take(pad256(batch * ns_flags_per((s + 127) / 128, (l + 127) / 128) * 4));
    // parts of A where its tiles are few and its contraction is long
    w.parts_bytes = s <= kSplitMaxSide && l >= kSplitMinLength ? x : 0;
    w.parts = take(w.parts_bytes);
    w.bytes = at;
    return w;
}

template <typename T, bool VECTOR>
cudaError_t ns_prepare(const PrepArgs &a, int64_t batch, cudaStream_t s) {
    // batch is the grid's second dim: at most 65535 matrices a launch
    for (int64_t z = 0; z < batch; z += 65535) {
        PrepArgs p = a;
        const int n = (int)std::min<int64_t>(65535, batch - z);
        p.g = reinterpret_cast<const T *>(a.g) + z * a.bsg;
        p.sums += z * a.parts;
        p.hi += z * (int64_t)a.rows * a.ldx;
        p.lo += z * (int64_t)a.rows * a.ldx;
        p.flags += z * a.flags_per;
        cudaError_t e = launch_pdl(ns_square_kernel<T, VECTOR>, dim3(a.parts, n), kPrepThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        e = launch_pdl(ns_scale_kernel<T, VECTOR>, dim3(a.parts, n), kPrepThreads, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int64_t orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, bool precise) {
    return ns_layout(batch, rows, cols, precise).bytes;
}

cudaError_t launch_orthogonalize(const Orthogonalize &o, cudaStream_t s, const char **why) {
    if (o.batch == 0 || o.rows == 0 || o.cols == 0) return cudaSuccess;
    const int64_t S = std::min(o.rows, o.cols), L = std::max(o.rows, o.cols);
    const NsLayout w = ns_layout(o.batch, o.rows, o.cols, o.precise);
    uint8_t *base = reinterpret_cast<uint8_t *>(o.workspace);
    auto half = [&](int64_t off) { return reinterpret_cast<__half *>(base + off); };

    // Tiles of 256 by CTA pairs or of 128 by single CTAs, whichever is done
    // sooner: a step's tiles over the workers, but no fewer than one tile of
    // each product after another, times the blocks of 64 of the contraction
    // and the time of one (375 ns a pair's, 297 ns a CTA's: those are bound by
    // their loads).
    int pairs = 0, singles = 0;
    cudaError_t e = o.precise ? ns_resident<2, true>(&pairs) : ns_resident<2, false>(&pairs);
    if (e != cudaSuccess) return e;
    e = o.precise ? ns_resident<1, true>(&singles) : ns_resident<1, false>(&singles);
    if (e != cudaSuccess) return e;
    // Parts of A's contraction for the single CTAs: as many as give idle ones
    // work, leave each enough to do and fit the memory for their sums.
    int64_t splits = 1;
    {
        const int64_t T = (S + 127) / 128, tiles = o.batch * (T * (T + 1) / 2);
        splits = std::min<int64_t>(singles / tiles, (L + 63) / 64 / kSplitMinBlocks);
        splits = std::min<int64_t>(splits, kSplitMost);
        splits = std::min<int64_t>(splits, w.parts_bytes / (tiles * 128 * 128 * 4));
        if (splits < 2) splits = 1;
        const int64_t panels = (L + 127) / 128, per = (panels + splits - 1) / splits;
        splits = (panels + per - 1) / per;  // none without a panel
    }
    auto cost = [&](int bt, int workers, double block, int64_t parts) {
        const int64_t T = (S + bt - 1) / bt, U = (L + bt - 1) / bt;
        const double tri = (double)(o.batch * T * (T + 1) / 2) / workers,
                     upd = (double)(o.batch * T * U) / workers;
        return block * (std::max(tri, 1. / parts) * L + std::max(tri, 1.) * S + std::max(upd, 1.) * S);
    };
    const bool pair = cost(256, pairs, 375, 1) <= cost(128, singles, 297, splits);
    const int bt = pair ? 256 : 128;

    NsPlan p = {};
    p.rows = (int)o.rows, p.cols = (int)o.cols, p.batch = (int)o.batch, p.steps = o.steps;
    p.tall = o.rows > o.cols;
    p.T = (int)((S + bt - 1) / bt);
    p.U = (int)((L + bt - 1) / bt);
    p.tri = p.T * (p.T + 1) / 2;
    p.upd = p.T * p.U;
    p.splits = pair ? 1 : (int)splits;
    p.parts = reinterpret_cast<float *>(base + w.parts);
    const int64_t per_step = o.batch * ((int64_t)p.tri * (p.splits + 1) + p.upd);
    if (per_step * o.steps > 0x7FFFFFFF) {
        *why = "too many tiles";
        return cudaErrorInvalidValue;
    }
    p.per_step = (int)per_step;
    p.tiles = (int)(per_step * o.steps);
    p.flags = reinterpret_cast<uint32_t *>(base + w.flags);
    p.flags_per = (int)ns_flags_per(p.T, p.U);
    for (int i = 0; i < 3 * o.steps; ++i) p.coefficients[i] = o.coefficients[i];
    for (int i = 0; i < o.steps; ++i) {
        const float *abc = o.coefficients + 3 * i;
        p.b_scale[i] = poly_scale(!o.precise && folded(i, o.steps) ? abc[0] : 0.f, abc[1], abc[2]);
    }
    p.scale = o.scale;
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.status = device_status_word();

    NsMaps maps = {};
    const bool out_map = o.cols % 8 == 0 && aligned_to(o.out, 16);
    if (!out_map) p.direct = o.out;
    bool ok = true;
    for (int i = 0; i < 2; ++i)
        ok = ok && ns_operand(&maps.x[i], half(w.x[i]), o.batch, o.rows, o.cols, w.ldx) &&
             ns_operand_mn(&maps.xm[i], half(w.x[i]), o.batch, o.rows, o.cols, w.ldx) &&
             ns_output(&maps.dx[i], half(w.x[i]), o.batch, o.rows, o.cols, w.ldx) &&
             ns_output(&maps.dlo[i], half(w.lo[i]), o.batch, o.rows, o.cols, w.ldx);
    if (o.precise) {
        for (int i = 0; i < 2; ++i)
            ok = ok && ns_operand(&maps.xl[i], half(w.lo[i]), o.batch, o.rows, o.cols, w.ldx) &&
                 ns_operand_mn(&maps.xml[i], half(w.lo[i]), o.batch, o.rows, o.cols, w.ldx);
        ok = ok && ns_operand(&maps.al, half(w.alo), o.batch, S, S, w.lds) &&
             ns_operand(&maps.bl, half(w.blo), o.batch, S, S, w.lds) &&
             ns_output(&maps.dal, half(w.alo), o.batch, S, S, w.lds) &&
             ns_output(&maps.dbl, half(w.blo), o.batch, S, S, w.lds);
    }
    ok = ok && ns_operand(&maps.a, half(w.a), o.batch, S, S, w.lds) &&
         ns_operand(&maps.b, half(w.b), o.batch, S, S, w.lds) &&
         ns_output(&maps.da, half(w.a), o.batch, S, S, w.lds) &&
         ns_output(&maps.db, half(w.b), o.batch, S, S, w.lds) &&
         (out_map ? ns_output(&maps.dout, o.out, o.batch, o.rows, o.cols, o.cols)
                  : ns_output(&maps.dout, half(w.x[0]), o.batch, o.rows, o.cols, w.ldx));
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }

    PrepArgs a = {};
    a.g = o.g, a.ldg = o.ldg, a.bsg = o.bsg;
    a.rows = (int)o.rows, a.cols = (int)o.cols, a.ldx = (int)w.ldx;
    a.eps = o.eps;
    a.lo_scale = lo_scale(o.precise);
    a.sums = reinterpret_cast<SquareSums *>(base + w.sums);
    a.hi = half(w.x[0]), a.lo = half(w.lo[0]);
    a.flags = p.flags;
    a.flags_per = p.flags_per;
    const int es = o.g_f32 ? 4 : 2;
    const bool vec = aligned_to(o.g, 16) && o.ldg * es % 16 == 0 && o.bsg * es % 16 == 0 &&
                     o.cols * es % 16 == 0;
    const int64_t groups = vec ? o.cols * es / 16 : o.cols;
    a.tx = 8;
    while (a.tx < kPrepThreads && a.tx < groups) a.tx *= 2;
    const int64_t row_blocks = (o.rows + kPrepThreads / a.tx - 1) / (kPrepThreads / a.tx);
    // eight blocks to an SM over the batch; more would add up more partial sums
    const int64_t share = 8 * (int64_t)num_sms() / o.batch;
    a.parts = (int)std::min<int64_t>(std::min<int64_t>(row_blocks, prep_parts(o.batch, o.rows)),
                                     share > 16 ? share : 16);
    e = o.g_f32 ? (vec ? ns_prepare<float, true>(a, o.batch, s) : ns_prepare<float, false>(a, o.batch, s))
                : (vec ? ns_prepare<uint16_t, true>(a, o.batch, s)
                       : ns_prepare<uint16_t, false>(a, o.batch, s));
    if (e != cudaSuccess) return e;
    const int workers = std::min(pair ? pairs : singles, p.per_step);
    if (pair)
        return ns_launch(o.precise ? ns_pair_kernel<true> : ns_pair_kernel<false>, 2 * workers, s,
                         maps, p);
    return ns_launch(o.precise ? ns_kernel<true> : ns_kernel<false>, workers, s, maps, p);
}

}  // namespace fp8
