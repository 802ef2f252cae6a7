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
// enough because the values are bounded: X, A and B are stored times 2^12,
// 2^12 and 2^10, which leaves room for singular values up to 4 and keeps
// entries down to 2^-26 (2^-24) normal.  Rounding X itself to fp16 would cost
// more than the products' roundings do: its error lies in all directions
// alike, and the first steps multiply small singular values by `a` each.  So X
// is held as the sum of two fp16 numbers (22 bits) until the last two steps,
// and a X is added from that sum in the epilogue; only the products see the
// rounded X.  In the last two steps the singular values are all of order 1
// and a X goes through the product instead, as (a I + B) X, which rounds less
// and reads nothing in the epilogue.  Measured in 64 bits against the formula,
// the result is 0.4e-3 to 1.3e-3 off (2-norm, matrices of 128 and more), below
// the 1.7e-3 of the bf16 output's own rounding; bf16 operands: 1e-2 and more.
//
// Neither operand is ever transposed in memory: the tensor core reads X with
// either of its dims as the contraction, straight from its row-major tiles.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "rowops.cuh"
#include "tmap.h"

namespace fp8 {

extern std::atomic<uint64_t> g_wait_limit_ns;

namespace {

constexpr float kXScale = 4096.f, kAScale = 4096.f, kBScale = 1024.f, kLoScale = 2048.f;
constexpr int kFoldedSteps = 2;

// ---------------------------------------------------------------- scaling ---

// The input's sum of squares by parts: of x, of x 2^-64 and of x 2^64, so
// that one of them neither overflows nor loses its small terms.
struct SquareSums {
    float mid, big, small;
};

struct PrepArgs {
    const void *g;
    int64_t ldg, bsg;  // row and batch strides in elements
    int rows, cols, ldx;
    float eps;
    SquareSums *sums;  // [batch][parts]
    int parts;
    int tx;            // threads along a row (a power of two)
    __half *hi, *lo;   // [batch][rows][ldx]
};

constexpr int kPrepThreads = 256;

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kPrepThreads) ns_square_kernel(const PrepArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V;
    __shared__ float red[3 * kPrepThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    const T *g = reinterpret_cast<const T *>(a.g) + blockIdx.y * a.bsg;
    const int ty = kPrepThreads / a.tx;
    float s[3] = {0.f, 0.f, 0.f};
    for (int64_t r = (int64_t)blockIdx.x * ty + threadIdx.x / a.tx; r < a.rows;
         r += (int64_t)a.parts * ty)
        for (int c = (threadIdx.x & (a.tx - 1)) * V; c < a.cols; c += a.tx * V) {
            float f[V];
            RV::unpack(RV::load(g + r * a.ldg + c), f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float b = f[i] * 0x1p-64f, l = f[i] * 0x1p64f;
                s[0] = fmaf(f[i], f[i], s[0]);
                s[1] = fmaf(b, b, s[1]);
                s[2] = fmaf(l, l, s[2]);
            }
        }
    row_sum<kPrepThreads, 3>(s, red);
    if (threadIdx.x == 0)
        a.sums[(int64_t)blockIdx.y * a.parts + blockIdx.x] = SquareSums{s[0], s[1], s[2]};
}

// X 2^12 = hi + lo 2^-11; every block adds the partial sums itself, in the
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
    if (!(s[0] < 0x1p100f)) pre = 0x1p-64f, sum = s[1];
    else if (s[0] < 0x1p-60f) pre = 0x1p64f, sum = s[2];
    const float den = sqrtf(sum) + a.eps * pre;
    const float mul = kXScale / den;
    const T *g = reinterpret_cast<const T *>(a.g) + blockIdx.y * a.bsg;
    const int64_t at = (int64_t)blockIdx.y * a.rows;
    const int ty = kPrepThreads / a.tx;
    for (int64_t r = (int64_t)blockIdx.x * ty + threadIdx.x / a.tx; r < a.rows;
         r += (int64_t)gridDim.x * ty)
        for (int c = (threadIdx.x & (a.tx - 1)) * V; c < a.cols; c += a.tx * V) {
            float f[V];
            RV::unpack(RV::load(g + r * a.ldg + c), f);
            struct alignas(2 * V) Halves {
                __half v[V];
            } hi, lo;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = (f[i] * pre) * mul;
                hi.v[i] = __float2half_rn(x);
                lo.v[i] = __float2half_rn((x - __half2float(hi.v[i])) * kLoScale);
            }
            const int64_t o = (at + r) * a.ldx + c;
            *reinterpret_cast<Halves *>(a.hi + o) = hi;
            *reinterpret_cast<Halves *>(a.lo + o) = lo;
        }
}

// ---------------------------------------------------------------- products ---

enum NsMode { kGram, kPoly, kUpdate };

struct NsArgs {
    int M, N, K;
    int m_tiles, n_tiles, tiles_per, tiles;  // per matrix, over the batch
    float acc_mul;                           // output = acc_mul * acc + ...
    float e_mul;                             //   e_mul * (E + lo 2^-11)
    float diag;                              //   + diag on the diagonal
    const __half *e, *e_lo;                  // [batch][M][lde]; e_lo nullable
    int64_t lde, bse;
    int last;                                // the output is bf16
    uint16_t *direct;                        // bf16 output without a tensor map (nullable)
    int write_lo;
    uint64_t wait_limit_ns;
    unsigned int *status;
};

constexpr int NS_EPI_WARPS = 8;                // two to each quarter of the lanes
constexpr int NS_THREADS = 64 + 32 * NS_EPI_WARPS;
constexpr int NS_BOX = 2048;                   // a 32 x 32 box of 2-byte outputs
constexpr int NS_STAGING = NS_EPI_WARPS * 2 * NS_BOX;  // an output and a second one
constexpr int NS_OPERAND = 128 * 128;          // 128 rows of 64 fp16
constexpr int NS_STAGE = 2 * NS_OPERAND;
constexpr int NS_STAGES = 6;
constexpr size_t NS_SMEM = 1024 + (size_t)NS_STAGES * NS_STAGE + 1024 + NS_STAGING;
static_assert(NS_SMEM <= 227 * 1024, "shared memory");

// Instruction descriptor, kind::f16: D fp32, A and B fp16; bits 15 / 16 set
// for an operand whose M (N) dim is the contiguous one.
constexpr uint32_t idesc_f16_f32(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
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

template <int CG>
__device__ __forceinline__ void ns_load(void *dst, const void *tmap, uint64_t *bar,
                                        uint32_t leader_bar, int x, int y, int z) {
    if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
            "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(leader_bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
            : "memory");
}

__device__ __forceinline__ void ns_store(const void *tmap, uint32_t src, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
}

// Tile index -> matrix, row tile, column tile.  Symmetric products walk the
// tiles with tn <= tm, row by row.
template <bool SYM>
__device__ __forceinline__ void ns_locate(const NsArgs &p, int tile, int &z, int &tm, int &tn) {
    z = tile / p.tiles_per;
    const int t = tile - z * p.tiles_per;
    if constexpr (SYM) {
        tm = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
        while (tm * (tm + 1) / 2 > t) --tm;
        tn = t - tm * (tm + 1) / 2;
    } else {
        grouped_tile(t, p.m_tiles, p.n_tiles, 8 / 2, tm, tn);
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 half2_floats(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// D = A·Bᵀ tiles of 128*CG x BN by one CTA (CG = 1) or a pair on two SMs
// (CG = 2): warp 0 loads, warp 1 issues the MMAs, the others write the output
// from the other of two accumulators.  A_MN / B_MN: the operand's M (N) dim,
// not K, is contiguous in memory.
template <int CG, int BN, bool A_MN, bool B_MN, int MODE>
__device__ __forceinline__ void ns_gemm_body(const CUtensorMap &tma_a, const CUtensorMap &tma_b,
                                             const CUtensorMap &tma_d, const CUtensorMap &tma_lo,
                                             const NsArgs &p) {
    constexpr bool SYM = MODE != kUpdate;
    constexpr int BM = 128 * CG, BNH = BN / CG;
    static_assert(!SYM || BM == BN, "a symmetric product takes square tiles");
    constexpr uint32_t TMEM_COLS = 256 * CG;  // two accumulators
    constexpr uint32_t IDESC = idesc_f16_f32(BM, BN, A_MN, B_MN);
    // an N-contiguous B is loaded 128 columns wide whatever BN is
    constexpr uint32_t STAGE_TX = NS_OPERAND + (B_MN ? NS_OPERAND : BNH * 128);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + NS_STAGES * NS_OPERAND;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NS_STAGES * NS_STAGE);
    uint64_t *full = bars, *empty = bars + NS_STAGES, *tfull = bars + 2 * NS_STAGES;
    uint64_t *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    uint8_t *staging = smem + NS_STAGES * NS_STAGE + 1024;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int worker = blockIdx.x / CG, workers = gridDim.x / CG;

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
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tma_a);
        tma_prefetch_desc(&tma_b);
        tma_prefetch_desc(&tma_d);
        tma_prefetch_desc(&tma_lo);
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
    pdl_wait_prior();
    pdl_allow_next();

    const int nk = (p.K + 63) / 64;
    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = worker; tile < p.tiles && ok; tile += workers) {
                int z, tm, tn;
                ns_locate<SYM>(p, tile, z, tm, tn);
                const int arow = tm * BM + (int)rank * 128, brow = tn * BN + (int)rank * BNH;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, p.wait_limit_ns,
                                           kStatusTimeoutTma, p.status)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * STAGE_TX);
                    const uint32_t lead = CG == 2 ? mapa_shared(smem_u32(&full[stage]), 0) : 0u;
                    uint8_t *da = sA + stage * NS_OPERAND, *db = sB + stage * NS_OPERAND;
                    if constexpr (A_MN) {
                        ns_load<CG>(da, &tma_a, &full[stage], lead, arow, kb * 64, z);
                        ns_load<CG>(da + 8192, &tma_a, &full[stage], lead, arow + 64, kb * 64, z);
                    } else {
                        ns_load<CG>(da, &tma_a, &full[stage], lead, kb * 64, arow, z);
                    }
                    if constexpr (B_MN) {
                        ns_load<CG>(db, &tma_b, &full[stage], lead, brow, kb * 64, z);
                        ns_load<CG>(db + 8192, &tma_b, &full[stage], lead, brow + 64, kb * 64, z);
                    } else {
                        ns_load<CG>(db, &tma_b, &full[stage], lead, kb * 64, brow, z);
                    }
                    if (++stage == NS_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && rank == 0) {
                // wait (bounded) for the copies in flight before teardown
                for (int s = 0; s < NS_STAGES; ++s) {
                    stage = stage == 0 ? NS_STAGES - 1 : stage - 1;
                    if (stage == NS_STAGES - 1) phase ^= 1u;
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&full[stage], phase, &no_abort, 10000000ull,
                                      kStatusTimeoutTma, p.status);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint64_t a_desc0 = A_MN ? smem_desc_mn128(smem_u32(sA)) : smem_desc_sw128(smem_u32(sA));
            const uint64_t b_desc0 = B_MN ? smem_desc_mn128(smem_u32(sB)) : smem_desc_sw128(smem_u32(sB));
            constexpr int A_STEP = A_MN ? 2048 : 32, B_STEP = B_MN ? 2048 : 32;
            for (int tile = worker; tile < p.tiles && ok; tile += workers, ++it) {
                const int acc = it & 1;
                const uint32_t acc_phase = (it >> 1) & 1;
                if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, p.wait_limit_ns,
                                       kStatusTimeoutMma, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_bounded(&full[stage], phase, abort_flag, p.wait_limit_ns,
                                           kStatusTimeoutMma, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a_desc0 + (uint64_t)((stage * NS_OPERAND) >> 4);
                    const uint64_t bd = b_desc0 + (uint64_t)((stage * NS_OPERAND) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16<CG>(d_tmem, ad + (uint64_t)((k * A_STEP) >> 4),
                                    bd + (uint64_t)((k * B_STEP) >> 4), IDESC, (kb | k) != 0);
                    if constexpr (CG == 2) mma_commit_pair(&empty[stage], 0x3);
                    else mma_commit(&empty[stage]);
                    if (++stage == NS_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) {
                    if constexpr (CG == 2) mma_commit_pair(&tfull[acc], 0x3);
                    else mma_commit(&tfull[acc]);
                }
            }
            if constexpr (CG == 2) mma_commit_pair(drain, 0x1);
            else mma_commit(drain);
            volatile int no_abort = 0;
            mbar_wait_bounded(drain, 0, &no_abort, p.wait_limit_ns, kStatusTimeoutMma, p.status);
        }
    } else {
        // Two warps to each quarter of the accumulator's lanes (rows): chunks
        // of 32 columns go to them in turn.
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t *box = staging + (warp - 2) * 2 * NS_BOX, *box2 = box + NS_BOX;
        int it = 0;
        for (int tile = worker; tile < p.tiles; tile += workers, ++it) {
            const int acc = it & 1;
            const uint32_t acc_phase = (it >> 1) & 1;
            int z, tm, tn;
            ns_locate<SYM>(p, tile, z, tm, tn);
            const int row0 = tm * BM + (int)rank * 128 + quarter * 32, row = row0 + lane;
            const bool mirror = SYM && tm != tn;
            const int width = row0 < p.M ? min(BN, p.N - tn * BN) : 0;
            // The added matrix's values of a chunk, 8 columns at a time (rows
            // are padded to a multiple of 8, so a group that starts inside
            // the matrix is inside its row), loaded one chunk ahead of the
            // accumulator: the first before the tile's products are done.
            const int64_t at = z * p.bse + (int64_t)row * p.lde;
            const bool add = MODE != kGram && p.e != nullptr && row < p.M;
            uint4 eh[4], el[4];
            auto fetch = [&](int c) {
                if constexpr (MODE != kGram) {
                    const int col = tn * BN + c * 32;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const bool in = add && c * 32 < BN && col + 8 * q < p.N;
                        eh[q] = in ? *reinterpret_cast<const uint4 *>(p.e + at + col + 8 * q)
                                   : make_uint4(0, 0, 0, 0);
                        if constexpr (MODE == kUpdate)
                            el[q] = in && p.e_lo != nullptr
                                        ? *reinterpret_cast<const uint4 *>(p.e_lo + at + col + 8 * q)
                                        : make_uint4(0, 0, 0, 0);
                    }
                }
            };
            fetch(half);
            const bool ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, p.wait_limit_ns,
                                              kStatusTimeoutEpilogue, p.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = half; c * 32 < width; c += 2) {
                const int col = tn * BN + c * 32;
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                       (uint32_t)(acc * BN + c * 32),
                                   r);
                tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * p.acc_mul;
                if constexpr (MODE != kGram) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t hw[4] = {eh[q].x, eh[q].y, eh[q].z, eh[q].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = 8 * q + 2 * i;
                            float2 e = half2_floats(hw[i]);
                            if constexpr (MODE == kUpdate) {
                                const uint32_t lw[4] = {el[q].x, el[q].y, el[q].z, el[q].w};
                                const float2 l = half2_floats(lw[i]);
                                e.x = fmaf(l.x, 1.f / kLoScale, e.x);
                                e.y = fmaf(l.y, 1.f / kLoScale, e.y);
                            }
                            v[j] = fmaf(p.e_mul, e.x, v[j]);
                            v[j + 1] = fmaf(p.e_mul, e.y, v[j + 1]);
                        }
                    }
                    fetch(c + 2);
                }
                if constexpr (MODE == kPoly) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += row == col + j ? p.diag : 0.f;
                }
                uint32_t packed[16];
                if (MODE == kUpdate && p.last) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = pack_half2(v[2 * j], v[2 * j + 1]);
                }
                if (lane == 0) bulk_wait_group_read<0>();  // the last copies have read the boxes
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(box + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) =
                        make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2],
                                   packed[4 * q + 3]);
                if (mirror) {
                    // box row j holds column j: lane's value at place `lane`
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        *reinterpret_cast<uint16_t *>(box2 + j * 64 +
                                                      16 * ((lane >> 3) ^ ((j >> 1) & 3)) +
                                                      2 * (lane & 7)) =
                            (uint16_t)(packed[j >> 1] >> (16 * (j & 1)));
                }
                if (MODE == kUpdate && p.write_lo) {
                    uint32_t plo[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 h = half2_floats(packed[j]);
                        plo[j] = pack_half2((v[2 * j] - h.x) * kLoScale,
                                            (v[2 * j + 1] - h.y) * kLoScale);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(box2 + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) =
                            make_uint4(plo[4 * q], plo[4 * q + 1], plo[4 * q + 2], plo[4 * q + 3]);
                }
                if (MODE == kUpdate && p.direct != nullptr) {
                    // an output whose rows no tensor map can describe: row by
                    // row, 32 neighbouring values to a store
                    __syncwarp();
                    for (int i = 0; i < 32; ++i)
                        if (row0 + i < p.M && col + lane < p.N)
                            p.direct[((int64_t)z * p.M + row0 + i) * p.N + col + lane] =
                                *reinterpret_cast<const uint16_t *>(
                                    box + i * 64 + 16 * ((lane >> 3) ^ ((i >> 1) & 3)) +
                                    2 * (lane & 7));
                    __syncwarp();
                    continue;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ns_store(&tma_d, smem_u32(box), col, row0, z);
                    if (mirror) ns_store(&tma_d, smem_u32(box2), row0, col, z);
                    if (MODE == kUpdate && p.write_lo) ns_store(&tma_lo, smem_u32(box2), col, row0, z);
                    bulk_commit_group();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
                else mbar_arrive(&tempty[acc]);
            }
        }
        if (lane == 0) bulk_wait_group_all();
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

template <bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(NS_THREADS, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                   const __grid_constant__ CUtensorMap tma_d,
                   const __grid_constant__ CUtensorMap tma_lo, const NsArgs p) {
    ns_gemm_body<1, 128, A_MN, B_MN, MODE>(tma_a, tma_b, tma_d, tma_lo, p);
}

template <int BN, bool A_MN, bool B_MN, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NS_THREADS, 1)
    ns_gemm_pair_kernel(const __grid_constant__ CUtensorMap tma_a,
                        const __grid_constant__ CUtensorMap tma_b,
                        const __grid_constant__ CUtensorMap tma_d,
                        const __grid_constant__ CUtensorMap tma_lo, const NsArgs p) {
    ns_gemm_body<2, BN, A_MN, B_MN, MODE>(tma_a, tma_b, tma_d, tma_lo, p);
}

// A batch of row-major 2-byte matrices [rows, cols] in memory, `ld` elements
// from row to row and rows * ld from matrix to matrix.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

bool ns_tmap(CUtensorMap *m, const Mat &a, int64_t batch, int box_cols, int box_rows,
             CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promo) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {(cuuint64_t)(a.ld * 2), (cuuint64_t)(a.rows * a.ld * 2)};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(a.p), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promo,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ns_operand(CUtensorMap *m, const Mat &a, int64_t batch, bool mn, int box_rows) {
    return ns_tmap(m, a, batch, 64, mn ? 64 : box_rows, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bool ns_output(CUtensorMap *m, const Mat &a, int64_t batch) {
    return ns_tmap(m, a, batch, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

int64_t ns_tiles(const NsArgs &p, int bm, int bn, bool sym) {
    const int64_t mt = (p.M + bm - 1) / bm, nt = (p.N + bn - 1) / bn;
    return sym ? mt * (mt + 1) / 2 : mt * nt;
}

template <auto KERNEL>
cudaError_t ns_launch_kernel(int grid, cudaStream_t s, const CUtensorMap &a, const CUtensorMap &b,
                             const CUtensorMap &d, const CUtensorMap &lo, const NsArgs &p) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)NS_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    return launch_pdl(KERNEL, grid, NS_THREADS, NS_SMEM, s, a, b, d, lo, p);
}

// One product of the whole batch: d [M, N] from a and b (see ns_gemm_body).
template <bool A_MN, bool B_MN, int MODE>
cudaError_t ns_gemm(NsArgs p, int64_t batch, const Mat &a, const Mat &b, const Mat &d, const Mat &lo,
                    cudaStream_t s, const char **why) {
    constexpr bool SYM = MODE != kUpdate;
    // Tiles of 256 x bn by a CTA pair or of 128 x 128 by one CTA (bn = 0):
    // the least waves times a tile's time, which goes by the rows that each
    // CTA loads for 64 of K, 128 + bn/2 of a pair's tile (375 ns measured at
    // 256) and, with less to do between two loads, 205 to 256 of the single
    // CTA's (297 ns).
    const int64_t sms = num_sms(), pairs = sms / 2 > 0 ? sms / 2 : 1;
    int bn = 0;
    int64_t best = ((ns_tiles(p, 128, 128, SYM) * batch + sms - 1) / sms) * 205;
    for (int c : {256, 224, 192}) {
        if (SYM && c != 256) break;
        const int64_t cost = ((ns_tiles(p, 256, c, SYM) * batch + pairs - 1) / pairs) * (128 + c / 2);
        if (cost < best) best = cost, bn = c;
    }
    const int bm = bn ? 256 : 128, bw = bn ? bn : 128;
    p.m_tiles = (p.M + bm - 1) / bm;
    p.n_tiles = (p.N + bw - 1) / bw;
    p.tiles_per = (int)ns_tiles(p, bm, bw, SYM);
    p.tiles = (int)(p.tiles_per * batch);
    p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    p.status = device_status_word();
    CUtensorMap ta, tb, td, tl;
    if (!ns_operand(&ta, a, batch, A_MN, 128) || !ns_operand(&tb, b, batch, B_MN, bn ? bn / 2 : 128) ||
        !ns_output(&td, d, batch) || !ns_output(&tl, lo, batch)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    const int grid = (int)(bn ? 2 * std::min<int64_t>(p.tiles, pairs) : std::min<int64_t>(p.tiles, sms));
    if (bn == 0) return ns_launch_kernel<ns_gemm_kernel<A_MN, B_MN, MODE>>(grid, s, ta, tb, td, tl, p);
    if constexpr (!SYM) {
        if (bn == 224)
            return ns_launch_kernel<ns_gemm_pair_kernel<224, A_MN, B_MN, MODE>>(grid, s, ta, tb, td, tl, p);
        if (bn == 192)
            return ns_launch_kernel<ns_gemm_pair_kernel<192, A_MN, B_MN, MODE>>(grid, s, ta, tb, td, tl, p);
    }
    return ns_launch_kernel<ns_gemm_pair_kernel<256, A_MN, B_MN, MODE>>(grid, s, ta, tb, td, tl, p);
}

int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }

constexpr int kPrepParts = 1024;  // blocks a matrix's sum of squares is split over, at most

struct NsLayout {
    int64_t ldx, lds, hi0, hi1, lo0, lo1, a, b, sums, bytes;
};

NsLayout ns_layout(int64_t batch, int64_t rows, int64_t cols) {
    NsLayout w;
    const int64_t s = std::min(rows, cols);
    w.ldx = pad8(cols);
    w.lds = pad8(s);
    const int64_t x = pad256(batch * rows * w.ldx * 2), q = pad256(batch * s * w.lds * 2);
    w.hi0 = 0;
    w.hi1 = w.hi0 + x;
    w.lo0 = w.hi1 + x;
    w.lo1 = w.lo0 + x;
    w.a = w.lo1 + x;
    w.b = w.a + q;
    w.sums = w.b + q;
    w.bytes = w.sums + pad256(batch * kPrepParts * (int64_t)sizeof(SquareSums));
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
        cudaError_t e = launch_pdl(ns_square_kernel<T, VECTOR>, dim3(a.parts, n), kPrepThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        const int ty = kPrepThreads / a.tx;
        const int64_t blocks = std::min<int64_t>((a.rows + ty - 1) / ty, 16 * (int64_t)num_sms());
        e = launch_pdl(ns_scale_kernel<T, VECTOR>, dim3((unsigned)blocks, n), kPrepThreads, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int64_t orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return ns_layout(batch, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const Orthogonalize &o, cudaStream_t s, const char **why) {
    if (o.batch == 0 || o.rows == 0 || o.cols == 0) return cudaSuccess;
    const bool tall = o.rows > o.cols;
    const int64_t S = std::min(o.rows, o.cols), L = std::max(o.rows, o.cols);
    const NsLayout w = ns_layout(o.batch, o.rows, o.cols);
    uint8_t *base = reinterpret_cast<uint8_t *>(o.workspace);
    auto half = [&](int64_t off) { return reinterpret_cast<__half *>(base + off); };

    PrepArgs p = {};
    p.g = o.g, p.ldg = o.ldg, p.bsg = o.bsg;
    p.rows = (int)o.rows, p.cols = (int)o.cols, p.ldx = (int)w.ldx;
    p.eps = o.eps;
    p.sums = reinterpret_cast<SquareSums *>(base + w.sums);
    p.hi = half(w.hi0), p.lo = half(w.lo0);
    const int es = o.g_f32 ? 4 : 2;
    const bool vec = aligned_to(o.g, 16) && o.ldg * es % 16 == 0 && o.bsg * es % 16 == 0 &&
                     o.cols * es % 16 == 0;
    const int64_t groups = vec ? o.cols * es / 16 : o.cols;
    p.tx = 8;
    while (p.tx < kPrepThreads && p.tx < groups) p.tx *= 2;
    const int64_t row_blocks = (o.rows + kPrepThreads / p.tx - 1) / (kPrepThreads / p.tx);
    p.parts = (int)std::min<int64_t>(row_blocks, kPrepParts);
    cudaError_t e = o.g_f32 ? (vec ? ns_prepare<float, true>(p, o.batch, s)
                                   : ns_prepare<float, false>(p, o.batch, s))
                            : (vec ? ns_prepare<uint16_t, true>(p, o.batch, s)
                                   : ns_prepare<uint16_t, false>(p, o.batch, s));
    if (e != cudaSuccess) return e;

    const Mat A = {half(w.a), S, S, w.lds}, B = {half(w.b), S, S, w.lds};
    int cur = 0;
    for (int i = 0; i < o.steps; ++i) {
        const float a = o.coefficients[3 * i], b = o.coefficients[3 * i + 1],
                    c = o.coefficients[3 * i + 2];
        const bool fold = i >= o.steps - kFoldedSteps, last = i == o.steps - 1;
        const Mat X = {half(cur ? w.hi1 : w.hi0), o.rows, o.cols, w.ldx};
        const Mat Y = {half(cur ? w.hi0 : w.hi1), o.rows, o.cols, w.ldx};
        const Mat Ylo = {half(cur ? w.lo0 : w.lo1), o.rows, o.cols, w.ldx};

        NsArgs q = {};  // A = X Xᵀ (tall: Xᵀ X)
        q.M = q.N = (int)S;
        q.K = (int)L;
        q.acc_mul = kAScale / (kXScale * kXScale);
        e = tall ? ns_gemm<true, true, kGram>(q, o.batch, X, X, A, A, s, why)
                 : ns_gemm<false, false, kGram>(q, o.batch, X, X, A, A, s, why);
        if (e != cudaSuccess) return e;

        q.K = (int)S;  // B = b A + c A A (+ a I); A is its own transpose
        q.acc_mul = c * (kBScale / (kAScale * kAScale));
        q.e = half(w.a), q.lde = w.lds, q.bse = S * w.lds;
        q.e_mul = b * (kBScale / kAScale);
        q.diag = fold ? a * kBScale : 0.f;
        e = ns_gemm<false, false, kPoly>(q, o.batch, A, A, B, B, s, why);
        if (e != cudaSuccess) return e;

        q = {};  // X <- a X + B X (tall: a X + X B)
        q.M = (int)o.rows, q.N = (int)o.cols, q.K = (int)S;
        q.acc_mul = last ? o.scale / (kBScale * kXScale) : 1.f / kBScale;
        if (!fold) {
            q.e = reinterpret_cast<const __half *>(X.p);
            q.e_lo = half(cur ? w.lo1 : w.lo0);
            q.lde = w.ldx, q.bse = o.rows * w.ldx;
            q.e_mul = a;
            q.write_lo = i + 1 < o.steps - kFoldedSteps;
        }
        Mat D = Y;
        if (last) {
            q.last = 1;
            if (o.cols % 8 == 0 && aligned_to(o.out, 16)) D = Mat{o.out, o.rows, o.cols, o.cols};
            else q.direct = o.out;
        }
        e = tall ? ns_gemm<false, false, kUpdate>(q, o.batch, X, B, D, Ylo, s, why)
                 : ns_gemm<false, true, kUpdate>(q, o.batch, B, X, D, Ylo, s, why);
        if (e != cudaSuccess) return e;
        cur ^= 1;
    }
    return cudaSuccess;
}

}  // namespace fp8
