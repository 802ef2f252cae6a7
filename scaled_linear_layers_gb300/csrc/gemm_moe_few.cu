// The experts' FP8 products (fprop and dgrad, block recipe) where an expert has
// few rows, as in serving: bound by the weights' bytes.
//
// The weights are the tensor cores' rows: a CTA takes 128 of an expert's output
// columns (rows of W) and up to 64 of its tokens, so that one token costs a
// 128 x 16 product and a promotion of 16 columns, not of 256, and most of what
// is copied are weights.  The instruction's width follows the tile's tokens (16
// to 64).  The contraction goes in groups of four 128-deep blocks: a ring stage,
// a copy of the weights and one of the tokens, and a hand-off each.  With a block
// a hand-off the single threads that issue copies and products bound it, at 600
// to 850 cycles a block where the bandwidth leaves 700 (8 tokens to 8 of 64
// experts, each expert's rows padded to 16, 4096 x 2048: 71 us); warps that issue as a
// whole, by an elected lane, and a copy for four blocks leave them time: 60 us, 52 of
// them the weights' bytes.  Contractions of few groups do not fill that pipeline
// (few_rows in gemm_moe.cu chooses by them).  The MMA warp writes the blocks'
// partial products into TMEM slots, and four epilogue warps fold them into fp32
// registers, each column with its token's scale times the weights'.  A warp of
// its own brings those scales into shared memory, 16 blocks at a time and ahead
// of their use, another finds the tiles.  The numbers and their order are those
// of the kernel for many rows.  Every wait is bounded.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "moe_tiles.cuh"
#include "rowops.cuh"
#include "tmap.h"

namespace fp8 {

namespace {

constexpr int BW = kMoeBlock, BT = kMoeFewRows, BK = kMoeBlock;  // weight rows, tokens, depth of a block
constexpr int KG = 4;  // blocks of a group
constexpr int TOKENS = 16;  // of a step of the instruction's width
constexpr int W_BYTES = BW * BK, T_BYTES = BT * BK;
constexpr int STAGE_BYTES = KG * (W_BYTES + T_BYTES), STAGES = 2;
constexpr int SLOTS = 2;  // TMEM slots of a group, KG * BT columns
constexpr int EPI_WARPS = 4, EPI0 = 4, THREADS = 32 * (EPI0 + EPI_WARPS);
constexpr int PANEL = 16;          // blocks of one panel of scales
constexpr int PANEL_ROW = BT + 4;  // tokens' scales of a block, then the weights'
constexpr int PANEL_FLOATS = PANEL * PANEL_ROW;
constexpr int TILES = 4, READERS = 3 + EPI_WARPS;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 2 * PANEL_FLOATS * sizeof(float) +
                        512 + kMoeSegmentBytes;
static_assert(SLOTS * KG * BT == 512, "the slots fill TMEM");
static_assert(PANEL % KG == 0, "a group lies in one panel");
static_assert(SMEM <= 227 * 1024, "smem");

__device__ __forceinline__ MoeTile find_tile(const MoeArgs &p, const MoeSegments &g, int index) {
    const int w_tiles = p.cols_out / BW;
    MoeTile t;
    t.expert = moe_expert_of(g, p.experts, index / w_tiles);
    const int t_tiles = g.first[t.expert + 1] - g.first[t.expert];
    const int in = index - g.first[t.expert] * w_tiles;
    // an expert's tokens one after the other against the same weights
    t.n = in / t_tiles * BW;
    t.row0 = g.lo[t.expert] + in % t_tiles * BT;
    t.rows = min(BT, g.hi[t.expert] - t.row0);
    t.kb0 = t.bad = t.unused = 0;
    t.nk = p.depth;
    return t;
}

// Copies of a group: of 128 weight rows, and of 16, 32 or 64 tokens.
struct Maps {
    CUtensorMap w, t[3];
};

__global__ void __launch_bounds__(THREADS, 1)
    moe_few_kernel(const __grid_constant__ Maps maps, const MoeArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint8_t *sW = smem;
    uint8_t *sT = smem + STAGES * KG * W_BYTES;
    float *panels = reinterpret_cast<float *>(smem + STAGES * STAGE_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(panels + 2 * PANEL_FLOATS);  // [STAGES]
    uint64_t *empty = full + STAGES;    // [STAGES]
    uint64_t *sfull = empty + STAGES;   // [SLOTS] MMA -> epilogue
    uint64_t *sempty = sfull + SLOTS;   // [SLOTS] epilogue -> MMA
    uint64_t *tfull = sempty + SLOTS;   // [TILES] search -> readers
    uint64_t *tempty = tfull + TILES;   // [TILES] readers -> search
    uint64_t *pfull = tempty + TILES;   // [2] scales -> epilogue
    uint64_t *pempty = pfull + 2;       // [2] epilogue -> scales
    uint64_t *drain = pempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    MoeTile *tiles = reinterpret_cast<MoeTile *>(full + 48);  // [TILES]
    const MoeSegments seg(reinterpret_cast<int32_t *>(full) + 128, p.experts);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&sempty[s], EPI_WARPS);
        }
        for (int s = 0; s < TILES; ++s) {
            mbar_init(&tfull[s], 1);
            mbar_init(&tempty[s], READERS);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&pfull[s], 32);
            mbar_init(&pempty[s], EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.t[0]);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    pdl_wait_prior();  // the offsets are the previous kernels' result
    pdl_allow_next();
    if (warp == 2) moe_count_tiles<BT>(p, seg, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    auto wait = [&](uint64_t *bar, uint32_t parity, unsigned int code) {
        return mbar_wait_bounded<true>(bar, parity, abort_flag, p.wait_limit_ns, code, p.status);
    };
    // The i-th tile of this CTA is in its place; false when none is left or the
    // wait gave up.
    auto have_tile = [&](uint32_t i) {
        return wait(&tfull[i % TILES], (i / TILES) & 1u, kStatusTimeoutTma) &&
               tiles[i % TILES].nk >= 0;
    };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        const bool leader = elect_one();
        for (uint32_t i = 0; ok && __all_sync(0xFFFFFFFFu, have_tile(i)); ++i) {
            const MoeTile &t = tiles[i % TILES];
            const int nk = __shfl_sync(0xFFFFFFFFu, t.nk, 0), rows = t.rows;
            const int size = __shfl_sync(0xFFFFFFFFu, rows > 32 ? 2 : rows > 16 ? 1 : 0, 0);
            const int w_row = __shfl_sync(0xFFFFFFFFu, t.expert * p.by + t.n, 0);
            const int w_k = __shfl_sync(0xFFFFFFFFu, t.expert * p.bx / BK, 0);
            const int row0 = __shfl_sync(0xFFFFFFFFu, t.row0, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
            const uint32_t bytes = KG * BK * (BW + (TOKENS << size));
            for (int q = 0; q < nk; q += KG) {
                ok = __all_sync(0xFFFFFFFFu, wait(&empty[stage], phase ^ 1u, kStatusTimeoutTma));
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    if (!(p.lose && i == 0 && q == 2 * KG)) {
                        tma_load_3d(sW + stage * KG * W_BYTES, &maps.w, &full[stage], 0, w_row, w_k + q);
                        tma_load_3d(sT + stage * KG * T_BYTES, &maps.t[size], &full[stage], 0, row0, q);
                    }
                }
                __syncwarp();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // wait (bounded) for the copies still in flight before teardown
        for (int s = 0; s < STAGES; ++s) {
            stage = stage == 0 ? STAGES - 1 : stage - 1;
            if (stage == STAGES - 1) phase ^= 1u;
            volatile int no_abort = 0;
            mbar_wait_bounded(&full[stage], phase, &no_abort, 10000000ull, kStatusTimeoutTma,
                              p.status);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t g = 0;  // groups issued so far (across tiles)
        bool ok = true;
        const bool leader = elect_one();
        const uint64_t w_desc = smem_desc_sw128(smem_u32(sW)), t_desc = smem_desc_sw128(smem_u32(sT));
        for (uint32_t i = 0; ok && __all_sync(0xFFFFFFFFu, have_tile(i)); ++i) {
            const int nk = __shfl_sync(0xFFFFFFFFu, tiles[i % TILES].nk, 0);
            const int rows = __shfl_sync(0xFFFFFFFFu, tiles[i % TILES].rows, 0);
            const uint32_t t_block = (rows > 32 ? 64 : rows > 16 ? 32 : 16) * BK;  // bytes
            const uint32_t idesc = idesc_f8_f32(BW, (rows + TOKENS - 1) / TOKENS * TOKENS);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
            for (int q = 0; q < nk; q += KG, ++g) {
                const uint32_t slot = g % SLOTS, sphase = (g / SLOTS) & 1u;
                ok = __all_sync(0xFFFFFFFFu, wait(&sempty[slot], sphase ^ 1u, kStatusTimeoutMma) &&
                                                 wait(&full[stage], phase, kStatusTimeoutMma));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int j = 0; j < KG; ++j) {
                        if (q + j >= nk) break;
                        const uint64_t w0 = w_desc + ((stage * KG + j) * W_BYTES >> 4);
                        const uint64_t t0 = t_desc + ((stage * KG * T_BYTES + j * t_block) >> 4);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            mma_f8(tmem_base + (slot * KG + j) * BT, w0 + 2 * k, t0 + 2 * k, idesc,
                                   k != 0);
                    }
                    mma_commit(&empty[stage]);
                    mma_commit(&sfull[slot]);
                }
                __syncwarp();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (leader) mma_commit(drain);
        volatile int no_abort = 0;  // a short limit must not cut this wait short
        mbar_wait_bounded(drain, 0, &no_abort, kDefaultWaitLimitNs, kStatusTimeoutMma, p.status);
    } else if (warp == 2) {
        if (lane == 0) {
            // -------------------------------------------- search for tiles
            const int num_tiles = seg.first[p.experts] * (p.cols_out / BW);
            int index = blockIdx.x;
            for (uint32_t i = 0;; ++i, index += gridDim.x) {
                MoeTile t;
                t.nk = -1;
                if (index < num_tiles) t = find_tile(p, seg, index);
                if (!mbar_wait_bounded<true>(&tempty[i % TILES], ((i / TILES) & 1u) ^ 1u, abort_flag,
                                             p.wait_limit_ns + moe_tile_ns(p.depth),
                                             kStatusTimeoutTma, p.status))
                    break;
                tiles[i % TILES] = t;
                mbar_arrive(&tfull[i % TILES]);
                if (t.nk < 0) break;
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------ scales, a panel ahead
        uint32_t n = 0;  // panels so far (across tiles)
        bool ok = true;
        for (uint32_t i = 0; ok && __all_sync(0xFFFFFFFFu, have_tile(i)); ++i) {
            const MoeTile &t = tiles[i % TILES];
            const int rows = t.rows, nk = t.nk;
            const float *sa = p.sa + (int64_t)t.row0 * p.sa_row;
            const float *sb = p.sb + t.expert * p.sb_expert + (int64_t)(t.n / BK) * p.sb_col;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
            for (int q0 = 0; q0 < nk; q0 += PANEL, ++n) {
                ok = wait(&pempty[n & 1], ((n >> 1) & 1u) ^ 1u, kStatusTimeoutTma);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                float *panel = panels + (n & 1) * PANEL_FLOATS;
                // 16 blocks of two tokens at a time; those behind the last go unused
                const int q = lane & (PANEL - 1);
                if (q0 + q < nk) {
                    for (int r = lane / PANEL; r < rows; r += 2)
                        cp_async4(panel + q * PANEL_ROW + r,
                                  sa + (int64_t)r * p.sa_row + (int64_t)(q0 + q) * p.sa_k);
                    if (lane < PANEL)
                        cp_async4(panel + q * PANEL_ROW + BT, sb + (int64_t)(q0 + q) * p.sb_k);
                }
                cp_async_arrive_noinc(&pfull[n & 1]);
            }
        }
        cp_async_wait_all();
    } else {
        // ------------------------------------------------- epilogue (4 warps)
        const int quarter = warp & 3;  // TMEM lanes 32*quarter .. +31: weight rows
        bool ok = true;
        uint32_t g = 0, n = 0;
        for (uint32_t i = 0;; ++i) {
            ok = __all_sync(0xFFFFFFFFu, ok && have_tile(i));
            if (!ok) break;
            const MoeTile &t = tiles[i % TILES];
            const int nk = t.nk, rows = t.rows, chunks = (rows + 15) / 16;
            float acc[BT];
#pragma unroll
            for (int j = 0; j < BT; ++j) acc[j] = 0.f;
            for (int q = 0; q < nk; q += KG, ++g) {
                if (q % PANEL == 0) {
                    ok = wait(&pfull[n & 1], (n >> 1) & 1u, kStatusTimeoutEpilogue);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                }
                const float *scales = panels + (n & 1) * PANEL_FLOATS + q % PANEL * PANEL_ROW;
                const uint32_t slot = g % SLOTS, sphase = (g / SLOTS) & 1u;
                ok = wait(&sfull[slot], sphase, kStatusTimeoutEpilogue);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t taddr =
                    tmem_base + ((uint32_t)(quarter * 32) << 16) + slot * KG * BT;
                const int blocks = min(KG, nk - q);
#pragma unroll
                for (int c = 0; c < BT / 16; ++c) {
                    if (c >= chunks) break;
                    uint32_t r[KG][16];
#pragma unroll
                    for (int j = 0; j < KG; ++j)
                        if (j < blocks) tmem_ld_32x32b_x16(taddr + j * BT + 16 * c, r[j]);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < KG; ++j) {
                        if (j >= blocks) break;
                        tmem_regs_ready(r[j]);
                        const float *row = scales + j * PANEL_ROW;
                        const float ws = row[BT];
                        const float4 *ts = reinterpret_cast<const float4 *>(row + 16 * c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 s = ts[k];
                            float *a = acc + 16 * c + 4 * k;
                            const uint32_t *v = r[j] + 4 * k;
                            a[0] = __fmaf_rn(__uint_as_float(v[0]), __fmul_rn(s.x, ws), a[0]);
                            a[1] = __fmaf_rn(__uint_as_float(v[1]), __fmul_rn(s.y, ws), a[1]);
                            a[2] = __fmaf_rn(__uint_as_float(v[2]), __fmul_rn(s.z, ws), a[2]);
                            a[3] = __fmaf_rn(__uint_as_float(v[3]), __fmul_rn(s.w, ws), a[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[slot]);
                if ((q + KG) % PANEL == 0 || q + KG >= nk) {
                    if (lane == 0) mbar_arrive(&pempty[n & 1]);
                    ++n;
                }
            }
            if (!ok) break;
            // a token's 32 neighbouring outputs by one warp: 64 bytes
            uint16_t *d = p.d + (int64_t)t.row0 * p.cols_out + t.n + quarter * 32 + lane;
#pragma unroll
            for (int j = 0; j < BT; ++j)
                if (j < rows) float_to_elem(d + (int64_t)j * p.cols_out, acc[j]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
        }
    }

    __syncwarp();  // lanes that skipped a role wait here for their warp's lane 0
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, 512);
    }
}

}  // namespace

cudaError_t launch_moe_few(const MoeArgs &p, const uint8_t *a, int64_t a_cols, const uint8_t *b,
                           int64_t b_rows, int64_t b_cols, cudaStream_t s, const char **why) {
    Maps maps;
    bool made = make_tmap_k128_blocks(&maps.w, b, b_rows, b_cols, BW, KG);
    for (int i = 0; i < 3; ++i)
        made = made && make_tmap_k128_blocks(&maps.t[i], a, p.capacity, a_cols, TOKENS << i, KG);
    if (!made) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    static std::atomic<bool> attr_done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(moe_few_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    // every expert may end in a tile of its own
    const int64_t ends = p.experts < p.capacity ? p.experts : p.capacity;
    const int64_t most = (p.capacity / BT + ends) * (p.cols_out / BW), sms = num_sms();
    return launch_pdl(moe_few_kernel, (unsigned)(most < sms ? most : sms), THREADS, SMEM, s, maps, p);
}

}  // namespace fp8
