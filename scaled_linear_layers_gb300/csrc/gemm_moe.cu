// The FP8 linears of all experts in one launch, block recipe: rows sorted by
// expert in segments offsets[e] .. offsets[e + 1] - 1 (on the device), and for
// the rows r of expert e
//
//   fprop: y[r, n]  = sum_kb xs(r, kb) ws(e, n/128, kb) sum_{k in kb} x[r, k] w[e, n, k]
//   dgrad: dx[r, k] = sum_nb gs(r, nb) ws(e, nb, k/128) sum_{n in nb} g[r, n] w[e, n, k]
//   wgrad: dw[e, n, k] = sum_b gs(b, n) xs(b, k) sum_{r in b} g[r, n] x[r, k],
//          b the 128-row blocks of e's segment
//
// The pipeline is that of the single block-scaled GEMM (one persistent CTA an
// SM, 128 x 256 output tiles; TMA ring, an MMA warp that writes each 128-deep
// partial into one of two TMEM slots, eight epilogue warps that fold it into
// fp32 registers with its scales).  What differs is that a tile's rows,
// weights and contraction depend on offsets that only the device knows: every
// CTA reads them once, keeps them in shared memory with the row tiles before
// each expert, and a warp of its own finds the tiles' experts by bisection, a
// few tiles ahead of the producer, MMA and epilogue warps: the host launches
// without waiting for the sort.  Tiles go expert by expert, so that an expert's
// weights are in L2 while its rows pass.  Rows of a tile past its segment are
// computed from what lies there and not stored.
//
// wgrad is bound by the promotion: a block's 32768 partials an SM take a packed
// multiply-add and a packed product of scales for two of them, by two warps a scheduler
// that wait for each 16 columns' load from TMEM.  fprop and dgrad, whose partials take
// the multiply-add alone, are bound by the tensor cores' feed and the hand-offs (a copy
// of fprop without the promotion's arithmetic takes 1414 us of 1541) and by a tile's
// end, in which nothing is folded.  Measured, us: 16384 rows of 8 experts to
// 28672 columns, 4096 deep; dgrad of 65536 rows of 64 experts to 4096 columns,
// 2048 deep; wgrad 14336 x 4096 of 8 experts' 32768 rows:
//   16 (fprop) or 4 bytes of a row stored at a time, first scales read as a
//   tile begins                                               1705   632   2715
//   outputs through a box in shared memory, the next tile's first scales read
//   before them                                               1596   534   2644
//   wgrad in pairs: accumulators, partials and scales in register pairs, a
//   chunk's scales read a chunk ahead                         1547   501   2468
// and, not taken: loads of 32 columns 1989, 599, 3168 (registers spilled) and for
// wgrad alone 2783; the next block's first load asked for before the last chunk's
// products 1845, 602, 3340; two products of 128 columns a block, each with TMEM
// slots of its own, 1842, 585, 2461 (A is read twice from shared memory); pairs of
// CTAs on 256 x 256 tiles 1537, 528; whole boxes stored by the copy engine 1512, 495,
// with 8 KB a warp for them and three stages 1509, 522.  A copy of the kernel that
// stores nothing takes 1368 and 409: a block is about 0.44 us, a tile's end 2.3.
#include <cuda.h>

#include <atomic>
#include <cstdlib>

#include "common.cuh"
#include "kernels.h"
#include "moe_tiles.cuh"
#include "rowops.cuh"
#include "tmap.h"

namespace fp8 {

extern std::atomic<uint64_t> g_wait_limit_ns;

namespace {

constexpr int BM = kMoeBlock, BN = 256, BK = kMoeBlock;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int SLOTS = 2;  // TMEM slots of BN columns
constexpr int EPI_WARPS = 8, EPI0 = 4;
constexpr int THREADS = 32 * (EPI0 + EPI_WARPS);
constexpr int COLS = BN * 4 / EPI_WARPS;  // accumulator columns of a one-row thread
constexpr int REGS_LOW = 40, REGS_HIGH = 232;
constexpr uint32_t IDESC = idesc_f8_f32(BM, BN);
// Shared memory of an epilogue warp: the box that a tile's output goes through
// (wgrad: half of it; the other half holds column scales, two blocks of them).
constexpr int WARP_BYTES = 2048;
static_assert(2 * COLS * sizeof(float) == WARP_BYTES / 2, "two blocks' column scales");
constexpr int TILES = 4;  // tiles found ahead of their use
constexpr int READERS = 2 + EPI_WARPS;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_WARPS * WARP_BYTES + 512 +
                        kMoeSegmentBytes;
static_assert(SLOTS * BN == 512, "the slots fill TMEM");
static_assert(SMEM <= 227 * 1024, "smem");

using Args = MoeArgs;
using Tile = MoeTile;

template <bool kWgrad>
__device__ __forceinline__ int total_tiles(const Args &p, const MoeSegments &g) {
    const int n_tiles = (p.cols_out + BN - 1) / BN;
    if (kWgrad) return p.experts * (p.rows_out / BM) * n_tiles;
    return g.first[p.experts] * n_tiles;
}

template <bool kWgrad>
__device__ __forceinline__ Tile find_tile(const Args &p, const MoeSegments &g, int index) {
    const int n_tiles = (p.cols_out + BN - 1) / BN;
    Tile t;
    int m_tiles, lo, hi, in;
    if (kWgrad) {
        m_tiles = p.rows_out / BM;
        const int per = m_tiles * n_tiles;
        t.expert = index / per;
        in = index - t.expert * per;
    } else {
        t.expert = moe_expert_of(g, p.experts, index / n_tiles);
        m_tiles = g.first[t.expert + 1] - g.first[t.expert];
        in = index - g.first[t.expert] * n_tiles;
    }
    lo = g.lo[t.expert];
    hi = g.hi[t.expert];
    int tm, tn;
    grouped_tile(in, m_tiles, n_tiles, 16, tm, tn);
    t.n = tn * BN;
    t.unused = 0;
    if (kWgrad) {
        t.bad = ((lo | hi) & (BK - 1)) != 0;
        t.row0 = tm * BM;
        t.rows = BM;
        t.kb0 = lo / BK;
        t.nk = t.bad ? 0 : (hi - lo) / BK;
    } else {
        t.bad = 0;
        t.row0 = lo + tm * BM;
        t.rows = min(BM, hi - t.row0);
        t.kb0 = 0;
        t.nk = p.depth;
    }
    return t;
}

// acc += p * f on a pair of neighbouring columns
__device__ __forceinline__ void fold(uint64_t &acc, uint32_t p0, uint32_t p1, uint64_t f) {
    uint64_t pv;
    asm("mov.b64 %0, {%1, %2};" : "=l"(pv) : "r"(p0), "r"(p1));
    acc = pair_fma(pv, f, acc);
}

__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
    const float2 f = pair_split(v);
    return pack_bf16x2(f.x, f.y);
}

template <bool kWgrad>
__global__ void __launch_bounds__(THREADS, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tma_a,
                    const __grid_constant__ CUtensorMap tma_b, const Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint8_t *sA = smem;
    uint8_t *sB = smem + STAGES * A_BYTES;
    uint8_t *boxes = smem + STAGES * STAGE_BYTES;  // [EPI_WARPS]
    uint64_t *full = reinterpret_cast<uint64_t *>(boxes + EPI_WARPS * WARP_BYTES);  // [STAGES] TMA -> MMA
    uint64_t *empty = full + STAGES;                               // [STAGES] MMA -> TMA
    uint64_t *sfull = empty + STAGES;                              // [SLOTS] MMA -> epilogue
    uint64_t *sempty = sfull + SLOTS;                              // [SLOTS] epilogue -> MMA
    uint64_t *tfull = sempty + SLOTS;                              // [TILES] search -> readers
    uint64_t *tempty = tfull + TILES;                              // [TILES] readers -> search
    uint64_t *drain = tempty + TILES;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    Tile *tiles = reinterpret_cast<Tile *>(full + 32);  // [TILES]
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
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tma_a);
        tma_prefetch_desc(&tma_b);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, SLOTS * BN);
        tmem_relinquish();
    }
    pdl_wait_prior();  // the offsets are the previous kernels' result
    pdl_allow_next();
    if (warp == 2) moe_count_tiles<BM>(p, seg, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // The i-th tile of this CTA is in its place; false when none is left or the
    // wait gave up.
    auto have_tile = [&](uint32_t i) {
        return mbar_wait_bounded<true>(&tfull[i % TILES], (i / TILES) & 1u, abort_flag,
                                       p.wait_limit_ns, kStatusTimeoutTma, p.status) &&
               tiles[i % TILES].nk >= 0;
    };
    // each warp of the first warpgroup gives registers back as it enters its
    // role, each epilogue warp takes more
    auto regs_low = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_LOW)); };

    if (warp == 0) {
        regs_low();
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        const bool leader = elect_one();
        for (uint32_t i = 0; ok && __all_sync(0xFFFFFFFFu, have_tile(i)); ++i) {
            const Tile &t = tiles[i % TILES];
            const int nk = __shfl_sync(0xFFFFFFFFu, t.nk, 0);
            const int arow = __shfl_sync(0xFFFFFFFFu, t.row0, 0);
            const int brow = __shfl_sync(0xFFFFFFFFu, t.expert * p.by + t.n, 0);
            int ax = __shfl_sync(0xFFFFFFFFu, t.kb0 * BK, 0);
            int bx = ax + __shfl_sync(0xFFFFFFFFu, t.expert * p.bx, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
            for (int q = 0; q < nk; ++q, ax += BK, bx += BK) {
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait_bounded<true>(&empty[stage], phase ^ 1u, abort_flag,
                                                        p.wait_limit_ns, kStatusTimeoutTma, p.status));
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
                    if (!(p.lose && i == 0 && q == 2)) {
                        tma_load_2d(sA + stage * A_BYTES, &tma_a, &full[stage], ax, arow);
                        tma_load_2d(sB + stage * B_BYTES, &tma_b, &full[stage], bx, brow);
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
        regs_low();
        // ------------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t g = 0;  // blocks issued so far (across tiles)
        bool ok = true;
        const bool leader = elect_one();
        const uint64_t a_desc = smem_desc_sw128(smem_u32(sA)), b_desc = smem_desc_sw128(smem_u32(sB));
        for (uint32_t i = 0; ok && __all_sync(0xFFFFFFFFu, have_tile(i)); ++i) {
            const int nk = __shfl_sync(0xFFFFFFFFu, tiles[i % TILES].nk, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
            for (int q = 0; q < nk; ++q, ++g) {
                const uint32_t slot = g % SLOTS, sphase = (g / SLOTS) & 1u;
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait_bounded<true>(&sempty[slot], sphase ^ 1u, abort_flag,
                                                        p.wait_limit_ns, kStatusTimeoutMma, p.status) &&
                                    mbar_wait_bounded<true>(&full[stage], phase, abort_flag,
                                                            p.wait_limit_ns, kStatusTimeoutMma, p.status));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t a0 = a_desc + (stage * A_BYTES >> 4);
                    const uint64_t b0 = b_desc + (stage * B_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_f8(tmem_base + slot * BN, a0 + 2 * k, b0 + 2 * k, IDESC, k != 0);
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
        regs_low();
        if (lane == 0) {
            // -------------------------------------------- search for tiles
            const int num_tiles = total_tiles<kWgrad>(p, seg);
            // a place is free once the tile before is done: far from its end where
            // the contraction is long
            const uint64_t limit_ns =
                p.wait_limit_ns + moe_tile_ns(kWgrad ? p.capacity / BK : p.depth);
            int index = blockIdx.x;
            for (uint32_t i = 0;; ++i, index += gridDim.x) {
                const uint32_t at = i % TILES;
                Tile t;
                t.nk = -1;
                if (index < num_tiles) t = find_tile<kWgrad>(p, seg, index);
                if (!mbar_wait_bounded<true>(&tempty[at], ((i / TILES) & 1u) ^ 1u, abort_flag,
                                             limit_ns, kStatusTimeoutTma, p.status))
                    break;
                tiles[at] = t;
                mbar_arrive(&tfull[at]);
                if (t.nk < 0) break;
            }
        }
    } else if (warp < EPI0) {
        regs_low();  // an idle warp of the first warpgroup
    } else {
        // ------------------------------------------------- epilogue (8 warps)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_HIGH));
        const int quarter = warp & 3;          // TMEM lanes 32*quarter .. +31
        const int half = (warp - EPI0) >> 2;   // columns half*COLS .. +COLS-1 of the tile
        bool ok = true;
        uint32_t g = 0;
        auto wait_block = [&](uint32_t h) {  // block h of all
            if (ok)
                ok = mbar_wait_bounded<true>(&sfull[h % SLOTS], (h / SLOTS) & 1u, abort_flag, p.wait_limit_ns,
                                             kStatusTimeoutEpilogue, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) tc_fence_after();
        };
        // A tile stays in its place until the warp is done with it, so that what
        // the stores need is read again rather than kept in registers.
        auto next_tile = [&](uint32_t i) {
            ok = __all_sync(0xFFFFFFFFu, ok && have_tile(i));
            return ok;
        };
        auto free_tile = [&](uint32_t i) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[i % TILES]);
        };
        auto hand_back = [&](uint32_t slot) {  // the block's partial is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[slot]);
        };
        uint8_t *box = boxes + (warp - EPI0) * WARP_BYTES;
        if constexpr (kWgrad) {
            // Four rows x 32 columns a thread (16-lane TMEM loads): thread l
            // holds rows 8i + l/4 (i = 0..3) of its lane quarter and, of every
            // 8 columns, 2(l%4) and +1, so it needs 32 column scales a block
            // instead of 128; they are staged by cp.async, one block ahead.
            float *wbuf = reinterpret_cast<float *>(box + WARP_BYTES / 2);
            const int fr = lane >> 2, fc = lane & 3;
            const float *sa = nullptr, *sb = nullptr;
            float next[4] = {};
            constexpr int NC = COLS / 16;  // 16 columns a load
            // Chunk c of the block in work: the partials of rows 0..15 and 16..31
            // and the scales of this thread's columns, with those of chunk c + 1
            // under way while it is folded in.
            uint32_t ra[2][8], rb[2][8];
            uint64_t sc[2][2];
            // block h of all: its scales into its half of wbuf
            auto fetch = [&](uint32_t h, bool there) {
                if (there) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) next[i] = sa[8 * i];
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                                     smem_u32(wbuf + (h & 1) * COLS + 4 * lane)),
                                 "l"(sb)
                                 : "memory");
                    sa += p.sa_k;
                    sb += p.sb_k;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            auto scales = [&](uint32_t h, int c) {
                const float *buf = wbuf + (h & 1) * COLS + 2 * fc + 16 * c;
                sc[c & 1][0] = *reinterpret_cast<const uint64_t *>(buf);
                sc[c & 1][1] = *reinterpret_cast<const uint64_t *>(buf + 8);
            };
            auto load = [&](uint32_t h, int c) {
                const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                       (h % SLOTS) * BN + (uint32_t)(half * COLS) + 16 * c;
                tmem_ld_16x256b_x2(taddr, ra[c & 1]);
                tmem_ld_16x256b_x2(taddr + (16u << 16), rb[c & 1]);
            };
            auto loaded = [&](int c) {
                tmem_ld_wait();
                tmem_regs_ready(ra[c & 1]);
                tmem_regs_ready(rb[c & 1]);
            };
            auto begin = [&](uint32_t at) {
                const Tile &t = tiles[at % TILES];
                sa = p.sa + (int64_t)t.kb0 * p.sa_k + t.row0 + quarter * 32 + fr;
                sb = p.sb + (int64_t)t.kb0 * p.sb_k +
                     min(t.n + half * COLS + 4 * lane, p.cols_out - 4);
                fetch(g, t.nk > 0);
            };
            bool more = next_tile(0);
            if (more) begin(0);
            for (uint32_t at = 0; more; ++at) {
                const Tile &t = tiles[at % TILES];
                const int nk = t.nk;
                const float start = t.bad ? __uint_as_float(0x7FFFFFFFu) : 0.f;
                uint64_t acc[4][COLS / 8];  // [i][j]: columns 8 j + 2 fc and + 1
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < COLS / 8; ++j) acc[i][j] = pair_of(start, start);
                for (int q = 0; q < nk; ++q, ++g) {
                    uint64_t cur[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) cur[i] = pair_of(next[i], next[i]);
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                    fetch(g + 1, q + 1 < nk);
                    wait_block(g);
                    if (!ok) break;
                    scales(g, 0);
                    load(g, 0);
                    loaded(0);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (c + 1 < NC) {
                            load(g, c + 1);
                            scales(g, c + 1);
                        }
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t *v = (i < 2 ? ra : rb)[c & 1] + 4 * jj + 2 * (i & 1);
                                fold(acc[i][2 * c + jj], v[0], v[1], pair_mul(sc[c & 1][jj], cur[i]));
                            }
                        if (c + 1 < NC) {
                            loaded(c + 1);
                            if (c + 2 == NC) hand_back(g % SLOTS);
                        }
                    }
                }
                const bool done = ok;
                more = next_tile(at + 1);
                if (more) begin(at + 1);
                const int j0 = t.n + half * COLS;
                if (done && j0 < p.cols_out) {
                    // eight rows of 64 columns at a time through the box (16-byte
                    // groups, group j of row r at j ^ r): 128 bytes of a row a store
                    uint16_t *d = p.d +
                                  ((int64_t)t.expert * p.rows_out + t.row0 + quarter * 32 + (lane >> 3)) *
                                      p.cols_out +
                                  j0 + 8 * (lane & 7);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<uint32_t *>(box + fr * 128 + ((j ^ fr) * 16) + 4 * fc) =
                                    pack_pair(acc[i][8 * h + j]);
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int r = 4 * k + (lane >> 3);
                                const uint4 v = *reinterpret_cast<const uint4 *>(
                                    box + r * 128 + (((lane & 7) ^ r) * 16));
                                *reinterpret_cast<uint4 *>(d + (int64_t)(8 * i + 4 * k) * p.cols_out +
                                                           64 * h) = v;
                            }
                            __syncwarp();
                        }
                }
                free_tile(at);
            }
            cp_async_wait_all();
        } else {
            // one row x 128 columns a thread: a block's scale is one product
            const float *sa = nullptr, *sb = nullptr;
            float sa_next = 0.f, sb_next = 0.f;
            constexpr int NC = COLS / 16;
            uint32_t r[2][16];  // chunk c of the block in work and, under way, c + 1
            auto load = [&](uint32_t h, int c) {
                tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(quarter * 32) << 16) + (h % SLOTS) * BN +
                                       (uint32_t)(half * COLS) + 16 * c,
                                   r[c & 1]);
            };
            auto loaded = [&](int c) {
                tmem_ld_wait();
                tmem_regs_ready(r[c & 1]);
            };
            auto begin = [&](uint32_t at) {
                const Tile &t = tiles[at % TILES];
                sa = p.sa + (int64_t)min(t.row0 + quarter * 32 + lane, p.capacity - 1) * p.sa_row;
                sb = p.sb + t.expert * p.sb_expert +
                     (int64_t)(min(t.n + half * COLS, p.cols_out - 1) / BK) * p.sb_col;
                sa_next = *sa;
                sb_next = *sb;
            };
            bool more = next_tile(0);
            if (more) begin(0);
            for (uint32_t at = 0; more; ++at) {
                const Tile &t = tiles[at % TILES];
                const int nk = t.nk;
                uint64_t acc[COLS / 2];
#pragma unroll
                for (int j = 0; j < COLS / 2; ++j) acc[j] = 0ull;
                for (int q = 0; q < nk; ++q, ++g) {
                    const float f = sa_next * sb_next;
                    const uint64_t ff = pair_of(f, f);
                    if (q + 1 < nk) {
                        sa += p.sa_k;
                        sb += p.sb_k;
                    }
                    sa_next = *sa;
                    sb_next = *sb;
                    wait_block(g);
                    if (!ok) break;
                    load(g, 0);
                    loaded(0);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (c + 1 < NC) load(g, c + 1);
#pragma unroll
                        for (int a = 0; a < 8; ++a)
                            fold(acc[8 * c + a], r[c & 1][2 * a], r[c & 1][2 * a + 1], ff);
                        if (c + 1 < NC) {
                            loaded(c + 1);
                            if (c + 2 == NC) hand_back(g % SLOTS);
                        }
                    }
                }
                const bool done = ok;
                more = next_tile(at + 1);
                if (more) begin(at + 1);
                const int j0 = t.n + half * COLS, there = t.rows - quarter * 32;
                if (done && there > 0 && j0 < p.cols_out) {
                    // 32 columns at a time through the box (16-byte groups, group c
                    // of row r at c ^ r/2): 64 bytes of eight rows a store
                    uint16_t *d = p.d + (int64_t)(t.row0 + quarter * 32 + (lane >> 2)) * p.cols_out + j0 +
                                  8 * (lane & 3);
#pragma unroll
                    for (int c = 0; c < COLS / 32; ++c) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = pack_pair(acc[16 * c + 4 * b + e]);
                            *reinterpret_cast<uint4 *>(box + lane * 64 + ((b ^ ((lane >> 1) & 3)) * 16)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = 8 * k + (lane >> 2);
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                box + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) * 16));
                            if (r < there)
                                *reinterpret_cast<uint4 *>(d + (int64_t)(8 * k) * p.cols_out + 32 * c) = v;
                        }
                        __syncwarp();
                    }
                }
                free_tile(at);
            }
        }
    }

    __syncwarp();  // lanes that skipped a role wait here for their warp's lane 0
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, SLOTS * BN);
    }
}

template <bool kWgrad>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const Args &args, int64_t tiles,
                   cudaStream_t s, const char **why) {
    static std::atomic<bool> attr_done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        // setmaxnreg.inc waits until the launch's own registers can supply the
        // raised counts: a build with fewer than the split needs is refused
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, moe_gemm_kernel<kWgrad>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs * THREADS < 128 * REGS_LOW + (THREADS - 128) * REGS_HIGH) {
            *why = "the register split does not fit the kernel's launch allocation";
            return cudaErrorInvalidConfiguration;
        }
        e = cudaFuncSetAttribute(moe_gemm_kernel<kWgrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    const int64_t sms = num_sms();
    return launch_pdl(moe_gemm_kernel<kWgrad>, (unsigned)(tiles < sms ? tiles : sms), THREADS, SMEM,
                      s, ta, tb, args);
}

Args common_args(const MoeGemm &m) {
    Args a = {};
    a.offsets = m.offsets;
    a.experts = (int)m.experts;
    a.capacity = (int)m.capacity;
    a.sa = m.sa;
    a.sb = m.sb;
    a.d = m.d;
    a.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
    a.status = device_status_word();
    a.lose = take_lost_copies();
    return a;
}

// Whether the kernel that puts the weights on the tensor cores' rows takes a
// call, by the rows an expert on average (what the host knows of the routing is
// the capacity, padding included) and the contraction's blocks.  That kernel's time
// over this one's, mean of 8 to 256 experts and 512 to 8192 columns, rows routed at
// random (fprop / dgrad):
//   rows            0.25          1            4            8           16           24
//    4 blocks      - / 1.27    - / 1.72    - / 1.86     - / 1.88     - / 1.94     - / 2.01
//    8 blocks   0.99 / 0.97  1.10 / 1.05  1.15 / 1.11  1.17 / 1.13  1.26 / 1.22  1.37 / 1.33
//   10          0.88 / 0.89  0.94 / 0.97  1.00 / 1.02                1.16 / 1.15
//   14          0.81 / 0.83  0.87 / 0.89  0.97 / 0.98                1.06 / 1.07
//   16          0.87 / 0.85  0.93 / 0.95  0.99 / 1.00  1.01 / 1.01  1.05 / 1.04  1.11 / 1.10
//   32          0.80 / 0.80  0.91 / 0.90  0.98 / 0.97  0.99 / 0.98  1.02 / 1.01  1.06 / 1.05
//   64             - / 0.76    - / 0.87    - / 0.95     - / 0.96     - / 0.98     - / 1.03
// Single shapes lie up to a fifth to either side; the limit of 16 leaves room for the
// padding.  With 24 rows at any depth as the rule, 832 calls took 1.08 times the
// better kernel's time on average and 2.2 at most; so, 1.01 and 1.23.
// FP8LINEAR_MOE_FEW=0/1 overrides.
bool few_rows(const MoeGemm &m, int depth) {
    const char *env = getenv("FP8LINEAR_MOE_FEW");
    if (env != nullptr) return atoi(env) == 1;
    return m.capacity <= (depth >= 16 ? 16 : depth >= 10 ? 1 : 0) * m.experts;
}

// Output tiles of fprop and dgrad at most: every expert may end in a tile of its own.
int64_t most_tiles(const MoeGemm &m, int64_t cols) {
    const int64_t ends = m.experts < m.capacity ? m.experts : m.capacity;
    return (m.capacity / BM + ends) * ((cols + BN - 1) / BN);
}

}  // namespace

namespace {

// fprop and dgrad: A [capacity, K] times each expert's K-deep rows of B
// [b_rows, b_cols].
cudaError_t launch_rows(const MoeGemm &m, const Args &p, int64_t K, int64_t b_rows, int64_t b_cols,
                        cudaStream_t s, const char **why) {
    if (few_rows(m, p.depth)) return launch_moe_few(p, m.a, K, m.b, b_rows, b_cols, s, why);
    CUtensorMap ta, tb;
    if (!make_tmap_k128(&ta, m.a, m.capacity, K, BM) ||
        !make_tmap_k128(&tb, m.b, b_rows, b_cols, BN)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    return launch<false>(ta, tb, p, most_tiles(m, p.cols_out), s, why);
}

}  // namespace

cudaError_t launch_moe_fprop(const MoeGemm &m, cudaStream_t s, const char **why) {
    if (m.capacity == 0) return cudaSuccess;
    Args a = common_args(m);
    a.cols_out = (int)m.N;
    a.depth = (int)(m.K / BK);
    a.by = (int)m.N;
    a.sa_row = m.K / BK;
    a.sa_k = 1;
    a.sb_expert = (m.N / BK) * (m.K / BK);
    a.sb_col = m.K / BK;
    a.sb_k = 1;
    return launch_rows(m, a, m.K, m.experts * m.N, m.K, s, why);
}

cudaError_t launch_moe_dgrad(const MoeGemm &m, cudaStream_t s, const char **why) {
    if (m.capacity == 0) return cudaSuccess;
    Args a = common_args(m);
    a.cols_out = (int)m.K;
    a.depth = (int)(m.N / BK);
    a.bx = (int)m.N;
    a.sa_row = m.N / BK;
    a.sa_k = 1;
    a.sb_expert = (m.N / BK) * (m.K / BK);
    a.sb_col = 1;
    a.sb_k = m.K / BK;
    return launch_rows(m, a, m.N, m.K, m.experts * m.N, s, why);
}

cudaError_t launch_moe_wgrad(const MoeGemm &m, cudaStream_t s, const char **why) {
    if (m.capacity == 0)
        return cudaMemsetAsync(m.d, 0, (size_t)(m.experts * m.N * m.K) * sizeof(uint16_t), s);
    CUtensorMap ta, tb;
    if (!make_tmap_k128(&ta, m.a, m.N, m.capacity, BM) ||
        !make_tmap_k128(&tb, m.b, m.K, m.capacity, BN)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    Args a = common_args(m);
    a.rows_out = (int)m.N;
    a.cols_out = (int)m.K;
    a.sa_k = m.N;
    a.sb_k = m.K;
    const int64_t tiles = m.experts * (m.N / BM) * ((m.K + BN - 1) / BN);
    return launch<true>(ta, tb, a, tiles, s, why);
}

}  // namespace fp8
