// Layer norm of the rows of x [rows, cols]:
//
//   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps)
//   xhat = (x - mean) rstd,  y = xhat w + b
//
// with y stored in x's type and / or as E4M3 bytes of y * scale_inv (with
// max |y|, for the next step's scale), and its gradient
//
//   dx = rstd (w dy - mean_c(w dy) - xhat mean_c(w dy xhat))
//   dw = sum_r dy xhat,  db = sum_r dy.
//
// Both directions move every element once, so HBM bounds them: 4 (bf16), 3
// (bf16 -> E4M3) and 6 (bf16 backward) bytes an element.  A row is shared by a
// team of TPR threads, EPT elements each, always the same columns: w and b
// stay in registers, and the backward's column sums too.  The mean, the
// squares about the mean (a second sum over registers: no cancellation) and
// the output need one read of the row.  Many rows (norm_*_ring_kernel) come
// through a ring of bulk copies in shared memory, several rows ahead of the
// sums, so the loads in flight do not depend on registers; few rows are loaded
// straight into registers one row ahead.  The backward of wide rows, whose sums
// by column alone would fill the registers, shares a row between the blocks of a
// cluster.  All sums are fp32; the mean's, whose terms cancel, adds leading bits
// and rests apart.
//
// Measured at 16384 x 4096 (device time; share of the copy bandwidth): bf16
// forward 48 us (0.83), to E4M3 40 us (0.75, its amax cleared in a launch of
// its own), backward 68 us (0.88, 5 us of it the reduction over the blocks'
// column sums); fp32 forward 94 us (0.84), backward 132 us (0.90); 8192 columns
// within 0.05 of that; 4096 x 16384 backward bf16 80 us (0.74), fp32 125 us
// (0.95).  What keeps the E4M3 form from its 30 us is the work on a row between
// two barriers (issue slots 60 % busy, DRAM 62 %), which is why elements are
// worked on in pairs and a thread holds as many as fit.  Rows of odd width move
// single elements: bf16 8192 x 8191 forward 74 us (0.53), fp32 89 us (0.89).  One
// row of 4096: 3.5 us, a launch's latency.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

extern std::atomic<uint64_t> g_wait_limit_ns;

namespace {

constexpr int kWideThreads = 1024;  // of the kernels for rows too wide for a team
constexpr int kMaxStages = 8;
constexpr size_t kRingBytes = 208 * 1024;  // of an SM's shared memory, for its blocks' rings

struct NormArgs {
    const void *x;
    int64_t ldx;
    const void *w, *b;  // nullable
    int param_f32;
    int64_t rows;
    int cols;
    float eps;
    void *y;                 // nullable
    uint8_t *yq;             // nullable
    const float *scale_inv;  // with yq
    float *amax;             // nullable, zero on entry
    float *mean, *rstd;      // nullable
    int stages;              // of the ring
    int lose;                // (tests) rows are waited for but not copied
    uint64_t wait_limit_ns;
    unsigned int *status;
};

struct NormBwdArgs {
    const void *dy, *x;
    int64_t lddy, ldx;
    const void *w;  // nullable
    int param_f32;
    int64_t rows;
    int cols, width;  // worked on by the block; of the rows
    const float *mean, *rstd;
    void *dx;        // [rows, width]; nullable
    float *partial;  // [2][parts][width]: dw then db of each part of the rows; nullable
    int stages;
    int lose;        // (tests) rows are waited for but not copied
    uint64_t wait_limit_ns;
    unsigned int *status;
};

// A block is one team, or eight teams of a warp.
constexpr int block_threads(int tpr) { return tpr == 32 ? 256 : tpr; }
constexpr int teams(int tpr) { return block_threads(tpr) / tpr; }
// Blocks an SM should hold, by the registers that a thread needs; the
// backward's also by the partial sums that each block leaves.
constexpr int fwd_blocks(int tpr, int ept) {
    return tpr > 512 ? 1 : (ept > 16 ? 512 : ept > 8 ? 768 : 1024) / block_threads(tpr);
}
constexpr int bwd_blocks(int tpr) { return tpr > 256 ? 1 : tpr == 128 ? 3 : 2; }

__device__ __forceinline__ void amax_commit(float v, float *amax) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
    if ((threadIdx.x & 31) == 0 && m != 0)
        atomicMax(reinterpret_cast<unsigned int *>(amax), m);
}

// 16-byte-multiple copy global -> shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A team's ring: `stages` slots of `slot` bytes with a barrier each.  The
// dynamic shared memory holds all teams' slots, then their barriers, then the
// block's give-up flag.  After a wait that ran out the status word says so and
// the block walks on, without further copies, over what the slots hold: its
// outputs are invalid, but its barriers stay paired; the copies on their way
// are waited for at the end.
struct Ring {
    uint8_t *data;
    uint64_t *bars;
    volatile int *abort;
    int stages;
    uint32_t slot;
    int failed_slot;  // of this thread's first wait that ran out; -1: none did
    uint32_t failed_phase;

    __device__ __forceinline__ void wait(int at, uint32_t phase, uint64_t limit_ns,
                                         unsigned int *status) {
        if (!mbar_wait_bounded(&bars[at], phase, abort, limit_ns, kStatusTimeoutTma, status) &&
            failed_slot < 0) {
            failed_slot = at;
            failed_phase = phase;
        }
    }

    // (leader, which requests nothing after a wait of its own that ran out)
    __device__ __forceinline__ bool open() const { return failed_slot < 0; }

    // The leader waited for all it requested, or, after a failure, for all but
    // what went into the slots from that one on: bounded waits for those.
    __device__ __forceinline__ void settle(unsigned int *status) {
        if (failed_slot < 0) return;
        volatile int no_abort = 0;
        for (int i = 0; i < stages; ++i) {
            const int at = failed_slot + i;
            const bool wrapped = at >= stages;
            mbar_wait_bounded(&bars[wrapped ? at - stages : at], failed_phase ^ (wrapped ? 1u : 0u),
                              &no_abort, 10000000ull, kStatusTimeoutTma, status);
        }
    }

    template <int TEAMS>
    __device__ __forceinline__ void init(uint8_t *smem, int n, uint32_t slot_bytes, int team,
                                         bool leader) {
        stages = n;
        slot = slot_bytes;
        failed_slot = -1;
        data = smem + (size_t)team * n * slot_bytes;
        uint64_t *all = reinterpret_cast<uint64_t *>(smem + (size_t)TEAMS * n * slot_bytes);
        bars = all + team * n;
        abort = reinterpret_cast<volatile int *>(all + TEAMS * n);
        if (leader) {
            for (int i = 0; i < n; ++i) mbar_init(&bars[i], 1);
            if (team == 0) *abort = 0;
            fence_mbarrier_init();
        }
        __syncthreads();
    }
};

size_t ring_bytes(int team_count, int stages, size_t slot) {
    return (size_t)team_count * stages * (slot + sizeof(uint64_t)) + 16;
}

// A row's place in a slot.  Rows that 16-byte copies fit are copied as they
// are; of others the whole aligned 16-byte groups that hold them, so the row
// starts up to 15 bytes into the slot.  A row whose groups reach past its
// tensor (its first or last) is not copied: it is read where it is.
template <typename T, bool VECTOR>
struct RowSource {
    const T *p;
    int64_t ld;
    uint32_t bytes;     // of a row
    uintptr_t lo, hi;   // of the tensor

    __device__ __forceinline__ RowSource(const void *base, int64_t rows, int64_t stride, int cols) {
        p = reinterpret_cast<const T *>(base);
        ld = stride;
        bytes = (uint32_t)cols * sizeof(T);
        lo = reinterpret_cast<uintptr_t>(p);
        hi = reinterpret_cast<uintptr_t>(p + (rows - 1) * ld + cols);
    }
    static __host__ __device__ __forceinline__ uint32_t slot(uint32_t row_bytes) {
        return VECTOR ? row_bytes : ((row_bytes + 15u) & ~15u) + 16u;
    }
    __device__ __forceinline__ bool copied(int64_t r, uintptr_t &first, uintptr_t &end) const {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p + r * ld);
        first = VECTOR ? at : at & ~uintptr_t(15);
        end = VECTOR ? at + bytes : (at + bytes + 15) & ~uintptr_t(15);
        return VECTOR || (first >= lo && end <= hi);
    }
    // (leader) bytes that request() will bring
    __device__ __forceinline__ uint32_t size(int64_t r) const {
        uintptr_t first, end;
        return copied(r, first, end) ? (uint32_t)(end - first) : 0u;
    }
    __device__ __forceinline__ void request(int64_t r, uint8_t *to, uint64_t *bar) const {
        uintptr_t first, end;
        if (copied(r, first, end))
            bulk_load(to, reinterpret_cast<const void *>(first), (uint32_t)(end - first), bar);
    }
    __device__ __forceinline__ const T *row(int64_t r, const uint8_t *from) const {
        uintptr_t first, end;
        if (VECTOR) return reinterpret_cast<const T *>(from);
        const T *global = p + r * ld;
        return copied(r, first, end)
                   ? reinterpret_cast<const T *>(from + (reinterpret_cast<uintptr_t>(global) & 15u))
                   : global;
    }
};

// Columns of a row that each block of a cluster works on, the last of them the
// rest: whole 16-byte groups, and groups of 8 parameters.
__host__ __device__ constexpr int cluster_share(int width, int ctas) {
    return ((width + ctas - 1) / ctas + 15) / 16 * 16;
}

// 8 bytes to the shared memory of a block of the cluster, counted there.
__device__ __forceinline__ void st_async64(uint32_t to, uint64_t v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                     to),
                 "l"(v), "r"(bar)
                 : "memory");
}

// After a wait for the phase: what other blocks wrote before it is seen.
__device__ __forceinline__ void mbar_acquire_cluster(uint64_t *bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(parity)
        : "memory");
}

// Arms a slot's barrier for `bytes` (a phase without a copy completes at once).
__device__ __forceinline__ void slot_expect(uint64_t *bar, uint32_t bytes) {
    if (bytes > 0) mbar_arrive_expect_tx(bar, bytes);
    else mbar_arrive(bar);
}

// ---------------------------------------------------------------- forward ---

// What a team member does with its elements of one row, two at a time (one at
// a time 16384 x 4096 to E4M3 took 61 us).
// FULL: the row has exactly TPR * EPT columns, so no group is past its end
// (the tests and branches for that are a fifth of the instructions).
template <typename T, bool VECTOR, int TPR, int EPT, bool FULL>
struct NormRow {
    using RV = RowVec<T, VECTOR>;
    static constexpr int V = RV::V, NV = EPT / V, P = EPT / 2;
    uint64_t w[P], b[P];
    float inv_c, si, amax;
    int t;

    static __device__ __forceinline__ int column(int e) {
        return ((e / V) * TPR + threadIdx.x % TPR) * V + e % V;
    }

    static __device__ __forceinline__ bool inside(int cols, int e) {
        return FULL || column(e) < cols;
    }

    __device__ __forceinline__ void init(const NormArgs &a) {
        t = threadIdx.x % TPR;
        inv_c = 1.f / (float)a.cols;
        si = a.yq != nullptr ? *a.scale_inv : 0.f;
        amax = 0.f;
        auto param = [&](const void *p, float none, uint64_t (&to)[P]) {
            float f[EPT];
#pragma unroll
            for (int e = 0; e < EPT; ++e) f[e] = none;
            if (p != nullptr) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (inside(a.cols, j * V))
                        load_params<V>(p, a.param_f32, column(j * V),
                                       reinterpret_cast<float(&)[V]>(f[j * V]));
            }
#pragma unroll
            for (int i = 0; i < P; ++i) to[i] = pair_of(f[2 * i], f[2 * i + 1]);
        };
        param(a.w, 1.f, w);
        param(a.b, 0.f, b);
    }

    // mean of f (columns past the row's end hold zero), leaving f - mean
    __device__ __forceinline__ float centre(const NormArgs &a, uint64_t (&f)[P], float *red) const {
        float s, e = 0.f;
        if constexpr (sizeof(T) == 2) {
            // 8-bit significands: short sums of them rarely round in fp32
            uint64_t p[P];
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = f[i];
#pragma unroll
            for (int h = P / 2; h > 0; h /= 2)
#pragma unroll
                for (int i = 0; i < h; ++i) p[i] = pair_add(p[i], p[i + h]);
            const float2 v = pair_split(p[0]);
            s = v.x + v.y;
        } else {
            s = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 v = pair_split(f[i]);
                add_exact(s, e, v.x);
                add_exact(s, e, v.y);
            }
        }
        const float mean = row_sum_split<TPR>(s, e, red) * inv_c;
        const uint64_t minus = pair_of(-mean, -mean);
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = pair_add(f[i], minus);
        return mean;
    }

    __device__ __forceinline__ float spread(const NormArgs &a, const uint64_t (&f)[P],
                                            float *red) const {
        uint64_t q = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            uint64_t d = f[i];
            if constexpr (V == 1) {
                float2 v = pair_split(d);
                if (!inside(a.cols, 2 * i)) v.x = 0.f;
                if (!inside(a.cols, 2 * i + 1)) v.y = 0.f;
                d = pair_of(v.x, v.y);
            } else if (!inside(a.cols, 2 * i)) {
                continue;
            }
            q = pair_fma(d, d, q);
        }
        const float2 v = pair_split(q);
        float s[1] = {v.x + v.y};
        row_sum<TPR, 1>(s, red);
        return 1.f / sqrtf(fmaf(s[0], inv_c, a.eps));
    }

    __device__ __forceinline__ void store(const NormArgs &a, int64_t row, const uint64_t (&f)[P],
                                          float mean, float rstd) {
        if (t == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        const uint64_t r2 = pair_of(rstd, rstd), s2 = pair_of(si, si);
        float o[EPT];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 v = pair_split(pair_fma(pair_mul(f[i], r2), w[i], b[i]));
            o[2 * i] = v.x, o[2 * i + 1] = v.y;
        }
        auto each = [&](auto act) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (inside(a.cols, j * V))
                    act(row * a.cols + column(j * V), reinterpret_cast<float(&)[V]>(o[j * V]));
        };
        if (a.y != nullptr)
            each([&](int64_t at, float(&u)[V]) { RV::store(reinterpret_cast<T *>(a.y) + at, u); });
        if (a.amax != nullptr)
            each([&](int64_t, float(&u)[V]) {
#pragma unroll
                for (int i = 0; i < V; ++i) amax = max_abs_nan(amax, u[i]);
            });
        if (a.yq != nullptr)
            each([&](int64_t at, float(&u)[V]) {
                if constexpr (V == 1) {
                    u[0] = __fmul_rn(u[0], si);
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float2 v = pair_split(pair_mul(pair_of(u[i], u[i + 1]), s2));
                        u[i] = v.x, u[i + 1] = v.y;
                    }
                }
                RV::store_e4m3(a.yq + at, u);
            });
    }

    // f = the row's elements, from load(j) of each group
    template <typename L>
    static __device__ __forceinline__ void unpack(L load, uint64_t (&f)[P]) {
        float u[EPT];
#pragma unroll
        for (int j = 0; j < NV; ++j) RV::unpack(load(j), reinterpret_cast<float(&)[V]>(u[j * V]));
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = pair_of(u[2 * i], u[2 * i + 1]);
    }
};

// Every thread of a block makes the same number of turns in the loops below
// (the sums may be block-wide); a row past the end is computed from zeros and
// not stored.

template <typename T, bool VECTOR, int TPR, int EPT>
__global__ void __launch_bounds__(block_threads(TPR), fwd_blocks(TPR, EPT))
    norm_fwd_kernel(const NormArgs a) {
    using RV = RowVec<T, VECTOR>;
    using Row = NormRow<T, VECTOR, TPR, EPT, false>;
    __shared__ float red[2][2 * (TPR > 32 ? TPR / 32 : 1)];
    pdl_wait_prior();
    pdl_allow_next();
    const T *x = reinterpret_cast<const T *>(a.x);
    const int64_t step = (int64_t)gridDim.x * teams(TPR);
    int64_t row = (int64_t)blockIdx.x * teams(TPR) + threadIdx.x / TPR;
    typename RV::Raw nxt[Row::NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < Row::NV; ++j) {
            const int c = Row::column(j * Row::V);
            nxt[j] = r < a.rows && c < a.cols ? RV::load(x + r * a.ldx + c) : RV::zero();
        }
    };
    fetch(row);
    Row n;
    n.init(a);
    for (int64_t first = (int64_t)blockIdx.x * teams(TPR); first < a.rows;
         first += step, row += step) {
        uint64_t f[Row::P];
        Row::unpack([&](int j) { return nxt[j]; }, f);
        fetch(row + step);
        const float mean = n.centre(a, f, red[0]);
        const float rstd = n.spread(a, f, red[1]);
        if (row < a.rows) n.store(a, row, f, mean, rstd);
    }
    if (a.amax != nullptr) amax_commit(n.amax, a.amax);
}

template <typename T, bool VECTOR, int TPR, int EPT, bool FULL>
__global__ void __launch_bounds__(block_threads(TPR), fwd_blocks(TPR, EPT))
    norm_fwd_ring_kernel(const NormArgs a) {
    using RV = RowVec<T, VECTOR>;
    using Row = NormRow<T, VECTOR, TPR, EPT, FULL>;
    using Source = RowSource<T, VECTOR>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][2 * (TPR > 32 ? TPR / 32 : 1)];
    const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const Source x(a.x, a.rows, a.ldx, a.cols);
    Ring ring = {};
    ring.init<teams(TPR)>(smem, a.stages, Source::slot(x.bytes), team, t == 0);
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t step = (int64_t)gridDim.x * teams(TPR);
    int64_t row = (int64_t)blockIdx.x * teams(TPR) + team;
    auto request = [&](int64_t r, int slot) {
        if (r < a.rows && ring.open()) {
            slot_expect(&ring.bars[slot], x.size(r));
            if (!a.lose) x.request(r, ring.data + slot * ring.slot, &ring.bars[slot]);
        }
    };
    if (t == 0)
        for (int i = 0; i < a.stages; ++i) request(row + i * step, i);
    Row n;
    n.init(a);
    int slot = 0;
    uint32_t phase = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams(TPR); first < a.rows;
         first += step, row += step) {
        const bool in = row < a.rows;
        if (in)
            ring.wait(slot, phase, a.wait_limit_ns, a.status);
        const T *src = x.row(row, ring.data + slot * ring.slot);
        uint64_t f[Row::P];
        Row::unpack(
            [&](int j) {
                return in && Row::inside(a.cols, j * Row::V) ? RV::load(src + Row::column(j * Row::V))
                                                             : RV::zero();
            },
            f);
        const float mean = n.centre(a, f, red[0]);
        // the sum needed every member's elements, so the slot has been read
        if (t == 0) request(row + a.stages * step, slot);
        const float rstd = n.spread(a, f, red[1]);
        if (in) n.store(a, row, f, mean, rstd);
        if (++slot == a.stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (t == 0) ring.settle(a.status);
    if (a.amax != nullptr) amax_commit(n.amax, a.amax);
}

// Rows too wide for a team: one block to a row, three passes over it (the
// second and third find it in L2).  Columns are unsigned here and below: up to
// 2^31 - 1 of them, the step past the last passes 2^31.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_fwd_wide_kernel(const NormArgs a) {
    __shared__ float red[2][2 * kWideThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    const unsigned C = a.cols;
    const float inv_c = 1.f / (float)C;
    const float si = a.yq != nullptr ? *a.scale_inv : 0.f;
    float m = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
        float s = 0.f, e = 0.f;
        for (unsigned c = threadIdx.x; c < C; c += kWideThreads) add_exact(s, e, elem_to_float(x[c]));
        const float mean = row_sum_split<kWideThreads>(s, e, red[0]) * inv_c;
        float q[1] = {0.f};
        for (unsigned c = threadIdx.x; c < C; c += kWideThreads) {
            const float d = elem_to_float(x[c]) - mean;
            q[0] = fmaf(d, d, q[0]);
        }
        row_sum<kWideThreads, 1>(q, red[1]);
        const float rstd = 1.f / sqrtf(fmaf(q[0], inv_c, a.eps));
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        for (unsigned c = threadIdx.x; c < C; c += kWideThreads) {
            const float w = a.w != nullptr ? load_param(a.w, a.param_f32, c) : 1.f;
            const float b = a.b != nullptr ? load_param(a.b, a.param_f32, c) : 0.f;
            float o[1] = {fmaf((elem_to_float(x[c]) - mean) * rstd, w, b)};
            if (a.y != nullptr) float_to_elem(reinterpret_cast<T *>(a.y) + row * C + c, o[0]);
            m = max_abs_nan(m, o[0]);
            if (a.yq != nullptr) {
                o[0] = __fmul_rn(o[0], si);
                RowVec<T, false>::store_e4m3(a.yq + row * C + c, o);
            }
        }
    }
    if (a.amax != nullptr) amax_commit(m, a.amax);
}

// The statistics of rows without columns: 0 / 0.
__global__ void __launch_bounds__(256) norm_no_columns_kernel(float *mean, float *rstd,
                                                              int64_t rows) {
    pdl_wait_prior();
    pdl_allow_next();
    const float nan = __int_as_float(0x7FFFFFFF);
    for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows;
         r += (int64_t)gridDim.x * 256) {
        if (mean != nullptr) mean[r] = nan;
        if (rstd != nullptr) rstd[r] = nan;
    }
}

// --------------------------------------------------------------- backward ---

// A team member's part of the gradient: its columns' sums so far.
template <typename T, bool VECTOR, int TPR, int EPT, bool FULL>
struct NormBwdRow {
    using RV = RowVec<T, VECTOR>;
    using Raw = typename RV::Raw;
    static constexpr int V = RV::V, NV = EPT / V, P = EPT / 2;
    // pairs of elements come from one group, or from two single elements
    static constexpr int STEP = V > 1 ? 1 : 2, PAIRS = V > 1 ? V / 2 : 1;
    // 32 columns' sums leave no registers for their weights: L1 holds them
    static constexpr bool W_IN_REGISTERS = EPT <= 16;
    uint64_t w[W_IN_REGISTERS ? P : 1], dw[P], db[P];
    float inv_c;

    static __device__ __forceinline__ int column(int e) {
        return ((e / V) * TPR + threadIdx.x % TPR) * V + e % V;
    }

    static __device__ __forceinline__ bool inside(int cols, int e) {
        return FULL || column(e) < cols;
    }

    // the weights of the elements of groups j to j + STEP - 1
    __device__ __forceinline__ void weights(const NormBwdArgs &a, int j, uint64_t (&p)[PAIRS]) const {
        if constexpr (W_IN_REGISTERS) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) p[i] = w[j * V / 2 + i];
        } else {
            load_weights(a, j, p);
        }
    }

    static __device__ __forceinline__ void load_weights(const NormBwdArgs &a, int j,
                                                        uint64_t (&p)[PAIRS]) {
        float f[V * STEP];
#pragma unroll
        for (int e = 0; e < V * STEP; ++e) f[e] = 1.f;
        if (a.w != nullptr) {
            if constexpr (VECTOR) {
                if (inside(a.cols, j * V)) load_params<V>(a.w, a.param_f32, column(j * V), f);
            } else {
#pragma unroll
                for (int e = 0; e < STEP; ++e)
                    if (inside(a.cols, j + e)) f[e] = load_param(a.w, a.param_f32, column(j + e));
            }
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) p[i] = pair_of(f[2 * i], f[2 * i + 1]);
    }

    __device__ __forceinline__ void init(const NormBwdArgs &a) {
        inv_c = 1.f / (float)a.width;
#pragma unroll
        for (int i = 0; i < P; ++i) dw[i] = db[i] = 0;
        if constexpr (W_IN_REGISTERS) {
#pragma unroll
            for (int j = 0; j < NV; j += STEP)
                load_weights(a, j, reinterpret_cast<uint64_t(&)[PAIRS]>(w[j * V / 2]));
        }
    }

    // the elements of groups j to j + STEP - 1, which load() gives
    template <typename L>
    static __device__ __forceinline__ void unpack(L load, int j, uint64_t (&p)[PAIRS]) {
        float f[V * STEP];
        RV::unpack(load(j), reinterpret_cast<float(&)[V]>(f[0]));
        if constexpr (STEP == 2) RV::unpack(load(j + 1), reinterpret_cast<float(&)[V]>(f[1]));
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) p[i] = pair_of(f[2 * i], f[2 * i + 1]);
    }

    // the row's sums of w dy and w dy xhat, and its share of the columns' (a
    // row or column past the end holds dy = 0)
    template <typename LX, typename LG>
    __device__ __forceinline__ void sums(const NormBwdArgs &a, LX load_x, LG load_dy, float mean,
                                         float rstd, float (&s)[2]) {
        const uint64_t minus = pair_of(-mean, -mean), r2 = pair_of(rstd, rstd);
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int j = 0; j < NV; j += STEP) {
            uint64_t x[PAIRS], g[PAIRS], wt[PAIRS];
            unpack(load_x, j, x);
            unpack(load_dy, j, g);
            weights(a, j, wt);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const int e = j * V / 2 + i;
                const uint64_t h = pair_mul(pair_add(x[i], minus), r2);
                const uint64_t wg = pair_mul(wt[i], g[i]);
                s0 = pair_add(s0, wg);
                s1 = pair_fma(wg, h, s1);
                dw[e] = pair_fma(g[i], h, dw[e]);
                db[e] = pair_add(db[e], g[i]);
            }
        }
        const float2 u = pair_split(s0), v = pair_split(s1);
        s[0] = u.x + u.y;
        s[1] = v.x + v.y;
    }

    template <typename LX, typename LG>
    __device__ __forceinline__ void store(const NormBwdArgs &a, int64_t row, LX load_x, LG load_dy,
                                          float mean, float rstd, const float (&s)[2]) const {
        const float m1 = -(s[0] * inv_c), m2 = -(s[1] * inv_c);
        const uint64_t minus = pair_of(-mean, -mean), r2 = pair_of(rstd, rstd);
        const uint64_t m12 = pair_of(m1, m1), m22 = pair_of(m2, m2);
#pragma unroll
        for (int j = 0; j < NV; j += STEP) {
            uint64_t x[PAIRS], g[PAIRS], wt[PAIRS];
            unpack(load_x, j, x);
            unpack(load_dy, j, g);
            weights(a, j, wt);
            float o[V * STEP];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const uint64_t h = pair_mul(pair_add(x[i], minus), r2);
                const uint64_t d = pair_fma(h, m22, pair_fma(wt[i], g[i], m12));
                const float2 v = pair_split(pair_mul(r2, d));
                o[2 * i] = v.x, o[2 * i + 1] = v.y;
            }
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
                if (inside(a.cols, (j + k) * V))
                    RV::store(reinterpret_cast<T *>(a.dx) + row * a.width + column((j + k) * V),
                              reinterpret_cast<float(&)[V]>(o[k * V]));
            }
        }
    }

    // group j of the sums; 16 bytes at a time (rows of groups of V > 1 have a
    // multiple of 4 columns and start on 16 bytes, and so do their sums)
    static __device__ __forceinline__ void put(float *to, const uint64_t (&sum)[P], int j) {
        if constexpr (V == 1) {
            const float2 v = pair_split(sum[j / 2]);
            *to = j % 2 ? v.y : v.x;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float2 u = pair_split(sum[(j * V + i) / 2]);
                const float2 v = pair_split(sum[(j * V + i) / 2 + 1]);
                *reinterpret_cast<float4 *>(to + i) = make_float4(u.x, u.y, v.x, v.y);
            }
        }
    }

    // the column sums of part `part` of the rows; with several teams in a block
    // theirs meet in `meet` [teams][TPR * EPT] first
    __device__ __forceinline__ void commit(const NormBwdArgs &a, int part, int parts,
                                           float *meet) const {
        float *pw = a.partial + (int64_t)part * a.width;
        float *pb = pw + (int64_t)parts * a.width;
        if constexpr (teams(TPR) == 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!inside(a.cols, j * V)) continue;
                put(pw + column(j * V), dw, j);
                put(pb + column(j * V), db, j);
            }
        } else {
            constexpr int WIDTH = TPR * EPT;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    const float2 v = pair_split(which ? db[e / 2] : dw[e / 2]);
                    meet[(threadIdx.x / TPR) * WIDTH + column(e)] = e % 2 ? v.y : v.x;
                }
                __syncthreads();
                for (int c = threadIdx.x; c < a.cols; c += block_threads(TPR)) {
                    float v = 0.f;
#pragma unroll
                    for (int r = 0; r < teams(TPR); ++r) v += meet[r * WIDTH + c];
                    (which ? pb : pw)[c] = v;
                }
            }
        }
    }
};

template <typename T, bool VECTOR, int TPR, int EPT>
__global__ void __launch_bounds__(block_threads(TPR), bwd_blocks(TPR))
    norm_bwd_kernel(const NormBwdArgs a) {
    using Row = NormBwdRow<T, VECTOR, TPR, EPT, false>;
    using RV = typename Row::RV;
    using Raw = typename Row::Raw;
    __shared__ float red[2][2 * (TPR > 32 ? TPR / 32 : 1)];
    __shared__ float meet[teams(TPR) > 1 ? teams(TPR) * TPR * EPT : 1];
    pdl_wait_prior();
    pdl_allow_next();
    const int t = threadIdx.x % TPR;
    const T *x = reinterpret_cast<const T *>(a.x), *dy = reinterpret_cast<const T *>(a.dy);
    const int64_t step = (int64_t)gridDim.x * teams(TPR);
    int64_t row = (int64_t)blockIdx.x * teams(TPR) + threadIdx.x / TPR;
    Raw nx[Row::NV], ng[Row::NV];
    float nmean, nrstd;
    auto fetch = [&](int64_t r) {
        const bool in = r < a.rows;
        nmean = in ? a.mean[r] : 0.f;
        nrstd = in ? a.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < Row::NV; ++j) {
            const int c = (j * TPR + t) * Row::V;
            nx[j] = in && c < a.cols ? RV::load(x + r * a.ldx + c) : RV::zero();
            ng[j] = in && c < a.cols ? RV::load(dy + r * a.lddy + c) : RV::zero();
        }
    };
    fetch(row);
    Row n;
    n.init(a);
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams(TPR); first < a.rows;
         first += step, row += step, ++turn) {
        Raw cx[Row::NV], cg[Row::NV];
#pragma unroll
        for (int j = 0; j < Row::NV; ++j) cx[j] = nx[j], cg[j] = ng[j];
        const float mean = nmean, rstd = nrstd;
        fetch(row + step);
        auto lx = [&](int j) { return cx[j]; };
        auto lg = [&](int j) { return cg[j]; };
        float s[2];
        n.sums(a, lx, lg, mean, rstd, s);
        row_sum<TPR, 2>(s, red[turn & 1]);
        if (a.dx != nullptr && row < a.rows) n.store(a, row, lx, lg, mean, rstd, s);
    }
    if (a.partial != nullptr) n.commit(a, blockIdx.x, gridDim.x, meet);
}

// A slot holds the row's x, then its dy; it is read twice, for the sums and
// for dx, and asked to be filled again one turn later, when the next row's
// sums show that every member is past it.
template <typename T, bool VECTOR, int TPR, int EPT, bool FULL>
__global__ void __launch_bounds__(block_threads(TPR), bwd_blocks(TPR))
    norm_bwd_ring_kernel(const NormBwdArgs a) {
    using Row = NormBwdRow<T, VECTOR, TPR, EPT, FULL>;
    using RV = typename Row::RV;
    using Source = RowSource<T, VECTOR>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][2 * (TPR > 32 ? TPR / 32 : 1)];
    const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const Source x(a.x, a.rows, a.ldx, a.cols), dy(a.dy, a.rows, a.lddy, a.cols);
    const uint32_t half = Source::slot(x.bytes);
    Ring ring = {};
    ring.init<teams(TPR)>(smem, a.stages, 2 * half, team, t == 0);
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t step = (int64_t)gridDim.x * teams(TPR);
    int64_t row = (int64_t)blockIdx.x * teams(TPR) + team;
    auto request = [&](int64_t r, int slot) {
        if (r < a.rows && ring.open()) {
            uint8_t *to = ring.data + slot * ring.slot;
            slot_expect(&ring.bars[slot], x.size(r) + dy.size(r));
            if (a.lose) return;
            x.request(r, to, &ring.bars[slot]);
            dy.request(r, to + half, &ring.bars[slot]);
        }
    };
    if (t == 0)
        for (int i = 0; i < a.stages; ++i) request(row + i * step, i);
    float nmean = row < a.rows ? a.mean[row] : 0.f, nrstd = row < a.rows ? a.rstd[row] : 0.f;
    Row n;
    n.init(a);
    int slot = 0, before = a.stages - 1, turn = 0;
    uint32_t phase = 0;
    for (int64_t first = (int64_t)blockIdx.x * teams(TPR); first < a.rows;
         first += step, row += step, ++turn) {
        const bool in = row < a.rows;
        const float mean = nmean, rstd = nrstd;
        if (row + step < a.rows) nmean = a.mean[row + step], nrstd = a.rstd[row + step];
        if (in)
            ring.wait(slot, phase, a.wait_limit_ns, a.status);
        const T *sx = x.row(row, ring.data + slot * ring.slot);
        const T *sg = dy.row(row, ring.data + slot * ring.slot + half);
        auto load = [&](const T *p, int j) {
            return in && Row::inside(a.cols, j * Row::V) ? RV::load(p + Row::column(j * Row::V))
                                                         : RV::zero();
        };
        auto lx = [&](int j) { return load(sx, j); };
        auto lg = [&](int j) { return load(sg, j); };
        float s[2];
        n.sums(a, lx, lg, in ? mean : 0.f, in ? rstd : 0.f, s);
        row_sum<TPR, 2>(s, red[turn & 1]);
        if (t == 0 && turn > 0) request(row + (a.stages - 1) * step, before);
        if (a.dx != nullptr && in) n.store(a, row, lx, lg, mean, rstd, s);
        before = slot;
        if (++slot == a.stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (t == 0) ring.settle(a.status);
    // every copy has arrived and been read: the teams' sums meet in the ring
    if (a.partial != nullptr) n.commit(a, blockIdx.x, gridDim.x, reinterpret_cast<float *>(smem));
}

// Rows too wide for one block's registers and ring: each is shared by a
// cluster of CTAS blocks, a block's columns always the same, which tell each
// other their parts of the row's two sums.  A row's sums are told before the
// row before it is finished, so their way between the blocks is not waited for.
// Sums of up to four turns are on their way: a block tells those of turn i + 2
// when it has turn i's from all, who then are past turn i - 2.
template <typename T, bool VECTOR, int CTAS, int TPR, int EPT, bool FULL>
__global__ void __launch_bounds__(TPR, 1) __cluster_dims__(CTAS, 1, 1)
    norm_bwd_cluster_kernel(NormBwdArgs a) {
    using Row = NormBwdRow<T, VECTOR, TPR, EPT, FULL>;
    using RV = typename Row::RV;
    using Source = RowSource<T, VECTOR>;
    static_assert(teams(TPR) == 1, "one row at a time");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][2 * (TPR / 32)];
    __shared__ __align__(16) uint64_t theirs[4][CTAS];
    __shared__ uint64_t told[4];
    const int t = threadIdx.x, rank = (int)cluster_ctarank();
    const int first = rank * cluster_share(a.width, CTAS);
    a.cols = min(cluster_share(a.width, CTAS), a.width - first);
    a.x = reinterpret_cast<const T *>(a.x) + first;
    a.dy = reinterpret_cast<const T *>(a.dy) + first;
    if (a.w != nullptr)
        a.w = reinterpret_cast<const uint8_t *>(a.w) + (size_t)first * (a.param_f32 ? 4 : 2);
    if (a.dx != nullptr) a.dx = reinterpret_cast<T *>(a.dx) + first;
    if (a.partial != nullptr) a.partial += first;
    const Source x(a.x, a.rows, a.ldx, a.cols), dy(a.dy, a.rows, a.lddy, a.cols);
    const uint32_t half = Source::slot(x.bytes);
    if (t == 0)
        for (int i = 0; i < 4; ++i) mbar_init(&told[i], 1);
    Ring ring = {};
    ring.init<1>(smem, a.stages, 2 * half, 0, t == 0);
    cluster_sync_all();
    pdl_wait_prior();
    pdl_allow_next();
    const int64_t step = gridDim.x / CTAS;
    int64_t row = blockIdx.x / CTAS;
    auto request = [&](int64_t r, int slot) {
        if (r < a.rows && ring.open()) {
            uint8_t *to = ring.data + slot * ring.slot;
            slot_expect(&ring.bars[slot], x.size(r) + dy.size(r));
            if (a.lose && rank == 0) return;  // the others then wait for this block's sums
            x.request(r, to, &ring.bars[slot]);
            dy.request(r, to + half, &ring.bars[slot]);
        }
    };
    if (t == 0)
        for (int i = 0; i < a.stages; ++i) request(row + i * step, i);
    Row n;
    n.init(a);
    auto load = [&](const T *p, int j) {
        return Row::inside(a.cols, j * Row::V) ? RV::load(p + Row::column(j * Row::V)) : RV::zero();
    };
    auto in_x = [&](int64_t r, int slot) { return x.row(r, ring.data + slot * ring.slot); };
    auto in_dy = [&](int64_t r, int slot) { return dy.row(r, ring.data + slot * ring.slot + half); };
    int ahead = 0;  // slot of the next row to tell the sums of
    uint32_t phase = 0;
    auto tell = [&](int64_t r, float mean, float rstd, int turn) {
        ring.wait(ahead, phase, a.wait_limit_ns, a.status);
        const T *sx = in_x(r, ahead), *sg = in_dy(r, ahead);
        float s[2];
        n.sums(a, [&](int j) { return load(sx, j); }, [&](int j) { return load(sg, j); }, mean, rstd,
               s);
        // (after a wait that ran out, up to the turn before, the barrier may not
        // have turned, and nothing paces this block: it tells no more, and the
        // others' waits run out in turn)
        const bool tells = t < CTAS && !*ring.abort;
        row_sum<TPR, 2>(s, red[turn & 1]);
        if (t == 0 && tells)
            mbar_arrive_expect_tx(&told[turn & 3], CTAS * sizeof(uint64_t));
        if (tells)
            st_async64(mapa_shared(smem_u32(&theirs[turn & 3][rank]), t), pair_of(s[0], s[1]),
                       mapa_shared(smem_u32(&told[turn & 3]), t));
        if (++ahead == a.stages) {
            ahead = 0;
            phase ^= 1u;
        }
    };
    float mean = row < a.rows ? a.mean[row] : 0.f, rstd = row < a.rows ? a.rstd[row] : 0.f;
    float nmean = 0.f, nrstd = 0.f;
    if (row + step < a.rows) nmean = a.mean[row + step], nrstd = a.rstd[row + step];
    if (row < a.rows) tell(row, mean, rstd, 0);
    int slot = 0, before = 0;
    for (int turn = 0; row < a.rows; row += step, ++turn) {
        const float hmean = nmean, hrstd = nrstd;
        if (row + 2 * step < a.rows) nmean = a.mean[row + 2 * step], nrstd = a.rstd[row + 2 * step];
        if (row + step < a.rows) {
            tell(row + step, hmean, hrstd, turn + 1);
            // every member is past the row before
            if (t == 0 && turn > 0) request(row + (a.stages - 1) * step, before);
        }
        const uint32_t parity = (uint32_t)(turn >> 2) & 1u;
        if (mbar_wait_bounded(&told[turn & 3], parity, ring.abort, a.wait_limit_ns,
                              kStatusTimeoutTma, a.status))
            mbar_acquire_cluster(&told[turn & 3], parity);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CTAS; ++i) {
            const float2 v = pair_split(*(volatile uint64_t *)&theirs[turn & 3][i]);
            s[0] += v.x;
            s[1] += v.y;
        }
        if (a.dx != nullptr) {
            const T *sx = in_x(row, slot), *sg = in_dy(row, slot);
            n.store(a, row, [&](int j) { return load(sx, j); }, [&](int j) { return load(sg, j); },
                    mean, rstd, s);
        }
        mean = hmean, rstd = hrstd;
        before = slot;
        if (++slot == a.stages) slot = 0;
    }
    if (t == 0) ring.settle(a.status);
    if (a.partial != nullptr) n.commit(a, blockIdx.x / CTAS, gridDim.x / CTAS, nullptr);
    cluster_sync_all();  // no block leaves while another may still write to it
    // A block that has had every row's sums has nothing on its way to it.  One
    // that gave up may have: what the others told before they came here lands
    // within a few us.
    if (t == 0 && *ring.abort) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) __nanosleep(1000);
    }
}

// Rows too wide for a team: dx with one block to a row (two passes), the
// column sums by blocks of 256 columns x a share of the rows.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_bwd_wide_kernel(const NormBwdArgs a) {
    __shared__ float red[2][2 * kWideThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    const unsigned C = a.cols;
    const float inv_c = 1.f / (float)C;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
        const T *dy = reinterpret_cast<const T *>(a.dy) + row * a.lddy;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.f, 0.f};
        for (unsigned c = threadIdx.x; c < C; c += kWideThreads) {
            const float w = a.w != nullptr ? load_param(a.w, a.param_f32, c) : 1.f;
            const float wg = w * elem_to_float(dy[c]);
            s[0] += wg;
            s[1] = fmaf(wg, (elem_to_float(x[c]) - mean) * rstd, s[1]);
        }
        row_sum<kWideThreads, 2>(s, red[turn & 1]);
        const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
        for (unsigned c = threadIdx.x; c < C; c += kWideThreads) {
            const float w = a.w != nullptr ? load_param(a.w, a.param_f32, c) : 1.f;
            const float h = (elem_to_float(x[c]) - mean) * rstd;
            float_to_elem(reinterpret_cast<T *>(a.dx) + row * C + c,
                          rstd * (fmaf(w, elem_to_float(dy[c]), -m1) - h * m2));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) norm_colsum_wide_kernel(const NormBwdArgs a) {
    pdl_wait_prior();
    pdl_allow_next();
    const unsigned c = blockIdx.x * 256 + threadIdx.x;
    if (c >= (unsigned)a.cols) return;
    const T *x = reinterpret_cast<const T *>(a.x), *dy = reinterpret_cast<const T *>(a.dy);
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float g = elem_to_float(dy[r * a.lddy + c]);
        dw = fmaf(g, (elem_to_float(x[r * a.ldx + c]) - a.mean[r]) * a.rstd[r], dw);
        db += g;
    }
    float *pw = a.partial + (int64_t)blockIdx.y * a.cols;
    pw[c] = dw;
    pw[(int64_t)gridDim.y * a.cols + c] = db;
}

// dw, db = the partial sums of `parts` blocks, added in a fixed order: warp w
// of a block takes partials w, w + 32, ... of 32 columns, then the warps' sums
// are added in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *partial, int parts,
                                                           int cols, void *dw, void *db,
                                                           int param_f32) {
    __shared__ float acc[32][33];
    pdl_wait_prior();
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned c = blockIdx.x * 32 + lane;
    void *out = blockIdx.y ? db : dw;
    if (out == nullptr) return;
    const float *p = partial + (int64_t)blockIdx.y * parts * cols;
    float v = 0.f;
    if (c < (unsigned)cols) {
#pragma unroll 8
        for (int i = warp; i < parts; i += 32) v += p[(int64_t)i * cols + c];
    }
    acc[warp][lane] = v;
    __syncthreads();
    // transposed: warp w sums column w
    v = warp_sum(acc[lane][warp]);
    const unsigned col = blockIdx.x * 32 + warp;
    if (lane == 0 && col < (unsigned)cols) {
        if (param_f32)
            reinterpret_cast<float *>(out)[col] = v;
        else
            float_to_elem(reinterpret_cast<uint16_t *>(out) + col, v);
    }
}

// ------------------------------------------------------------------- host ---

// Threads to a row: the fewest, up to `most`, that hold it with `ept` elements
// each (0: none do).  A team of one warp needs no barrier for its sums.
int threads_for(int64_t cols, int ept, int most) {
    for (int tpr : {32, 128, 256, 512, 1024})
        if (tpr <= most && cols <= (int64_t)tpr * ept) return tpr;
    return 0;
}

// Blocks of a persistent walk over `units` groups of rows: what fits the GPU
// at once.
template <auto KERNEL>
cudaError_t walk_grid(int threads, int64_t units, int *grid) {
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(threads, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t g = (int64_t)num_sms() * per_sm;
    *grid = (int)(g < units ? g : units);
    return cudaSuccess;
}

struct RingPlan {
    int grid, stages;  // stages 0: no ring
    size_t bytes;
};

// A ring pays once every team has more than one row, and needs room for two
// slots; blocks that would leave fewer than three are traded for slots.  The
// dynamic shared memory is at least `least` bytes.
template <auto KERNEL>
cudaError_t plan_ring(int threads, int team_count, int64_t rows, size_t slot, RingPlan *r,
                      size_t least = 0) {
    r->stages = 0;
    int blocks = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(threads, &blocks);
    if (e != cudaSuccess) return e;
    int64_t stages = 0;
    for (;; --blocks) {
        stages = ((int64_t)(kRingBytes / blocks) - 1024) / (int64_t)(team_count * (slot + 8));
        if (stages >= 3 || blocks == 1) break;
    }
    const int64_t units = (rows + team_count - 1) / team_count;
    const int64_t grid = (int64_t)num_sms() * blocks;
    if (stages < 2 || units <= grid) return cudaSuccess;
    r->grid = (int)grid;
    r->stages = (int)std::min<int64_t>(stages, kMaxStages);
    r->bytes = std::max(ring_bytes(team_count, r->stages, slot), least);
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kRingBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    return cudaSuccess;
}

template <typename T, bool VECTOR, int TPR, int EPT, bool FULL = false>
cudaError_t run_fwd_ring(NormArgs a, cudaStream_t s, bool *done) {
    if constexpr (VECTOR && !FULL && TPR * EPT % 1024 == 0)
        if (a.cols == TPR * EPT) return run_fwd_ring<T, true, TPR, EPT, true>(a, s, done);
    constexpr auto ring = norm_fwd_ring_kernel<T, VECTOR, TPR, EPT, FULL>;
    RingPlan r;
    cudaError_t e = plan_ring<ring>(block_threads(TPR), teams(TPR), a.rows,
                                    RowSource<T, VECTOR>::slot(a.cols * sizeof(T)), &r);
    if (e != cudaSuccess || r.stages == 0) return e;
    a.stages = r.stages;
    *done = true;
    return launch_pdl(ring, r.grid, block_threads(TPR), r.bytes, s, a);
}

// Many rows: 32 elements to a thread where the row fills them, so that the
// sums over the team cost less an element (16384 x 4096 to E4M3: 39 us; with 16 elements 53).
// Rows that 16-byte copies do not fit gain by the ring (bf16 16384 x 333: 13 us,
// straight into registers 21; 8192 x 8191: 74 and 97) except where a warp would
// work on 32 single elements a thread (16384 x 1001: 30 and 23).
template <typename T, bool VECTOR>
cudaError_t pick_fwd_ring(const NormArgs &a, cudaStream_t s, bool *done) {
    if (a.cols <= 512) return run_fwd_ring<T, VECTOR, 32, 16>(a, s, done);
    if (a.cols <= 1024) {
        if constexpr (VECTOR) return run_fwd_ring<T, VECTOR, 32, 32>(a, s, done);
        else return cudaSuccess;
    }
    if (a.cols <= 2048) return run_fwd_ring<T, VECTOR, 128, 16>(a, s, done);
    if (a.cols <= 4096) return run_fwd_ring<T, VECTOR, 128, 32>(a, s, done);
    if (a.cols <= 8192) return run_fwd_ring<T, VECTOR, 256, 32>(a, s, done);
    if (a.cols <= 16384) return run_fwd_ring<T, VECTOR, 512, 32>(a, s, done);
    return cudaSuccess;
}

template <typename T, bool VECTOR, int TPR, int EPT>
cudaError_t run_fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int THREADS = block_threads(TPR);
    constexpr auto kernel = norm_fwd_kernel<T, VECTOR, TPR, EPT>;
    int grid = 0;
    cudaError_t e = walk_grid<kernel>(THREADS, (a.rows + teams(TPR) - 1) / teams(TPR), &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, THREADS, 0, s, a);
}

template <typename T, bool VECTOR>
cudaError_t pick_fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int EPT = VECTOR ? 16 : 8;
    bool done = false;
    cudaError_t re = pick_fwd_ring<T, VECTOR>(a, s, &done);
    if (re != cudaSuccess || done) return re;
    switch (threads_for(a.cols, EPT, 1024)) {
    case 32: return run_fwd<T, VECTOR, 32, EPT>(a, s);
    case 128: return run_fwd<T, VECTOR, 128, EPT>(a, s);
    case 256: return run_fwd<T, VECTOR, 256, EPT>(a, s);
    case 512: return run_fwd<T, VECTOR, 512, EPT>(a, s);
    case 1024: return run_fwd<T, VECTOR, 1024, EPT>(a, s);
    }
    int grid = 0;
    cudaError_t e = walk_grid<norm_fwd_wide_kernel<T>>(kWideThreads, a.rows, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_fwd_wide_kernel<T>, grid, kWideThreads, 0, s, a);
}

template <typename T, bool VECTOR, int TPR, int EPT, bool FULL = false>
cudaError_t run_bwd_ring(NormBwdArgs a, int *parts, cudaStream_t s, bool *done) {
    if constexpr (VECTOR && !FULL && TPR * EPT % 1024 == 0)
        if (a.cols == TPR * EPT) return run_bwd_ring<T, true, TPR, EPT, true>(a, parts, s, done);
    constexpr auto ring = norm_bwd_ring_kernel<T, VECTOR, TPR, EPT, FULL>;
    RingPlan r;
    cudaError_t e =
        plan_ring<ring>(block_threads(TPR), teams(TPR), a.rows,
                        2 * (size_t)RowSource<T, VECTOR>::slot(a.cols * sizeof(T)), &r,
                        teams(TPR) > 1 ? teams(TPR) * TPR * EPT * sizeof(float) : 0);
    if (e != cudaSuccess || r.stages == 0) return e;
    a.stages = r.stages;
    *parts = r.grid = std::min(r.grid, kNormMaxPartials);
    *done = true;
    return launch_pdl(ring, r.grid, block_threads(TPR), r.bytes, s, a);
}

// Rows that 16-byte copies do not fit: narrow ones gain by the ring (bf16 16384
// x 333: 18 us, straight into registers 28), wide ones only in fp32 (16384 x
// 1999: 66 and 77; bf16 66 and 56, whose single elements are taken apart twice
// from a slot but once from registers; at 1001 columns neither gains).
template <typename T, bool VECTOR>
cudaError_t pick_bwd_ring(const NormBwdArgs &a, int *parts, cudaStream_t s, bool *done) {
    if (a.cols <= 512) return run_bwd_ring<T, VECTOR, 32, 16>(a, parts, s, done);
    if constexpr (VECTOR) {
        if (a.cols <= 1024) {
            if constexpr (sizeof(T) == 2) return run_bwd_ring<T, VECTOR, 32, 32>(a, parts, s, done);
            else return run_bwd_ring<T, VECTOR, 128, 8>(a, parts, s, done);
        }
    }
    if constexpr (VECTOR || sizeof(T) == 4) {
        if (a.cols <= 1024) return cudaSuccess;
        if (a.cols <= 2048) return run_bwd_ring<T, VECTOR, 128, 16>(a, parts, s, done);
        if (a.cols <= 4096) return run_bwd_ring<T, VECTOR, 256, 16>(a, parts, s, done);
        if (a.cols <= 8192) return run_bwd_ring<T, VECTOR, 512, 16>(a, parts, s, done);
    }
    return cudaSuccess;
}

// Slots of the ring of a cluster's block.
template <typename T, bool VECTOR>
int cluster_slots(int width, int ctas, size_t *slot) {
    *slot = 2 * (size_t)RowSource<T, VECTOR>::slot(cluster_share(width, ctas) * sizeof(T));
    return (int)std::min<size_t>((kRingBytes - 1024) / (*slot + sizeof(uint64_t)), kMaxStages);
}

// A cluster of CTAS blocks to a row.  Its ring has three slots or more: the row
// told about, the row finished, one on its way.
template <typename T, bool VECTOR, int CTAS, int TPR, int EPT, bool FULL = false>
cudaError_t run_bwd_cluster(NormBwdArgs a, int *parts, cudaStream_t s) {
    if constexpr (VECTOR && !FULL)
        if (a.width == CTAS * TPR * EPT)
            return run_bwd_cluster<T, true, CTAS, TPR, EPT, true>(a, parts, s);
    constexpr auto kernel = norm_bwd_cluster_kernel<T, VECTOR, CTAS, TPR, EPT, FULL>;
    static_assert(3 * (2 * (TPR * EPT * sizeof(T) + 16) + 8) + 1024 <= kRingBytes, "three slots");
    size_t slot = 0;
    a.stages = cluster_slots<T, VECTOR>(a.width, CTAS, &slot);
    int clusters = 0;
    cudaError_t e = clusters_resident<kernel>(CTAS, TPR, kRingBytes, &clusters);
    if (e != cudaSuccess) return e;
    *parts = (int)std::min<int64_t>(std::min(clusters, kNormMaxPartials), a.rows);
    return launch_pdl(kernel, *parts * CTAS, TPR, ring_bytes(1, a.stages, slot), s, a);
}

// Two blocks as far as their registers go; four also where two leave only three
// slots (fp32 4096 x 16384: 125 us, by two 151; x 12000: by two 98, by four
// 127), unless single elements bound the row (x 16383: 187 and 184).
template <typename T, bool VECTOR>
cudaError_t pick_bwd_cluster(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    if (a.width > 16384) return run_bwd_cluster<T, VECTOR, 4, 512, 16>(a, parts, s);
    if constexpr (VECTOR && sizeof(T) == 4) {
        size_t slot = 0;
        if (cluster_slots<T, VECTOR>(a.width, 2, &slot) < 4)
            return run_bwd_cluster<T, VECTOR, 4, 512, 8>(a, parts, s);
    }
    return run_bwd_cluster<T, VECTOR, 2, 512, 16>(a, parts, s);
}

template <typename T, bool VECTOR, int TPR, int EPT>
cudaError_t run_bwd(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    constexpr int THREADS = block_threads(TPR);
    constexpr auto kernel = norm_bwd_kernel<T, VECTOR, TPR, EPT>;
    int grid = 0;
    cudaError_t e = walk_grid<kernel>(THREADS, (a.rows + teams(TPR) - 1) / teams(TPR), &grid);
    if (e != cudaSuccess) return e;
    *parts = grid = std::min(grid, kNormMaxPartials);
    return launch_pdl(kernel, grid, THREADS, 0, s, a);
}

template <typename T, bool VECTOR>
cudaError_t pick_bwd(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    constexpr int EPT = VECTOR ? 16 : 8;
    bool done = false;
    cudaError_t re = pick_bwd_ring<T, VECTOR>(a, parts, s, &done);
    if (re != cudaSuccess || done) return re;
    if (a.cols > 8192 && a.cols <= 32768) return pick_bwd_cluster<T, VECTOR>(a, parts, s);
    // 1024 threads leave 64 registers each, too few for the column sums
    switch (threads_for(a.cols, EPT, 512)) {
    case 32: return run_bwd<T, VECTOR, 32, EPT>(a, parts, s);
    case 128: return run_bwd<T, VECTOR, 128, EPT>(a, parts, s);
    case 256: return run_bwd<T, VECTOR, 256, EPT>(a, parts, s);
    case 512: return run_bwd<T, VECTOR, 512, EPT>(a, parts, s);
    }
    if constexpr (!VECTOR)
        if (a.cols <= 8192) return run_bwd<T, VECTOR, 512, 2 * EPT>(a, parts, s);
    // the column sums first: dx may be written over dy or x
    cudaError_t e = cudaSuccess;
    if (a.partial != nullptr) {
        *parts = a.rows < 64 ? (int)a.rows : 64;
        e = launch_pdl(norm_colsum_wide_kernel<T>, dim3((a.cols + 255u) / 256, *parts), 256, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    if (a.dx == nullptr) return cudaSuccess;
    int grid = 0;
    e = walk_grid<norm_bwd_wide_kernel<T>>(kWideThreads, a.rows, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_bwd_wide_kernel<T>, grid, kWideThreads, 0, s, a);
}

// Whether rows of T at p, `ld` apart, can be read 16 bytes at a time.
template <typename T>
bool row_vectors(const void *p, int64_t ld, int64_t cols) {
    return aligned_to(p, 16) && ld * sizeof(T) % 16 == 0 && cols * sizeof(T) % 16 == 0;
}

template <typename T>
cudaError_t norm_fwd_type(const NormArgs &a, cudaStream_t s) {
    const bool vec = row_vectors<T>(a.x, a.ldx, a.cols) && aligned_to(a.w, 16) &&
                     aligned_to(a.b, 16) &&
                     (a.y == nullptr || aligned_to(a.y, 16)) &&
                     (a.yq == nullptr || aligned_to(a.yq, RowVec<T, true>::V));
    return vec ? pick_fwd<T, true>(a, s) : pick_fwd<T, false>(a, s);
}

template <typename T>
cudaError_t norm_bwd_type(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    const bool vec = row_vectors<T>(a.x, a.ldx, a.cols) && row_vectors<T>(a.dy, a.lddy, a.cols) &&
                     aligned_to(a.w, 16) && (a.dx == nullptr || aligned_to(a.dx, 16));
    return vec ? pick_bwd<T, true>(a, parts, s) : pick_bwd<T, false>(a, parts, s);
}

int take_lost_copies() {
    if (tl_lose_copies == 0) return 0;
    --tl_lose_copies;
    return 1;
}

}  // namespace

cudaError_t launch_layer_norm(const NormForward &n, cudaStream_t s) {
    if (n.amax != nullptr) {
        cudaError_t e = launch_zero_f32(n.amax, 1, s);
        if (e != cudaSuccess) return e;
    }
    if (n.rows == 0) return cudaSuccess;
    if (n.cols == 0) {
        if (n.mean == nullptr && n.rstd == nullptr) return cudaSuccess;
        const int64_t grid = std::min<int64_t>((n.rows + 255) / 256, 8 * (int64_t)num_sms());
        return launch_pdl(norm_no_columns_kernel, (int)grid, 256, 0, s, n.mean, n.rstd, n.rows);
    }
    NormArgs a = {n.x, n.ldx, n.w, n.b, n.param_f32, n.rows, (int)n.cols, n.eps,
                  n.y, n.yq, n.scale_inv, n.amax, n.mean, n.rstd, 0, take_lost_copies(),
                  g_wait_limit_ns.load(std::memory_order_relaxed), device_status_word()};
    return n.x_f32 ? norm_fwd_type<float>(a, s) : norm_fwd_type<uint16_t>(a, s);
}

cudaError_t launch_layer_norm_backward(const NormBackward &n, cudaStream_t s) {
    if (n.cols == 0) return cudaSuccess;
    const bool sums = n.dw != nullptr || n.db != nullptr;
    int parts = 0;
    if (n.rows > 0) {
        NormBwdArgs a = {n.dy, n.x, n.lddy, n.ldx, n.w, n.param_f32, n.rows, (int)n.cols,
                         (int)n.cols, n.mean, n.rstd, n.dx, sums ? n.workspace : nullptr, 0,
                         take_lost_copies(),
                         g_wait_limit_ns.load(std::memory_order_relaxed), device_status_word()};
        cudaError_t e = n.x_f32 ? norm_bwd_type<float>(a, &parts, s)
                                : norm_bwd_type<uint16_t>(a, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!sums) return cudaSuccess;
    return launch_pdl(norm_reduce_kernel, dim3((unsigned)((n.cols + 31) / 32), 2), 1024, 0, s,
                      (const float *)n.workspace, parts, (int)n.cols, n.dw, n.db, n.param_f32);
}

}  // namespace fp8
