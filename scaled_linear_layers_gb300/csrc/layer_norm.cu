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
// (bf16 -> E4M3) and 6 (bf16 backward) bytes an element.  A row is held in
// the registers of TPR threads, EPT elements each, so it is read once for the
// mean, the squares about the mean (a second sum over registers: no
// cancellation) and the output.  The threads walk over rows with the same
// columns each time: w and b stay in registers, the backward's column sums
// too, and the next row's loads are issued before this row's sums are formed.
// All sums are fp32.
#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

// Elements of a row held by one thread in the register kernels.
constexpr int EPT = 16;
constexpr int kWideThreads = 1024;  // of the kernels for rows too wide for registers

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
};

struct NormBwdArgs {
    const void *dy, *x;
    int64_t lddy, ldx;
    const void *w;  // nullable
    int param_f32;
    int64_t rows;
    int cols;
    const float *mean, *rstd;
    void *dx;        // nullable
    float *partial;  // [2][ctas][cols]: dw then db of each CTA's rows; nullable
};

constexpr int block_threads(int tpr) { return tpr < 128 ? 128 : tpr; }

__device__ __forceinline__ void amax_commit(uint32_t m, float *amax) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0 && m != 0)
        atomicMax(reinterpret_cast<unsigned int *>(amax), m);
}

// TPR threads to a row; a block holds block_threads(TPR) / TPR rows at a time.
template <typename T, bool VECTOR, int TPR>
__global__ void __launch_bounds__(block_threads(TPR), TPR > 512 ? 1 : 512 / block_threads(TPR))
    norm_fwd_kernel(const NormArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V, NV = EPT / V, RPB = block_threads(TPR) / TPR;
    __shared__ float red[2][TPR > 32 ? TPR / 32 : 1];
    const int t = threadIdx.x % TPR;
    const int C = a.cols;
    const float inv_c = 1.f / (float)C;
    pdl_wait_prior();
    pdl_allow_next();

    const T *x = reinterpret_cast<const T *>(a.x);
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    typename RV::Raw nxt[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * V;
            nxt[j] = r < a.rows && c < C ? RV::load(x + r * a.ldx + c) : RV::zero();
        }
    };
    fetch(row);
    float w[EPT], b[EPT];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (j * TPR + t) * V + i;
            w[j * V + i] = a.w != nullptr && c < C ? load_param(a.w, a.param_f32, c) : 1.f;
            b[j * V + i] = a.b != nullptr && c < C ? load_param(a.b, a.param_f32, c) : 0.f;
        }
    const float si = a.yq != nullptr ? *a.scale_inv : 0.f;
    uint32_t m = 0;

    // every thread of a block makes the same number of turns (the sums below
    // are block-wide); a row past the end is computed from zeros, not stored
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.rows; first += step, row += step) {
        float f[EPT];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[V];
            RV::unpack(nxt[j], u);
#pragma unroll
            for (int i = 0; i < V; ++i) f[j * V + i] = u[i];
        }
        fetch(row + step);
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < EPT; ++e) s[0] += f[e];  // columns past C hold zero
        row_sum<TPR, 1>(s, red[0]);
        const float mean = s[0] * inv_c;
        float q[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = f[j * V + i] - mean;
                f[j * V + i] = d;
                if ((j * TPR + t) * V < C) q[0] = fmaf(d, d, q[0]);
            }
        row_sum<TPR, 1>(q, red[1]);
        const float rstd = 1.f / sqrtf(fmaf(q[0], inv_c, a.eps));
        if (row < a.rows) {
            if (t == 0) {
                if (a.mean != nullptr) a.mean[row] = mean;
                if (a.rstd != nullptr) a.rstd[row] = rstd;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + t) * V;
                if (c < C) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o[i] = fmaf(f[j * V + i] * rstd, w[j * V + i], b[j * V + i]);
                    if (a.y != nullptr) RV::store(reinterpret_cast<T *>(a.y) + row * C + c, o);
                    if (a.amax != nullptr) {
#pragma unroll
                        for (int i = 0; i < V; ++i) m = max(m, abs_bits(o[i]));
                    }
                    if (a.yq != nullptr) {
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = __fmul_rn(o[i], si);
                        RV::store_e4m3(a.yq + row * C + c, o);
                    }
                }
            }
        }
    }
    if (a.amax != nullptr) amax_commit(m, a.amax);
}

// Rows too wide for registers: one block to a row, three passes over it (the
// second and third find it in L2).
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_fwd_wide_kernel(const NormArgs a) {
    __shared__ float red[2][kWideThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    const int C = a.cols;
    const float inv_c = 1.f / (float)C;
    const float si = a.yq != nullptr ? *a.scale_inv : 0.f;
    uint32_t m = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < C; c += kWideThreads) s[0] += elem_to_float(x[c]);
        row_sum<kWideThreads, 1>(s, red[0]);
        const float mean = s[0] * inv_c;
        float q[1] = {0.f};
        for (int c = threadIdx.x; c < C; c += kWideThreads) {
            const float d = elem_to_float(x[c]) - mean;
            q[0] = fmaf(d, d, q[0]);
        }
        row_sum<kWideThreads, 1>(q, red[1]);
        const float rstd = 1.f / sqrtf(fmaf(q[0], inv_c, a.eps));
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < C; c += kWideThreads) {
            const float w = a.w != nullptr ? load_param(a.w, a.param_f32, c) : 1.f;
            const float b = a.b != nullptr ? load_param(a.b, a.param_f32, c) : 0.f;
            float o[1] = {fmaf((elem_to_float(x[c]) - mean) * rstd, w, b)};
            if (a.y != nullptr) float_to_elem(reinterpret_cast<T *>(a.y) + row * C + c, o[0]);
            m = max(m, abs_bits(o[0]));
            if (a.yq != nullptr) {
                o[0] = __fmul_rn(o[0], si);
                RowVec<T, false>::store_e4m3(a.yq + row * C + c, o);
            }
        }
    }
    if (a.amax != nullptr) amax_commit(m, a.amax);
}

// The same walk for the gradient; a block's column sums stay in registers and
// leave once, at its end.  With several rows in a block (TPR = 32) its warps'
// sums meet in shared memory first.
template <typename T, bool VECTOR, int TPR>
__global__ void __launch_bounds__(block_threads(TPR), TPR > 256 ? 1 : 512 / block_threads(TPR))
    norm_bwd_kernel(const NormBwdArgs a) {
    using RV = RowVec<T, VECTOR>;
    constexpr int V = RV::V, NV = EPT / V, RPB = block_threads(TPR) / TPR;
    __shared__ float red[2][2 * (TPR > 32 ? TPR / 32 : 1)];
    __shared__ float sums[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * EPT : 1];
    const int t = threadIdx.x % TPR;
    const int C = a.cols;
    const float inv_c = 1.f / (float)C;
    pdl_wait_prior();
    pdl_allow_next();

    const T *x = reinterpret_cast<const T *>(a.x), *dy = reinterpret_cast<const T *>(a.dy);
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    typename RV::Raw nx[NV], ng[NV];
    float nmean, nrstd;
    auto fetch = [&](int64_t r) {
        const bool in = r < a.rows;
        nmean = in ? a.mean[r] : 0.f;
        nrstd = in ? a.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * V;
            nx[j] = in && c < C ? RV::load(x + r * a.ldx + c) : RV::zero();
            ng[j] = in && c < C ? RV::load(dy + r * a.lddy + c) : RV::zero();
        }
    };
    fetch(row);
    float w[EPT], dw[EPT], db[EPT];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (j * TPR + t) * V + i;
            w[j * V + i] = a.w != nullptr && c < C ? load_param(a.w, a.param_f32, c) : 1.f;
            dw[j * V + i] = db[j * V + i] = 0.f;
        }

    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.rows;
         first += step, row += step, ++turn) {
        typename RV::Raw cx[NV], cg[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) cx[j] = nx[j], cg[j] = ng[j];
        const float mean = nmean, rstd = nrstd;
        fetch(row + step);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = (j * TPR + t) * V < C;
            float fx[V], fg[V];
            RV::unpack(cx[j], fx);
            RV::unpack(cg[j], fg);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = j * V + i;
                // columns and rows past the end hold dy = 0 and add nothing,
                // but their xhat is kept finite too
                const float h = in ? (fx[i] - mean) * rstd : 0.f;
                const float wg = w[e] * fg[i];
                s[0] += wg;
                s[1] = fmaf(wg, h, s[1]);
                dw[e] = fmaf(fg[i], h, dw[e]);
                db[e] += fg[i];
            }
        }
        row_sum<TPR, 2>(s, red[turn & 1]);
        if (a.dx != nullptr && row < a.rows) {
            const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + t) * V;
                if (c < C) {
                    float fx[V], fg[V], o[V];
                    RV::unpack(cx[j], fx);
                    RV::unpack(cg[j], fg);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float h = (fx[i] - mean) * rstd;
                        o[i] = rstd * (fmaf(w[j * V + i], fg[i], -m1) - h * m2);
                    }
                    RV::store(reinterpret_cast<T *>(a.dx) + row * C + c, o);
                }
            }
        }
    }
    if (a.partial == nullptr) return;
    float *pw = a.partial + (int64_t)blockIdx.x * C;
    float *pb = pw + (int64_t)gridDim.x * C;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (j * TPR + t) * V + i;
                if (c < C) pw[c] = dw[j * V + i], pb[c] = db[j * V + i];
            }
    } else {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    sums[threadIdx.x / TPR][(j * TPR + t) * V + i] =
                        which ? db[j * V + i] : dw[j * V + i];
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += block_threads(TPR)) {
                float v = 0.f;
#pragma unroll
                for (int r = 0; r < RPB; ++r) v += sums[r][c];
                (which ? pb : pw)[c] = v;
            }
        }
    }
}

// Rows too wide for registers: dx with one block to a row (two passes), the
// column sums by blocks of 256 columns x a share of the rows.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_bwd_wide_kernel(const NormBwdArgs a) {
    __shared__ float red[2][2 * kWideThreads / 32];
    pdl_wait_prior();
    pdl_allow_next();
    const int C = a.cols;
    const float inv_c = 1.f / (float)C;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
        const T *dy = reinterpret_cast<const T *>(a.dy) + row * a.lddy;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < C; c += kWideThreads) {
            const float w = a.w != nullptr ? load_param(a.w, a.param_f32, c) : 1.f;
            const float wg = w * elem_to_float(dy[c]);
            s[0] += wg;
            s[1] = fmaf(wg, (elem_to_float(x[c]) - mean) * rstd, s[1]);
        }
        row_sum<kWideThreads, 2>(s, red[turn & 1]);
        const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
        for (int c = threadIdx.x; c < C; c += kWideThreads) {
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
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
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
// of a block takes partials w, w + 8, ... of 32 columns, then the eight warps'
// sums are added in order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float *partial, int parts, int cols,
                                                          void *dw, void *db, int param_f32) {
    __shared__ float acc[8][33];
    pdl_wait_prior();
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    void *out = blockIdx.y ? db : dw;
    if (out == nullptr) return;
    const float *p = partial + (int64_t)blockIdx.y * parts * cols;
    float v = 0.f;
    if (c < cols)
        for (int i = warp; i < parts; i += 8) v += p[(int64_t)i * cols + c];
    acc[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < cols) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += acc[i][lane];
        if (param_f32)
            reinterpret_cast<float *>(out)[c] = v;
        else
            float_to_elem(reinterpret_cast<uint16_t *>(out) + c, v);
    }
}

// Threads to a row: the fewest that hold it (0: none do).  A row of up to 512
// columns is one warp's, so its sums need no barrier.
int threads_for(int64_t cols, int most) {
    for (int tpr : {32, 128, 256, 512, 1024})
        if (tpr <= most && cols <= (int64_t)tpr * EPT) return tpr;
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

template <typename T, bool VECTOR, int TPR>
cudaError_t run_fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int RPB = block_threads(TPR) / TPR;
    int grid = 0;
    cudaError_t e = walk_grid<norm_fwd_kernel<T, VECTOR, TPR>>(block_threads(TPR), (a.rows + RPB - 1) / RPB, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_fwd_kernel<T, VECTOR, TPR>, grid, block_threads(TPR), 0, s, a);
}

template <typename T, bool VECTOR>
cudaError_t pick_fwd(const NormArgs &a, cudaStream_t s) {
    switch (threads_for(a.cols, 1024)) {
    case 32: return run_fwd<T, VECTOR, 32>(a, s);
    case 128: return run_fwd<T, VECTOR, 128>(a, s);
    case 256: return run_fwd<T, VECTOR, 256>(a, s);
    case 512: return run_fwd<T, VECTOR, 512>(a, s);
    case 1024: return run_fwd<T, VECTOR, 1024>(a, s);
    }
    int grid = 0;
    cudaError_t e = walk_grid<norm_fwd_wide_kernel<T>>(kWideThreads, a.rows, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_fwd_wide_kernel<T>, grid, kWideThreads, 0, s, a);
}

template <typename T, bool VECTOR, int TPR>
cudaError_t run_bwd(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    constexpr int RPB = block_threads(TPR) / TPR;
    int grid = 0;
    cudaError_t e = walk_grid<norm_bwd_kernel<T, VECTOR, TPR>>(block_threads(TPR), (a.rows + RPB - 1) / RPB, &grid);
    if (e != cudaSuccess) return e;
    if (grid > kNormMaxPartials) grid = kNormMaxPartials;
    *parts = grid;
    return launch_pdl(norm_bwd_kernel<T, VECTOR, TPR>, grid, block_threads(TPR), 0, s, a);
}

template <typename T, bool VECTOR>
cudaError_t pick_bwd(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    // 1024 threads leave 64 registers each, too few for the column sums
    switch (threads_for(a.cols, 512)) {
    case 32: return run_bwd<T, VECTOR, 32>(a, parts, s);
    case 128: return run_bwd<T, VECTOR, 128>(a, parts, s);
    case 256: return run_bwd<T, VECTOR, 256>(a, parts, s);
    case 512: return run_bwd<T, VECTOR, 512>(a, parts, s);
    }
    int grid = 0;
    cudaError_t e = cudaSuccess;
    if (a.dx != nullptr) {
        e = walk_grid<norm_bwd_wide_kernel<T>>(kWideThreads, a.rows, &grid);
        if (e != cudaSuccess) return e;
        e = launch_pdl(norm_bwd_wide_kernel<T>, grid, kWideThreads, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    if (a.partial == nullptr) return cudaSuccess;
    *parts = a.rows < 64 ? (int)a.rows : 64;
    return launch_pdl(norm_colsum_wide_kernel<T>, dim3((a.cols + 255) / 256, *parts), 256, 0, s, a);
}

// Whether rows of T at p, `ld` apart, can be read 16 bytes at a time.
template <typename T>
bool row_vectors(const void *p, int64_t ld, int64_t cols) {
    return aligned_to(p, 16) && ld * sizeof(T) % 16 == 0 && cols * sizeof(T) % 16 == 0;
}

template <typename T>
cudaError_t norm_fwd_type(const NormArgs &a, cudaStream_t s) {
    const bool vec = row_vectors<T>(a.x, a.ldx, a.cols) &&
                     (a.y == nullptr || aligned_to(a.y, 16)) &&
                     (a.yq == nullptr || aligned_to(a.yq, RowVec<T, true>::V));
    return vec ? pick_fwd<T, true>(a, s) : pick_fwd<T, false>(a, s);
}

template <typename T>
cudaError_t norm_bwd_type(const NormBwdArgs &a, int *parts, cudaStream_t s) {
    const bool vec = row_vectors<T>(a.x, a.ldx, a.cols) && row_vectors<T>(a.dy, a.lddy, a.cols) &&
                     (a.dx == nullptr || aligned_to(a.dx, 16));
    return vec ? pick_bwd<T, true>(a, parts, s) : pick_bwd<T, false>(a, parts, s);
}

}  // namespace

cudaError_t launch_layer_norm(const NormForward &n, cudaStream_t s) {
    if (n.amax != nullptr) {
        cudaError_t e = launch_zero_f32(n.amax, 1, s);
        if (e != cudaSuccess) return e;
    }
    if (n.rows == 0 || n.cols == 0) return cudaSuccess;
    NormArgs a = {n.x, n.ldx, n.w, n.b, n.param_f32, n.rows, (int)n.cols, n.eps,
                  n.y, n.yq, n.scale_inv, n.amax, n.mean, n.rstd};
    return n.x_f32 ? norm_fwd_type<float>(a, s) : norm_fwd_type<uint16_t>(a, s);
}

cudaError_t launch_layer_norm_backward(const NormBackward &n, cudaStream_t s) {
    if (n.cols == 0) return cudaSuccess;
    const bool sums = n.dw != nullptr || n.db != nullptr;
    int parts = 0;
    if (n.rows > 0) {
        NormBwdArgs a = {n.dy, n.x, n.lddy, n.ldx, n.w, n.param_f32, n.rows, (int)n.cols,
                         n.mean, n.rstd, n.dx, sums ? n.workspace : nullptr};
        cudaError_t e = n.x_f32 ? norm_bwd_type<float>(a, &parts, s)
                                : norm_bwd_type<uint16_t>(a, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!sums) return cudaSuccess;
    return launch_pdl(norm_reduce_kernel, dim3((unsigned)((n.cols + 31) / 32), 2), 256, 0, s,
                      (const float *)n.workspace, parts, (int)n.cols, n.dw, n.db, n.param_f32);
}

}  // namespace fp8
