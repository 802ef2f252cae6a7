// The gated activation between an expert's two linears, and its gradient from
// an 8-bit checkpoint of its input.
//
//   h = (gate | up), each cols wide;  s = 1 / (1 + exp(-gate))
//   forward:   y = gate s up, as rows and/or as E4M3 under a scale for each
//              1x128 tile (the next linear's operand under the block recipe);
//              h as E4M3 under 1x128 scales (the checkpoint)
//   backward:  dgate = dy up (s + gate s (1 - s)),  dup = dy gate s,  and y
//              again, from the checkpoint or from h
//
// A tile's scales are those of fp8_quantize's block recipe (amax/448, taken as
// a multiply by 448/amax); y is quantised before its rounding to rows, so the
// cast adds the only rounding.  All arithmetic is fp32; bf16 rows take the
// hardware's exponential and division (2^-21 or so, far below bf16's 2^-9),
// fp32 rows the exact ones.
//
// Everything moves once and is bound by HBM: 7.1 bytes an element forward to
// E4M3 with the checkpoint, 10.1 backward from it (bf16).  Sixteen lanes share
// a tile, eight neighbouring columns each, so that a tile's maximum is four
// shuffles and a bf16 lane's loads are 16 bytes; rows that do not lie on 16
// bytes go element by element, a tile's columns dealt out to the lanes in turn.
#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kTile = 128, kLanes = 16, kPer = kTile / kLanes;
constexpr int kThreads = 256, kTeams = kThreads / kLanes;

__device__ __forceinline__ float sigmoid(float x, uint16_t) {
    return __fdividef(1.f, 1.f + __expf(-x));
}
__device__ __forceinline__ float sigmoid(float x, float) { return __fdiv_rn(1.f, 1.f + expf(-x)); }

// Two e4m3 bytes as fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{.reg .b16 l, u; mov.b32 {l, u}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, u;}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// A lane's eight columns of one tile: neighbours when VECTOR, else every 16th
// from `lane` on, those below `left` (the tile's columns).
template <typename T, bool VECTOR>
__device__ __forceinline__ void load_cols(const T *p, int lane, int left, float (&f)[kPer]) {
    if constexpr (VECTOR) {
        using R = RowVec<T, true>;
#pragma unroll
        for (int i = 0; i < kPer; i += R::V) {
            typename R::Raw raw = R::zero();
            if (kPer * lane < left) raw = R::load(p + kPer * lane + i);
            float v[R::V];
            R::unpack(raw, v);
#pragma unroll
            for (int k = 0; k < R::V; ++k) f[i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            f[i] = lane + kLanes * i < left ? elem_to_float(p[lane + kLanes * i]) : 0.f;
    }
}

template <typename T, bool VECTOR>
__device__ __forceinline__ void store_cols(T *p, int lane, int left, const float (&f)[kPer]) {
    if constexpr (VECTOR) {
        using R = RowVec<T, true>;
        if (kPer * lane >= left) return;
#pragma unroll
        for (int i = 0; i < kPer; i += R::V) {
            float v[R::V];
#pragma unroll
            for (int k = 0; k < R::V; ++k) v[k] = f[i + k];
            R::store(p + kPer * lane + i, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + kLanes * i < left) float_to_elem(p + lane + kLanes * i, f[i]);
    }
}

template <bool VECTOR>
__device__ __forceinline__ void store_e4m3(uint8_t *p, int lane, int left, const float (&f)[kPer],
                                           float inv) {
    uint32_t two[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i)
        two[i] = cvt_e4m3x2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
    if constexpr (VECTOR) {
        if (kPer * lane < left)
            *reinterpret_cast<uint2 *>(p + kPer * lane) =
                make_uint2(two[0] | (two[1] << 16), two[2] | (two[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + kLanes * i < left)
                p[lane + kLanes * i] = (uint8_t)(two[i / 2] >> (8 * (i & 1)));
    }
}

template <bool VECTOR>
__device__ __forceinline__ void load_e4m3(const uint8_t *p, int lane, int left, float scale,
                                          float (&f)[kPer]) {
    uint32_t two[kPer / 2] = {};
    if constexpr (VECTOR) {
        if (kPer * lane < left) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p + kPer * lane);
            two[0] = w.x & 0xFFFFu, two[1] = w.x >> 16, two[2] = w.y & 0xFFFFu, two[3] = w.y >> 16;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + kLanes * i < left)
                two[i / 2] |= (uint32_t)p[lane + kLanes * i] << (8 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const float2 v = e4m3x2_to_float2(two[i]);
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// The largest |v| of a tile, as a bit pattern, in all of its sixteen lanes.
__device__ __forceinline__ uint32_t tile_amax(const float (&f)[kPer]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, abs_bits(f[i]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
}

// Walks the tiles of [rows, tiles] in steps of the grid's teams: a division at
// the start, then whole rows and the rest of a step at a time.
struct TileWalk {
    int64_t row;
    int tile;
    __device__ __forceinline__ TileWalk(int tiles) {
        const int64_t first = (int64_t)blockIdx.x * kTeams + threadIdx.x / kLanes;
        row = first / tiles;
        tile = (int)(first - row * tiles);
    }
    __device__ __forceinline__ void next(int tiles, int64_t step_rows, int step_tiles) {
        row += step_rows;
        tile += step_tiles;
        if (tile >= tiles) {
            tile -= tiles;
            ++row;
        }
    }
};

struct Walk {
    int tiles, step_tiles;
    int64_t step_rows;
};

__device__ __forceinline__ int64_t live_rows(const int32_t *live, int64_t rows) {
    return live == nullptr ? rows : min(rows, (int64_t)max(0, *live));
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluForward a, const Walk w) {
    pdl_wait_prior();
    pdl_allow_next();
    const int lane = threadIdx.x % kLanes, lane32 = threadIdx.x & 31;
    const int64_t rows = live_rows(a.live, a.rows);
    const T *h = reinterpret_cast<const T *>(a.h);
    T *y = reinterpret_cast<T *>(a.y);
    TileWalk at(w.tiles);
    // both halves of a warp go on until neither has a tile left
    while (__any_sync(0xFFFFFFFFu, at.row < rows)) {
        const bool on = at.row < rows;
        const int64_t c0 = (int64_t)at.tile * kTile;
        const int left = on ? (int)min((int64_t)kTile, a.cols - c0) : 0;
        float g[kPer], u[kPer], v[kPer];
        load_cols<T, VECTOR>(h + at.row * a.ldh + c0, lane, left, g);
        load_cols<T, VECTOR>(h + at.row * a.ldh + a.cols + c0, lane, left, u);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = g[i] * sigmoid(g[i], T()) * u[i];
        if (y != nullptr) store_cols<T, VECTOR>(y + at.row * a.cols + c0, lane, left, v);
        // the three tiles' scales are formed by three lanes side by side
        const uint32_t mg = a.hq != nullptr ? tile_amax(g) : 0u;
        const uint32_t mu = a.hq != nullptr ? tile_amax(u) : 0u;
        const uint32_t mv = a.yq != nullptr ? tile_amax(v) : 0u;
        float s, inv;
        scales_from_amax(__uint_as_float(lane == 0 ? mg : lane == 1 ? mu : mv), s, inv);
        const float ig = __shfl_sync(0xFFFFFFFFu, inv, lane32 & 16);
        const float iu = __shfl_sync(0xFFFFFFFFu, inv, (lane32 & 16) + 1);
        const float iv = __shfl_sync(0xFFFFFFFFu, inv, (lane32 & 16) + 2);
        if (a.hq != nullptr) {
            uint8_t *q = a.hq + at.row * 2 * a.cols + c0;
            store_e4m3<VECTOR>(q, lane, left, g, ig);
            store_e4m3<VECTOR>(q + a.cols, lane, left, u, iu);
            if (on && lane < 2) a.h_scale[(at.row * 2 + lane) * w.tiles + at.tile] = s;
        }
        if (a.yq != nullptr) {
            store_e4m3<VECTOR>(a.yq + at.row * a.cols + c0, lane, left, v, iv);
            if (on && lane == 2) a.y_scale[at.row * w.tiles + at.tile] = s;
        }
        at.next(w.tiles, w.step_rows, w.step_tiles);
    }
}

template <typename T, bool VECTOR, bool SAVED>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const SwigluBackward a, const Walk w) {
    pdl_wait_prior();
    pdl_allow_next();
    const int lane = threadIdx.x % kLanes;
    const int64_t rows = live_rows(a.live, a.rows);
    const T *dy = reinterpret_cast<const T *>(a.dy);
    T *dh = reinterpret_cast<T *>(a.dh), *y = reinterpret_cast<T *>(a.y);
    TileWalk at(w.tiles);
    for (; at.row < rows; at.next(w.tiles, w.step_rows, w.step_tiles)) {
        const int64_t c0 = (int64_t)at.tile * kTile;
        const int left = (int)min((int64_t)kTile, a.cols - c0);
        float g[kPer], u[kPer], d[kPer];
        load_cols<T, VECTOR>(dy + at.row * a.lddy + c0, lane, left, d);
        if constexpr (SAVED) {
            const uint8_t *q = reinterpret_cast<const uint8_t *>(a.h) + at.row * a.ldh + c0;
            const float *s = a.h_scale + at.row * 2 * w.tiles + at.tile;
            load_e4m3<VECTOR>(q, lane, left, s[0], g);
            load_e4m3<VECTOR>(q + a.cols, lane, left, s[w.tiles], u);
        } else {
            const T *h = reinterpret_cast<const T *>(a.h) + at.row * a.ldh + c0;
            load_cols<T, VECTOR>(h, lane, left, g);
            load_cols<T, VECTOR>(h + a.cols, lane, left, u);
        }
        float v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float s = sigmoid(g[i], T()), act = g[i] * s;
            v[i] = act * u[i];
            g[i] = d[i] * u[i] * (s + act * (1.f - s));
            u[i] = d[i] * act;
        }
        T *out = dh + at.row * 2 * a.cols + c0;
        store_cols<T, VECTOR>(out, lane, left, g);
        store_cols<T, VECTOR>(out + a.cols, lane, left, u);
        if (y != nullptr) store_cols<T, VECTOR>(y + at.row * a.cols + c0, lane, left, v);
    }
}

// As many blocks as the device holds at once, or fewer for fewer tiles.
template <auto KERNEL>
cudaError_t plan(int64_t rows, int64_t cols, Walk *w, int *grid) {
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(kThreads, &per_sm);
    if (e != cudaSuccess) return e;
    w->tiles = (int)((cols + kTile - 1) / kTile);
    const int64_t blocks = (rows * w->tiles + kTeams - 1) / kTeams;
    const int64_t most = (int64_t)per_sm * num_sms();
    *grid = (int)(blocks < most ? blocks : most);
    const int64_t step = (int64_t)*grid * kTeams;
    w->step_rows = step / w->tiles;
    w->step_tiles = (int)(step % w->tiles);
    return cudaSuccess;
}

template <typename T, bool VECTOR>
cudaError_t forward(const SwigluForward &a, cudaStream_t s) {
    Walk w;
    int grid = 0;
    cudaError_t e = plan<swiglu_kernel<T, VECTOR>>(a.rows, a.cols, &w, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(swiglu_kernel<T, VECTOR>, grid, kThreads, 0, s, a, w);
}

template <typename T, bool VECTOR, bool SAVED>
cudaError_t backward(const SwigluBackward &a, cudaStream_t s) {
    Walk w;
    int grid = 0;
    cudaError_t e = plan<swiglu_backward_kernel<T, VECTOR, SAVED>>(a.rows, a.cols, &w, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(swiglu_backward_kernel<T, VECTOR, SAVED>, grid, kThreads, 0, s, a, w);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluForward &a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const int size = a.f32 ? 4 : 2;
    // eight columns a lane: whole 16-byte groups of rows, 8-byte ones of bytes
    const bool vector = a.cols % kPer == 0 && a.ldh * size % 16 == 0 && aligned_to(a.h, 16) &&
                        aligned_to(a.y, 16) && aligned_to(a.yq, 8) && aligned_to(a.hq, 8);
    if (a.f32) return vector ? forward<float, true>(a, s) : forward<float, false>(a, s);
    return vector ? forward<uint16_t, true>(a, s) : forward<uint16_t, false>(a, s);
}

cudaError_t launch_swiglu_backward(const SwigluBackward &a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const int size = a.f32 ? 4 : 2;
    const bool saved = a.h_scale != nullptr;
    const int unit = saved ? 8 : 16;  // bytes of eight columns, or of a load
    const bool vector = a.cols % kPer == 0 && a.lddy * size % 16 == 0 && aligned_to(a.dy, 16) &&
                        a.ldh * (saved ? 1 : size) % unit == 0 && aligned_to(a.h, unit) &&
                        aligned_to(a.dh, 16) && aligned_to(a.y, 16);
    if (a.f32) {
        if (saved) return vector ? backward<float, true, true>(a, s) : backward<float, false, true>(a, s);
        return vector ? backward<float, true, false>(a, s) : backward<float, false, false>(a, s);
    }
    if (saved)
        return vector ? backward<uint16_t, true, true>(a, s) : backward<uint16_t, false, true>(a, s);
    return vector ? backward<uint16_t, true, false>(a, s) : backward<uint16_t, false, false>(a, s);
}

}  // namespace fp8
