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
// hardware's exponential and reciprocal, whose error in s is 2^-21 (1 + |gate|/8), far
// below bf16's 2^-8, and whose s is zero for gates below -87.3; fp32 rows take expf
// and a division (zero below -88.7).  Of 2.9e7 E4M3 values of y, 14 take the other
// neighbour of a border than with expf and a division, which bring scales and bytes no
// nearer to 64 bits (scales 5e-8 either way) and take 370 us where this takes 281 (expf
// alone 290).
//
// Everything moves once and is bound by HBM: 7.1 bytes an element forward to
// E4M3 with the checkpoint, 10.1 backward from it (bf16).  Sixteen lanes share
// a tile, eight neighbouring columns each, so that a tile's maximum is four
// shuffles and a bf16 lane's loads are 16 bytes; rows that do not lie on 16
// bytes go element by element, a tile's columns dealt out to the lanes in turn.
// 16384 x 14336 bf16: forward to E4M3 with the checkpoint 282 us, 0.87 of the
// measured bandwidth (376 when a team took one tile after another, a division for
// each scale and its inverse in every lane); backward with y again 363 us, 0.96.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "occupancy.h"
#include "rowops.cuh"

namespace fp8 {

namespace {

constexpr int kTile = 128, kLanes = 16, kPer = kTile / kLanes;
constexpr int kThreads = 256, kTeams = kThreads / kLanes;

// Blocks an SM, so that the next item's loads are held in registers beside the
// one at work.  Two, three and four blocks, us: 16384 x 14336 bf16 forward 330, 291
// and 310, backward from the checkpoint 417, 371 and 361; 8192 x 8192, forward fp32
// 125, 111 and 129, backward fp32 from the checkpoint 185, 245 and 226, bf16 from h
// 136, 120 and 135; fp32 rows of odd width, backward of 3001 x 1001: 11.9, 13.6 and
// 22.6.
template <bool VECTOR>
constexpr int kForwardBlocks = VECTOR ? 3 : 2;
template <typename T, bool VECTOR, bool SAVED>
constexpr int kBackwardBlocks = !VECTOR || sizeof(T) == 4 ? 2 : SAVED ? 4 : 3;

__device__ __forceinline__ float sigmoid(float x, uint16_t) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
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
// from `lane` on, those below `left` (the tile's columns).  Loaded and then
// unpacked, so that all loads of an item are under way before the first is used.
template <typename T, bool VECTOR>
struct Cols;
template <>
struct Cols<uint16_t, true> {
    uint4 raw;
    __device__ __forceinline__ void load(const uint16_t *p, int lane, int left) {
        raw = kPer * lane < left ? *reinterpret_cast<const uint4 *>(p + kPer * lane)
                                 : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void unpack(float (&f)[kPer]) const {
        RowVec<uint16_t, true>::unpack(raw, f);
    }
};
template <>
struct Cols<float, true> {
    float4 raw[2];
    __device__ __forceinline__ void load(const float *p, int lane, int left) {
        const float4 *q = reinterpret_cast<const float4 *>(p + kPer * lane);
        const bool on = kPer * lane < left;
        raw[0] = on ? q[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        raw[1] = on ? q[1] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void unpack(float (&f)[kPer]) const {
        f[0] = raw[0].x, f[1] = raw[0].y, f[2] = raw[0].z, f[3] = raw[0].w;
        f[4] = raw[1].x, f[5] = raw[1].y, f[6] = raw[1].z, f[7] = raw[1].w;
    }
};
template <typename T>
struct Cols<T, false> {
    T raw[kPer];
    __device__ __forceinline__ void load(const T *p, int lane, int left) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            raw[i] = lane + kLanes * i < left ? p[lane + kLanes * i] : T(0);
    }
    __device__ __forceinline__ void unpack(float (&f)[kPer]) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = elem_to_float(raw[i]);
    }
};

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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The larger of a lane's and the other lanes' of its tile.
__device__ __forceinline__ float team_max(float m) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        m = max_abs_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
}

// The largest |v| of a tile in all of its sixteen lanes (NaN if any is).
__device__ __forceinline__ float tile_amax(const float (&f)[kPer]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max_abs_nan(m, f[i]);
    return team_max(m);
}

// Those of the gate's and the up's tile.
template <typename T, bool VECTOR>
__device__ __forceinline__ void tile_amax2(const Cols<T, VECTOR> &, const Cols<T, VECTOR> &,
                                           const float (&g)[kPer], const float (&u)[kPer],
                                           float &mg, float &mu) {
    mg = tile_amax(g);
    mu = tile_amax(u);
}
// bf16 magnitudes order as 16-bit whole numbers: both maxima in one register
template <>
__device__ __forceinline__ void tile_amax2<uint16_t, true>(const Cols<uint16_t, true> &g,
                                                           const Cols<uint16_t, true> &u,
                                                           const float (&)[kPer],
                                                           const float (&)[kPer], float &mg,
                                                           float &mu) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t a = max_u16x2(max_u16x2(g.raw.x & kAbs, g.raw.y & kAbs),
                                max_u16x2(g.raw.z & kAbs, g.raw.w & kAbs));
    const uint32_t b = max_u16x2(max_u16x2(u.raw.x & kAbs, u.raw.y & kAbs),
                                max_u16x2(u.raw.z & kAbs, u.raw.w & kAbs));
    uint32_t m = max_u16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    mg = bf16_lo(m);
    mu = bf16_hi(m);
}

// Every team of sixteen lanes keeps a tile's columns and goes down the rows, so
// that its addresses move by constants: `width` teams side by side (a tile each,
// or each width-th of more tiles than there are teams), `row_step` rows of them.
struct Walk {
    int tiles, width;
    int64_t row_step;
};

struct Team {
    int lane;
    int64_t tile, row0;
    __device__ __forceinline__ explicit Team(const Walk &w) {
        const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / kLanes;
        lane = threadIdx.x % kLanes;
        row0 = team / w.width;
        tile = team - row0 * w.width;
    }
};

__device__ __forceinline__ int64_t live_rows(const int32_t *live, int64_t rows) {
    return live == nullptr ? rows : min(rows, (int64_t)max(0, *live));
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads, kForwardBlocks<VECTOR>)
    swiglu_kernel(const SwigluForward a, const Walk w) {
    pdl_wait_prior();
    pdl_allow_next();
    Team at(w);
    const int lane = at.lane, first = threadIdx.x & 16;  // the team's first lane of the warp
    const int64_t rows = live_rows(a.live, a.rows);
    const int64_t h_step = w.row_step * a.ldh, y_step = w.row_step * a.cols;
    // Lanes 0..2 form and store the scales of the gate's, the up's and y's tile,
    // lanes 3..5 their inverses: one division a lane.
    const bool of_gate = lane % 3 == 0, of_up = lane % 3 == 1, forward = lane < 3;
    const bool has_scale = lane == 2 ? a.yq != nullptr : lane < 2 && a.hq != nullptr;
    const int64_t s_step = w.row_step * w.tiles * (lane == 2 ? 1 : 2);
    // both teams of a warp go on until neither has anything left
    for (; __any_sync(0xFFFFFFFFu, at.tile < w.tiles); at.tile += w.width) {
        const int64_t c0 = at.tile * kTile, row = at.row0;
        const int left = (int)max((int64_t)0, min((int64_t)kTile, a.cols - c0));
        const int own = at.row0 < w.row_step && left > 0 && row < rows
                            ? (int)((rows - row + w.row_step - 1) / w.row_step) : 0;
        const int most = max(own, __shfl_xor_sync(0xFFFFFFFFu, own, 16));
        const T *h = reinterpret_cast<const T *>(a.h) + row * a.ldh + c0;
        T *y = reinterpret_cast<T *>(a.y) + row * a.cols + c0;
        uint8_t *yq = a.yq + row * a.cols + c0, *hq = a.hq + 2 * row * a.cols + c0;
        float *scale = lane == 2 ? a.y_scale + row * w.tiles + at.tile
                                 : a.h_scale + (2 * row + lane) * w.tiles + at.tile;
        Cols<T, VECTOR> next_gate, next_up;
        next_gate.load(h, lane, 0 < own ? left : 0);
        next_up.load(h + a.cols, lane, 0 < own ? left : 0);
        for (int i = 0; i < most; ++i) {
            const Cols<T, VECTOR> gate = next_gate, up = next_up;
            const int cols = i < own ? left : 0;
            h += h_step;
            next_gate.load(h, lane, i + 1 < own ? left : 0);
            next_up.load(h + a.cols, lane, i + 1 < own ? left : 0);
            float g[kPer], u[kPer], v[kPer];
            gate.unpack(g);
            up.unpack(u);
#pragma unroll
            for (int k = 0; k < kPer; ++k) v[k] = g[k] * sigmoid(g[k], T()) * u[k];
            if (a.y != nullptr) {
                store_cols<T, VECTOR>(y, lane, cols, v);
                y += y_step;
            }
            float mg = 0.f, mu = 0.f, mv = 0.f;
            if (a.hq != nullptr) tile_amax2<T, VECTOR>(gate, up, g, u, mg, mu);
            if (a.yq != nullptr) mv = tile_amax(v);
            // scales_from_amax
            const float m = of_gate ? mg : of_up ? mu : mv, top = m < 1e-12f ? 1e-12f : m;
            const float s = __fdiv_rn(forward ? top : 448.f, forward ? 448.f : top);
            if (has_scale && i < own) *scale = s;
            scale += s_step;
            if (a.hq != nullptr) {
                store_e4m3<VECTOR>(hq, lane, cols, g, __shfl_sync(0xFFFFFFFFu, s, first + 3));
                store_e4m3<VECTOR>(hq + a.cols, lane, cols, u,
                                   __shfl_sync(0xFFFFFFFFu, s, first + 4));
                hq += 2 * y_step;
            }
            if (a.yq != nullptr) {
                store_e4m3<VECTOR>(yq, lane, cols, v, __shfl_sync(0xFFFFFFFFu, s, first + 5));
                yq += y_step;
            }
        }
    }
}

// The bytes of a lane's columns of one checkpoint tile.
template <bool VECTOR>
struct Bytes;
template <>
struct Bytes<true> {
    uint2 raw;
    __device__ __forceinline__ void load(const uint8_t *p, int lane, int left) {
        raw = kPer * lane < left ? *reinterpret_cast<const uint2 *>(p + kPer * lane)
                                 : make_uint2(0, 0);
    }
    __device__ __forceinline__ uint32_t two(int i) const {
        return ((i & 2) ? raw.y : raw.x) >> (16 * (i & 1));
    }
};
template <>
struct Bytes<false> {
    uint8_t raw[kPer];
    __device__ __forceinline__ void load(const uint8_t *p, int lane, int left) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            raw[i] = lane + kLanes * i < left ? p[lane + kLanes * i] : (uint8_t)0;
    }
    __device__ __forceinline__ uint32_t two(int i) const {
        return raw[2 * i] | ((uint32_t)raw[2 * i + 1] << 8);
    }
};
template <bool VECTOR>
__device__ __forceinline__ void decode(const Bytes<VECTOR> &b, float scale, float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const float2 v = e4m3x2_to_float2(b.two(i));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// One team's input of the backward pass: dy, and h from its bytes or as it is.
template <typename T, bool VECTOR, bool SAVED>
struct BackwardInput {
    Cols<T, VECTOR> grad;
    typename std::conditional<SAVED, Bytes<VECTOR>, Cols<T, VECTOR>>::type gate, up;
    float gate_scale, up_scale;
    template <typename H>
    __device__ __forceinline__ void load(const T *dy, const H *h, const float *scale, int64_t cols,
                                         int tiles, int lane, int left) {
        grad.load(dy, lane, left);
        gate.load(h, lane, left);
        up.load(h + cols, lane, left);
        if constexpr (SAVED) {
            gate_scale = left > 0 ? scale[0] : 0.f;
            up_scale = left > 0 ? scale[tiles] : 0.f;
        }
    }
    __device__ __forceinline__ void unpack(float (&d)[kPer], float (&g)[kPer], float (&u)[kPer]) const {
        grad.unpack(d);
        if constexpr (SAVED) {
            decode(gate, gate_scale, g);
            decode(up, up_scale, u);
        } else {
            gate.unpack(g);
            up.unpack(u);
        }
    }
};

template <typename T, bool VECTOR, bool SAVED>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks<T, VECTOR, SAVED>)
    swiglu_backward_kernel(const SwigluBackward a, const Walk w) {
    using H = typename std::conditional<SAVED, uint8_t, T>::type;
    pdl_wait_prior();
    pdl_allow_next();
    Team at(w);
    const int lane = at.lane;
    const int64_t rows = live_rows(a.live, a.rows);
    const int64_t h_step = w.row_step * a.ldh, dy_step = w.row_step * a.lddy;
    const int64_t y_step = w.row_step * a.cols, s_step = w.row_step * 2 * w.tiles;
    if (at.row0 >= w.row_step) return;
    for (; at.tile < w.tiles; at.tile += w.width) {
        const int64_t c0 = at.tile * kTile;
        const int left = (int)min((int64_t)kTile, a.cols - c0);
        int64_t row = at.row0, to = row * a.cols + c0;
        const T *dy = reinterpret_cast<const T *>(a.dy) + row * a.lddy + c0;
        const H *h = reinterpret_cast<const H *>(a.h) + row * a.ldh + c0;
        const float *scale = a.h_scale + row * 2 * w.tiles + at.tile;
        BackwardInput<T, VECTOR, SAVED> next;
        next.load(dy, h, scale, a.cols, w.tiles, lane, row < rows ? left : 0);
        for (; row < rows; to += y_step) {
            const BackwardInput<T, VECTOR, SAVED> in = next;
            row += w.row_step;
            dy += dy_step;
            h += h_step;
            scale += s_step;
            next.load(dy, h, scale, a.cols, w.tiles, lane, row < rows ? left : 0);
            float d[kPer], g[kPer], u[kPer], v[kPer];
            in.unpack(d, g, u);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float s = sigmoid(g[i], T()), act = g[i] * s;
                v[i] = act * u[i];
                g[i] = d[i] * u[i] * (s + act * (1.f - s));
                u[i] = d[i] * act;
            }
            T *out = reinterpret_cast<T *>(a.dh) + 2 * to - c0;
            store_cols<T, VECTOR>(out, lane, left, g);
            store_cols<T, VECTOR>(out + a.cols, lane, left, u);
            if (a.y != nullptr)
                store_cols<T, VECTOR>(reinterpret_cast<T *>(a.y) + to, lane, left, v);
        }
    }
}

// As many blocks as the device holds at once, or fewer for fewer tiles.
template <auto KERNEL>
cudaError_t plan(int64_t rows, int64_t cols, Walk *w, int *grid) {
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<KERNEL>(kThreads, &per_sm);
    if (e != cudaSuccess) return e;
    w->tiles = (int)((cols + kTile - 1) / kTile);
    const int64_t want = (rows * w->tiles + kTeams - 1) / kTeams;
    const int64_t most = (int64_t)per_sm * num_sms();
    *grid = (int)(want < most ? want : most);
    const int64_t teams = (int64_t)*grid * kTeams;
    w->width = (int)(w->tiles < teams ? w->tiles : teams);
    w->row_step = teams / w->width;
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
        // columns dealt out in turn are whole lines at each load: 8192 x 8192 with y
        // again 255 us, by eight neighbouring columns a lane 280
        return backward<float, false, false>(a, s);
    }
    if (saved)
        return vector ? backward<uint16_t, true, true>(a, s) : backward<uint16_t, false, true>(a, s);
    return vector ? backward<uint16_t, true, false>(a, s) : backward<uint16_t, false, false>(a, s);
}

}  // namespace fp8
