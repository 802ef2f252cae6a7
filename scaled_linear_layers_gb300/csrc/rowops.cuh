// Row-wise helpers shared by the layer-norm and expert-dispatch kernels:
// 16-byte and single-element access to bf16 and fp32 rows, and sums over the
// threads that share a row.
#pragma once

#include "common.cuh"

namespace fp8 {

// A row's elements in groups of V: 16 bytes when VECTOR, else one element.
// The raw form is what a load leaves in registers.
template <typename T, bool VECTOR>
struct RowVec;

template <>
struct RowVec<uint16_t, true> {
    static constexpr int V = 8;
    using Raw = uint4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ Raw load(const uint16_t *p) {
        return *reinterpret_cast<const uint4 *>(p);
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[V]) {
        f[0] = bf16_lo(r.x), f[1] = bf16_hi(r.x), f[2] = bf16_lo(r.y), f[3] = bf16_hi(r.y);
        f[4] = bf16_lo(r.z), f[5] = bf16_hi(r.z), f[6] = bf16_lo(r.w), f[7] = bf16_hi(r.w);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&f)[V]) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ void store_raw(uint16_t *p, const Raw &r) {
        *reinterpret_cast<uint4 *>(p) = r;
    }
    static __device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[V]) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16),
                       cvt_e4m3x2(f[4], f[5]) | (cvt_e4m3x2(f[6], f[7]) << 16));
    }
};

template <>
struct RowVec<float, true> {
    static constexpr int V = 4;
    using Raw = float4;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ Raw load(const float *p) {
        return *reinterpret_cast<const float4 *>(p);
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[V]) {
        f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[V]) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
    static __device__ __forceinline__ void store_raw(float *p, const Raw &r) {
        *reinterpret_cast<float4 *>(p) = r;
    }
    static __device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[V]) {
        *reinterpret_cast<uint32_t *>(p) = cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16);
    }
};

__device__ __forceinline__ float elem_to_float(uint16_t v) {
    return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ float elem_to_float(float v) { return v; }
__device__ __forceinline__ void float_to_elem(uint16_t *p, float v) {
    *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
}
__device__ __forceinline__ void float_to_elem(float *p, float v) { *p = v; }

template <typename T>
struct RowVec<T, false> {
    static constexpr int V = 1;
    using Raw = T;
    static __device__ __forceinline__ Raw zero() { return T(0); }
    static __device__ __forceinline__ Raw load(const T *p) { return *p; }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[V]) {
        f[0] = elem_to_float(r);
    }
    static __device__ __forceinline__ void store(T *p, const float (&f)[V]) {
        float_to_elem(p, f[0]);
    }
    static __device__ __forceinline__ void store_raw(T *p, const Raw &r) { *p = r; }
    static __device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[V]) {
        *p = (uint8_t)(cvt_e4m3x2(f[0], 0.f) & 0xFFu);
    }
};

// One element of a bf16 or fp32 parameter vector as fp32.
__device__ __forceinline__ float load_param(const void *p, int f32, int64_t i) {
    return f32 ? reinterpret_cast<const float *>(p)[i]
               : elem_to_float(reinterpret_cast<const uint16_t *>(p)[i]);
}

// Sum over a warp; every lane gets the same value.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of N values over the TPR threads that share a row (TPR = 32: a warp;
// else the whole block).  `red` holds N * (TPR/32) floats; a caller that
// reduces again alternates between two such arrays, so one barrier per call
// is enough (a warp can be at most one call ahead of the slowest).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *red) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[i * W + warp] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = lane < W ? red[i * W + lane] : 0.f;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
            v[i] = __shfl_sync(0xFFFFFFFFu, t, 0);
        }
    }
}

// |v|'s bit pattern (patterns of non-negative floats order like the values,
// and a NaN's sorts above infinity's).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

inline bool aligned_to(const void *p, size_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace fp8
