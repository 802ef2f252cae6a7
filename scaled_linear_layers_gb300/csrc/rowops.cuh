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

// 4-byte words of a row from an address aligned only to its elements: an fp32
// element, or two bf16 ones, shifted together from the two aligned words that
// hold them when they lie across two.  Word i then also reads the element
// before its first and the one after its second.
template <typename T>
struct WordRow {
    static constexpr int V = 4 / sizeof(T);
    const uint32_t *at, *next;
    uint32_t shift;  // bits

    __device__ __forceinline__ WordRow() {}
    __device__ __forceinline__ explicit WordRow(const T *p) {
        const uint32_t u = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
        at = reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(p) - u);
        next = at + (u != 0);
        shift = u * 8u;
    }

    // what word i lies in; zeros unless `on`.  Shifted together apart from the
    // loads, so that none of them is waited for before the next is issued.
    struct Raw {
        uint32_t lo, hi;
    };
    __device__ __forceinline__ Raw load(int64_t i, bool on) const {
        Raw r;
        r.lo = on ? at[i] : 0u;
        r.hi = V == 2 && on ? next[i] : 0u;
        return r;
    }
    __device__ __forceinline__ uint32_t word(const Raw &r) const {
        return V == 1 ? r.lo : __funnelshift_r(r.lo, r.hi, shift);
    }

    static __device__ __forceinline__ void unpack(uint32_t w, float (&f)[V]) {
        if constexpr (V == 1) {
            f[0] = __uint_as_float(w);
        } else {
            f[0] = __uint_as_float(w << 16);
            f[1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint32_t pack(const float (&f)[V]) {
        if constexpr (V == 1) return __float_as_uint(f[0]);
        else return pack_bf16x2(f[0], f[1]);
    }
};

// Two fp32 values in one 64-bit register, and arithmetic on both in one
// instruction (each lane rounds as the single one does).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 pair_split(uint64_t p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The larger of a and |b|; NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// One element of a bf16 or fp32 parameter vector as fp32.
__device__ __forceinline__ float load_param(const void *p, int f32, int64_t i) {
    return f32 ? reinterpret_cast<const float *>(p)[i]
               : elem_to_float(reinterpret_cast<const uint16_t *>(p)[i]);
}

// V neighbouring ones from a multiple of V on (V > 1: p is 16-byte aligned).
template <int V>
__device__ __forceinline__ void load_params(const void *p, int f32, int64_t i, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = load_param(p, f32, i);
    } else if (f32) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i + k);
            f[k] = bf16_lo(v.x), f[k + 1] = bf16_hi(v.x);
            f[k + 2] = bf16_lo(v.y), f[k + 3] = bf16_hi(v.y);
        }
    }
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

// The sum of one value whose terms may cancel: each is split into its leading
// 12 bits and the rest, which are added apart.  Sums of the leading parts of
// values within 2^12 of each other are exact in fp32, and what the rests lose
// is 2^-12 of what a plain sum would.
template <int TPR>
__device__ __forceinline__ float row_sum_split(float v, float rest, float *red) {
    float s[2];
    s[0] = __uint_as_float(__float_as_uint(v) & 0xFFFFF000u);
    s[1] = fabsf(v) < INFINITY ? (v - s[0]) + rest : 0.f;  // an infinity or NaN is in s[0]
    row_sum<TPR, 2>(s, red);
    return s[0] + s[1];
}

// sum += v, with the addition's rounding error added to err.
__device__ __forceinline__ void add_exact(float &sum, float &err, float v) {
    const float t = __fadd_rn(sum, v);
    const float z = __fsub_rn(t, sum);
    err += __fadd_rn(__fsub_rn(sum, __fsub_rn(t, z)), __fsub_rn(v, z));
    sum = t;
}

// |v|'s bit pattern (patterns of non-negative floats order like the values,
// and a NaN's sorts above infinity's).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

inline bool aligned_to(const void *p, size_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace fp8
