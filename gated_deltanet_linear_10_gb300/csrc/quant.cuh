// 8-bit outputs (e4m3) with one fp32 scale per row, and the vector accesses
// and reductions the row kernels share (internal header).
//
//   scale = max(max_j |y_j| / 448, 2^-126),   q_j = rn_e4m3(y_j / scale)
//
// 448 is the largest e4m3 value.  The lower bound keeps 1 / scale finite, so
// a row of zeros gives q = 0.  Nothing is hidden: a NaN among the y_j makes the
// scale and every q_j of the row NaN, an infinite y_j makes the scale infinite.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gdn {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

// max(a, b), NaN when either is (fmaxf would drop it); of |a|, |b|, |c|.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Pairs of fp32 values, two to an instruction.
using F2 = uint64_t;
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2_bits(uint32_t lo, uint32_t hi) { return f2(__uint_as_float(lo), __uint_as_float(hi)); }
__device__ __forceinline__ float2 f2_get(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The hardware's reciprocal and power of two (a few ulp; results below 2^-126
// flushed to 0).
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504089f;

__device__ __forceinline__ float e4m3_scale(float amax) {
    return max_nan(amax * (1.0f / kE4m3Max), kMinScale);
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// One e4m3 value.
struct E4m3 {
    uint8_t v;
};

// N elements of T as registers: raw bytes as loaded (so that a row can be
// requested while another is worked on), unpacked to fp32 where used.
// N = 1: one element; otherwise N * sizeof(T) is 16 or 32 bytes, moved as
// 16-byte accesses (or, with `half`, 8-byte ones).
template <typename T, int N> struct RawVec {
    uint4 r[N * sizeof(T) / 16];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) r[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void load_half(const T *p) {   // 8-byte aligned p
        uint2 *d = reinterpret_cast<uint2 *>(r);
#pragma unroll
        for (int i = 0; i < (int)(N * sizeof(T) / 8); ++i) d[i] = reinterpret_cast<const uint2 *>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // elements lo .. hi - 1 of the vector at p, the others left as they are
    __device__ __forceinline__ void load_part(const T *p, int lo, int hi) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= lo && i < hi) reinterpret_cast<T *>(r)[i] = p[i];
    }
    // as N / 2 pairs
    __device__ __forceinline__ void pairs(F2 *out) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(r);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) out[i] = f2_bits(w[2 * i], w[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) out[i] = f2_bits(w[i] << 16, w[i] & 0xffff0000u);
        }
    }
};
template <typename T> struct RawVec<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T *p) { r = *p; }
    __device__ __forceinline__ void load_part(const T *, int, int) {}
    __device__ __forceinline__ void zero() { Io<T>::store(&r, 0.f); }
    __device__ __forceinline__ void pairs(F2 *out) const { out[0] = f2(Io<T>::load(&r), 0.f); }
};

// N values out of (N + 1) / 2 pairs.
template <int N> __device__ __forceinline__ void unpair(const F2 *in, float *out) {
#pragma unroll
    for (int i = 0; i < (N + 1) / 2; ++i) {
        const float2 v = f2_get(in[i]);
        out[2 * i] = v.x;
        if (2 * i + 1 < N) out[2 * i + 1] = v.y;
    }
}

// Stores N fp32 values as O (N = 1, 4 or 8; vectors aligned to their size).
template <int N> __device__ __forceinline__ void store_row(float *p, const float *v) {
    if constexpr (N == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) Vec16<float>::store(p + i, v + i);
    }
}
template <int N> __device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float *v) {
    if constexpr (N == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        static_assert(N == 8, "bf16 vectors are 16 bytes");
        Vec16<__nv_bfloat16>::store(p, v);
    }
}
template <int N> __device__ __forceinline__ void store_row(E4m3 *p, const float *v) {
    if constexpr (N == 1) {
        p->v = (uint8_t)__nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint32_t *>(p) = pack_e4m3x4(v[0], v[1], v[2], v[3]);
    } else {
        static_assert(N == 8, "e4m3 vectors are 4 or 8 bytes");
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_e4m3x4(v[0], v[1], v[2], v[3]),
                                                   pack_e4m3x4(v[4], v[5], v[6], v[7]));
    }
}

// Bytes lo .. of a vector of W words (lo > 0), or its bytes .. hi - 1 (lo <= 0), at
// most four stores; p on the vector's size.
template <int W> __device__ __forceinline__ void store_bytes(uint8_t *p, const uint32_t (&w)[W], int lo, int hi) {
    auto word = [&](int b) {
        uint32_t v = w[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = b >= 4 * i ? w[i] : v;
        return v;
    };
    int b = lo > 0 ? lo : 0;
    if (lo > 0) {
        if (b & 1) {
            p[b] = (uint8_t)(word(b) >> (b & 2 ? 24 : 8));
            b += 1;
        }
        if (b & 2) {
            *reinterpret_cast<uint16_t *>(p + b) = (uint16_t)(word(b) >> 16);
            b += 2;
        }
        if (W > 1 && (b & 4)) {
            *reinterpret_cast<uint32_t *>(p + b) = word(b);
            b += 4;
        }
        if (W > 2 && (b & 8)) *reinterpret_cast<uint2 *>(p + 8) = make_uint2(w[W - 2], w[W - 1]);
    } else {
        if (W > 2 && (hi & 8)) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[W > 1 ? 1 : 0]);
            b = 8;
        }
        if (W > 1 && (hi & 4)) {
            *reinterpret_cast<uint32_t *>(p + b) = word(b);
            b += 4;
        }
        if (hi & 2) {
            *reinterpret_cast<uint16_t *>(p + b) = (uint16_t)word(b);
            b += 2;
        }
        if (hi & 1) p[b] = (uint8_t)(word(b) >> (hi & 2 ? 16 : 0));
    }
}

// An end of a row: values lo .. of such a vector (lo > 0), or its values .. hi - 1.
template <int N> __device__ __forceinline__ void store_part(float *p, const float *v, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i >= lo && i < hi) store_row<1>(p + i, v + i);
}
template <int N> __device__ __forceinline__ void store_part(__nv_bfloat16 *p, const float *v, int lo, int hi) {
    if constexpr (N > 1) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        store_bytes(reinterpret_cast<uint8_t *>(p), w, 2 * lo, 2 * hi);
    }
}
template <int N> __device__ __forceinline__ void store_part(E4m3 *p, const float *v, int lo, int hi) {
    if constexpr (N > 1) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = pack_e4m3x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        store_bytes(reinterpret_cast<uint8_t *>(p), w, lo, hi);
    }
}

// (sum, NaN-keeping max) over the block; every thread gets both.  `part` is
// one of two shared arrays of 32 float2 used alternately, so that one barrier
// per call is enough: a thread is at most one call ahead of the slowest.
__device__ __forceinline__ float2 block_sum_max(float sum, float mx, float2 *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    if (warps == 1) return make_float2(sum, mx);
    if (lane == 0) part[warp] = make_float2(sum, mx);
    __syncthreads();
    const float2 p = lane < warps ? part[lane] : make_float2(0.f, 0.f);
    sum = p.x;
    mx = p.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    return make_float2(sum, mx);
}

// The NaN-keeping max alone, in the same way.
__device__ __forceinline__ float block_max(float mx, float2 *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (warps == 1) return mx;
    if (lane == 0) part[warp].x = mx;
    __syncthreads();
    mx = lane < warps ? part[lane].x : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    return mx;
}

}  // namespace gdn
