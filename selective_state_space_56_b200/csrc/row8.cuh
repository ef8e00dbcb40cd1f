// row8.cuh -- rows of any length read and written in vectors of eight elements.
//
// The operators around the scan walk rows (rows, L) of several arrays of the same sizes.
// Vectors start at multiples of 8 elements of the whole array, so every access of a whole
// vector is 16-byte aligned in all of them, whatever the row's length and the element type;
// a row's first and last vector may hold elements of the neighbouring rows, which are read
// (never past the array), ignored, and not written.
#pragma once

#include "s6_device.cuh"

namespace s6 {

constexpr int kE = 8;

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ f2 pair(int i) const {
        return bf16pair(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    }
    __device__ __forceinline__ void to_f(float (&o)[kE]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 lo, hi;
    __device__ __forceinline__ void load(const float* p) {
        lo = *reinterpret_cast<const float4*>(p);
        hi = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { lo = hi = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ f2 pair(int i) const {
        return i == 0 ? pack2(lo.x, lo.y) : i == 1 ? pack2(lo.z, lo.w) : i == 2 ? pack2(hi.x, hi.y) : pack2(hi.z, hi.w);
    }
    __device__ __forceinline__ void to_f(float (&o)[kE]) const {
        o[0] = lo.x, o[1] = lo.y, o[2] = lo.z, o[3] = lo.w;
        o[4] = hi.x, o[5] = hi.y, o[6] = hi.z, o[7] = hi.w;
    }
};

__device__ __forceinline__ void store_all(__nv_bfloat16* p, const float (&v)[kE]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_all(float* p, const float (&v)[kE]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// A row's place in the arrays: its elements are [lo, hi), its vector v starts at base + 8 v.
struct Row {
    int64_t lo, hi, base, total;
    int64_t vectors;
};
__device__ __forceinline__ Row row_of(int64_t r, int64_t rows, int64_t L) {
    Row w;
    w.lo = r * L;
    w.hi = w.lo + L;
    w.base = w.lo & ~(int64_t)(kE - 1);
    w.total = rows * L;
    w.vectors = (w.hi - w.base + kE - 1) / kE;
    return w;
}

// The 8 elements from element e (a multiple of 8) on.  Nothing is read past the array or for
// vectors beyond the row; what belongs to a neighbouring row is read and masked by the caller.
template <typename T>
__device__ __forceinline__ void fetch(Raw8<T>& r, const void* p, int64_t e, const Row& w) {
    const T* q = static_cast<const T*>(p) + e;
    if (e < w.hi && e + kE <= w.total) {
        r.load(q);
    } else {
        r.zero();
        if (e < w.hi) {  // the array's last, partial vector
            T* o = reinterpret_cast<T*>(&r);
            for (int j = 0; j < kE; ++j)
                if (e + j < w.total) o[j] = q[j];
        }
    }
}

template <typename T>
__device__ __forceinline__ void put(void* p, int64_t e, const Row& w, const float (&v)[kE]) {
    T* q = static_cast<T*>(p) + e;
    if (e >= w.lo && e + kE <= w.hi) {
        store_all(q, v);
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j)
            if (e + j >= w.lo && e + j < w.hi) q[j] = io<T>::from_f(v[j]);
    }
}

// Eight fp32 values to e4m3 (round to nearest even, values beyond 448 saturate).
__device__ __forceinline__ uint2 to_e4m3(const float (&v)[kE]) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;  // keeps the scale of a group of zeros positive
constexpr int kGroup = 128;           // values that share a scale

// 448 v / m for the values v of a group with largest magnitude m.  Where v and m have few bits the
// quotient is often exactly half way between two values of e4m3, and v * (448 / m), rounded twice,
// then lies beside it (bf16 groups of normal values: 2.4e-4 of the e4m3 outputs off by a step).  So
// 448 / m is kept in two pieces (as in Dekker, "A floating-point technique for extending the
// available precision"): hi = 448 / m rounded, lo = (448 - hi m) / m, whose numerator one fused
// multiply-add gives exactly.  v hi + v lo is then rounded once, from within 2^-46 of the quotient,
// so a quotient that fp32 holds comes out exactly.  m infinite: hi = lo = 0, so finite values give 0
// and infinite ones NaN.
struct Quotient {
    f2 hi, lo;
    // The halves of a pair in groups of their own.
    __device__ __forceinline__ Quotient(float m0, float m1) {
        const float h0 = kE4m3Max / m0, h1 = kE4m3Max / m1;
        hi = pack2(h0, h1);
        lo = pack2(rest(h0, m0), rest(h1, m1));
    }
    __device__ __forceinline__ explicit Quotient(float m) {
        const float h = kE4m3Max / m, l = rest(h, m);
        hi = pack2(h, h);
        lo = pack2(l, l);
    }
    static constexpr float kLargest = 3.40282347e38f;  // of fp32
    __device__ __forceinline__ static float rest(float h, float m) {
        return fmaf(-h, fminf(m, kLargest), kE4m3Max) * (h * (1.f / kE4m3Max));
    }
    __device__ __forceinline__ f2 operator()(f2 v) const { return fma2(v, hi, mul2(v, lo)); }
    // Eight values of a group, in place.
    __device__ __forceinline__ void operator()(float (&v)[kE]) const {
#pragma unroll
        for (int i = 0; i < kE; i += 2) unpack2((*this)(pack2(v[i], v[i + 1])), v[i], v[i + 1]);
    }
};

}  // namespace s6
