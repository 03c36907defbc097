// kda_layer_device.h -- device helpers of the layer operators.
#pragma once

#include "kda_device.h"

namespace kda {

// Eight consecutive channels as fp32, from any element-aligned address.  A row of D
// channels is cut into ceil(D / 8) vectors; where 8 does not divide D the last vector is
// moved back to end with the row (vec_channel), so its first channels are also another
// vector's: both compute the same values.  The copies below let the compiler use 16-byte
// accesses, which gfx950 serves at every address.
struct Raw16 { uint32_t w[4]; };

// Two values rounded to bf16 by one instruction (two single conversions cost a third to join).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    Raw16 r;
    __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(&r, p, 16); }
    __device__ __forceinline__ void zero() { r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0; }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(r.w[i] << 16);
            o[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = pack_bf(x[2 * i], x[2 * i + 1]);
    }
    __device__ __forceinline__ void store(uint16_t *p) const { __builtin_memcpy(p, &r, 16); }
    __device__ __forceinline__ void part(const uint16_t *p, int n) {  // n < 8 elements, the others 0
        uint16_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (uint16_t)0;
        __builtin_memcpy(&r, v, 16);
    }
    __device__ __forceinline__ void store_part(uint16_t *p, int n) const {
        uint16_t v[8];
        __builtin_memcpy(v, &r, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
};
template <> struct Vec8<float> {
    Raw16 r[2];
    __device__ __forceinline__ void load(const float *p) { __builtin_memcpy(r, p, 32); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i >> 2].w[i & 3] = 0;
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(r[i >> 2].w[i & 3]);
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i >> 2].w[i & 3] = __float_as_uint(x[i]);
    }
    __device__ __forceinline__ void store(float *p) const { __builtin_memcpy(p, r, 32); }
    __device__ __forceinline__ void part(const float *p, int n) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
        __builtin_memcpy(r, v, 32);
    }
    __device__ __forceinline__ void store_part(float *p, int n) const {
        float v[8];
        __builtin_memcpy(v, r, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
};

__host__ __device__ __forceinline__ int vec_count(int D) { return (D + 7) >> 3; }
// First channel of vector i (D >= 8), or 0 with D < 8, where a vector has D channels.
__device__ __forceinline__ int vec_channel(int i, int D) {
    const int c = 8 * i;
    return D < 8 ? 0 : (c + 8 <= D ? c : D - 8);
}
template <typename T> __device__ __forceinline__ void vec_load(Vec8<T> &v, const T *row, int c, int D) {
    if (D >= 8) v.load(row + c);
    else v.part(row, D);
}
template <typename T> __device__ __forceinline__ void vec_store(const Vec8<T> &v, T *row, int c, int D) {
    if (D >= 8) v.store(row + c);
    else v.store_part(row, D);
}

__device__ __forceinline__ float load_f32(const void *p, int64_t i, int bf16) {
    return bf16 ? bf2f(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// 1 / (1 + e^-x): e^-x overflows to inf for x < -88, whose reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// Sequence of token t (flattened over the batch), its first token and the token after its
// last: batch rows, or packed sequences by binary search (empty ones hold no token).
struct SeqSpan { int n; int64_t first, end; };
template <typename P> __device__ __forceinline__ SeqSpan seq_span(const P &p, int n) {
    if (p.cu_seqlens) {  // held to the tokens there are, whatever the device's copy says
        const int64_t a = p.cu_seqlens[n], b = p.cu_seqlens[n + 1];
        const int64_t first = a < 0 ? 0 : a < p.tokens ? a : p.tokens;
        return {n, first, b < first ? first : b < p.tokens ? b : p.tokens};
    }
    return {n, (int64_t)n * p.T, (int64_t)(n + 1) * p.T};
}
template <typename P> __device__ __forceinline__ SeqSpan seq_of(const P &p, int64_t t) {
    if (!p.cu_seqlens) return seq_span(p, (int)(t / p.T));
    int lo = 0, hi = p.N - 1;  // last n with cu[n] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return seq_span(p, lo);
}

}  // namespace kda
