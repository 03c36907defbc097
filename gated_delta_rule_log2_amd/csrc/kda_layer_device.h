// kda_layer_device.h -- device helpers of the layer operators.
#pragma once

#include "kda_device.h"

namespace kda {

// Two values rounded to bf16 by one instruction (two single conversions cost a third to join).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// V consecutive channels as fp32, from any element-aligned address.  A row of D channels is cut
// into ceil(D / V) vectors; where V does not divide D the last vector is moved back to end with
// the row (vec_channel), so its first channels are also another vector's: both compute the same
// values.  The copies below let the compiler use wide accesses, which gfx950 serves at every
// address.
template <typename T, int V> struct Vec {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(w, p, sizeof(w)); }
    __device__ __forceinline__ void store(T *p) const { __builtin_memcpy(p, w, sizeof(w)); }
    // Past the caches: for inputs that nothing reads again, and outputs that only a later kernel reads
    // (there the read costs what the store saved, no more).  Vectors of one access only: those of two
    // (fp32, V = 8) fetch their lines twice.
    typedef uint32_t Raw __attribute__((ext_vector_type(V * sizeof(T) / 4), aligned(sizeof(T))));
    __device__ __forceinline__ void load_stream(const T *p) {
        if constexpr (sizeof(w) <= 16) {
            const Raw r = __builtin_nontemporal_load(reinterpret_cast<const Raw *>(p));
            __builtin_memcpy(w, &r, sizeof(w));
        } else {
            load(p);
        }
    }
    __device__ __forceinline__ void store_stream(T *p) const {
        static_assert(sizeof(w) <= 16, "a vector of one access");
        Raw r;
        __builtin_memcpy(&r, w, sizeof(w));
        __builtin_nontemporal_store(r, reinterpret_cast<Raw *>(p));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (unsigned i = 0; i < V * sizeof(T) / 4; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void get(float (&o)[V]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                o[2 * i] = __uint_as_float(w[i] << 16);
                o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[V]) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = pack_bf(x[2 * i], x[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        }
    }
    __device__ __forceinline__ void part(const T *p, int n) {  // n < V elements, the others 0
        T v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? p[i] : T(0);
        __builtin_memcpy(w, v, sizeof(w));
    }
    __device__ __forceinline__ void store_part(T *p, int n) const {
        T v[V];
        __builtin_memcpy(v, w, sizeof(w));
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = v[i];
    }
};
template <typename T> using Vec8 = Vec<T, 8>;

template <int V = 8> __host__ __device__ __forceinline__ int vec_count(int D) { return (D + V - 1) / V; }
// First channel of vector i (D >= V), or 0 with D < V, where a vector has D channels.
template <int V = 8> __device__ __forceinline__ int vec_channel(int i, int D) {
    const int c = V * i;
    return D < V ? 0 : (c + V <= D ? c : D - V);
}
template <typename T, int V> __device__ __forceinline__ void vec_load(Vec<T, V> &v, const T *row, int c, int D) {
    if (D >= V) v.load(row + c);
    else v.part(row, D);
}
template <typename T, int V> __device__ __forceinline__ void vec_store(const Vec<T, V> &v, T *row, int c, int D) {
    if (D >= V) v.store(row + c);
    else v.store_part(row, D);
}
template <typename T, int V> __device__ __forceinline__ void vec_load_stream(Vec<T, V> &v, const T *row, int c, int D) {
    if (D >= V) v.load_stream(row + c);
    else v.part(row, D);
}
template <typename T, int V> __device__ __forceinline__ void vec_store_stream(const Vec<T, V> &v, T *row, int c, int D) {
    if (D >= V) v.store_stream(row + c);
    else v.store_part(row, D);
}

__device__ __forceinline__ float load_f32(const void *p, int64_t i, int bf16) {
    return bf16 ? bf2f(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// 1 / (1 + e^-x): e^-x overflows to inf for x < -88, whose reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// Sum of column i over rows [rows][n], by a workgroup of 64 columns by 16 groups of rows: in a fixed
// order, so results do not depend on scheduling.  The first 64 threads have it.
__device__ __forceinline__ float sum_rows(const float *rows_of, int rows, int64_t n, int64_t i) {
    __shared__ float part[16][64];
    const int g = threadIdx.x >> 6, c = threadIdx.x & 63;
    float s = 0.f;
    if (i < n) {
        int b = g;
        for (; b + 7 * 16 < rows; b += 8 * 16) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = rows_of[(int64_t)(b + 16 * k) * n + i];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
        for (; b < rows; b += 16) s += rows_of[(int64_t)b * n + i];
    }
    part[g][c] = s;
    __syncthreads();
    if (g == 0)
#pragma unroll
        for (int k = 1; k < 16; ++k) s += part[k][c];
    return s;
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
