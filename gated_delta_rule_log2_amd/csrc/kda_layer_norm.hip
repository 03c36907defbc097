// kda_layer_norm.hip -- RMS norm with the residual's addition in front and, on request, an
// output in 8 bits (e4m3) with scales; and its gradients.
//
//   h = x + residual, rounded to the type it is stored in (the residual stream)
//   y = h r w,  r = (mean(h^2) + eps)^(-1/2)
//   e4m3: over each group of values (the row, or `group` of them) scale = max|y| / 448 and
//         q = round(y / scale), the largest value landing on e4m3's largest, 448
//   dx = r g - h r^3 mean(g h) + dh with g = dy w;   dweight = sum over rows of dy h r
//
// Bound by HBM: each value is read once and written once per output, with about ten
// operations (8192 rows of 4096 in bf16: to 8 bits 236 MB in 52 us, 4.5 TB/s; backward 268 MB
// in 51 us, 5.3 TB/s, where loads that stay in the caches took 71).  A row stays in the
// registers of one wave (D <= 1024) or one workgroup between the sum of squares and the output;
// sums are fp32.
#include "kda_layer.h"
#include "kda_layer_device.h"

namespace kda {

namespace {

constexpr float kE4m3Max = 448.f;

// Sum (or largest value, NaN if there is one) over the TPR threads of a row: lanes first,
// then the row's waves through LDS.  Every thread gets the result; rows of one wave need no
// barrier.
__device__ __forceinline__ float nan_max(float a, float b) { return a > b || a != a ? a : b; }

template <int TPR, bool MAX> __device__ __forceinline__ float row_reduce(float v, float *lds) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = MAX ? nan_max(v, shfl_xor(v, m)) : v + shfl_xor(v, m);
    if constexpr (TPR > 64) {
        const int w = (threadIdx.x % TPR) >> 6;
        __syncthreads();  // the previous reduction's values have been read
        if ((threadIdx.x & 63) == 0) lds[w] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v = MAX ? nan_max(v, lds[i]) : v + lds[i];
    }
    return v;
}

// First element of vector i that no earlier vector holds (a moved-back last vector shares
// its first ones), for sums.
__device__ __forceinline__ int own_from(int i, int c) { return 8 * i - c; }

template <typename T> __device__ __forceinline__ void load_weights(const NormParams &p, int c, float (&w)[8]) {
    if (p.D >= 8) {
        if (p.w_bf16) {
            Vec8<uint16_t> v;
            v.load(static_cast<const uint16_t *>(p.weight) + c);
            v.get(w);
        } else {
            Vec8<float> v;
            v.load(static_cast<const float *>(p.weight) + c);
            v.get(w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = j < p.D ? load_f32(p.weight, j, p.w_bf16) : 0.f;
    }
}

// A workgroup of `THREADS`, TPR of them for a row, NV vectors of eight values a thread:
// thread r of a row holds vectors r, r + TPR, ...
template <typename T, int TPR, int NV, bool FP8>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_fwd_kernel(NormParams p) {
    constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
    __shared__ float lds[THREADS / 64];
    const int r = threadIdx.x % TPR;
    int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool live = row < p.rows;  // the last workgroup's spare rows repeat its last row's reads
    if (!live) row = p.rows - 1;
    const int nv = vec_count(p.D);
    const T *x = static_cast<const T *>(p.x) + row * p.D;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.D : nullptr;

    Vec8<T> vx[NV], vr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = r + k * TPR;
        if (i < nv) {
            vec_load(vx[k], x, vec_channel(i, p.D), p.D);
            if (res) vec_load(vr[k], res, vec_channel(i, p.D), p.D);
        }
    }
    float h[NV][8];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = r + k * TPR;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
        if (i < nv) {
            const int c = vec_channel(i, p.D);
            vx[k].get(h[k]);
            if (res) {
                float e[8];
                vr[k].get(e);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[k][j] += e[j];
                vx[k].set(h[k]);  // the stored sum is what the norm is of
                vx[k].get(h[k]);
            }
            if (live && p.h) vec_store(vx[k], static_cast<T *>(p.h) + row * p.D, c, p.D);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= own_from(i, c)) s += h[k][j] * h[k][j];
        }
    }
    s = row_reduce<TPR, false>(s, lds);
    // 1 / sqrt by the correctly rounded operations: v_rsq's error would show in fp32 outputs
    const float rs = 1.f / sqrtf(s / (float)p.D + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = r + k * TPR;
        if (i < nv) {
            float w[8];
            load_weights<T>(p, vec_channel(i, p.D), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] = h[k][j] * rs * w[j];
        }
    }
    if constexpr (!FP8) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = r + k * TPR;
            if (live && i < nv) {
                Vec8<T> o;
                o.set(h[k]);
                vec_store(o, static_cast<T *>(p.y) + row * p.D, vec_channel(i, p.D), p.D);
            }
        }
    } else {
        float mx[NV];
        float all = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            mx[k] = 0.f;
            if (r + k * TPR < nv)
#pragma unroll
                for (int j = 0; j < 8; ++j) mx[k] = nan_max(mx[k], fabsf(h[k][j]));
            all = nan_max(all, mx[k]);
        }
        if (p.group == 0) {
            all = row_reduce<TPR, true>(all, lds);
#pragma unroll
            for (int k = 0; k < NV; ++k) mx[k] = all;
        } else {  // group / 8 neighbouring lanes, a power of two of at most 64
            for (int m = p.group / 16; m >= 1; m >>= 1)
#pragma unroll
                for (int k = 0; k < NV; ++k) mx[k] = nan_max(mx[k], shfl_xor(mx[k], m));
        }
        const int groups = p.group ? p.D / p.group : 1;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = r + k * TPR;
            if (!live || i >= nv) continue;
            const int c = vec_channel(i, p.D);
            const float big = mx[k] < 1e-30f ? 1e-30f : mx[k];  // a group of zeros has a scale too
            const float scale = big / kE4m3Max;
            if (p.group ? (8 * i) % p.group == 0 : i == 0) p.scales[row * groups + (p.group ? 8 * i / p.group : 0)] = scale;
            uint32_t o[2] = {0, 0};
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = h[k][j] / scale;
                q[j] = q[j] > kE4m3Max ? kE4m3Max : q[j] < -kE4m3Max ? -kE4m3Max : q[j];
            }
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                int v = 0;
                v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * d], q[4 * d + 1], v, false);
                v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * d + 2], q[4 * d + 3], v, true);
                o[d] = (uint32_t)v;
            }
            uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.D;
            if (p.D >= 8) __builtin_memcpy(y + c, o, 8);
            else
                for (int j = 0; j < p.D; ++j) y[j] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// A workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps its sums of dy h r for the
// weights in registers; one partial row leaves at the end.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, TPR > 256 ? 1 : 3) norm_bwd_kernel(NormParams p) {
    constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
    __shared__ float2 lds[2][THREADS / 64];
    __shared__ float join[ROWS > 1 ? THREADS * 8 : 8];
    const int r = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int nv = vec_count(p.D);
    constexpr bool KEEP = NV < 4;  // the weights, where the registers allow
    float kept[KEEP ? NV : 1][8], dw[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
        if (KEEP) load_weights<T>(p, vec_channel(r + k * TPR < nv ? r + k * TPR : nv - 1, p.D), kept[KEEP ? k : 0]);
    }
    auto weights = [&](int k, float (&w)[8]) {
        if (KEEP)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = kept[KEEP ? k : 0][j];
        else load_weights<T>(p, vec_channel(r + k * TPR < nv ? r + k * TPR : nv - 1, p.D), w);
    };
    const int64_t steps = (p.rows + ROWS - 1) / ROWS;
    // raw vectors of this row and, where the registers allow, of the next one
    constexpr bool AHEAD = TPR <= 256;
    Vec8<T> vh[NV], vd[NV], ve[NV];
    auto request = [&](int64_t b) {
        int64_t row = b * ROWS + sub;
        if (row >= p.rows) row = p.rows - 1;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = r + k * TPR < nv ? r + k * TPR : nv - 1, c = vec_channel(i, p.D);
            vec_load_stream(vh[k], static_cast<const T *>(p.x) + row * p.D, c, p.D);
            vec_load_stream(vd[k], static_cast<const T *>(p.dy) + row * p.D, c, p.D);
            vec_load_stream(ve[k], static_cast<const T *>(p.dh ? p.dh : p.x) + row * p.D, c, p.D);
        }
    };
    if (AHEAD && (int64_t)blockIdx.x < steps) request(blockIdx.x);
    int turn = 0;  // the row's sums alternate between two places, so that one barrier a row is enough
    for (int64_t b = blockIdx.x; b < steps; b += gridDim.x, turn ^= 1) {
        const int64_t row = b * ROWS + sub;
        const bool live = row < p.rows;
        if (!AHEAD) request(b);
        Vec8<T> ch[NV], cd[NV], ce[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) ch[k] = vh[k], cd[k] = vd[k], ce[k] = ve[k];
        if (AHEAD) request(b + gridDim.x < steps ? b + gridDim.x : b);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = r + k * TPR;
            float h[8], g[8], w[8];
            ch[k].get(h);
            cd[k].get(g);
            weights(k, w);
            if (i < nv) {
                const int from = own_from(i, vec_channel(i, p.D));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j >= from) {
                        ss += h[j] * h[j];
                        sg += g[j] * w[j] * h[j];
                    }
            }
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            ss += shfl_xor(ss, m);
            sg += shfl_xor(sg, m);
        }
        if constexpr (TPR > 64) {
            const int wv = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) lds[turn][wv] = make_float2(ss, sg);
            __syncthreads();
            float2 a = lds[turn][0];
#pragma unroll
            for (int i = 1; i < TPR / 64; ++i) {
                const float2 o = lds[turn][i];
                a.x += o.x;
                a.y += o.y;
            }
            ss = a.x;
            sg = a.y;
        }
        const float rs = 1.f / sqrtf(ss / (float)p.D + p.eps);
        const float m = rs * rs * rs * (sg / (float)p.D);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = r + k * TPR;
            if (live && i < nv) {
                float h[8], g[8], e[8], d[8], w[8];
                weights(k, w);
                ch[k].get(h);
                cd[k].get(g);
                ce[k].get(e);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[j] = rs * (g[j] * w[j]) - h[j] * m;
                    dw[k][j] += g[j] * (h[j] * rs);
                    if (p.dh) d[j] += e[j];
                }
                Vec8<T> o;
                o.set(d);
                vec_store(o, static_cast<T *>(p.dx) + row * p.D, vec_channel(i, p.D), p.D);
            }
        }
    }
    if constexpr (ROWS > 1) {  // the workgroup's rows, in order
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) join[threadIdx.x * 8 + j] = dw[k][j];
            __syncthreads();
            if (sub == 0)
                for (int q = 1; q < ROWS; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) dw[k][j] += join[(q * TPR + r) * 8 + j];
        }
        if (sub != 0) return;
    }
    float *out = p.partial + (int64_t)blockIdx.x * p.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = r + k * TPR;
        if (i < nv) {
            const int c = vec_channel(i, p.D);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= own_from(i, c) && c + j < p.D) out[c + j] = dw[k][j];
        }
    }
}

// dweight from the workgroups' partials.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float *partial, float *out, int blocks, int n) {
    const int i = blockIdx.x * 64 + (threadIdx.x & 63);
    const float s = sum_rows(partial, blocks, n, i);
    if (threadIdx.x < 64 && i < n) out[i] = s;
}

// Threads of a row and vectors of a thread for D values: one wave up to 1024, so that a
// row's sums need no barrier; then a workgroup of 256, then of 1024.
struct Shape { int tpr, nv; };
Shape shape_of(int D) {
    const int v = vec_count(D);
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    if (v <= 256) return {256, 1};
    if (v <= 512) return {256, 2};
    if (v <= 1024) return {256, 4};
    return v <= 2048 ? Shape{1024, 2} : Shape{1024, 4};
}

template <typename T, int TPR, int NV> hipError_t fwd(const NormParams &p, bool fp8, hipStream_t s) {
    constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
    const int64_t grid = (p.rows + ROWS - 1) / ROWS;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (fp8) hipLaunchKernelGGL((norm_fwd_kernel<T, TPR, NV, true>), dim3((unsigned)grid), dim3(THREADS), 0, s, p);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, TPR, NV, false>), dim3((unsigned)grid), dim3(THREADS), 0, s, p);
    return hipGetLastError();
}
template <typename T, int TPR, int NV> hipError_t bwd(const NormParams &p, hipStream_t s) {
    constexpr int THREADS = TPR > 256 ? TPR : 256;
    const int blocks = norm_bwd_blocks(p);
    if (blocks > 0) {
        hipLaunchKernelGGL((norm_bwd_kernel<T, TPR, NV>), dim3(blocks), dim3(THREADS), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_sum_kernel, dim3((p.D + 63) / 64), dim3(1024), 0, s, (const float *)p.partial, p.dweight,
                       blocks, p.D);
    return hipGetLastError();
}

#define KDA_NORM_SHAPES(T, CALL)                                       \
    switch (q.tpr * 16 + q.nv) {                                       \
    case 64 * 16 + 1: return CALL<T, 64, 1>;                           \
    case 64 * 16 + 2: return CALL<T, 64, 2>;                           \
    case 256 * 16 + 1: return CALL<T, 256, 1>;                         \
    case 256 * 16 + 2: return CALL<T, 256, 2>;                         \
    case 256 * 16 + 4: return CALL<T, 256, 4>;                         \
    case 1024 * 16 + 2: return CALL<T, 1024, 2>;                       \
    default: return CALL<T, 1024, 4>;                                  \
    }

typedef hipError_t (*FwdFn)(const NormParams &, bool, hipStream_t);
typedef hipError_t (*BwdFn)(const NormParams &, hipStream_t);
template <typename T> FwdFn fwd_fn(const Shape &q) { KDA_NORM_SHAPES(T, fwd) }
template <typename T> BwdFn bwd_fn(const Shape &q) { KDA_NORM_SHAPES(T, bwd) }

}  // namespace

// Three workgroups for each CU, what the registers hold at once (D <= 4096 in bf16): 8192 rows of
// 4096 took 75 us; 1024 workgroups, a third of them in a second turn, 101 us.
int norm_bwd_blocks(const NormParams &p) {
    const Shape q = shape_of(p.D);
    const int rows = q.tpr >= 256 ? 1 : 256 / q.tpr;
    const int64_t steps = (p.rows + rows - 1) / rows;
    return (int)(steps < 768 ? steps : 768);
}

hipError_t launch_norm_fwd(const NormParams &p, bool fp8, hipStream_t s) {
    const Shape q = shape_of(p.D);
    return p.x_bf16 ? fwd_fn<uint16_t>(q)(p, fp8, s) : fwd_fn<float>(q)(p, fp8, s);
}

hipError_t launch_norm_bwd(const NormParams &p, hipStream_t s) {
    const Shape q = shape_of(p.D);
    return p.x_bf16 ? bwd_fn<uint16_t>(q)(p, s) : bwd_fn<float>(q)(p, s);
}

}  // namespace kda
