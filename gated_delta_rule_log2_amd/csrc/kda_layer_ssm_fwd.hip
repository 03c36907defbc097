// kda_layer_ssm_fwd.hip -- the state space scan: preparation, joining of segments, the
// forward's scan and the single-token step (the scan itself is in kda_layer_ssm.h).
#include "kda_layer_ssm.h"

namespace kda {

namespace {

// d = softplus(dt + bias) or dt + bias; softplus by max(x, 0) + log(1 + e^-|x|).
__device__ __forceinline__ float step_of(float raw, int softplus) {
    return softplus ? fmaxf(raw, 0.f) + log1pf(expf(-fabsf(raw))) : raw;
}

// For each token of a chunk and head, [chunk][head][L]: the step d, and the sum of log2 decays
// up to the token, ch + cl, in two floats (the sums run in 64 bits: differences of near tokens
// keep fp32 precision however large the chunk's whole decay is).  Tokens past the chunk's end
// have d = 0 and the last token's sum.  A token's log2 decay is held to -200, where 2^x is 0 in
// fp32, so that sums stay finite.
// One workgroup per chunk and eight heads, a wave for two of them, a lane for a token: latency, 6 us for
// 128 chunks of 32 heads (dt is read in runs of eight heads).
constexpr int kPrepHeads = 8;
__global__ void __launch_bounds__(256) ssm_prep_kernel(SsmParams p, int hblocks) {
    const int c = blockIdx.x / hblocks, h0 = (blockIdx.x % hblocks) * kPrepHeads;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const Unit u = locate<256, false>(p, c);
    const SeqSpan q = seq_span(p, u.n);
    const int64_t tok0 = q.first + (int64_t)u.local * p.L;
    const int len = u.chunks == 0 ? 0 : (int)(q.end - tok0 < p.L ? q.end - tok0 : p.L);
    constexpr int K = kPrepHeads / 4;
    float raw[K];
    double a[K];
    const bool in = lane < len;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int h = h0 + K * w + k;
        raw[k] = in && h < p.H ? load_f32(p.dt, (tok0 + lane) * p.dt_stride + h, p.dt_bf16) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int h = h0 + K * w + k < p.H ? h0 + K * w + k : p.H - 1;
        raw[k] = in ? step_of(raw[k] + (p.dt_bias ? p.dt_bias[h] : 0.f), p.softplus) : 0.f;
        a[k] = -exp((double)p.A_log[h]) * 1.4426950408889634 * (double)raw[k];
        if (a[k] < -200.) a[k] = -200.;
        if (!in) a[k] = 0.;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const double b = __shfl_up(a[k], o, 64);
            if (lane >= o) a[k] += b;
        }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int h = h0 + K * w + k;
        if (h >= p.H || lane >= p.L) continue;
        const size_t i = ((size_t)c * p.H + h) * p.L + lane;
        const float hi = (float)a[k];
        p.d[i] = raw[k];
        p.ch[i] = hi;
        p.cl[i] = (float)(a[k] - (double)hi);
    }
}

// The first states of segments from their ends: in place, seg_state[seg] becomes the state that
// reaches the segment, from the sequence's (or dht) on.  Four values to a thread; the next
// segment's end is requested before this one's start is stored.  Bound by memory: 16 segments of 32 heads
// of 128 x 128 are 34 MB read and written in 13.5 us (5 TB/s), 134 MB in 22 us for both directions.
__global__ void __launch_bounds__(256) ssm_join_kernel(SsmParams p) {
    const int state = p.N * p.P, blocks = state / 1024 > 0 ? state / 1024 : 1;
    int64_t b = blockIdx.x;
    const int e4 = ((int)(b % blocks) * 256 + threadIdx.x) * 4;
    b /= blocks;
    const int h = (int)(b % p.H);
    b /= p.H;
    const int n = (int)(b % p.NS);
    const bool rev = b / p.NS;
    // the sequence's first segment and their number
    __shared__ int before[4];
    int seg0 = 0, segs;
    auto count = [&](int m) {
        const SeqSpan q = seq_span(p, m);
        const int chunks = (int)((q.end - q.first + p.L - 1) / p.L);
        return chunks > p.seg ? (chunks + p.seg - 1) / p.seg : 1;
    };
    segs = count(n);
    if (!p.cu_seqlens) {
        seg0 = n * segs;
    } else {
        int s = 0;
        for (int m = threadIdx.x; m < n; m += 256) s += count(m);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
        if ((threadIdx.x & 63) == 0) before[threadIdx.x >> 6] = s;
        __syncthreads();
        seg0 = before[0] + before[1] + before[2] + before[3];
    }
    if (seg0 + segs > p.total_segs) return;  // only where the device's offsets are not the host's
    if (e4 >= state) return;
    const float *init = rev ? p.dht : p.h0;
    f32x4 run = zero4(), next = zero4();
    if (init) run = *reinterpret_cast<const f32x4 *>(init + ((size_t)n * p.H + h) * state + e4);
    auto at = [&](int s) { return (size_t)((rev ? p.total_segs + seg0 + segs - 1 - s : seg0 + s)) * p.H + h; };
    if (segs > 1) next = *reinterpret_cast<const f32x4 *>(p.seg_state + at(0) * state + e4);
    for (int s = 0; s < segs; ++s) {
        const f32x4 end = next;
        if (s + 2 < segs) next = *reinterpret_cast<const f32x4 *>(p.seg_state + at(s + 1) * state + e4);
        *reinterpret_cast<f32x4 *>(p.seg_state + at(s) * state + e4) = run;
        if (s + 1 < segs) run = run * p.seg_dec[at(s)] + end;
    }
}

__device__ __forceinline__ float4 stream4(const float *p) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    return make_float4(v[0], v[1], v[2], v[3]);
}

// One token for each row, its state [N][P] read and written once: bound by HBM, or by latency
// where there are few rows.  A workgroup has a (row, head) and `cols` of the P columns, four to
// a thread; the threads' rows of the state are 256 / (cols / 4) apart.  A slot below 0 or past
// the pool marks a padding row: y = 0 and no state is touched.  The states are loaded past the caches,
// which other layers' states have filled by the next token: 64 rows of 32 heads, 128 x 128 (270 MB) take
// 51 us so (5.3 TB/s), 59 without (states that the last call left in the caches: 32 rows 24 us, 22 without).
template <typename T, int COLS>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmParams p) {
    constexpr int CT = COLS / 4, RT = 256 / CT;
    __shared__ float4 red[256];
    __shared__ float bc[2][128];
    const int ptiles = (p.P + COLS - 1) / COLS;
    int b = blockIdx.x;
    const int p0 = (b % ptiles) * COLS;
    b /= ptiles;
    const int h = b % p.H, row = b / p.H, grp = h / (p.H / p.G);
    const int tid = threadIdx.x, col = p0 + 4 * (tid % CT), n0 = tid / CT;
    T *y = static_cast<T *>(p.y) + ((int64_t)row * p.H + h) * p.P;
    const int slot = p.slots ? p.slots[row] : row;
    if (slot < 0 || slot >= p.num_slots) {
        if (n0 == 0 && col < p.P)
            for (int j = 0; j < 4; ++j) y[col + j] = Store<T>::to(0.f);
        return;
    }
    if (tid < p.N) {
        bc[0][tid] = load_f32(p.Bm, row * p.b_stride + (int64_t)grp * p.N + tid, p.x_bf16);
        bc[1][tid] = load_f32(p.C, row * p.c_stride + (int64_t)grp * p.N + tid, p.x_bf16);
    }
    const float d = step_of(load_f32(p.dt, row * p.dt_stride + h, p.dt_bf16) + (p.dt_bias ? p.dt_bias[h] : 0.f), p.softplus);
    const float a = expf(-expf(p.A_log[h]) * d);
    float x[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
    float *st = p.state + ((int64_t)slot * p.H + h) * p.N * p.P + col;
    constexpr int K = 128 / RT;
    float4 s[K];
    if (col < p.P) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k * RT < p.N) s[k] = stream4(st + (int64_t)(n0 + k * RT) * p.P);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = load_f32(p.x, row * p.x_stride + (int64_t)h * p.P + col + j, p.x_bf16);
    }
    __syncthreads();
    if (col < p.P)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int n = n0 + k * RT;
            if (n < p.N) {
                const float bn = d * bc[0][n], cn = bc[1][n];
                s[k].x = a * s[k].x + bn * x[0];
                s[k].y = a * s[k].y + bn * x[1];
                s[k].z = a * s[k].z + bn * x[2];
                s[k].w = a * s[k].w + bn * x[3];
                *reinterpret_cast<float4 *>(st + (int64_t)n * p.P) = s[k];
                o[0] += cn * s[k].x;
                o[1] += cn * s[k].y;
                o[2] += cn * s[k].z;
                o[3] += cn * s[k].w;
            }
        }
    red[tid] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (n0 == 0 && col < p.P) {
        for (int q = 1; q < RT; ++q) {
            const float4 e = red[q * CT + tid];
            o[0] += e.x;
            o[1] += e.y;
            o[2] += e.z;
            o[3] += e.w;
        }
        const float D = p.D ? p.D[h] : 0.f;
        for (int j = 0; j < 4; ++j) y[col + j] = Store<T>::to(o[j] + D * x[j]);
    }
}

template <typename T> hipError_t step(const SsmParams &p, hipStream_t s) {
    // narrow tiles where whole heads would leave CUs idle
    const bool narrow = (int64_t)p.B * p.H * ((p.P + 127) / 128) < 512;
    const int64_t grid = (int64_t)p.B * p.H * (narrow ? p.P / 32 : (p.P + 127) / 128);
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (narrow) hipLaunchKernelGGL((ssm_step_kernel<T, 32>), dim3((unsigned)grid), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((ssm_step_kernel<T, 128>), dim3((unsigned)grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_prep(const SsmParams &p, hipStream_t s) {
    if (p.total_chunks == 0) return hipSuccess;
    const int hblocks = (p.H + kPrepHeads - 1) / kPrepHeads;
    const int64_t grid = (int64_t)p.total_chunks * hblocks;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ssm_prep_kernel, dim3((unsigned)grid), dim3(256), 0, s, p, hblocks);
    return hipGetLastError();
}

hipError_t launch_ssm_join(const SsmParams &p, int dirs, hipStream_t s) {
    const int64_t state = (int64_t)p.N * p.P, blocks = state / 1024 > 0 ? state / 1024 : 1;
    const int64_t grid = (int64_t)dirs * p.NS * p.H * blocks;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

namespace {
template <typename T> hipError_t fwd(const SsmParams &p, hipStream_t s) {
    const hipError_t e = launch_segments<T>(p, 1, s);
    return e == hipSuccess ? launch_scan<T, kY>(p, 1, s) : e;
}
}  // namespace

hipError_t launch_ssm_fwd(const SsmParams &p, hipStream_t s) { return p.x_bf16 ? fwd<uint16_t>(p, s) : fwd<float>(p, s); }
hipError_t launch_ssm_step(const SsmParams &p, hipStream_t s) { return p.x_bf16 ? step<uint16_t>(p, s) : step<float>(p, s); }

}  // namespace kda
