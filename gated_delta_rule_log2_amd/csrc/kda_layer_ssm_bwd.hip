// kda_layer_ssm_bwd.hip -- gradients of the state space scan: the scans of dC, dB and dx (see
// kda_layer_ssm.h), and the gradients of the steps and decays from what they leave.
//
// A decay e^{d_t A} lies between tokens a < t <= b.  Inside a chunk, with the scans' terms
//   W_ba = (C_b . B_a) e^{cum_b - cum_a} (dy_b . x_a) (a < b),   o_b = e^{cum_b} C_b . S0 dy_b,
//   q_a = d_a e^{cum_L - cum_a} B_a . R x_a,   K = e^{cum_L} <R, S0>  (R behind the chunk):
//   dl_t = sum_{a < t <= b} d_a W_ba + sum_{b >= t} o_b + sum_{a < t} q_a + K
//   dd_t = A dl_t + sum_b W_bt + (C_t . B_t) (dy_t . x_t) + q_t / d_t      (formed without dividing)
//   dA_log = sum W_ba d_a (cum_b - cum_a) + sum o_b cum_b + sum q_a (cum_L - cum_a) + K cum_L
// (no difference of large sums in the last), ddt_bias = sum ddt, dD = sum dy . x.  Across chunks
//   K = <R, S0'> - sum q,   <R, S0'> of the chunk before = K + sum o,
// from the product <R, S> behind the segment that the scan of dB formed (S0' the state behind the
// chunk).  Each step of this chain adds the sums' fp32 rounding, which reaches all of a chunk's steps.
// Where the chain ends at a known value (the product behind the segment before, 0 in front of a
// sequence without an initial state, K = 0 of a chunk that forgets its start), what it is off by
// there is taken back in proportion to the steps.
#include "kda_layer_ssm.h"

namespace kda {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += shfl_xor(v, m);
    return v;
}
// Sum over this lane and the later ones, in 64 bits: it is subtracted from another such sum.
__device__ __forceinline__ double suffix_sum(double v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double a = __shfl_down(v, o, 64);
        if (lane + o < 64) v += a;
    }
    return v;
}

// One workgroup per (segment, head), from the last chunk to the first, a chunk to a wave and a
// token to a lane: ddt, and the chunk's terms of dA_log, ddt_bias and dD.  Bound by latency: 13 us at 8192
// tokens of 32 heads (23 MB) with eight waves, a segment's chunks at once; 19 with four.
constexpr int kStepWaves = 8;
__global__ void __launch_bounds__(64 * kStepWaves) ssm_step_grad_kernel(SsmParams p) {
    __shared__ double o_sum[kStepWaves], q_sum[kStepWaves];
    __shared__ int forgets[kStepWaves];
    const int seg = blockIdx.x / p.H, h = blockIdx.x % p.H, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const Segment sg = segment_of<64 * kStepWaves>(p, seg, true);
    const int tiles = p.N / 16, L = p.L;
    double behind = 0.;  // <R, S0'> behind the last chunk not yet done
    for (int k = 0; k < tiles; ++k) behind += p.w_dot[((size_t)seg * p.H + h) * tiles + k];
    // <R, S> in front of the segment, where it is known
    const bool inner = sg.rank + 1 < sg.segs, anchored = inner || !p.h0;
    double before = 0.;
    if (inner)
        for (int k = 0; k < tiles; ++k) before += p.w_dot[((size_t)(seg - 1) * p.H + h) * tiles + k];
    const float A = -expf(p.A_log[h]);
    for (int k0 = 0; k0 < sg.count; k0 += kStepWaves) {
        const bool mine = k0 + w < sg.count;
        const int c = sg.first + sg.count - 1 - (mine ? k0 + w : k0);
        const size_t chn = (size_t)c * p.H + h;
        const int token = sg.token + (c - sg.first) * L, len = sg.end - token < L ? sg.end - token : L;
        const bool in = lane < L;
        const size_t at = chn * L + (in ? lane : 0);
        float inner_dl = p.w_dl[at], cols = p.w_cols[at], diag = p.w_diag[at], dyx = p.w_qdiag[at];
        const float d = p.d[at], ch = p.ch[at], cl = p.cl[at], lh = p.ch[chn * L + L - 1], ll = p.cl[chn * L + L - 1];
        float o = 0.f, qd = 0.f;
        float os[8], qs[8];  // of at most eight tiles, all requested at once
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const size_t from = (chn * tiles + (k < tiles ? k : 0)) * L + (in ? lane : 0);
            os[k] = p.w_o[from];
            qs[k] = p.w_q[from];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < tiles) o += os[k], qd += qs[k];
        const bool real = lane < len;
        if (!real) inner_dl = cols = diag = dyx = o = qd = 0.f;
        const float q = d * qd;
        const double q_from = suffix_sum(q, lane), q_all = __shfl(q_from, 0, 64);
        const double o_from = suffix_sum(o, lane), o_all = __shfl(o_from, 0, 64);
        // K is a difference, off by some 1e-7 of the sums; where the chunk's whole decay is below
        // fp32's rounding it is 0 to that precision, and the sums' errors end there too
        if (lane == 0) {
            o_sum[w] = o_all;
            q_sum[w] = q_all;
            forgets[w] = lh + ll < -24.f;
        }
        __syncthreads();
        // the chain over these chunks; own: K of this wave's, and the chunk after the last known place
        double K = 0.;
        int from = 0, own_from = 0;
        bool open = false;
        const int m = sg.count - k0 < kStepWaves ? sg.count - k0 : kStepWaves;
        for (int k = 0; k < m; ++k) {
            double through = behind - q_sum[k];
            if (forgets[k]) {
                if (open) K -= through * (2 * (w - own_from) + 1) / (2 * (k - own_from) + 1);
                open = false;
                through = 0.;
                from = k + 1;
            }
            if (k == w) K = through, own_from = from, open = !forgets[k];
            behind = through + o_sum[k];
        }
        if (open && anchored && k0 + m == sg.count) K += (before - behind) * (2 * (w - own_from) + 1) / (2 * (m - own_from));
        const double dl = (double)inner_dl + o_from + (q_all - q_from) + K;
        const float dd = (float)(A * dl) + (cols + diag + qd);
        const float raw = p.softplus ? -dd * expm1f(-d) : dd;  // sigmoid(dt) = 1 - e^-softplus(dt)
        constexpr float kLn2 = 0.6931471805599453f;
        const float s0 = wave_sum(o * (ch + cl) + q * ((lh - ch) + (ll - cl)));
        const float s1 = wave_sum(real ? raw : 0.f), s2 = wave_sum(dyx);
        if (mine) {
            if (real) {
                const int64_t to = ((int64_t)token + lane) * p.H + h;
                if (p.dt_bf16) static_cast<uint16_t *>(p.ddt)[to] = f2bf(raw);
                else static_cast<float *>(p.ddt)[to] = raw;
            }
            if (lane == 0) {
                p.sums[chn * 4] = kLn2 * (p.w_decay[chn] + s0 + (float)K * (lh + ll));
                p.sums[chn * 4 + 1] = s1;
                p.sums[chn * 4 + 2] = s2;
            }
        }
        __syncthreads();
    }
}

// dA_log, ddt_bias and dD: one workgroup per head sums its chunks' terms in a fixed order (latency, 4.5 us).
__global__ void __launch_bounds__(256) ssm_head_sum_kernel(SsmParams p) {
    __shared__ float red[3][256];
    const int h = blockIdx.x, tid = threadIdx.x;
    float s[3] = {0.f, 0.f, 0.f};
    for (int c = tid; c < p.total_chunks; c += 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += p.sums[((size_t)c * p.H + h) * 4 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) red[k][tid] = s[k];
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if (tid < o)
#pragma unroll
            for (int k = 0; k < 3; ++k) red[k][tid] += red[k][tid + o];
        __syncthreads();
    }
    if (tid == 0) {
        p.dA_log[h] = red[0][0];
        if (p.ddt_bias) p.ddt_bias[h] = red[1][0];
        if (p.dD) p.dD[h] = red[2][0];
    }
}

// dB and dC from the parts of the heads, in order.
template <typename T>
__global__ void __launch_bounds__(256) ssm_part_sum_kernel(SsmParams p) {
    const int64_t n = p.tokens * p.G * p.N, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    float b[8], c[8], e[8];
    load8(p.dBp + i, b);
    load8(p.dCp + i, c);
    for (int k = 1; k < p.split; ++k) {
        load8(p.dBp + k * n + i, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] += e[j];
        load8(p.dCp + k * n + i, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] += e[j];
    }
    store8(static_cast<T *>(p.dB) + i, b);
    store8(static_cast<T *>(p.dC) + i, c);
}

template <typename T> hipError_t bwd(const SsmParams &p, hipStream_t s) {
    hipError_t e = launch_segments<T>(p, 2, s);
    if (e == hipSuccess) e = launch_scan<T, kDc>(p, 1, s);
    if (e == hipSuccess) e = launch_scan<T, kDb>(p, 1, s);
    if (e == hipSuccess) e = launch_scan<T, kDx>(p, 1, s);
    if (e != hipSuccess) return e;
    if (p.total_chunks > 0) {
        const int64_t grid = (int64_t)p.total_segs * p.H;
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL(ssm_step_grad_kernel, dim3((unsigned)grid), dim3(64 * kStepWaves), 0, s, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (p.split > 1) {
            const int64_t n = (p.tokens * p.G * p.N + 2047) / 2048;
            if (n > INT32_MAX) return hipErrorInvalidValue;
            hipLaunchKernelGGL(ssm_part_sum_kernel<T>, dim3((unsigned)n), dim3(256), 0, s, p);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    hipLaunchKernelGGL(ssm_head_sum_kernel, dim3(p.H), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_bwd(const SsmParams &p, hipStream_t s) { return p.x_bf16 ? bwd<uint16_t>(p, s) : bwd<float>(p, s); }

}  // namespace kda
