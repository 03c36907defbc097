// kda_layer_ssm_fwd.hip -- the state space scan: chunk preparation, the chunk outputs and the
// single-token step (the pass over chunks is in kda_layer_ssm.h, with the formulas).
#include "kda_layer_ssm.h"

namespace kda {

namespace {

// d = softplus(dt + bias) or dt + bias; softplus by max(x, 0) + log(1 + e^-|x|).
__device__ __forceinline__ float step_of(float raw, int softplus) {
    return softplus ? fmaxf(raw, 0.f) + log1pf(expf(-fabsf(raw))) : raw;
}

// For each token of a chunk and head, [chunk][head][L]:
//   d   the step;  ch + cl  the sum of log2 decays up to the token, in two floats (the sums
//   run in 64 bits: differences of near tokens keep fp32 precision however long the chunk's
//   decay is);  fs = d e^{cum_L - cum};  fe = e^{cum};  and dec = e^{cum_L}.
// Tokens past the chunk's end have d = fs = 0 and the last token's sum.  A token's log2 decay
// is held to -200, where 2^x is 0 in fp32, so that sums stay finite.
// One workgroup per chunk and 64 heads: dt comes in rows of heads and leaves in rows of tokens.
__global__ void __launch_bounds__(256) ssm_prep_kernel(SsmParams p, int hblocks) {
    __shared__ float raw[64][65];
    const int c = blockIdx.x / hblocks, h0 = (blockIdx.x % hblocks) * 64;
    const Unit u = locate<256, false>(p, c);
    const SeqSpan q = seq_span(p, u.n);
    const int64_t tok0 = q.first + (int64_t)u.local * p.L;
    const int len = u.chunks == 0 ? 0 : (int)(q.end - tok0 < p.L ? q.end - tok0 : p.L);
    if (threadIdx.x == 0 && h0 == 0) p.chunk[c] = make_int4((int)tok0, len, u.n, u.local);
    for (int e = threadIdx.x; e < p.L * 64; e += 256) {
        const int row = e >> 6, h = h0 + (e & 63);
        raw[row][e & 63] = row < len && h < p.H ? load_f32(p.dt, (tok0 + row) * p.dt_stride + h, p.dt_bf16) : 0.f;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int k = 0; k < 16; ++k) {
        const int h = h0 + 16 * w + k;
        if (h >= p.H) break;
        const bool in = lane < len;
        const float d = in ? step_of(raw[lane < p.L ? lane : 0][16 * w + k] + (p.dt_bias ? p.dt_bias[h] : 0.f), p.softplus) : 0.f;
        double a = -exp((double)p.A_log[h]) * 1.4426950408889634 * (double)d;
        if (a < -200.) a = -200.;
        if (!in) a = 0.;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double b = __shfl_up(a, o, 64);
            if (lane >= o) a += b;
        }
        const double whole = __shfl(a, 63, 64);
        if (lane < p.L) {
            const size_t i = ((size_t)c * p.H + h) * p.L + lane;
            const float hi = (float)a;
            p.d[i] = d;
            p.ch[i] = hi;
            p.cl[i] = (float)(a - (double)hi);
            p.fs[i] = d * __builtin_amdgcn_exp2f((float)(whole - a));
            p.fe[i] = __builtin_amdgcn_exp2f(hi);
        }
        if (lane == 0) p.dec[(size_t)c * p.H + h] = __builtin_amdgcn_exp2f((float)whole);
    }
}

template <typename T> struct OutLds {
    static constexpr int L = ChunkLen<T>::value, PAD = sizeof(T) == 2 ? 8 : 4, XPAD = sizeof(T) == 2 ? 16 : 4;
    static constexpr int LD = 128 + PAD, XLD = 128 + XPAD, MLD = L + PAD;
    T c[L * LD];
    T b[L * LD];  // B, then the masked products M
    T x[L * XLD];
    float d[L], ch[L], cl[L], fe[L];
};

// y of one chunk and head.  Four waves: first the products B_j . C_i of the 16x16 blocks at or
// below the diagonal, dealt to the waves in turn, whose accumulators (a lane has one i and four
// j) become M_ij = (C_i . B_j) e^{cum_i - cum_j} d_j in LDS; then a wave takes 32 columns of y
// (all i, or a share of them where P is small) and adds x^T M^T and, scaled by e^{cum_i}, S0^T C^T,
// whose S0 comes as fragments straight from memory.  Rows of the products are columns of y, so a
// lane ends with eight consecutive values of one token.
template <typename T>
__global__ void __launch_bounds__(256) ssm_out_kernel(SsmParams p) {
    using M = OutLds<T>;
    constexpr int L = M::L, IT = L / 16;
    __shared__ M lds;
    const int64_t b = xcd_order();
    if (b >= (int64_t)p.total_chunks * p.H) return;
    const int h = (int)(b % p.H), c = (int)(b / p.H);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
    const int4 ci = p.chunk[c];
    const int64_t tok0 = ci.x;
    const int len = ci.y, grp = h / (p.H / p.G), n8 = p.N / 8, x8 = p.P / 8;
    {
        Tile<T, L, 16, 256> tb, tc, tx;
        tb.request(static_cast<const T *>(p.Bm) + tok0 * p.b_stride + (int64_t)grp * p.N, p.b_stride, n8, len);
        tc.request(static_cast<const T *>(p.C) + tok0 * p.c_stride + (int64_t)grp * p.N, p.c_stride, n8, len);
        tx.request(static_cast<const T *>(p.x) + tok0 * p.x_stride + (int64_t)h * p.P, p.x_stride, x8, len);
        const size_t i = ((size_t)c * p.H + h) * L;
        for (int k = tid; k < 4 * L; k += 256) {
            const float *from = k < L ? p.d : k < 2 * L ? p.ch : k < 3 * L ? p.cl : p.fe;
            float *to = k < L ? lds.d : k < 2 * L ? lds.ch : k < 3 * L ? lds.cl : lds.fe;
            to[k % L] = from[i + k % L];
        }
        tb.put(lds.b, M::LD, n8);
        tc.put(lds.c, M::LD, n8);
        tx.put(lds.x, M::XLD, x8);
    }
    __syncthreads();
    constexpr int BLOCKS = IT == 4 ? 12 : 4, MAXB = BLOCKS / 4;
    f32x4 gm[MAXB];
    T *m = lds.b;
#pragma unroll
    for (int k = 0; k < MAXB; ++k) {
        int it, jt;
        causal_block(w + 4 * k, it, jt);
        f32x4 acc = zero4();
        if (jt <= it) {
            for (int nb = 0; nb < p.N; nb += 32)
                acc = mma(acc, row_frag<false>(lds.b + (16 * jt + r) * M::LD + nb, g),
                          row_frag<false>(lds.c + (16 * it + r) * M::LD + nb, g));
            const int i = 16 * it + r;
            const float hi = lds.ch[i], lo = lds.cl[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * jt + 4 * g + e;
                const float decay = __builtin_amdgcn_exp2f((hi - lds.ch[j]) + (lo - lds.cl[j]));
                acc[e] = j <= i ? acc[e] * (decay * lds.d[j]) : 0.f;
            }
        }
        gm[k] = acc;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MAXB; ++k) {
        int it, jt;
        causal_block(w + 4 * k, it, jt);
        store4(m + (16 * it + r) * M::MLD + 16 * jt + 4 * g, gm[k][0], gm[k][1], gm[k][2], gm[k][3]);
    }
    __syncthreads();

    const int pblocks = p.P / 32, split = pblocks == 1 ? 4 : pblocks == 2 ? 2 : 1;
    const int pb = w / split, its = (IT + split - 1) / split, it0 = (w % split) * its;
    if (pb >= pblocks) return;
    const T *S0 = static_cast<const T *>(p.S[0]) + ((size_t)c * p.H + h) * p.N * p.P;
    const float D = p.D ? p.D[h] : 0.f;
    f32x4 am[2][IT], as[2][IT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < IT; ++q) am[t][q] = as[t][q] = zero4();
#pragma unroll
    for (int kb = 0; kb < L / 32; ++kb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const Frag<T> fx = col_frag<false, true>(lds.x + 32 * kb * M::XLD, M::XLD, 32 * pb + 4 * t, r, g);
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int it = it0 + q;
                if (q < its && it < IT && it >= 2 * kb)
                    am[t][q] = mma(am[t][q], fx, row_frag<false>(m + (16 * it + r) * M::MLD + 32 * kb, g));
            }
        }
    for (int nb = 0; nb < p.N / 32; ++nb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const Frag<T> fs = load_frag(S0 + ((size_t)nb * (p.P / 16) + 2 * pb + t) * 512 + lane * 8);
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int it = it0 + q;
                if (q < its && it < IT)
                    as[t][q] = mma(as[t][q], fs, row_frag<true>(lds.c + (16 * it + r) * M::LD + 32 * nb, g));
            }
        }
    T *y = static_cast<T *>(p.y) + (tok0 * p.H + h) * p.P + 32 * pb + 8 * g;
#pragma unroll
    for (int q = 0; q < IT; ++q) {
        const int i = 16 * (it0 + q) + r;
        if (q >= its || it0 + q >= IT || i >= len) continue;
        float xv[8], o[8];
        Vec8<T> vx;
        __builtin_memcpy(&vx, lds.x + i * M::XLD + 32 * pb + 8 * g, sizeof(vx));
        vx.get(xv);
        const float fe = lds.fe[i];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * t + e] = am[t][q][e] + fe * as[t][q][e] + D * xv[4 * t + e];
        store8(y + (int64_t)i * p.H * p.P, o);
    }
}

// One token for each row, its state [N][P] read and written once: bound by HBM, or by latency
// where there are few rows.  A workgroup has a (row, head) and `cols` of the P columns, four to
// a thread; the threads' rows of the state are 256 / (cols / 4) apart.  A slot below 0 or past
// the pool marks a padding row: y = 0 and no state is touched.
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
            if (n0 + k * RT < p.N) s[k] = *reinterpret_cast<const float4 *>(st + (int64_t)(n0 + k * RT) * p.P);
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

template <typename T> hipError_t fwd(const SsmParams &p, hipStream_t s) {
    hipError_t e = launch_ssm_prep(p, s);
    if (e == hipSuccess) e = launch_carry<T, false, false>(p, false, s);
    if (e != hipSuccess || p.total_chunks == 0) return e;
    hipLaunchKernelGGL(ssm_out_kernel<T>, dim3(xcd_grid((int64_t)p.total_chunks * p.H)), dim3(256), 0, s, p);
    return hipGetLastError();
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
    const int hblocks = (p.H + 63) / 64;
    const int64_t grid = (int64_t)p.total_chunks * hblocks;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ssm_prep_kernel, dim3((unsigned)grid), dim3(256), 0, s, p, hblocks);
    return hipGetLastError();
}

hipError_t launch_ssm_fwd(const SsmParams &p, hipStream_t s) { return p.x_bf16 ? fwd<uint16_t>(p, s) : fwd<float>(p, s); }
hipError_t launch_ssm_step(const SsmParams &p, hipStream_t s) { return p.x_bf16 ? step<uint16_t>(p, s) : step<float>(p, s); }

}  // namespace kda
