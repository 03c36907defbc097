// kda_layer_ssm_bwd.hip -- gradients of the state space scan.
//
// The states S0 in front of every chunk and the gradients R behind it come from the passes
// over chunks (kda_layer_ssm.h), fp32 values in two bf16 parts.  With G = C B^T, E_ij =
// e^{cum_i - cum_j} (j <= i), Q = dy x^T and V = dy S0^T, Z = x R^T, a chunk and head has
//   dx_j = d_j (sum_i G_ij E_ij dy_i + e^{cum_L - cum_j} R^T B_j) + D dy_j
//   dC_i = sum_j E_ij d_j Q_ij B_j + e^{cum_i} V_i
//   dB_j = sum_i E_ij d_j Q_ij C_i + d_j e^{cum_L - cum_j} Z_j         (both summed over the group)
// and, for the step and the decay, the terms that hold a decay between two tokens,
//   W_ij = G_ij E_ij Q_ij d_j (j < i),  o_i = e^{cum_i} C_i . V_i,
//   q_j = d_j e^{cum_L - cum_j} B_j . Z_j,  e^{cum_L} <R, S0>:
//   dl_t = sum_{i >= t} (sum_j W_ij + o_i) - sum_{j >= t} sum_i W_ij + sum_{j < t} q_j + e^{cum_L} <R, S0>
//   dd_t = A dl_t + (sum_{i > t} W_it + G_tt Q_tt d_t + q_t) / d_t     (formed without dividing)
//   dA_log = sum_t dl_t d_t A,  ddt_bias = sum_t ddt_t,  dD = sum_t Q_tt
// The sums over decays keep fp32 throughout (the products' operands are inputs, or states in two
// parts); only what ends in dx, dB and dC, which leave in the input's type, is rounded to it
// before its last product.
#include "kda_layer_ssm.h"

namespace kda {

namespace {

constexpr int kBwdThreads = 512, kBwdWaves = kBwdThreads / 64;

template <typename T> struct BwdLds {
    static constexpr int L = ChunkLen<T>::value, IT = L / 16, PAD = sizeof(T) == 2 ? 8 : 4;
    static constexpr int LD = 128 + PAD, GLD = L + PAD;
    T b[L * LD], c[L * LD], x[L * LD], dy[L * LD];
    T rt[128 * LD];          // R [n][p], its high part
    T dg[L * GLD], m[L * GLD];  // E d Q and G E, [i][j]
    float tok[5][L];         // d, ch, cl, fs, fe
    float rows[IT][L], cols[IT][L], diag[L], qdiag[L];  // sums of W by block
    float o[4][L], q[4][L];  // C . V and B . Z by block of n
    float dot[kBwdWaves];    // <R, S0>
};

// Suffix sum (inclusive) over the wave's lanes.
__device__ __forceinline__ float suffix_sum(float v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float a = __shfl_down(v, o, 64);
        if (lane + o < 64) v += a;
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += shfl_xor(v, m);
    return v;
}

// One workgroup per (chunk, group, part of the group's heads); dB and dC stay in registers over
// its heads.  Eight waves: the 16x16 blocks of G and Q are dealt to them in turn; for V, Z, dB
// and dC a wave has 32 columns of n and its share of the tokens, for dx 32 columns of p.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) ssm_bwd_kernel(SsmParams p) {
    using M = BwdLds<T>;
    constexpr int L = M::L, IT = M::IT, LD = M::LD, GLD = M::GLD, PARTS = sizeof(T) == 2 ? 2 : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    M &lds = *reinterpret_cast<M *>(smem);
    int64_t b = xcd_order();
    if (b >= (int64_t)p.total_chunks * p.G * p.split) return;
    const int part = (int)(b % p.split);
    b /= p.split;
    const int grp = (int)(b % p.G), c = (int)(b / p.G);
    const int hg = p.H / p.G, per_part = (hg + p.split - 1) / p.split;
    const int h_first = grp * hg + part * per_part;
    const int h_last = part * per_part + per_part < hg ? h_first + per_part : grp * hg + hg;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
    const int4 ci = p.chunk[c];
    const int64_t tok0 = ci.x;
    const int len = ci.y, n8 = p.N / 8, x8 = p.P / 8, nblocks = p.N / 32, pblocks = p.P / 32;
    {
        Tile<T, L, 16, kBwdThreads> tb, tc;
        tb.request(static_cast<const T *>(p.Bm) + tok0 * p.b_stride + (int64_t)grp * p.N, p.b_stride, n8, len);
        tc.request(static_cast<const T *>(p.C) + tok0 * p.c_stride + (int64_t)grp * p.N, p.c_stride, n8, len);
        tb.put(lds.b, LD, n8);
        tc.put(lds.c, LD, n8);
    }
    __syncthreads();
    // G's blocks (jt <= it, and for the zeros right of the diagonal jt = it | 1): lane has i = 16 it + r,
    // j = 16 jt + 4 g + e
    constexpr int BLOCKS = IT == 4 ? 12 : 4, MAXB = (BLOCKS + kBwdWaves - 1) / kBwdWaves;
    f32x4 gacc[MAXB];
    auto blocks = [&](auto f) {
#pragma unroll
        for (int k = 0; k < MAXB; ++k) {
            int it, jt;
            causal_block(w + kBwdWaves * k, it, jt);
            if (w + kBwdWaves * k < BLOCKS) f(it, jt, gacc[k]);
        }
    };
    blocks([&](int it, int jt, f32x4 &acc) {
        acc = zero4();
        if (jt <= it)
            for (int nb = 0; nb < p.N; nb += 32)
                acc = mma(acc, row_frag<false>(lds.b + (16 * jt + r) * LD + nb, g),
                          row_frag<false>(lds.c + (16 * it + r) * LD + nb, g));
    });
    // a wave's share of [32 columns] x [tokens]: block w / share, tiles it0 .. it0 + its - 1
    struct Share { int block, it0, its; bool live; };
    auto share = [&](int nb) {
        const int by = 8 / nb < IT ? 8 / nb : IT;
        return Share{w / by, (w % by) * ((IT + by - 1) / by), (IT + by - 1) / by, w / by < nb};
    };
    constexpr int QM = IT > 2 ? 2 : 1;  // at least two waves have a block (8 / 4): its <= IT / 2
    const Share sn = share(nblocks), sp = share(pblocks);
    f32x4 db[2][QM], dc[2][QM];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < QM; ++q) db[t][q] = dc[t][q] = zero4();
    const size_t state = (size_t)p.N * p.P;

    for (int h = h_first; h < h_last; ++h) {
        const size_t ch = (size_t)c * p.H + h;
        __syncthreads();  // the previous head's tiles have been read
        {
            Tile<T, L, 16, kBwdThreads> tx, ty;
            tx.request(static_cast<const T *>(p.x) + tok0 * p.x_stride + (int64_t)h * p.P, p.x_stride, x8, len);
            ty.request(static_cast<const T *>(p.dy) + (tok0 * p.H + h) * p.P, (int64_t)p.H * p.P, x8, len);
            if (tid < 5 * L) {
                const int a = tid / L;
                const float *from = a == 0 ? p.d : a == 1 ? p.ch : a == 2 ? p.cl : a == 3 ? p.fs : p.fe;
                lds.tok[a][tid % L] = from[ch * L + tid % L];
            }
            tx.put(lds.x, LD, x8);
            ty.put(lds.dy, LD, x8);
        }
        __syncthreads();

        // Q, W and the two [i][j] matrices
        blocks([&](int it, int jt, const f32x4 &gm) {
            f32x4 q = zero4();
            float mv[4] = {0.f, 0.f, 0.f, 0.f}, dgv[4] = {0.f, 0.f, 0.f, 0.f};
            const int i = 16 * it + r;
            if (jt <= it) {
                for (int pb = 0; pb < p.P; pb += 32)
                    q = mma(q, row_frag<false>(lds.x + (16 * jt + r) * LD + pb, g),
                            row_frag<false>(lds.dy + (16 * it + r) * LD + pb, g));
                const float hi = lds.tok[1][i], lo = lds.tok[2][i];
                float rows = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * jt + 4 * g + e;
                    const float E = j <= i ? __builtin_amdgcn_exp2f((hi - lds.tok[1][j]) + (lo - lds.tok[2][j])) : 0.f;
                    const float dj = lds.tok[0][j];
                    mv[e] = j <= i ? gm[e] * E : 0.f;
                    dgv[e] = j <= i ? E * dj * q[e] : 0.f;
                    float w0 = j < i ? gm[e] * E * q[e] : 0.f;
                    rows += dj * w0;
                    if (it == jt && j == i) {
                        lds.diag[j] = gm[e] * q[e];
                        lds.qdiag[j] = q[e];
                    }
#pragma unroll
                    for (int s = 1; s < 16; s <<= 1) w0 += shfl_xor(w0, s);
                    if (r == 0) lds.cols[it][j] = w0;
                }
                rows = sum_col_groups(rows);
                if (g == 0) lds.rows[jt][i] = rows;
            }
            store4(lds.m + i * GLD + 16 * jt + 4 * g, mv[0], mv[1], mv[2], mv[3]);
            store4(lds.dg + i * GLD + 16 * jt + 4 * g, dgv[0], dgv[1], dgv[2], dgv[3]);
        });

        // V and Z; R goes to LDS on the way
        {
            f32x4 v[2][QM], z[2][QM];
            float dot = 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < QM; ++q) v[t][q] = z[t][q] = zero4();
            if (sn.live) {
                const int sub = sn.it0 / sn.its;
#pragma unroll 1
                for (int kb = 0; kb < pblocks; ++kb) {
                    Frag<T> fx[QM], fy[QM];
#pragma unroll
                    for (int q = 0; q < QM; ++q)
                        if (q < sn.its) {
                            fy[q] = row_frag<true>(lds.dy + (16 * (sn.it0 + q) + r) * LD + 32 * kb, g);
                            fx[q] = row_frag<true>(lds.x + (16 * (sn.it0 + q) + r) * LD + 32 * kb, g);
                        }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const size_t pos = ch * state + ((size_t)kb * (p.N / 16) + 2 * sn.block + t) * 512 + lane * 8;
                        Frag<T> fs[PARTS], fr[PARTS];
#pragma unroll
                        for (int s = 0; s < PARTS; ++s) {
                            fs[s] = load_frag(static_cast<const T *>(p.S[s]) + pos);
                            fr[s] = load_frag(static_cast<const T *>(p.R[s]) + pos);
                        }
#pragma unroll
                        for (int q = 0; q < QM; ++q)
                            if (q < sn.its)
#pragma unroll
                                for (int s = 0; s < PARTS; ++s) {
                                    v[t][q] = mma(v[t][q], fs[s], fy[q]);
                                    z[t][q] = mma(z[t][q], fr[s], fx[q]);
                                }
                        if (sub == t) {  // the block's first two waves share R's copy and <R, S0>
                            float sv[8], rv[8], e[8];
                            from_frag(fs[0], sv);
                            from_frag(fr[0], rv);
                            T *to = lds.rt + wide_col(2 * sn.block + t, r) * LD + 32 * kb + 4 * g;
                            store4(to, rv[0], rv[1], rv[2], rv[3]);
                            store4(to + 16, rv[4], rv[5], rv[6], rv[7]);
                            if constexpr (PARTS == 2) {
                                from_frag(fs[1], e);
#pragma unroll
                                for (int k = 0; k < 8; ++k) sv[k] += e[k];
                                from_frag(fr[1], e);
#pragma unroll
                                for (int k = 0; k < 8; ++k) rv[k] += e[k];
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k) dot += sv[k] * rv[k];
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < QM; ++q)
                    if (q < sn.its) {
                        const int i = 16 * (sn.it0 + q) + r;
                        float cv[8], bv[8], o = 0.f, s = 0.f;
                        load8(lds.c + i * LD + 32 * sn.block + 8 * g, cv);
                        load8(lds.b + i * LD + 32 * sn.block + 8 * g, bv);
                        const float fe = lds.tok[4][i], fsj = lds.tok[3][i];
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o += cv[4 * t + e] * v[t][q][e];
                                s += bv[4 * t + e] * z[t][q][e];
                                dc[t][q][e] += fe * v[t][q][e];
                                db[t][q][e] += fsj * z[t][q][e];
                            }
                        o = sum_col_groups(o);
                        s = sum_col_groups(s);
                        if (g == 0) lds.o[sn.block][i] = o, lds.q[sn.block][i] = s;
                    }
            }
            dot = wave_sum(dot);
            if (lane == 0) lds.dot[w] = dot;
        }
        __syncthreads();

        if (w == kBwdWaves - 1) {  // token scalars: lane t has token t
            const int t = lane < L ? lane : L - 1;
            float rows = 0.f, cols = 0.f, o = 0.f, s = 0.f, dot = 0.f;
            for (int k = 0; k <= t / 16; ++k) rows += lds.rows[k][t];
            for (int k = t / 16; k < IT; ++k) cols += lds.cols[k][t];
            for (int k = 0; k < nblocks; ++k) o += lds.o[k][t], s += lds.q[k][t];
#pragma unroll
            for (int k = 0; k < kBwdWaves; ++k) dot += lds.dot[k];
            const float d = lds.tok[0][t];
            const float after = __builtin_amdgcn_exp2f((lds.tok[1][L - 1] - lds.tok[1][t]) + (lds.tok[2][L - 1] - lds.tok[2][t]));
            const float qd = after * s, in = lane < L ? 1.f : 0.f;
            const float head = suffix_sum(in * (rows + lds.tok[4][t] * o - d * cols), lane);
            const float q = in * d * qd;
            const float before = wave_sum(q) - suffix_sum(q, lane);
            const float dl = head + before + p.dec[ch] * dot;
            const float A = -expf(p.A_log[h]);
            const float dd = A * dl + (cols + lds.diag[t] + qd);
            const float raw = p.softplus ? -dd * expm1f(-d) : dd;  // sigmoid(dt) = 1 - e^-softplus(dt)
            const bool real = lane < len;
            if (real) {
                const int64_t at = (tok0 + lane) * p.H + h;
                if (p.dt_bf16) static_cast<uint16_t *>(p.ddt)[at] = f2bf(raw);
                else static_cast<float *>(p.ddt)[at] = raw;
            }
            const float s0 = wave_sum(real ? dl * d * A : 0.f), s1 = wave_sum(real ? raw : 0.f);
            const float s2 = wave_sum(real ? lds.qdiag[t] : 0.f);
            if (lane == 0) {
                p.sums[ch * 4] = s0;
                p.sums[ch * 4 + 1] = s1;
                p.sums[ch * 4 + 2] = s2;
            }
        }
        // dC and dB: the chunk's own tokens
        if (sn.live)
#pragma unroll
            for (int kb = 0; kb < L / 32; ++kb)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Frag<T> fb = col_frag<false, true>(lds.b + 32 * kb * LD, LD, 32 * sn.block + 4 * t, r, g);
                    const Frag<T> fc = col_frag<false, true>(lds.c + 32 * kb * LD, LD, 32 * sn.block + 4 * t, r, g);
#pragma unroll
                    for (int q = 0; q < QM; ++q)
                        if (q < sn.its) {
                            const int it = sn.it0 + q;
                            if (2 * kb <= it) dc[t][q] = mma(dc[t][q], fb, row_frag<false>(lds.dg + (16 * it + r) * GLD + 32 * kb, g));
                            if (2 * kb + 1 >= it)
                                db[t][q] = mma(db[t][q], fc, col_frag<false, false>(lds.dg + 32 * kb * GLD, GLD, 16 * it, r, g));
                        }
                }
        // dx
        if (sp.live) {
            f32x4 am[2][QM], as[2][QM];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < QM; ++q) am[t][q] = as[t][q] = zero4();
#pragma unroll
            for (int kb = 0; kb < L / 32; ++kb)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Frag<T> fy = col_frag<false, true>(lds.dy + 32 * kb * LD, LD, 32 * sp.block + 4 * t, r, g);
#pragma unroll
                    for (int q = 0; q < QM; ++q)
                        if (q < sp.its && 2 * kb + 1 >= sp.it0 + q)
                            am[t][q] = mma(am[t][q], fy, col_frag<false, false>(lds.m + 32 * kb * GLD, GLD, 16 * (sp.it0 + q), r, g));
                }
#pragma unroll 1
            for (int kb = 0; kb < nblocks; ++kb)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Frag<T> fr = col_frag<false, true>(lds.rt + 32 * kb * LD, LD, 32 * sp.block + 4 * t, r, g);
#pragma unroll
                    for (int q = 0; q < QM; ++q)
                        if (q < sp.its)
                            as[t][q] = mma(as[t][q], fr, row_frag<false>(lds.b + (16 * (sp.it0 + q) + r) * LD + 32 * kb, g));
                }
            const float D = p.D ? p.D[h] : 0.f;
#pragma unroll
            for (int q = 0; q < QM; ++q) {
                const int j = 16 * (sp.it0 + q) + r;
                if (q >= sp.its || j >= len) continue;
                float yv[8], o[8];
                load8(lds.dy + j * LD + 32 * sp.block + 8 * g, yv);
                const float d = lds.tok[0][j], fsj = lds.tok[3][j];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[4 * t + e] = d * am[t][q][e] + fsj * as[t][q][e] + D * yv[4 * t + e];
                store8(static_cast<T *>(p.dx) + ((tok0 + j) * p.H + h) * p.P + 32 * sp.block + 8 * g, o);
            }
        }
    }
    if (!sn.live) return;
#pragma unroll
    for (int q = 0; q < QM; ++q) {
        const int i = 16 * (sn.it0 + q) + r;
        if (q >= sn.its || i >= len) continue;
        const float vb[8] = {db[0][q][0], db[0][q][1], db[0][q][2], db[0][q][3], db[1][q][0], db[1][q][1], db[1][q][2], db[1][q][3]};
        const float vc[8] = {dc[0][q][0], dc[0][q][1], dc[0][q][2], dc[0][q][3], dc[1][q][0], dc[1][q][1], dc[1][q][2], dc[1][q][3]};
        const int64_t at = ((tok0 + i) * p.G + grp) * p.N + 32 * sn.block + 8 * g;
        if (p.split > 1) {
            store8(p.dBp + part * p.tokens * p.G * p.N + at, vb);
            store8(p.dCp + part * p.tokens * p.G * p.N + at, vc);
        } else {
            store8(static_cast<T *>(p.dB) + at, vb);
            store8(static_cast<T *>(p.dC) + at, vc);
        }
    }
}

// dA_log, ddt_bias and dD: one workgroup per head sums its chunks' terms in a fixed order.
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
    hipError_t e = launch_ssm_prep(p, s);
    if (e == hipSuccess) e = launch_carry<T, true, true>(p, true, s);
    if (e != hipSuccess) return e;
    const int64_t grid = (int64_t)p.total_chunks * p.G * p.split;
    if (grid > INT32_MAX - 8) return hipErrorInvalidValue;
    if (grid > 0) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(ssm_bwd_kernel<T>), hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(BwdLds<T>));
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(ssm_bwd_kernel<T>, dim3(xcd_grid(grid)), dim3(kBwdThreads), sizeof(BwdLds<T>), s, p);
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
