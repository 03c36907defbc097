// kda_layer_ssm.h -- the state space scan's device code: tiles and fragments, the chunk
// preparation and the pass that carries states over chunks, shared by forward and backward.
//
// Per head (group g = head / (H / G) of B and C), with d_t the step and A = -exp(A_log):
//     S_t = e^{d_t A} S_{t-1} + d_t B_t x_t^T,   y_t = S_t^T C_t + D x_t
// In chunks of L tokens, cum_i the sum of d A up to token i inside the chunk, S0 its first
// state, all as matrix products:
//     y_i = sum_{j <= i} (C_i . B_j) e^{cum_i - cum_j} d_j x_j + e^{cum_i} S0^T C_i + D x_i
//     S0' = e^{cum_L} S0 + sum_j e^{cum_L - cum_j} d_j B_j x_j^T
#pragma once

#include "kda_layer.h"
#include "kda_layer_device.h"

namespace kda {

template <typename T> struct ChunkLen { static constexpr int value = sizeof(T) == 2 ? 64 : 32; };

// ------------------------------------------------------------------ fragments and products
// A fragment is a lane's eight contraction elements for one row (or column) of a 16x16
// product over 32 (see kda_device.h); lane l has row r = l & 15 and lane group g = l >> 4.
// "std" order: elements 8 g + i.  "perm" order: 4 g + i and 16 + 4 g + i (i < 4), the order
// in which a pair of accumulator tiles already lies.  Both operands of a product take the
// same order, so either gives the same sums.
template <typename T> struct Frag;
template <> struct Frag<uint16_t> { uint4 u; };
template <> struct Frag<float> { float a[8]; };

__device__ __forceinline__ f32x4 mma(f32x4 acc, const Frag<uint16_t> &a, const Frag<uint16_t> &b) {
    return mma32_bf16(acc, a.u, b.u);
}
__device__ __forceinline__ f32x4 mma(f32x4 acc, const Frag<float> &a, const Frag<float> &b) {
    return mma32<true>(acc, a.a, b.a);
}

// Rows of a row-major tile in LDS: p points at the lane's row and the block's first element.
template <bool PERM> __device__ __forceinline__ Frag<uint16_t> row_frag(const uint16_t *p, int g) {
    Frag<uint16_t> f;
    if constexpr (PERM) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p + 4 * g), b = *reinterpret_cast<const uint2 *>(p + 16 + 4 * g);
        f.u = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        f.u = *reinterpret_cast<const uint4 *>(p + 8 * g);
    }
    return f;
}
template <bool PERM> __device__ __forceinline__ Frag<float> row_frag(const float *p, int g) {
    Frag<float> f;
    const float4 a = *reinterpret_cast<const float4 *>(p + (PERM ? 4 : 8) * g);
    const float4 b = *reinterpret_cast<const float4 *>(p + (PERM ? 16 + 4 * g : 8 * g + 4));
    f.a[0] = a.x; f.a[1] = a.y; f.a[2] = a.z; f.a[3] = a.w;
    f.a[4] = b.x; f.a[5] = b.y; f.a[6] = b.z; f.a[7] = b.w;
    return f;
}

// Columns of a row-major tile: element i is row k + i of the lane's column.  Column of lane r:
// col + r, or with WIDE col + 8 (r / 4) + r % 4, so that two tiles (col and col + 4) give a
// lane group eight consecutive columns.  Two-byte columns come by the transposing LDS read:
// the 16 lanes of a group address a 4 x 16 block, each four columns of one row, and each
// receives one column's four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <bool PERM, bool WIDE>
__device__ __forceinline__ Frag<uint16_t> col_frag(const uint16_t *tile, int ld, int col, int r, int g) {
    const uint16_t *p = tile + (r >> 2) * ld + col + (WIDE ? 8 : 4) * (r & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + (PERM ? 4 : 8) * g * ld));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + (PERM ? 16 + 4 * g : 8 * g + 4) * ld));
    Frag<uint16_t> f;
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    f.u = make_uint4(x.x, x.y, y.x, y.y);
    return f;
}
template <bool PERM, bool WIDE>
__device__ __forceinline__ Frag<float> col_frag(const float *tile, int ld, int col, int r, int g) {
    const float *p = tile + col + (WIDE ? 8 * (r >> 2) + (r & 3) : r);
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.a[i] = p[(PERM ? 4 * g + (i & 3) + 16 * (i >> 2) : 8 * g + i) * ld];
    return f;
}

// Eight fp32 values as a fragment, and as two (high and low part) for two-byte types: the low
// part is the rounding error of the high one, rounded, so their sum keeps 17 bits.
__device__ __forceinline__ uint32_t pack_bf(float a, float b) { return (uint32_t)f2bf(a) | ((uint32_t)f2bf(b) << 16); }
__device__ __forceinline__ float rest_bf(float v) {
    const float d = v - bf2f(f2bf(v));
    return d == d ? d : 0.f;  // an infinity has no rest
}
__device__ __forceinline__ Frag<uint16_t> to_frag(const float (&v)[8], uint16_t) {
    Frag<uint16_t> f;
    f.u = make_uint4(pack_bf(v[0], v[1]), pack_bf(v[2], v[3]), pack_bf(v[4], v[5]), pack_bf(v[6], v[7]));
    return f;
}
__device__ __forceinline__ Frag<float> to_frag(const float (&v)[8], float) {
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.a[i] = v[i];
    return f;
}
__device__ __forceinline__ void from_frag(const Frag<uint16_t> &f, float (&v)[8]) {
    const uint32_t w[4] = {f.u.x, f.u.y, f.u.z, f.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void from_frag(const Frag<float> &f, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f.a[i];
}
__device__ __forceinline__ Frag<uint16_t> load_frag(const uint16_t *p) {
    Frag<uint16_t> f;
    f.u = *reinterpret_cast<const uint4 *>(p);
    return f;
}
__device__ __forceinline__ Frag<float> load_frag(const float *p) { return row_frag<false>(p, 0); }
__device__ __forceinline__ void store_frag(uint16_t *p, const Frag<uint16_t> &f) { *reinterpret_cast<uint4 *>(p) = f.u; }
__device__ __forceinline__ void store_frag(float *p, const Frag<float> &f) {
    *reinterpret_cast<float4 *>(p) = make_float4(f.a[0], f.a[1], f.a[2], f.a[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f.a[4], f.a[5], f.a[6], f.a[7]);
}

// -------------------------------------------------------------------- sequences and chunks
// Unit `idx` (a chunk, or a segment of `seg` chunks) of the batch: its sequence, its number
// there, the sequence's first chunk and number of chunks.  Packed batches search the offsets
// with the whole workgroup (a prefix sum over the sequences' counts); a sequence without a
// token has no chunk but one segment, which hands its state on.
struct Unit { int n, local, chunk0, chunks; };
template <int THREADS, bool SEGS>
__device__ Unit locate(const SsmParams &p, int idx) {
    if (!p.cu_seqlens) {
        const int chunks = (p.T + p.L - 1) / p.L;
        const int per = SEGS ? (chunks > p.seg ? (chunks + p.seg - 1) / p.seg : 1) : chunks;
        const int n = idx / per;
        return {n, idx % per, n * chunks, chunks};
    }
    __shared__ int wave_units[THREADS / 64], wave_chunks[THREADS / 64];
    __shared__ int found[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if (tid == 0) found[0] = -1;
    int units0 = 0, chunks0 = 0;
    for (int base = 0; base < p.NS; base += THREADS) {
        const int n = base + tid;
        int chunks = 0, units = 0;
        if (n < p.NS) {
            const SeqSpan q = seq_span(p, n);
            chunks = (int)((q.end - q.first + p.L - 1) / p.L);
            units = SEGS ? (chunks > p.seg ? (chunks + p.seg - 1) / p.seg : 1) : chunks;
        }
        int cu = units, cc = chunks;  // inclusive sums over the wave
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int a = __shfl_up(cu, o, 64), b = __shfl_up(cc, o, 64);
            if (lane >= o) cu += a, cc += b;
        }
        if (lane == 63) wave_units[w] = cu, wave_chunks[w] = cc;
        __syncthreads();
        int u = units0 + cu - units, c = chunks0 + cc - chunks;
        for (int i = 0; i < w; ++i) u += wave_units[i], c += wave_chunks[i];
        if (idx >= u && idx < u + units) found[0] = n, found[1] = idx - u, found[2] = c, found[3] = chunks;
        for (int i = 0; i < THREADS / 64; ++i) units0 += wave_units[i], chunks0 += wave_chunks[i];
        __syncthreads();
        if (found[0] >= 0) break;
    }
    if (found[0] < 0) return {0, 0, 0, 0};  // only where the device's offsets are not the host's
    return {found[0], found[1], found[2], found[3]};
}

// A tile [rows of L][W columns] of a matrix whose rows are tokens: each of the workgroup's
// threads has up to K vectors of eight columns.  Rows past `len` are 0.
template <typename T, int L, int W8MAX, int THREADS> struct Tile {
    static constexpr int K = (L * W8MAX + THREADS - 1) / THREADS;
    Vec8<T> v[K];
    __device__ __forceinline__ void request(const T *base, int64_t stride, int w8, int len) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = threadIdx.x + k * THREADS, row = e / w8, c = e - row * w8;
            if (row < len) v[k].load(base + row * stride + 8 * c);
            else v[k].zero();
        }
    }
    template <typename F> __device__ __forceinline__ void each(int w8, F f) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = threadIdx.x + k * THREADS, row = e / w8, c = e - row * w8;
            if (row < L) f(v[k], row, 8 * c, k);
        }
    }
    __device__ __forceinline__ void put(T *lds, int ld, int w8) const {
        each(w8, [&](const Vec8<T> &x, int row, int c, int) { __builtin_memcpy(lds + row * ld + c, &x, sizeof(x)); });
    }
};

// The 16x16 blocks (it, jt) of an [i][j] matrix of a chunk that a causal product needs, block k of
// L / 16 = 2 or 4 rows of blocks: jt <= it, and jt = it + 1 for even it, whose zeros share a
// 32-wide contraction block with the diagonal.
__device__ __forceinline__ void causal_block(int k, int &it, int &jt) {
    it = k < 4 ? k >> 1 : 2 + ((k - 4) >> 2);
    jt = k < 4 ? k & 1 : (k - 4) & 3;
}

// Column of accumulator row / fragment row r of tile t in a 32-wide block pair: tiles 2 b and
// 2 b + 1 share the block's columns in fours.
__device__ __forceinline__ int wide_col(int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); }

// ------------------------------------------------------------------------- states over chunks
// A workgroup carries the state of one (sequence, segment, head) over the segment's chunks,
// for a tile of the state: the whole contraction dimension c of the product that will read it
// (n for y, p in the backward) by 64 of the other, o.  With `rev` it is the gradient of the
// states, from the last chunk to the first: R' = e^{cum_L} R + sum_i e^{cum_i} C_i dy_i^T.
// FIRST: the segment's end from a zero start goes to seg_end (all segments but a sequence's
// last).  Otherwise it starts from the sequence's state joined with the ends of the segments
// before it, stores every chunk's first state in the order in which a lane reads it as a
// fragment, and the last segment writes the final state.
//
// State and sums are fp32.  With two-byte types the scaled x (or dy) is split into a high and
// a low part, two products instead of one, so that a state keeps the precision of an fp32
// one; LO also stores the states in two parts.
template <typename T, bool PC> struct CarryLds {  // PC: c is p
    static constexpr int L = ChunkLen<T>::value;
    static constexpr int PAD = sizeof(T) == 2 ? 16 : 4;
    static constexpr int CLD = 128 + PAD, OLD = 64 + PAD;
    static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    T c[PC ? PARTS : 1][L * CLD];
    T o[PC ? 1 : PARTS][L * OLD];
};

template <typename T, bool PC, bool LO, bool FIRST>
__device__ __forceinline__ void carry(const SsmParams &p, CarryLds<T, PC> &lds, int seg_idx, int h, int ob, bool rev) {
    using M = CarryLds<T, PC>;
    constexpr int L = M::L, PARTS = M::PARTS, KS = L / 32;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
    const int CD = PC ? p.P : p.N, OD = PC ? p.N : p.P;
    const int o0 = 64 * ob, ow = OD - o0 < 64 ? OD - o0 : 64;
    const Unit u = locate<256, true>(p, seg_idx);
    const int segs = u.chunks > p.seg ? (u.chunks + p.seg - 1) / p.seg : 1;
    const int rank = rev ? segs - 1 - u.local : u.local;  // segments that come before this one
    if (FIRST && rank == segs - 1) return;                // the last one's end is nobody's start
    const int first = u.local * p.seg, count = u.chunks - first < p.seg ? u.chunks - first : p.seg;

    // the wave's part: one block of 32 along c, and of the four o tiles all, two or one
    const int cblocks = CD / 32, osplit = cblocks == 1 ? 4 : cblocks == 2 ? 2 : 1, ot = 4 / osplit;
    const int cb = w / osplit, t0 = (w % osplit) * ot;
    const bool active = cb < cblocks;
    f32x4 acc[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[a][t] = zero4();
    // (c, o) of acc[a][t][j]
    auto c_of = [&](int a, int j) { return 32 * cb + 16 * a + 4 * g + j; };
    auto o_of = [&](int t) { return o0 + wide_col(t0 + t, r); };
    auto live = [&](int t) { return active && t < ot && o0 + 16 * (t0 + t) < OD; };
    const size_t state = (size_t)p.N * p.P;
    auto at = [&](int a, int t, int j) { return PC ? (size_t)o_of(t) * p.P + c_of(a, j) : (size_t)c_of(a, j) * p.P + o_of(t); };
    const size_t head_seg = ((size_t)(rev ? p.total_segs : 0) + seg_idx) * p.H + h;
    // Units of 32 (c) by 16 (o) in the order in which the next kernels read them; a unit is 512
    // values: 64 lanes' eight in a fragment.
    auto unit = [&](int t) { return ((size_t)cb * (OD / 16) + 4 * ob + t0 + t) * 512; };
    auto native = [&](size_t hs, int a, int t) { return p.seg_end + hs * state + unit(t) + a * 256 + lane * 4; };

    if constexpr (!FIRST) {
        const float *init = rev ? p.dht : p.h0;
        if (init)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (live(t))
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[a][t][j] = init[((size_t)u.n * p.H + h) * state + at(a, t, j)];
        for (int k = 0; k < rank; ++k) {
            const size_t hs = head_seg + (size_t)((rev ? rank - k : k - rank) * (int64_t)p.H);
            const float f = p.seg_dec[hs];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (live(t))
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float4 e = *reinterpret_cast<const float4 *>(native(hs, a, t));
                        acc[a][t][0] = acc[a][t][0] * f + e.x;
                        acc[a][t][1] = acc[a][t][1] * f + e.y;
                        acc[a][t][2] = acc[a][t][2] * f + e.z;
                        acc[a][t][3] = acc[a][t][3] * f + e.w;
                    }
        }
    }

    const int grp = h / (p.H / p.G);
    const T *xm = static_cast<const T *>(rev ? p.dy : p.x) + (int64_t)h * p.P + (PC ? 0 : o0);
    const int64_t xs = rev ? (int64_t)p.H * p.P : p.x_stride;
    const T *bm = static_cast<const T *>(rev ? p.C : p.Bm) + (int64_t)grp * p.N + (PC ? o0 : 0);
    const int64_t bs = rev ? p.c_stride : p.b_stride;
    const int xw8 = (PC ? CD : ow) / 8, bw8 = (PC ? ow : CD) / 8;
    Tile<T, L, PC ? 16 : 8, 256> tx;
    Tile<T, L, PC ? 8 : 16, 256> tb;
    const float *factors = rev ? p.fe : p.fs;
    float dec = 1.f, next_dec = 1.f, scale[decltype(tx)::K];
    auto request = [&](int i) {
        const int c = u.chunk0 + first + (rev ? count - 1 - i : i);
        const int4 ci = p.chunk[c];
        tx.request(xm + (int64_t)ci.x * xs, xs, xw8, ci.y);
        tb.request(bm + (int64_t)ci.x * bs, bs, bw8, ci.y);
        const float *f = factors + ((size_t)c * p.H + h) * L;
#pragma unroll
        for (int k = 0; k < decltype(tx)::K; ++k) {
            const int row = (tid + k * 256) / xw8;
            scale[k] = row < L ? f[row] : 0.f;
        }
        next_dec = p.dec[(size_t)c * p.H + h];
    };
    if (count > 0) request(0);
    float whole = 1.f;
    for (int i = 0; i < count; ++i) {
        const int c = u.chunk0 + first + (rev ? count - 1 - i : i);
        __syncthreads();
        {
            T *hi, *lo;
            if constexpr (PC) hi = lds.c[0], lo = lds.c[PARTS - 1];
            else hi = lds.o[0], lo = lds.o[PARTS - 1];
            const int ld = PC ? M::CLD : M::OLD;
            tx.each(xw8, [&](const Vec8<T> &v, int row, int col, int k) {
                float e[8];
                v.get(e);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] *= scale[k];
                Vec8<T> o;
                o.set(e);
                __builtin_memcpy(hi + row * ld + col, &o, sizeof(o));
                if constexpr (PARTS == 2) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = rest_bf(e[j]);
                    o.set(e);
                    __builtin_memcpy(lo + row * ld + col, &o, sizeof(o));
                }
            });
            tb.put(PC ? lds.o[0] : lds.c[0], PC ? M::OLD : M::CLD, bw8);
        }
        dec = next_dec;
        __syncthreads();
        if (i + 1 < count) request(i + 1);
        if constexpr (!FIRST) {  // the chunk's first state (or last gradient), as fragments over c
            void *const *out = rev ? p.R : p.S;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (live(t)) {
                    const float v[8] = {acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3],
                                        acc[1][t][0], acc[1][t][1], acc[1][t][2], acc[1][t][3]};
                    const size_t pos = ((size_t)c * p.H + h) * state + unit(t) + lane * 8;
                    store_frag(static_cast<T *>(out[0]) + pos, to_frag(v, T()));
                    if constexpr (LO && PARTS == 2) {
                        float e[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = rest_bf(v[j]);
                        store_frag(static_cast<T *>(out[1]) + pos, to_frag(e, T()));
                    }
                }
        } else {
            whole *= dec;
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[a][t] *= dec;
        if (active)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Frag<T> fc[PC ? PARTS : 1][2];
#pragma unroll
                for (int q = 0; q < (PC ? PARTS : 1); ++q)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                        fc[q][a] = col_frag<false, false>(lds.c[q] + 32 * ks * M::CLD, M::CLD, 32 * cb + 16 * a, r, g);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < ot && 16 * (t0 + t) < ow) {
#pragma unroll
                        for (int q = 0; q < (PC ? 1 : PARTS); ++q) {
                            const int tt = t0 + t;
                            const Frag<T> fo = col_frag<false, true>(lds.o[q] + 32 * ks * M::OLD, M::OLD,
                                                                     32 * (tt >> 1) + 4 * (tt & 1), r, g);
#pragma unroll
                            for (int s = 0; s < (PC ? PARTS : 1); ++s)
#pragma unroll
                                for (int a = 0; a < 2; ++a) acc[a][t] = mma(acc[a][t], fc[s][a], fo);
                        }
                    }
            }
    }
    if constexpr (FIRST) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (live(t))
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    *reinterpret_cast<float4 *>(native(head_seg, a, t)) =
                        make_float4(acc[a][t][0], acc[a][t][1], acc[a][t][2], acc[a][t][3]);
        if (tid == 0 && ob == 0) p.seg_dec[head_seg] = whole;
    } else {
        float *out = rev ? p.dh0 : p.ht;
        if (out && rank == segs - 1)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (live(t))
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j) out[((size_t)u.n * p.H + h) * state + at(a, t, j)] = acc[a][t][j];
    }
}

// Workgroups are dealt to the eight XCDs in turn.  Logical index of workgroup b of a grid
// padded to a multiple of eight, so that neighbours (which share B, C or states) run on one
// XCD and meet in its L2.
__device__ __forceinline__ int64_t xcd_order() {
    return (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
}
inline unsigned xcd_grid(int64_t n) { return (unsigned)((n + 7) / 8 * 8); }

// Logical order: direction, segment, head, tile along o (neighbouring heads share B and C).
template <typename T, bool PC, bool LO, bool FIRST>
__global__ void __launch_bounds__(256) ssm_carry_kernel(SsmParams p, int dirs, int otiles) {
    __shared__ CarryLds<T, PC> lds;
    int64_t b = xcd_order();
    if (b >= (int64_t)dirs * p.total_segs * p.H * otiles) return;
    const int ob = (int)(b % otiles);
    b /= otiles;
    const int h = (int)(b % p.H), seg = (int)(b / p.H);
    const bool rev = seg >= p.total_segs;
    carry<T, PC, LO, FIRST>(p, lds, rev ? seg - p.total_segs : seg, h, ob, rev);
}

hipError_t launch_ssm_prep(const SsmParams &p, hipStream_t s);

template <typename T, bool PC, bool LO> hipError_t launch_carry(const SsmParams &p, bool both, hipStream_t s) {
    const int otiles = ((PC ? p.N : p.P) + 63) / 64;
    const int dirs = both ? 2 : 1;
    const int64_t grid = (int64_t)dirs * p.total_segs * otiles * p.H;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX - 8) return hipErrorInvalidValue;
    if (p.max_segs > 1) {
        hipLaunchKernelGGL((ssm_carry_kernel<T, PC, LO, true>), dim3(xcd_grid(grid)), dim3(256), 0, s, p, dirs, otiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((ssm_carry_kernel<T, PC, LO, false>), dim3(xcd_grid(grid)), dim3(256), 0, s, p, dirs, otiles);
    return hipGetLastError();
}

}  // namespace kda
