// kda_layer_ssm.h -- the state space scan's device code: one kernel that carries a state over
// chunks of tokens as matrix products, which the forward and each gradient instantiate.
//
// Per head (group g = head / (H / G) of B and C), with d_t the step and A = -exp(A_log):
//     S_t = e^{d_t A} S_{t-1} + d_t B_t x_t^T,   y_t = S_t^T C_t + D x_t
// and, R_t the gradient of the state behind token t, from the last token to the first,
//     R_{t-1} = e^{d_t A} (R_t + C_t dy_t^T)
//     dx_t = d_t (R_t + C_t dy_t^T)^T B_t + D dy_t
//     dC_t = S_t dy_t,   dB_t = d_t (R_t + C_t dy_t^T) x_t     (both summed over a group's heads)
// So y, dx, dC and dB are all the same scan, of a query, a key and a value:
//            query  key  value   direction   state
//       y      C     B     x      forward    S    [n][p]
//       dx     B     C     dy     backward   R    [n][p]
//       dC     dy    x     B      forward    S^T  [p][n]
//       dB     x     dy    C      backward   R^T  [p][n]
// In chunks of L tokens, cum_i the sum of d A up to token i inside the chunk, Z the state in front
// of the chunk (behind it for the backward direction):
//     forward   out_a = sum_{b <= a} (q_a . k_b) e^{cum_a - cum_b} d_b v_b + e^{cum_a} Z^T q_a
//               Z'    = e^{cum_L} Z + sum_b k_b (d_b e^{cum_L - cum_b} v_b)^T
//     backward  out_a = d_a (sum_{b >= a} (q_a . k_b) e^{cum_b - cum_a} v_b + e^{cum_L - cum_a} Z^T q_a)
//               Z'    = e^{cum_L} Z + sum_b k_b (e^{cum_b} v_b)^T
#pragma once

#include <type_traits>

#include "kda_layer.h"
#include "kda_layer_device.h"

namespace kda {

template <typename T> struct ChunkLen { static constexpr int value = sizeof(T) == 2 ? 64 : 32; };

// ------------------------------------------------------------------ fragments and products
// A fragment is a lane's eight contraction elements for one row (or column) of a 16x16 product
// over 32 (see kda_device.h); lane l has row r = l & 15 and lane group g = l >> 4.  "std" order:
// elements 8 g + i.  "perm" order: 4 g + i and 16 + 4 g + i (i < 4), in which a pair of
// accumulator tiles already lies.  Both operands of a product take the same order.
template <typename T> struct Frag;
template <> struct Frag<uint16_t> { uint4 u; };
template <> struct Frag<float> { float a[8]; };

__device__ __forceinline__ f32x4 mma(f32x4 acc, const Frag<uint16_t> &a, const Frag<uint16_t> &b) {
    return mma32_bf16(acc, a.u, b.u);
}
__device__ __forceinline__ f32x4 mma(f32x4 acc, const Frag<float> &a, const Frag<float> &b) {
    return mma32<true>(acc, a.a, b.a);
}

// A tile [rows][W] in LDS (W = 64 or 128).  Two-byte rows fill the 64 banks once (W = 128) or
// half; their 16-byte units are permuted by a function of the row.  The banks serve 32 lanes of an
// 8-byte read at a time, and 16 of a 16-byte read, which are not neighbours: lanes 0-3, 12-15 and
// 20-27, or 4-11, 16-19 and 28-31.  So the function has 16 values over 16 rows, those of rows 0-3 and
// 12-15 in pairs that differ in the last bit (fragments of rows, where lanes 16-31 read the next
// unit), and eight neighbouring rows have it differ above that bit (fragments of columns, over two
// units).  fp32 rows are padded by four.
template <typename T, int W> struct Layout;
template <> struct Layout<uint16_t, 128> {
    static constexpr int LD = 128;
    static __device__ __forceinline__ int at(int row, int col) {
        return row * 128 + (col ^ ((((row & 7) << 1 | (row >> 3 & 1)) ^ (row & 8)) << 3));
    }
};
template <> struct Layout<uint16_t, 64> {
    static constexpr int LD = 64;
    static __device__ __forceinline__ int at(int row, int col) {
        return row * 64 + (col ^ ((((row >> 1 & 3) << 1 | (row >> 3 & 1)) ^ (row >> 1 & 4)) << 3));
    }
};
template <int W> struct Layout<float, W> {
    static constexpr int LD = W + 4;
    static __device__ __forceinline__ int at(int row, int col) { return row * LD + col; }
};

// Eight bytes of LDS by a read of its own: volatile, because two reads at one distance merge into one
// of twice the size, whose 16 lanes at a time then meet in their banks (gradients of 8192 tokens, 32
// heads: 497 us against 512, and half as many LDS cycles; packed forward 152 against 157).
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 read_one(const uint16_t *p) {
    return *(const volatile __attribute__((address_space(3))) u32x2 *)(p);
}

// Row `row`'s elements k0 .. k0 + 31 of the contraction.
template <bool PERM, int W> __device__ __forceinline__ Frag<uint16_t> row_frag(const uint16_t *tile, int row, int k0, int g) {
    using Y = Layout<uint16_t, W>;
    Frag<uint16_t> f;
    if constexpr (PERM) {
        const u32x2 a = read_one(tile + Y::at(row, k0 + 4 * g)), b = read_one(tile + Y::at(row, k0 + 16 + 4 * g));
        f.u = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        f.u = *reinterpret_cast<const uint4 *>(tile + Y::at(row, k0 + 8 * g));
    }
    return f;
}
template <bool PERM, int W> __device__ __forceinline__ Frag<float> row_frag(const float *tile, int row, int k0, int g) {
    const float *p = tile + Layout<float, W>::at(row, k0);
    Frag<float> f;
    const float4 a = *reinterpret_cast<const float4 *>(p + (PERM ? 4 : 8) * g);
    const float4 b = *reinterpret_cast<const float4 *>(p + (PERM ? 16 + 4 * g : 8 * g + 4));
    f.a[0] = a.x; f.a[1] = a.y; f.a[2] = a.z; f.a[3] = a.w;
    f.a[4] = b.x; f.a[5] = b.y; f.a[6] = b.z; f.a[7] = b.w;
    return f;
}

// The lane's column over rows k0 .. k0 + 31, in perm order.  Column of lane r: col + r, or with
// WIDE col + 8 (r / 4) + r % 4, so that two tiles (col and col + 4) give a lane group eight
// consecutive columns.  Two-byte columns come by the transposing LDS read: the 16 lanes of a
// group address a 4 x 16 block, each four columns of one row, and each receives one column's
// four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <bool WIDE, int W>
__device__ __forceinline__ Frag<uint16_t> col_frag(const uint16_t *tile, int k0, int col, int r, int g) {
    using Y = Layout<uint16_t, W>;
    const int row = k0 + 4 * g + (r >> 2), c = col + (WIDE ? 8 : 4) * (r & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(tile + Y::at(row, c)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(tile + Y::at(row + 16, c)));
    Frag<uint16_t> f;
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    f.u = make_uint4(x.x, x.y, y.x, y.y);
    return f;
}
template <bool WIDE, int W>
__device__ __forceinline__ Frag<float> col_frag(const float *tile, int k0, int col, int r, int g) {
    const float *p = tile + Layout<float, W>::at(k0 + 4 * g, col + (WIDE ? 8 * (r >> 2) + (r & 3) : r));
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.a[i] = p[((i & 3) + 16 * (i >> 2)) * Layout<float, W>::LD];
    return f;
}

// Eight fp32 values as a fragment.  For two-byte types a value can be kept in parts, each the
// rounding error of those before it, rounded: two parts hold 16 bits, three all 24 (an infinity
// becomes NaN).
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
template <int PARTS> __device__ __forceinline__ void split(float (&v)[8], Frag<uint16_t> (&f)[PARTS]) {
#pragma unroll
    for (int s = 0; s < PARTS; ++s) {
        f[s] = to_frag(v, uint16_t());
        if (s + 1 < PARTS) {
            float h[8];
            from_frag(f[s], h);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] -= h[j];
        }
    }
}
__device__ __forceinline__ void split(float (&v)[8], Frag<float> (&f)[1]) { f[0] = to_frag(v, float()); }

// Eight tokens' values of one column (perm order from token 0 of `factors`) times their factors.
template <typename T, int PARTS>
__device__ __forceinline__ void scaled(const Frag<T> &f, const float *factors, Frag<T> (&out)[PARTS]) {
    float v[8];
    from_frag(f, v);
    const float4 a = *reinterpret_cast<const float4 *>(factors), b = *reinterpret_cast<const float4 *>(factors + 16);
    v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
    v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
    split(v, out);
}

// Four or eight consecutive values.
__device__ __forceinline__ void load_run(const uint16_t *p, float (&o)[4]) {
    uint2 u;
    __builtin_memcpy(&u, p, 8);
    o[0] = __uint_as_float(u.x << 16); o[1] = __uint_as_float(u.x & 0xffff0000u);
    o[2] = __uint_as_float(u.y << 16); o[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load_run(const float *p, float (&o)[4]) { __builtin_memcpy(o, p, 16); }
template <typename T> __device__ __forceinline__ void load_run(const T *p, float (&o)[8]) {
    Vec8<T> v;
    __builtin_memcpy(&v, p, sizeof(v));
    v.get(o);
}
__device__ __forceinline__ void store_run(uint16_t *p, const float (&o)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf(o[0], o[1]), pack_bf(o[2], o[3]));
}
__device__ __forceinline__ void store_run(float *p, const float (&o)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(o[0], o[1], o[2], o[3]); }
__device__ __forceinline__ void store_run(uint16_t *p, const float (&o)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf(o[0], o[1]), pack_bf(o[2], o[3]), pack_bf(o[4], o[5]), pack_bf(o[6], o[7]));
}
__device__ __forceinline__ void store_run(float *p, const float (&o)[8]) { store8(p, o); }

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

// The 16x16 blocks (it, jt) of an [i][j] matrix of a chunk that a causal product needs, block k of
// L / 16 = 2 or 4 rows of blocks: jt <= it, and jt = it + 1 for even it, whose zeros share a
// 32-wide contraction block with the diagonal.
__device__ __forceinline__ void causal_block(int k, int &it, int &jt) {
    it = k < 4 ? k >> 1 : 2 + ((k - 4) >> 2);
    jt = k < 4 ? k & 1 : (k - 4) & 3;
}

// Element `off` behind a uniform address: a scalar base and 32 bits to a lane, which is how the
// memory instructions take it (64-bit addresses to a lane, kept over the loop, spill).
template <typename T> __device__ __forceinline__ T *behind(T *base, unsigned off) {
    typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
    return reinterpret_cast<T *>(reinterpret_cast<Byte *>(base) + off * (unsigned)sizeof(T));
}

// A tile [rows of L][W columns] of a matrix whose rows are tokens, on its way to LDS: a thread has
// K vectors of eight columns, 256 / (W / 8) rows apart.  Rows past `len` and columns past `cols`
// are read from places inside and become 0.
template <typename T, int L, int W> struct Tile {
    static constexpr int W8 = W / 8, STEP = 256 / W8, K = L / STEP;
    Vec8<T> v[K];
    int len, cols;
    // One sequence of loads for full and partial tiles: behind a branch each tile's loads would wait
    // for the one's before.
    __device__ __forceinline__ void request(const T *base, int stride, int columns, int length) {
        const unsigned row = threadIdx.x / W8, c = 8 * (threadIdx.x % W8);
        len = length;
        cols = columns;
        const unsigned at = (int)c < cols ? c : 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const unsigned from = row + k * STEP < (unsigned)len ? row + k * STEP : len - 1;
            v[k].load(behind(base, __umul24(from, stride) + at));
        }
    }
    __device__ __forceinline__ void put(T *lds) {
        const int row = threadIdx.x / W8, c = 8 * (threadIdx.x % W8);
        if (len != L || cols != W)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (row + k * STEP >= len || c >= cols) v[k].zero();
#pragma unroll
        for (int k = 0; k < K; ++k) __builtin_memcpy(lds + Layout<T, W>::at(row + k * STEP, c), &v[k], sizeof(v[k]));
    }
};

// Column of accumulator row / fragment row r of tile t in a 32-wide block pair: tiles 2 b and
// 2 b + 1 share the block's columns in fours.
__device__ __forceinline__ int wide_col(int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); }

// A chunk's token factors in LDS, for the forward (backward) direction: the step d, the sum of
// log2 decays in two parts, the value's factor d e^{cum_L - cum} (e^{cum}) in the state's update
// and the state's factor e^{cum} (e^{cum_L - cum}) in the output; e^{cum_L} behind them.
template <int L> struct Tokens {
    float d, ch, cl, lh, ll;
    __device__ __forceinline__ void request(const SsmParams &p, size_t ch_idx) {
        if (threadIdx.x < L) {
            d = *behind(p.d + ch_idx * L, threadIdx.x);
            ch = *behind(p.ch + ch_idx * L, threadIdx.x);
            cl = *behind(p.cl + ch_idx * L, threadIdx.x);
            lh = *behind(p.ch + ch_idx * L + L - 1, 0u);
            ll = *behind(p.cl + ch_idx * L + L - 1, 0u);
        }
    }
    __device__ __forceinline__ void put(float (&tok)[5][L], float &dec, bool rev) const {
        if (threadIdx.x < L) {
            const float after = __builtin_amdgcn_exp2f((lh - ch) + (ll - cl)), before = __builtin_amdgcn_exp2f(ch);
            tok[0][threadIdx.x] = d;
            tok[1][threadIdx.x] = ch;
            tok[2][threadIdx.x] = cl;
            tok[3][threadIdx.x] = rev ? before : d * after;
            tok[4][threadIdx.x] = rev ? after : before;
            if (threadIdx.x == L - 1) dec = before;
        }
    }
};

// A segment's place, all of it uniform: its sequence, the sequence's segments and how many come
// before this one in the direction taken, its first chunk, their number, the first one's first
// token, and the token after the sequence's last.
struct Segment { int n, segs, rank, first, count, token, end; };
template <int THREADS> __device__ __forceinline__ Segment segment_of(const SsmParams &p, int seg, bool rev) {
    const Unit u = locate<THREADS, true>(p, seg);
    const SeqSpan q = seq_span(p, u.n);
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    Segment s;
    s.n = uniform(u.n);
    const int chunks = uniform(u.chunks), local = uniform(u.local);
    s.segs = chunks > p.seg ? (chunks + p.seg - 1) / p.seg : 1;
    s.rank = rev ? s.segs - 1 - local : local;
    s.first = uniform(u.chunk0) + local * p.seg;
    s.count = chunks - local * p.seg < p.seg ? chunks - local * p.seg : p.seg;
    s.token = uniform((int)q.first) + local * p.seg * p.L;
    s.end = uniform((int)q.end);
    return s;
}

// Workgroups are dealt to the eight XCDs in turn.  Logical index of workgroup b of a grid
// padded to a multiple of eight, so that neighbours (which share B, C or states) run on one
// XCD and meet in its L2.
__device__ __forceinline__ int64_t xcd_order() {
    return (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
}
inline unsigned xcd_grid(int64_t n) { return (unsigned)((n + 7) / 8 * 8); }

// ------------------------------------------------------------------------------------ the scan
// The same value, of which the compiler knows nothing: addresses that are formed from it are formed
// anew where they are used (in LDS some 60 for each step, in the final state 64), where kept ones
// would not fit the registers.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
// Instructions stay on their side: without it the scheduler starts so many fragments' reads early
// that registers spill, and a spill's reload waits for every tile load issued before it.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

// Sum over this lane and the later ones of its 16, and the value of a row's first lane.
template <int N> __device__ __forceinline__ float row_shl(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x100 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_suffix16(float x) {
    x += row_shl<1>(x);
    x += row_shl<2>(x);
    x += row_shl<4>(x);
    x += row_shl<8>(x);
    return x;
}
template <int ROW> __device__ __forceinline__ float row_first(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * ROW));
}

enum ScanMode { kFirst, kY, kDx, kDc, kDb };

constexpr bool scan_sums(int mode) { return mode == kDc || mode == kDb; }  // outputs summed over a group's heads
constexpr bool scan_np(int mode) { return mode == kY || mode == kDx; }     // state [n][p], else [p][n]

template <typename T, int KW, int CT, int MODE> struct ScanLds {
    static constexpr int L = ChunkLen<T>::value, VW = 64 * CT;
    T key[L * Layout<T, KW>::LD], val[L * Layout<T, VW>::LD];
    T q[MODE == kFirst ? 4 : L * Layout<T, KW>::LD];
    static constexpr int MPARTS = sizeof(T) == 2 && scan_sums(MODE) ? 2 : 1, MSIZE = L * Layout<T, 64>::LD;
    T m[MODE == kFirst ? 4 : MPARTS * MSIZE];
    T other[MODE == kDx || scan_sums(MODE) ? L * Layout<T, VW>::LD : 4];  // x; or C, B for dC, dB
    float tok[5][L];
    float rows[MODE == kDx ? 4 : 1][L], cols[MODE == kDx ? 4 : 1][L], diag[L], qdiag[L];
    float wave[4], dec;
};

// One (sequence, segment) and head, or up to two heads of a group, and VW = 64 CT columns of the
// value: states Z in registers over the segment's chunks, 16 CT columns and all rows to a wave (KW
// of them; those past the key's columns stay 0).  For each chunk and head
//   - the 16x16 blocks of q k^T that the direction reaches, dealt to the waves in turn, become M,
//     with the decays, in LDS;
//   - out = M v + factor Z^T q, with v^T and Z^T as the left operands: a lane ends with consecutive
//     columns of one token, and the accumulators that hold Z are, in pairs, its fragments;
//   - Z' = decay Z + k^T (factor v).
// For y and dx, M and Z are rounded to the input's type for their products, as y and dx are at
// their store.  Z itself is carried in fp32 and its scaled v goes through the products in three
// bf16 parts, so that it is as exact as an fp32 sum; so does Z for dC and dB, whose dot products
// with C and B (w_o, w_q) are parts of the decays' gradients and leave in fp32.  M has two parts
// there: with one, sums over a group's few heads were off by 1.4 to 1.55 of their final rounding
// (two cost 504 us against 491 in the gradients of 8192 tokens, 32 heads).  The next chunk's tiles
// are requested before this one's products.
// Bound, at 8192 tokens and 32 heads of 128 x 128 in bf16 (512 workgroups, two for each CU by their
// registers, 4.6 TB/s and less): no unit alone.  y takes 75 us, the states before it 43; dx 101, dC and
// dB 150 each, the states of both directions 80.  Of the states' pass the matrix units are busy for 31 %
// and the vector units for 40 %, of dC's for 19 and 43 % with LDS at 23 %; the rest is waiting at the three
// barriers of a step and for operands, with two waves to a SIMD.  More waves with smaller tiles (16
// columns to a wave, three or four workgroups) took as long: they form q k^T twice.
// kFirst: the states of segments from zero to seg_state (all but a sequence's last segment), the
// scan of dC or, in the second half of the grid, of dB, without outputs.
// kDx also leaves, per chunk and head, the sums over W_ba = (C_b . B_a) e^{cum_b - cum_a} (dy_b . x_a),
// b > a: for each t over a < t <= b with d_a (w_dl), over b (w_cols), over both with d_a (cum_b - cum_a) in log2
// (w_decay), and its diagonal without and with only dy . x (w_diag, w_qdiag).
template <typename T, int KW, int CT, int MODE>
__global__ void __launch_bounds__(256, 2) ssm_scan_kernel(SsmParams p, int slices, int dirs) {
    using M = ScanLds<T, KW, CT, MODE>;
    constexpr int L = M::L, IT = L / 16, KS = L / 32, VW = M::VW, NT = KW / 16, RUN = 4 * CT;
    constexpr bool SUMS = scan_sums(MODE), NP = scan_np(MODE), OUT = MODE != kFirst, REV = MODE == kDx || MODE == kDb;
    constexpr int HN = SUMS ? 2 : 1, PARTS = sizeof(T) == 2 ? 3 : 1, ZPARTS = SUMS ? PARTS : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    M &lds = *reinterpret_cast<M *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane_g = lane >> 4, lane_r = lane & 15;
    int64_t idx = xcd_order();
    const int units = SUMS ? p.G * p.split : p.H;
    if (idx >= (int64_t)dirs * p.total_segs * units * slices) return;
    const int slice = (int)(idx % slices);
    idx /= slices;
    const int unit = (int)(idx % units), dseg = (int)(idx / units);
    const int seg = dseg >= p.total_segs ? dseg - p.total_segs : dseg;
    const bool rev = OUT ? REV : dseg >= p.total_segs;
    const Segment sg = segment_of<256>(p, seg, rev);
    if (!OUT && sg.rank == sg.segs - 1) return;  // the last one's end is nobody's start
    const int hg = p.H / p.G, per = (hg + p.split - 1) / p.split, part = SUMS ? unit % p.split : 0;
    const int h0 = SUMS ? unit / p.split * hg + part * per : unit;
    const int nheads = !SUMS ? 1 : per < hg - part * per ? per : hg - part * per;
    const int grp = h0 / hg;

    const int KD = NP ? p.N : p.P, VD = NP ? p.P : p.N, v0 = VW * slice, vcols = VD - v0 < VW ? VD - v0 : VW;
    const int c0 = v0 + 16 * CT * w, run0 = c0 + (CT == 2 ? 8 : 4) * lane_g;  // the wave's columns; the lane's in an output
    const int tile = c0 / 16;
    const bool active = c0 < VD;
    const size_t state = (size_t)p.N * p.P;
    // Z[.][i][ct][j] in an [n][p] state: a uniform part and the lane's
    const int col0 = c0 + (CT == 2 ? wide_col(0, lane_r) : lane_r), own = NP ? 4 * lane_g * p.P + col0 : col0 * p.P + 4 * lane_g;
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            if (16 * i < KD)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int j = 0; j < 4; ++j) f(i, ct, j, NP ? (16 * i + j) * p.P + 4 * ct : 4 * ct * p.P + 16 * i + j);
    };

    f32x4 Z[HN][NT][CT];
    const float *init = rev ? p.dht : p.h0;
#pragma unroll
    for (int hh = 0; hh < HN; ++hh) {
        const float *from = nullptr;
        if (OUT) {
            if (p.max_segs > 1) from = p.seg_state + ((size_t)(rev ? p.total_segs + seg : seg) * p.H + h0 + hh) * state;
            else if (init) from = init + ((size_t)sg.n * p.H + h0 + hh) * state;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) Z[hh][i][ct] = zero4();
        if (from && active && hh < nheads) each([&](int i, int ct, int j, int at) { Z[hh][i][ct][j] = *behind(from + at, own); });
    }
    if constexpr (MODE == kDb) {
        // <R, S> behind the segment: S is the next segment's first state, or the sequence's last one
#pragma unroll
        for (int hh = 0; hh < HN; ++hh) {
            float dot = 0.f;
            const float *s = sg.rank == 0 ? p.last_state + ((size_t)sg.n * p.H + h0 + hh) * state
                                          : p.seg_state + ((size_t)(seg + 1) * p.H + h0 + hh) * state;
            if (active && hh < nheads) each([&](int i, int ct, int j, int at) { dot += Z[hh][i][ct][j] * *behind(s + at, own); });
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) dot += shfl_xor(dot, m);
            if (active && hh < nheads && lane == 0) p.w_dot[((size_t)seg * p.H + h0 + hh) * (p.N / 16) + tile] = dot;
        }
    }

    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    const T *Bm = static_cast<const T *>(p.Bm) + (int64_t)grp * p.N, *Cm = static_cast<const T *>(p.C) + (int64_t)grp * p.N;
    const int xs = (int)p.x_stride, bs = (int)p.b_stride, cs = (int)p.c_stride, ys = p.H * p.P;
    Tile<T, L, KW> tk, tq;
    Tile<T, L, VW> tv, to;
    Tokens<L> tt;
    auto chunk_at = [&](int k) { return sg.first + (rev ? sg.count - 1 - k : k); };
    const float D = !SUMS && OUT && p.D ? p.D[h0] : 0.f;
    auto token_of = [&](int c) { return sg.token + (c - sg.first) * L; };
    auto length_of = [&](int c) { return sg.end - token_of(c) < L ? sg.end - token_of(c) : L; };
    auto request = [&](int c, int h, bool with_val) {
        const int64_t t0 = token_of(c);
        const int len = length_of(c);
        const T *xt = x + t0 * xs + (int64_t)h * p.P, *yt = dy + t0 * ys + (int64_t)h * p.P;
        const T *bt = Bm + t0 * bs, *ct = Cm + t0 * cs;
        if constexpr (MODE == kY) {
            tk.request(bt, bs, KD, len);
            tv.request(xt + v0, xs, vcols, len);
        } else if constexpr (MODE == kDx) {
            tk.request(ct, cs, KD, len);
            tv.request(yt + v0, ys, vcols, len);
            to.request(xt + v0, xs, vcols, len);
        } else {
            tk.request(rev ? yt : xt, rev ? ys : xs, KD, len);
            if (with_val) {
                tv.request((rev ? ct : bt) + v0, rev ? cs : bs, vcols, len);
                if constexpr (OUT) to.request((rev ? bt : ct) + v0, rev ? bs : cs, vcols, len);
            }
        }
        tt.request(p, (size_t)c * p.H + h);
    };
    auto request_q = [&](int c, int h) {  // later than the others: its registers are then free of products
        const int64_t t0 = token_of(c);
        const int len = length_of(c);
        if constexpr (MODE == kY) tq.request(Cm + t0 * cs, cs, KD, len);
        else if constexpr (MODE == kDx) tq.request(Bm + t0 * bs, bs, KD, len);
        else if constexpr (MODE == kDc) tq.request(dy + t0 * ys + (int64_t)h * p.P, ys, KD, len);
        else if constexpr (MODE == kDb) tq.request(x + t0 * xs + (int64_t)h * p.P, xs, KD, len);
    };
    if (sg.count > 0) {
        request(chunk_at(0), h0, true);
        request_q(chunk_at(0), h0);
    }
    float whole = 1.f;
    for (int k = 0; k < sg.count; ++k) {
        const int c = chunk_at(k), len = length_of(c);
        const int64_t t0 = token_of(c);
        f32x4 sum[SUMS ? IT : 1];
#pragma unroll
        for (int i = 0; i < (SUMS ? IT : 1); ++i) sum[i] = zero4();
#pragma unroll
        for (int hh = 0; hh < HN; ++hh) {
            if (hh >= nheads) continue;
            const int h = h0 + hh;
            const size_t chn = (size_t)c * p.H + h;
            const int r = fresh(lane_r) & 15, g = fresh(lane_g) & 3;
            __syncthreads();  // the previous step's tiles have been read
            tk.put(lds.key);
            if constexpr (OUT) tq.put(lds.q);
            if (hh == 0) tv.put(lds.val);
            if (hh == 0 && OUT && MODE != kY) to.put(lds.other);
            tt.put(lds.tok, lds.dec, rev);
            __syncthreads();
            if (hh + 1 < nheads) request(c, h + 1, false);
            else if (k + 1 < sg.count) request(chunk_at(k + 1), h0, true);

            if constexpr (OUT) {
                float wd = 0.f;
#pragma unroll
                for (int s = 0; s < (IT == 4 ? 3 : 1); ++s) {
                    int it, jt;  // block rows of the output's token a = 16 it + r and of the key's b
                    causal_block(w + 4 * s, it, jt);
                    const bool pad = jt > it, diagonal = it == jt;
                    if (REV) it = IT - 1 - it, jt = IT - 1 - jt;
                    f32x4 acc = zero4();
                    const int a = 16 * it + r, b0 = 16 * jt + 4 * g;
                    if (!pad) {
#pragma unroll
                        for (int kb = 0; kb < KW / 32; ++kb)
                            acc = mma(acc, row_frag<false, KW>(lds.key, 16 * jt + r, 32 * kb, g),
                                      row_frag<false, KW>(lds.q, a, 32 * kb, g));
                        f32x4 dyx = zero4();
                        if constexpr (MODE == kDx)
#pragma unroll
                            for (int vb = 0; vb < VW / 32; ++vb)
                                dyx = mma(dyx, row_frag<false, VW>(lds.val, 16 * jt + r, 32 * vb, g),
                                          row_frag<false, VW>(lds.other, a, 32 * vb, g));
                        const float hi = lds.tok[1][a], lo = lds.tok[2][a], da = lds.tok[0][a];
                        float ch[4], cl[4], db[4];
                        load_run(&lds.tok[1][b0], ch);
                        load_run(&lds.tok[2][b0], cl);
                        load_run(&lds.tok[0][b0], db);
                        float cols = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float diff = REV ? (ch[e] - hi) + (cl[e] - lo) : (hi - ch[e]) + (lo - cl[e]);
                            const bool off = diagonal && (REV ? b0 + e < a : b0 + e > a);
                            const float decay = off ? 0.f : __builtin_amdgcn_exp2f(diff);
                            if constexpr (MODE == kDx) {
                                const bool same = diagonal && b0 + e == a;
                                const float wba = off || same ? 0.f : acc[e] * decay * dyx[e];
                                cols += wba;
                                const float row = wba * da;
                                wd += off ? 0.f : row * diff;
                                const float rows = row_scan16(row);
                                if (r == 15) lds.rows[it][b0 + e] = rows;
                                if (same) lds.diag[a] = acc[e] * dyx[e], lds.qdiag[a] = dyx[e];
                            }
                            acc[e] = off ? 0.f : acc[e] * (REV ? decay : decay * db[e]);
                        }
                        if constexpr (MODE == kDx) {
                            cols = sum_col_groups(cols);
                            if (g == 0) lds.cols[jt][a] = cols;
                        }
                    }
                    const float m[4] = {acc[0], acc[1], acc[2], acc[3]};
                    store_run(lds.m + Layout<T, 64>::at(a, b0), m);
                    if constexpr (M::MPARTS == 2) {
                        float hi[4];
                        const uint32_t u[2] = {pack_bf(m[0], m[1]), pack_bf(m[2], m[3])};
                        load_run(reinterpret_cast<const uint16_t *>(u), hi);
                        store_run(lds.m + M::MSIZE + Layout<T, 64>::at(a, b0), {m[0] - hi[0], m[1] - hi[1], m[2] - hi[2], m[3] - hi[3]});
                    }
                    phase();
                }
                if constexpr (MODE == kDx) {
#pragma unroll
                    for (int m = 32; m >= 1; m >>= 1) wd += shfl_xor(wd, m);
                    if (lane == 0) lds.wave[w] = wd;
                }
                __syncthreads();
                if (MODE == kDx && tid < L) {
                    // the sum over a < t <= b for this thread's t, by blocks: sums of whole ones, of rows from t
                    // and columns before t of those in t's block row or column, and of its diagonal one, alone
                    // a difference (of rows and columns from t on)
                    const int own = tid / 16;
                    const float d = lds.tok[0][tid], own_col = lds.cols[own][tid];
                    float rows = lds.rows[own][tid] - d * own_col, far = 0.f;
                    for (int t = 0; t < own; ++t) rows += lds.rows[t][tid];
                    for (int t = own + 1; t < IT; ++t) far += lds.cols[t][tid];
                    const float cols = own_col + far;
                    float dl = row_suffix16(rows) + row_scan16(row_shr<1>(d * far));
                    if constexpr (IT == 4) {
                        const float r0 = row_suffix16(lds.rows[0][tid]), r1 = row_suffix16(lds.rows[1][tid]);
                        // read where every lane takes part: under the choice the sums would be formed by its lanes alone
                        const float b20 = row_first<2>(r0), b30 = row_first<3>(r0), b31 = row_first<3>(r1);
                        dl += own == 1 ? b20 + b30 : own == 2 ? b30 + b31 : 0.f;
                    }
                    *behind(p.w_dl + chn * L, tid) = dl;
                    *behind(p.w_cols + chn * L, tid) = cols;
                    *behind(p.w_diag + chn * L, tid) = lds.diag[tid];
                    *behind(p.w_qdiag + chn * L, tid) = lds.qdiag[tid];
                    if (tid == 0) p.w_decay[chn] = (lds.wave[0] + lds.wave[1]) + (lds.wave[2] + lds.wave[3]);
                }
            }
            Frag<T> fv[KS][CT];
            if (active) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        fv[ks][ct] = col_frag<CT == 2, VW>(lds.val, 32 * ks, 16 * CT * w + 4 * ct, r, g);
                if constexpr (OUT) {
                    f32x4 zq[IT][CT];
#pragma unroll
                    for (int it = 0; it < IT; ++it)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) zq[it][ct] = zero4();
#pragma unroll
                    for (int kb = 0; kb < KW / 32; ++kb) {
                        Frag<T> fz[CT][ZPARTS];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            const f32x4 lo = Z[hh][2 * kb][ct], hi = Z[hh][2 * kb + 1][ct];
                            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                            split(v, fz[ct]);
                        }
#pragma unroll
                        for (int it = 0; it < IT; ++it) {
                            const Frag<T> fq = row_frag<true, KW>(lds.q, 16 * it + r, 32 * kb, g);
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                                for (int s = 0; s < ZPARTS; ++s) zq[it][ct] = mma(zq[it][ct], fz[ct][s], fq);
                        }
                        phase();
                    }
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const int i = 16 * it + r;
                        f32x4 mv[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) mv[ct] = zero4();
#pragma unroll
                        for (int kb = REV ? it / 2 : 0; kb < (REV ? KS : it / 2 + 1); ++kb) {
#pragma unroll
                            for (int s = 0; s < M::MPARTS; ++s) {
                                const Frag<T> fm = row_frag<true, 64>(lds.m + s * M::MSIZE, i, 32 * kb, g);
#pragma unroll
                                for (int ct = 0; ct < CT; ++ct) mv[ct] = mma(mv[ct], fv[kb][ct], fm);
                            }
                        }
                        const float f = lds.tok[4][i], scale = REV ? lds.tok[0][i] : 1.f;
                        const bool real = i < len;
                        float o[RUN], v[RUN];
#pragma unroll
                        for (int e = 0; e < RUN; ++e) o[e] = scale * (mv[e / 4][e % 4] + f * zq[it][e / 4][e % 4]);
                        if constexpr (!SUMS) {
                            load_run(lds.val + Layout<T, VW>::at(i, run0 - v0), v);
#pragma unroll
                            for (int e = 0; e < RUN; ++e) o[e] += D * v[e];
                            if (real) store_run(behind(static_cast<T *>(MODE == kY ? p.y : p.dx) + (t0 * p.H + h) * p.P, i * ys + run0), o);
                        } else {
#pragma unroll
                            for (int e = 0; e < RUN; ++e) sum[it][e] += o[e];
                            float dot = 0.f;
                            load_run(lds.other + Layout<T, VW>::at(i, run0 - v0), v);
#pragma unroll
                            for (int e = 0; e < RUN; ++e) dot += v[e] * zq[it][0][e];
                            dot = sum_col_groups(dot);
                            if (g == 0) *behind((MODE == kDc ? p.w_o : p.w_q) + (chn * (p.N / 16) + tile) * L, i) = f * dot;
                        }
                        phase();
                    }
                }
            }
            if (hh + 1 < nheads) request_q(c, h + 1);
            else if (k + 1 < sg.count) request_q(chunk_at(k + 1), h0);
            if (active) {
                const float dec = lds.dec;
                whole *= dec;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) Z[hh][i][ct] *= dec;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    Frag<T> fu[CT][PARTS];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) scaled(fv[ks][ct], &lds.tok[3][32 * ks + 4 * g], fu[ct]);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const Frag<T> fk = col_frag<false, KW>(lds.key, 32 * ks, 16 * i, r, g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                            for (int s = 0; s < PARTS; ++s) Z[hh][i][ct] = mma(Z[hh][i][ct], fk, fu[ct][s]);
                        if (i % 4 == 3) phase();
                    }
                }
            }
        }
        if constexpr (SUMS) {
            if (active)
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int i = 16 * it + (fresh(lane_r) & 15);
                    if (i >= len) continue;
                    const int64_t base = (t0 * p.G + grp) * p.N;
                    const int at = i * p.G * p.N + run0;
                    const float o[4] = {sum[it][0], sum[it][1], sum[it][2], sum[it][3]};
                    if (p.split > 1) store_run(behind((MODE == kDc ? p.dCp : p.dBp) + (part * p.tokens * p.G * p.N + base), at), o);
                    else store_run(behind(static_cast<T *>(MODE == kDc ? p.dC : p.dB) + base, at), o);
                }
        }
    }
    // the state behind the segment
    if (!OUT && tid == 0) p.seg_dec[(size_t)dseg * p.H + h0] = whole;
#pragma unroll
    for (int hh = 0; hh < HN; ++hh) {
        float *to = nullptr;
        if (!OUT) to = p.seg_state + ((size_t)dseg * p.H + h0) * state;
        else if (sg.rank == sg.segs - 1) {
            to = MODE == kY ? p.ht : MODE == kDc ? p.last_state : MODE == kDb ? p.dh0 : nullptr;
            if (to) to += ((size_t)sg.n * p.H + h0 + hh) * state;
        }
        const int end = fresh(own);
        if (to && active && hh < nheads) each([&](int i, int ct, int j, int at) { *behind(to + at, end) = Z[hh][i][ct][j]; });
    }
}

template <typename T, int KW, int CT, int MODE> hipError_t launch_scan_as(const SsmParams &p, int slices, int dirs, hipStream_t s) {
    const int64_t grid = (int64_t)dirs * p.total_segs * (scan_sums(MODE) ? (int64_t)p.G * p.split : p.H) * slices;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX - 8) return hipErrorInvalidValue;
    constexpr int bytes = (int)sizeof(ScanLds<T, KW, CT, MODE>);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(ssm_scan_kernel<T, KW, CT, MODE>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((ssm_scan_kernel<T, KW, CT, MODE>), dim3(xcd_grid(grid)), dim3(256), bytes, s, p, slices, dirs);
    return hipGetLastError();
}
// Tiles of 64 or 128 columns of the key; the value's columns at 16 or 32 to a wave, 16 where a
// workgroup carries two heads.
template <typename T, int MODE> hipError_t launch_scan(const SsmParams &p, int dirs, hipStream_t s) {
    const int kd = scan_np(MODE) ? p.N : p.P, vd = scan_np(MODE) ? p.P : p.N;
    if constexpr (scan_sums(MODE)) {
        const int slices = (vd + 63) / 64;
        return kd <= 64 ? launch_scan_as<T, 64, 1, MODE>(p, slices, dirs, s) : launch_scan_as<T, 128, 1, MODE>(p, slices, dirs, s);
    } else if (vd <= 64) {
        return kd <= 64 ? launch_scan_as<T, 64, 1, MODE>(p, 1, dirs, s) : launch_scan_as<T, 128, 1, MODE>(p, 1, dirs, s);
    } else {
        return kd <= 64 ? launch_scan_as<T, 64, 2, MODE>(p, 1, dirs, s) : launch_scan_as<T, 128, 2, MODE>(p, 1, dirs, s);
    }
}

// kda_layer_ssm_fwd.hip
hipError_t launch_ssm_prep(const SsmParams &p, hipStream_t s);
hipError_t launch_ssm_join(const SsmParams &p, int dirs, hipStream_t s);

// The common start: the steps and decays, and with several segments their first states.
template <typename T> hipError_t launch_segments(const SsmParams &p, int dirs, hipStream_t s) {
    hipError_t e = launch_ssm_prep(p, s);
    if (e != hipSuccess || p.max_segs == 1) return e;
    e = launch_scan<T, kFirst>(p, dirs, s);
    return e == hipSuccess ? launch_ssm_join(p, dirs, s) : e;
}

}  // namespace kda
