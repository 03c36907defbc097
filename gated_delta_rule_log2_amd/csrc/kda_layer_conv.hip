// kda_layer_conv.hip -- the short causal convolution in front of the recurrence: each
// channel's last W inputs (W = 2, 3 or 4), an optional bias and SiLU.
//
//   pre_t = bias + sum_w weight[w] x_{t-W+1+w};   y_t = pre_t  or  pre_t sigmoid(pre_t)
//
// Inputs left of a sequence's first token are its initial state's rows (the last W - 1
// inputs before it, oldest first) or 0.  Sums in fp32 from the stored values, one rounding
// at the store.
//
// Forward bound by HBM: 2 W + 5 operations for each input read and output written (8192 tokens of 4096
// channels in bf16: 134 MB in 33 us, 4.1 TB/s).  Backward as much by its arithmetic, 32 vector
// instructions for each value of x and dy (the same size: 201 MB in 58 us, of which the vector units are
// busy for half; runs of 32 or 48 tokens, and uniform tokens and addresses in a wave, took as long).  A
// thread owns four channels and a run of tokens, and keeps the window of W inputs in registers, so x
// is read once but for the W - 1 tokens before each run, which the neighbouring run has just
// brought into L2.
#include "kda_layer.h"
#include "kda_layer_device.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

// A workgroup's threads: `lanes` vectors of channels (a power of two) by 256 / lanes runs.
struct Lanes { int lanes, col_blocks; };
template <int V> Lanes lanes_of(int D) {
    const int nv = vec_count<V>(D);
    int l = 1;
    while (l < nv && l < 64) l <<= 1;
    return {l, (nv + l - 1) / l};
}

template <int W, int V> struct Weights {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvParams &p, int c) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int ch = c + j < p.D ? c + j : p.D - 1;
            b[j] = p.bias ? load_f32(p.bias, ch, p.w_bf16) : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][j] = load_f32(p.weight, (int64_t)ch * W + k, p.w_bf16);
        }
    }
};

// Channels of a thread: with eight, whose windows and weights leave three waves to a SIMD forward and
// one backward, 8192 tokens of 4096 channels took 48 and 92 us, with four 42 and 59 (then streaming
// stores brought the forward to 33).
constexpr int kFwdV = 4, kBwdV = 4;
// Tokens of a batch: a multiple of W, for the turning windows.
template <int W> struct Batch { static constexpr int value = W == 3 ? 3 : 4; };

// Input at place `pos` of sequence n (first token s0): a token, an initial state's row
// (pos < 0), or 0.
template <typename T, int W, int V>
__device__ __forceinline__ void load_input(const ConvParams &p, int n, int64_t s0, int64_t pos, int c, Vec<T, V> &v) {
    if (pos >= 0) vec_load(v, static_cast<const T *>(p.x) + (s0 + pos) * p.x_stride, c, p.D);
    else if (p.h0) vec_load(v, static_cast<const T *>(p.h0) + ((int64_t)n * (W - 1) + (W - 1 + pos)) * p.D, c, p.D);
    else v.zero();
}

// Slot `first` of the window has the oldest input.
template <int W, int V>
__device__ __forceinline__ void pre_of(const float (&wd)[W][V], int first, const Weights<W, V> &wt, float (&pre)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) pre[j] = wt.b[j];
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) pre[j] += wt.w[k][j] * wd[(first + k) % W][j];
}

// y, and in the workgroups behind the first `main_blocks` the final states: row r of
// sequence n is its input at place len - (W - 1) + r.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvParams p, Lanes g, int run, int64_t main_blocks) {
    constexpr int V = kFwdV;
    const int lane = threadIdx.x & (g.lanes - 1), sub = threadIdx.x / g.lanes, subs = kThreads / g.lanes;
    const int64_t blk = blockIdx.x / g.col_blocks;
    const int vec = (int)(blockIdx.x % g.col_blocks) * g.lanes + lane;
    if (vec >= vec_count<V>(p.D)) return;
    const int c = vec_channel<V>(vec, p.D);
    if (blk >= main_blocks) {
        const int64_t i = (blk - main_blocks) * subs + sub;  // (sequence, row)
        if (i >= (int64_t)p.N * (W - 1)) return;
        const int n = (int)(i / (W - 1)), r = (int)(i % (W - 1));
        const SeqSpan q = seq_span(p, n);
        Vec<T, V> v;
        load_input<T, W, V>(p, n, q.first, (q.end - q.first) - (W - 1) + r, c, v);
        vec_store(v, static_cast<T *>(p.ht) + i * p.D, c, p.D);
        return;
    }
    int64_t t = (blk * subs + sub) * run;
    const int64_t stop = t + run < p.tokens ? t + run : p.tokens;
    if (t >= stop) return;
    Weights<W, V> wt;
    wt.load(p, c);
    SeqSpan q = seq_of(p, t);
    // The window turns through its W slots: in step u of a batch of U tokens (a multiple of W; all
    // requested before the first is used) the current token is in slot u % W, the one k before it
    // in slot (u - k) % W.
    constexpr int U = 2 * Batch<W>::value;
    float wd[W][V];
    const T *x = static_cast<const T *>(p.x);
    T *y = static_cast<T *>(p.y);
    bool fill = true;
    while (t < stop) {
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) vec_load(v[u], x + (t + u < stop ? t + u : stop - 1) * p.x_stride, c, p.D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t < stop) {
                if (fill || t >= q.end) {  // the tokens before a run's or a sequence's first
                    if (t >= q.end) q = seq_of(p, t);
                    fill = false;
#pragma unroll
                    for (int k = 1; k < W; ++k) {
                        Vec<T, V> e;
                        load_input<T, W, V>(p, q.n, q.first, t - q.first - k, c, e);
                        e.get(wd[(u - k + W) % W]);
                    }
                }
                v[u].get(wd[u % W]);
                float pre[V];
                pre_of(wd, u + 1, wt, pre);
                if (p.silu)
#pragma unroll
                    for (int j = 0; j < V; ++j) pre[j] *= sigmoid(pre[j]);
                Vec<T, V> o;
                o.set(pre);
                vec_store_stream(o, y + t * p.D, c, p.D);
                ++t;
            }
        }
    }
}

// dL/dpre from dy: SiLU'(x) = s + x s (1 - s) with s = sigmoid(x).
template <int V>
__device__ __forceinline__ void dpre_of(const float (&pre)[V], const float (&dy)[V], int silu, float (&d)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float s = sigmoid(pre[j]);
        d[j] = silu ? dy[j] * (s + pre[j] * s * (1.f - s)) : dy[j];
    }
}

// dx_t = sum_k weight[W-1-k] dpre_{t+k} over the sequence (plus dht's row where token t is
// one of the last W - 1), dweight[w] = sum_t dpre_t x_{t-W+1+w}, dbias = sum_t dpre_t.
// A run walks its tokens once, and W - 1 tokens beyond it for the last dx; the weight and
// bias sums of its own tokens stay in registers, are joined over the workgroup's runs in
// LDS in a fixed order and leave as one partial per workgroup.  Workgroups behind
// `main_blocks` compute dh0.
template <typename T, typename TY, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvParams p, Lanes g, int run, int64_t main_blocks) {
    constexpr int V = kBwdV;
    __shared__ float red[kThreads][V];
    const int lane = threadIdx.x & (g.lanes - 1), sub = threadIdx.x / g.lanes, subs = kThreads / g.lanes;
    const int64_t blk = blockIdx.x / g.col_blocks;
    const int vec = (int)(blockIdx.x % g.col_blocks) * g.lanes + lane;
    const bool live = vec < vec_count<V>(p.D);
    const int c = vec_channel<V>(live ? vec : 0, p.D);
    const T *x = static_cast<const T *>(p.x);
    const TY *dy = static_cast<const TY *>(p.dy);
    Weights<W, V> wt;
    wt.load(p, c);
    if (blk >= main_blocks) {
        const int64_t i = (blk - main_blocks) * subs + sub;  // (sequence, row of its initial state)
        if (!live || i >= (int64_t)p.N * (W - 1)) return;
        const int n = (int)(i / (W - 1)), r = (int)(i % (W - 1));
        const SeqSpan q = seq_span(p, n);
        const int64_t len = q.end - q.first;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            const int64_t pos = r - (W - 1) + k;  // the output that reads row r with weight W - 1 - k
            if (pos < 0 || pos >= len) continue;
            float wd[W][V], pre[V], gy[V], d[V];
#pragma unroll
            for (int m = 0; m < W; ++m) {
                Vec<T, V> v;
                load_input<T, W, V>(p, n, q.first, pos - (W - 1) + m, c, v);
                v.get(wd[m]);
            }
            pre_of(wd, 0, wt, pre);
            Vec<TY, V> v;
            vec_load(v, dy + (q.first + pos) * p.D, c, p.D);
            v.get(gy);
            dpre_of(pre, gy, p.silu, d);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += wt.w[W - 1 - k][j] * d[j];
        }
        if (p.dht && r - len >= 0) {  // a sequence shorter than the state hands the row on to the final state
            Vec<T, V> v;
            float d[V];
            vec_load(v, static_cast<const T *>(p.dht) + ((int64_t)n * (W - 1) + (r - len)) * p.D, c, p.D);
            v.get(d);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += d[j];
        }
        Vec<T, V> o;
        o.set(s);
        vec_store(o, static_cast<T *>(p.dh0) + i * p.D, c, p.D);
        return;
    }

    float dw[W][V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][j] = 0.f;
    }
    int64_t a = (blk * subs + sub) * run;
    const int64_t stop = a + run < p.tokens ? a + run : p.tokens;
    while (live && a < stop) {  // one sequence's part [a, b) of the run at a time
        const SeqSpan q = seq_of(p, a);
        const int64_t b = q.end < stop ? q.end : stop;
        if (b <= a) break;  // only where the device's offsets are not the host's
        const int64_t last = b + W - 1 < q.end ? b + W - 1 : q.end;
        // Window and unfinished dx turn through their slots as in the forward: in step u (token s)
        // slot (u + 1 + k) % W of wd has token s - (W - 1) + k, of pend that token's dx so far.
        constexpr int U = Batch<W>::value;
        float wd[W][V], pend[W][V];
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) pend[k][j] = 0.f;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            Vec<T, V> v;
            load_input<T, W, V>(p, q.n, q.first, a - q.first - k, c, v);
            v.get(wd[W - k]);
        }
        Vec<T, V> nx[U];
        Vec<TY, V> ny[U];
        auto request = [&](int64_t s) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = s + u < last ? s + u : last - 1;
                vec_load(nx[u], x + t * p.x_stride, c, p.D);
                vec_load(ny[u], dy + t * p.D, c, p.D);
            }
        };
        request(a);
        // past the tokens whose outputs read [a, b), steps without a dpre finish the last dx
        for (int64_t s = a; s < b + W - 1;) {
            Vec<T, V> vx[U];
            Vec<TY, V> vy[U];
#pragma unroll
            for (int u = 0; u < U; ++u) vx[u] = nx[u], vy[u] = ny[u];
            request(s + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s < b + W - 1) {
                    if (s < last) {
                        float pre[V], gy[V], d[V];
                        vx[u].get(wd[u % W]);
                        vy[u].get(gy);
                        pre_of(wd, u + 1, wt, pre);
                        dpre_of(pre, gy, p.silu, d);
                        if (s < b)
#pragma unroll
                            for (int j = 0; j < V; ++j) {
                                db[j] += d[j];
#pragma unroll
                                for (int k = 0; k < W; ++k) dw[k][j] += d[j] * wd[(u + 1 + k) % W][j];
                            }
#pragma unroll
                        for (int k = 0; k < W; ++k)
#pragma unroll
                            for (int j = 0; j < V; ++j) pend[(u + 1 + k) % W][j] += wt.w[k][j] * d[j];
                    }
                    const int64_t t = s - (W - 1), r = t - (q.end - (W - 1));
                    if (t >= a) {  // token t has all its terms; the final state's gradient joins them
                        float e[V];
                        if (p.dht && r >= 0) {
                            Vec<T, V> v;
                            vec_load(v, static_cast<const T *>(p.dht) + ((int64_t)q.n * (W - 1) + r) * p.D, c, p.D);
                            v.get(e);
#pragma unroll
                            for (int j = 0; j < V; ++j) pend[(u + 1) % W][j] += e[j];
                        }
                        Vec<T, V> o;
                        o.set(pend[(u + 1) % W]);
                        vec_store(o, static_cast<T *>(p.dx) + t * p.D, c, p.D);
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) pend[(u + 1) % W][j] = 0.f;
                    ++s;
                }
            }
        }
        a = b;
    }
    // join the runs of the workgroup, in order, one row of [W + 1][D] at a time
#pragma unroll
    for (int k = 0; k < W + 1; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) red[threadIdx.x][j] = k < W ? dw[k < W ? k : 0][j] : db[j];
        __syncthreads();
        if (sub == 0 && live) {
            float s[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = red[lane][j];
            for (int i = 1; i < subs; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += red[i * g.lanes + lane][j];
            float *out = p.partial + (blk * (W + 1) + k) * p.D;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < p.D) out[c + j] = s[j];
        }
        __syncthreads();
    }
}

// dweight [D][W] and dbias [D] from the workgroups' partials [blocks][W + 1][D].
template <int W> __global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(ConvParams p, int blocks) {
    const int64_t i = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const float s = sum_rows(p.partial, blocks, (int64_t)(W + 1) * p.D, i);
    if (threadIdx.x >= 64 || i >= (int64_t)(W + 1) * p.D) return;
    const int k = (int)(i / p.D), ch = (int)(i % p.D);
    if (k < W) p.dweight[(int64_t)ch * W + k] = s;
    else if (p.dbias) p.dbias[ch] = s;
}

// One token for each row; the row's state (its last W - 1 inputs) moves on in place.  A
// negative slot, or one past the pool, marks a padding row: y = 0 and no state is touched.
// Bound by launch latency at decoding sizes; one thread per (row, channel).
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvParams p) {
    const int cols = (p.D + kThreads - 1) / kThreads, row = blockIdx.x / cols;
    const int ch = (int)(blockIdx.x % cols) * kThreads + threadIdx.x;
    if (ch >= p.D) return;
    T *y = static_cast<T *>(p.y) + (int64_t)row * p.D + ch;
    const int slot = p.slots ? p.slots[row] : row;
    if (slot < 0 || slot >= p.num_slots) {
        *y = Store<T>::to(0.f);
        return;
    }
    T *st = static_cast<T *>(p.state) + (int64_t)slot * (W - 1) * p.D + ch;
    T in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k] = st[(int64_t)k * p.D];
    in[W - 1] = static_cast<const T *>(p.x)[(int64_t)row * p.x_stride + ch];
    float s = p.bias ? load_f32(p.bias, ch, p.w_bf16) : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += load_f32(p.weight, (int64_t)ch * W + k, p.w_bf16) * Store<T>::from(in[k]);
    if (p.silu) s *= sigmoid(s);
    *y = Store<T>::to(s);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) st[(int64_t)k * p.D] = in[k + 1];
}

// Tokens of one thread: longer runs repeat fewer window loads and leave fewer partial sums, shorter
// ones fill the chip where there are few vectors.  At 8192 tokens of 4096 channels in bf16 runs of 32
// took 42 us forward (33 with streaming stores, where 64 took 37) and 64 took 59 us backward; 16 took
// 47 and 72, and 128 backward 81.
int run_of(const ConvParams &p) {
    const int64_t vectors = vec_count<kFwdV>(p.D) * p.tokens;
    return vectors >= ((int64_t)1 << 22) ? 32 : vectors >= ((int64_t)1 << 20) ? 8 : 4;
}
int bwd_run_of(const ConvParams &p) { return vec_count<kBwdV>(p.D) * p.tokens >= ((int64_t)1 << 22) ? 64 : 16; }

template <typename T, int W> hipError_t fwd(const ConvParams &p, hipStream_t s) {
    const Lanes g = lanes_of<kFwdV>(p.D);
    const int subs = kThreads / g.lanes, run = run_of(p);
    const int64_t per = (int64_t)subs * run, main_blocks = (p.tokens + per - 1) / per;
    const int64_t tail = p.ht ? ((int64_t)p.N * (W - 1) + subs - 1) / subs : 0;
    const int64_t grid = (main_blocks + tail) * g.col_blocks;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((conv_fwd_kernel<T, W>), dim3((unsigned)grid), dim3(kThreads), 0, s, p, g, run, main_blocks);
    return hipGetLastError();
}
template <typename T, typename TY, int W> hipError_t bwd(const ConvParams &p, hipStream_t s) {
    const Lanes g = lanes_of<kBwdV>(p.D);
    const int subs = kThreads / g.lanes;
    const int64_t main_blocks = conv_bwd_blocks(p);
    const int64_t tail = p.dh0 ? ((int64_t)p.N * (W - 1) + subs - 1) / subs : 0;
    const int64_t grid = (main_blocks + tail) * g.col_blocks;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (grid > 0) {
        hipLaunchKernelGGL((conv_bwd_kernel<T, TY, W>), dim3((unsigned)grid), dim3(kThreads), 0, s, p, g, bwd_run_of(p),
                           main_blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t n = (int64_t)(W + 1) * p.D;
    hipLaunchKernelGGL(conv_bwd_sum_kernel<W>, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, s, p, (int)main_blocks);
    return hipGetLastError();
}
template <typename T, int W> hipError_t step(const ConvParams &p, hipStream_t s) {
    if (p.B == 0) return hipSuccess;
    const int64_t grid = (int64_t)((p.D + kThreads - 1) / kThreads) * p.B;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((conv_step_kernel<T, W>), dim3((unsigned)grid), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

int conv_bwd_blocks(const ConvParams &p) {
    const int64_t per = (int64_t)(kThreads / lanes_of<kBwdV>(p.D).lanes) * bwd_run_of(p);
    return (int)((p.tokens + per - 1) / per);
}

hipError_t launch_conv_fwd(const ConvParams &p, hipStream_t s) {
    switch (p.W) {
    case 2: return p.x_bf16 ? fwd<uint16_t, 2>(p, s) : fwd<float, 2>(p, s);
    case 3: return p.x_bf16 ? fwd<uint16_t, 3>(p, s) : fwd<float, 3>(p, s);
    case 4: return p.x_bf16 ? fwd<uint16_t, 4>(p, s) : fwd<float, 4>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_conv_bwd(const ConvParams &p, hipStream_t s) {
    // dy in x's type, or in fp32 beside a bf16 x (the recurrence's gradients are fp32)
#define KDA_CONV_BWD(W) \
    return !p.x_bf16 ? bwd<float, float, W>(p, s) : p.dy_bf16 ? bwd<uint16_t, uint16_t, W>(p, s) : bwd<uint16_t, float, W>(p, s)
    switch (p.W) {
    case 2: KDA_CONV_BWD(2);
    case 3: KDA_CONV_BWD(3);
    case 4: KDA_CONV_BWD(4);
    default: return hipErrorInvalidValue;
    }
#undef KDA_CONV_BWD
}

hipError_t launch_conv_step(const ConvParams &p, hipStream_t s) {
    switch (p.W) {
    case 2: return p.x_bf16 ? step<uint16_t, 2>(p, s) : step<float, 2>(p, s);
    case 3: return p.x_bf16 ? step<uint16_t, 3>(p, s) : step<float, 3>(p, s);
    case 4: return p.x_bf16 ? step<uint16_t, 4>(p, s) : step<float, 4>(p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace kda
