// kda_layer_abi.cpp -- the C ABI of the operators around the recurrence (short convolution,
// RMS norm, state space scan) declared in include/kda.h: argument checks, workspace layout, launches.  The
// checks come before any HIP call, descriptor first, then pointers, then the workspace.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <functional>

#include "../../include/kda.h"
#include "kda_layer.h"

namespace kda {
namespace {

bool dtype_ok(int32_t t) { return t == KDA_DTYPE_FP32 || t == KDA_DTYPE_BF16; }
kda_status to_status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// Batch rows or packed offsets, as kda_fwd_desc has them.
kda_status check_seqs(int32_t B, int32_t T, int32_t num_seqs, const int64_t *cu) {
    if (!cu) return num_seqs == B ? KDA_OK : KDA_ERR_SHAPE;
    if (B != 1 || num_seqs < 1 || cu[0] != 0 || cu[num_seqs] != T) return KDA_ERR_VARLEN;
    for (int32_t n = 0; n < num_seqs; ++n)
        if (cu[n + 1] < cu[n]) return KDA_ERR_VARLEN;
    return KDA_OK;
}

kda_status check_conv(const kda_conv_desc *d, ConvParams &p) {
    if (!d) return KDA_ERR_NULL_POINTER;
    if (d->B < 1 || d->T < 0 || d->D < 1 || d->W < 1 || d->num_seqs < 0 || d->x_stride < d->D) return KDA_ERR_SHAPE;
    if ((int64_t)d->B * d->T > (int64_t)INT32_MAX / 2) return KDA_ERR_SHAPE;
    if (d->W < 2 || d->W > 4 || (d->flags & ~(uint32_t)KDA_CONV_SILU)) return KDA_ERR_UNSUPPORTED;
    const kda_status st = check_seqs(d->B, d->T, d->num_seqs, d->cu_seqlens_host);
    if (st != KDA_OK) return st;
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->w_dtype) || !dtype_ok(d->dy_dtype)) return KDA_ERR_DTYPE;
    std::memset(&p, 0, sizeof(p));
    p.B = d->B; p.T = d->T; p.D = d->D; p.W = d->W; p.N = d->num_seqs;
    p.tokens = (int64_t)d->B * d->T;
    p.x_bf16 = d->x_dtype == KDA_DTYPE_BF16;
    p.w_bf16 = d->w_dtype == KDA_DTYPE_BF16;
    p.dy_bf16 = d->dy_dtype == KDA_DTYPE_BF16;
    p.silu = (d->flags & KDA_CONV_SILU) ? 1 : 0;
    p.x_stride = d->x_stride;
    return KDA_OK;
}

kda_status check_conv_bwd(const kda_conv_desc *d, ConvParams &p, size_t &bytes) {
    const kda_status st = check_conv(d, p);
    if (st != KDA_OK) return st;
    if (p.dy_bf16 && !p.x_bf16) return KDA_ERR_DTYPE;  // dy has x's type or fp32
    bytes = sizeof(float) * (size_t)conv_bwd_blocks(p) * (p.W + 1) * p.D;
    if (bytes == 0) bytes = 256;
    return KDA_OK;
}

kda_status check_norm(const kda_norm_desc *d, bool fp8, NormParams &p) {
    if (!d) return KDA_ERR_NULL_POINTER;
    if (d->rows < 0 || d->D < 1 || d->group_size < 0 || !(d->eps >= 0.f)) return KDA_ERR_SHAPE;
    if (d->rows > (int64_t)INT32_MAX / 2) return KDA_ERR_SHAPE;
    if (d->D > kNormMaxD) return KDA_ERR_UNSUPPORTED;
    const int32_t g = fp8 ? d->group_size : 0;
    if (g && (g < 8 || g > 512 || (g & (g - 1)) || d->D % g)) return KDA_ERR_UNSUPPORTED;
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->w_dtype)) return KDA_ERR_DTYPE;
    std::memset(&p, 0, sizeof(p));
    p.rows = d->rows; p.D = d->D; p.group = g;
    p.x_bf16 = d->x_dtype == KDA_DTYPE_BF16;
    p.w_bf16 = d->w_dtype == KDA_DTYPE_BF16;
    p.eps = d->eps;
    return KDA_OK;
}

constexpr int64_t kMaxStride = (1 << 24) - 1;  // a chunk's offsets stay in 32 bits
constexpr int64_t kCarryGroups = 512;  // workgroups of a pass over chunks at once: two for each CU

kda_status check_ssm(const kda_ssm_desc *d, SsmParams &p) {
    if (!d) return KDA_ERR_NULL_POINTER;
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->G < 1 || d->N < 1 || d->P < 1 || d->num_seqs < 0) return KDA_ERR_SHAPE;
    if ((int64_t)d->B * d->T > (int64_t)INT32_MAX / 2 || d->H > (1 << 20)) return KDA_ERR_SHAPE;
    if (d->N % 32 || d->N > 128 || d->P % 32 || d->P > 128 || (d->flags & ~(uint32_t)KDA_SSM_SOFTPLUS)) return KDA_ERR_UNSUPPORTED;
    if (d->H % d->G) return KDA_ERR_GVA;
    if (d->x_stride < (int64_t)d->H * d->P || d->dt_stride < d->H || d->b_stride < (int64_t)d->G * d->N ||
        d->c_stride < (int64_t)d->G * d->N)
        return KDA_ERR_SHAPE;
    if ((int64_t)d->H * d->P > kMaxStride || (int64_t)d->G * d->N > kMaxStride || d->x_stride > kMaxStride || d->b_stride > kMaxStride || d->c_stride > kMaxStride) return KDA_ERR_SHAPE;
    const kda_status st = check_seqs(d->B, d->T, d->num_seqs, d->cu_seqlens_host);
    if (st != KDA_OK) return st;
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->dt_dtype)) return KDA_ERR_DTYPE;
    std::memset(&p, 0, sizeof(p));
    p.B = d->B; p.T = d->T; p.H = d->H; p.G = d->G; p.N = d->N; p.P = d->P; p.NS = d->num_seqs;
    p.tokens = (int64_t)d->B * d->T;
    p.x_bf16 = d->x_dtype == KDA_DTYPE_BF16;
    p.dt_bf16 = d->dt_dtype == KDA_DTYPE_BF16;
    p.softplus = (d->flags & KDA_SSM_SOFTPLUS) ? 1 : 0;
    p.x_stride = d->x_stride; p.dt_stride = d->dt_stride; p.b_stride = d->b_stride; p.c_stride = d->c_stride;
    p.L = p.x_bf16 ? 64 : 32;
    return KDA_OK;
}

// Time of a pass over segments, in steps of a chunk, on `slots` workgroups at once: items(f) calls
// f(steps) for each of them, in their order.  A slot costs kItem steps for its states besides; the
// last ones run faster, with the GPU partly empty.  Few items are dealt out one by one, many fill
// the slots evenly but for the last.
constexpr int kDealt = 128;
template <typename F> double pass_time(F items, int64_t slots) {
    constexpr double kItem = 1.5, kTail = 0.62;
    double sum = 0., most = 0.;
    int64_t count = 0;
    items([&](int64_t steps) {
        const double t = (double)steps + kItem;
        sum += t;
        if (t > most) most = t;
        ++count;
    });
    const double even = sum / (double)slots;
    double last = even + 0.5 * most;
    if (count <= slots) {
        last = most;
    } else if (count <= kDealt) {
        double busy[kDealt], *end = busy + slots;  // a heap, the first slot to be free on top
        for (double *s = busy; s < end; ++s) *s = 0.;
        last = 0.;
        items([&](int64_t steps) {
            std::pop_heap(busy, end, std::greater<double>());
            end[-1] += (double)steps + kItem;
            if (end[-1] > last) last = end[-1];
            std::push_heap(busy, end, std::greater<double>());
        });
    }
    return last > even ? even + kTail * (last - even) : even;
}

// The chunks, and how many of them make a segment: the number that takes the least time by the above,
// of some about the one that gives every slot one segment, and of whole sequences.  Those need no
// first pass for the segments' states (0.45 of the forward's time for a chunk, which is 1 here) and no
// joining (2); the backward has both for two directions, and 4.5 of the forward's passes.
// Measured over 15 packed batches at nine lengths each (8192 or 6000 tokens, 5 to 30 sequences, 32 or
// 64 heads, forward and backward): 6 % behind the best length on average, where one segment for every
// slot is 28 % behind.  A segment has at least two chunks: fp32 gradients of 2 x 1003 tokens, 8 heads of
// 64 x 64, take 80 us at one, 85 at two and 113 at four.
// dC's and dB's scans sum two heads of a group in a workgroup, which shares the tiles of B and C and
// halves the parts to be summed (8192 tokens, 32 heads in 16 groups of 128 x 128: 494 us against 614
// with one head); where that leaves half the CUs without work, one (the fp32 case: 73 us against 85).
kda_status plan_ssm(const kda_ssm_desc *d, SsmParams &p, bool backward) {
    auto each = [&](auto f) {
        if (d->cu_seqlens_host)
            for (int32_t n = 0; n < p.NS; ++n) f((d->cu_seqlens_host[n + 1] - d->cu_seqlens_host[n] + p.L - 1) / p.L);
        else
            for (int32_t n = 0; n < p.NS; ++n) f((int64_t)(p.T + p.L - 1) / p.L);
    };
    int64_t chunks = 0, longest = 1, segs = 0, most = 1;
    each([&](int64_t c) {
        chunks += c;
        if (c > longest) longest = c;
    });
    if (chunks * p.H > INT32_MAX) return KDA_ERR_SHAPE;
    const int64_t slots = p.H < kCarryGroups ? (kCarryGroups + p.H / 2) / p.H : 1;
    auto parts = [](int64_t c, int64_t seg) { return c > seg ? (c + seg - 1) / seg : 1; };
    double best = 0.;
    p.seg = (int32_t)longest;
    for (int k = 0; k <= 6 && longest > 2; ++k) {
        static const double share[6] = {0.5, 0.75, 1., 1.25, 1.5, 2.};
        int64_t seg = longest;
        if (k > 0) {
            seg = (int64_t)(share[k - 1] * (double)chunks / (double)slots + 0.5);
            if (seg < 2) seg = 2;
            if (seg >= longest) break;
        }
        auto all = [&](auto f) {
            each([&](int64_t c) {
                const int64_t n = parts(c, seg);
                for (int64_t i = 0; i + 1 < n; ++i) f(seg);
                f(c - (n - 1) * seg);
            });
        };
        auto first = [&](auto f) {
            for (int dir = 0; dir < (backward ? 2 : 1); ++dir)
                each([&](int64_t c) {
                    for (int64_t i = 1; i < parts(c, seg); ++i) f(seg);
                });
        };
        double t = (backward ? 4.5 : 1.) * pass_time(all, slots);
        if (seg < longest) t += 0.45 * pass_time(first, slots) + (backward ? 4. : 2.);
        if (k == 0 || t < best) best = t, p.seg = (int32_t)seg;
    }
    each([&](int64_t c) {
        const int64_t s = parts(c, p.seg);
        segs += s;
        if (s > most) most = s;
    });
    if (segs * p.H * 8 > INT32_MAX - 8) return KDA_ERR_SHAPE;
    p.total_chunks = (int32_t)chunks; p.total_segs = (int32_t)segs; p.max_segs = (int32_t)most;
    const int32_t heads = p.H / p.G, pairs = (heads + 1) / 2;
    p.split = segs * p.G * pairs * ((p.N + 63) / 64) <= kCarryGroups / 2 ? heads : pairs;
    return KDA_OK;
}

}  // namespace

size_t ssm_workspace(SsmParams &p, void *ws, bool backward) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char *at = ws ? static_cast<unsigned char *>(ws) + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return static_cast<void *>(at);
    };
    const size_t ch = (size_t)p.total_chunks * p.H, tok = ch * p.L * sizeof(float);
    const size_t state = (size_t)p.N * p.P, dirs = backward ? 2 : 1;
    p.d = static_cast<float *>(take(tok));
    p.ch = static_cast<float *>(take(tok));
    p.cl = static_cast<float *>(take(tok));
    auto floats = [&](size_t n) { return static_cast<float *>(take(n * sizeof(float))); };
    if (p.max_segs > 1) {
        p.seg_state = floats(dirs * p.total_segs * p.H * state);
        p.seg_dec = floats(dirs * p.total_segs * p.H);
    }
    if (backward) {
        p.last_state = floats((size_t)p.NS * p.H * state);
        p.w_dl = floats(ch * p.L);
        p.w_cols = floats(ch * p.L);
        p.w_diag = floats(ch * p.L);
        p.w_qdiag = floats(ch * p.L);
        p.w_decay = floats(ch);
        p.w_o = floats(ch * p.L * (p.N / 16));
        p.w_q = floats(ch * p.L * (p.N / 16));
        p.w_dot = floats((size_t)p.total_segs * p.H * (p.N / 16));
        p.sums = floats(ch * 4);
        if (p.split > 1) {
            const size_t part = (size_t)p.split * p.tokens * p.G * p.N * sizeof(float);
            p.dBp = static_cast<float *>(take(part));
            p.dCp = static_cast<float *>(take(part));
        }
    }
    return off ? off : 256;
}

}  // namespace kda

using namespace kda;

static kda_status ssm_prepare(const kda_ssm_desc *d, SsmParams &p, bool backward) {
    const kda_status st = check_ssm(d, p);
    return st == KDA_OK ? plan_ssm(d, p, backward) : st;
}

static kda_status ssm_size(const kda_ssm_desc *d, size_t *bytes, bool backward) {
    SsmParams p;
    const kda_status st = ssm_prepare(d, p, backward);
    if (st != KDA_OK) return st;
    if (!bytes) return KDA_ERR_NULL_POINTER;
    *bytes = ssm_workspace(p, nullptr, backward);
    return KDA_OK;
}

extern "C" {

kda_status kda_short_conv_fwd(const kda_conv_desc *d, const void *x, const void *weight, const void *bias,
                              const void *initial_state, const int64_t *cu_seqlens, void *y, void *final_state,
                              hipStream_t stream) {
    ConvParams p;
    const kda_status st = check_conv(d, p);
    if (st != KDA_OK) return st;
    if (!weight || (p.tokens > 0 && (!x || !y))) return KDA_ERR_NULL_POINTER;
    if ((cu_seqlens == nullptr) != (d->cu_seqlens_host == nullptr)) return KDA_ERR_VARLEN;
    if (final_state && final_state == initial_state) return KDA_ERR_UNSUPPORTED;
    p.x = x; p.weight = weight; p.bias = bias; p.h0 = initial_state; p.cu_seqlens = cu_seqlens;
    p.y = y; p.ht = final_state;
    return to_status(launch_conv_fwd(p, stream));
}

kda_status kda_short_conv_bwd_workspace_size(const kda_conv_desc *d, size_t *bytes) {
    ConvParams p;
    size_t need = 0;
    const kda_status st = check_conv_bwd(d, p, need);
    if (st != KDA_OK) return st;
    if (!bytes) return KDA_ERR_NULL_POINTER;
    *bytes = need;
    return KDA_OK;
}

kda_status kda_short_conv_bwd(const kda_conv_desc *d, const void *x, const void *weight, const void *bias,
                              const void *initial_state, const int64_t *cu_seqlens, const void *dy, const void *dht,
                              void *dx, float *dweight, float *dbias, void *dh0, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    ConvParams p;
    size_t need = 0;
    const kda_status st = check_conv_bwd(d, p, need);
    if (st != KDA_OK) return st;
    if (!weight || !dweight || (p.tokens > 0 && (!x || !dy || !dx))) return KDA_ERR_NULL_POINTER;
    if ((cu_seqlens == nullptr) != (d->cu_seqlens_host == nullptr)) return KDA_ERR_VARLEN;
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    p.x = x; p.weight = weight; p.bias = bias; p.h0 = initial_state; p.cu_seqlens = cu_seqlens;
    p.dy = dy; p.dht = dht; p.dx = dx; p.dweight = dweight; p.dbias = dbias; p.dh0 = dh0;
    p.partial = static_cast<float *>(workspace);
    return to_status(launch_conv_bwd(p, stream));
}

kda_status kda_short_conv_step(const kda_conv_desc *d, const void *x, const void *weight, const void *bias,
                               void *state, const int32_t *slots, int32_t num_slots, void *y, hipStream_t stream) {
    ConvParams p;
    const kda_status st = check_conv(d, p);
    if (st != KDA_OK) return st;
    if (p.T != 1 || num_slots < 0 || (!slots && num_slots < p.B)) return KDA_ERR_SHAPE;
    if (d->cu_seqlens_host) return KDA_ERR_VARLEN;
    if (!x || !weight || !y || (num_slots > 0 && !state)) return KDA_ERR_NULL_POINTER;
    p.x = x; p.weight = weight; p.bias = bias; p.state = state; p.slots = slots; p.num_slots = num_slots;
    p.y = y;
    return to_status(launch_conv_step(p, stream));
}

kda_status kda_rms_norm_fwd(const kda_norm_desc *d, const void *x, const void *residual, const void *weight, void *y,
                            void *h, hipStream_t stream) {
    NormParams p;
    const kda_status st = check_norm(d, false, p);
    if (st != KDA_OK) return st;
    if (!weight || (p.rows > 0 && (!x || !y))) return KDA_ERR_NULL_POINTER;
    p.x = x; p.residual = residual; p.weight = weight; p.y = y; p.h = h;
    return to_status(launch_norm_fwd(p, false, stream));
}

kda_status kda_rms_norm_fp8(const kda_norm_desc *d, const void *x, const void *residual, const void *weight, void *q,
                            float *scales, void *h, hipStream_t stream) {
    NormParams p;
    const kda_status st = check_norm(d, true, p);
    if (st != KDA_OK) return st;
    if (!weight || (p.rows > 0 && (!x || !q || !scales))) return KDA_ERR_NULL_POINTER;
    p.x = x; p.residual = residual; p.weight = weight; p.y = q; p.scales = scales; p.h = h;
    return to_status(launch_norm_fwd(p, true, stream));
}

kda_status kda_rms_norm_bwd_workspace_size(const kda_norm_desc *d, size_t *bytes) {
    NormParams p;
    const kda_status st = check_norm(d, false, p);
    if (st != KDA_OK) return st;
    if (!bytes) return KDA_ERR_NULL_POINTER;
    const size_t need = sizeof(float) * (size_t)norm_bwd_blocks(p) * p.D;
    *bytes = need ? need : 256;
    return KDA_OK;
}

kda_status kda_rms_norm_bwd(const kda_norm_desc *d, const void *h, const void *weight, const void *dy, const void *dh,
                            void *dx, float *dweight, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    NormParams p;
    size_t need = 0;
    kda_status st = check_norm(d, false, p);
    if (st != KDA_OK) return st;
    if (!weight || !dweight || (p.rows > 0 && (!h || !dy || !dx))) return KDA_ERR_NULL_POINTER;
    st = kda_rms_norm_bwd_workspace_size(d, &need);
    if (st != KDA_OK) return st;
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    p.x = h; p.weight = weight; p.dy = dy; p.dh = dh; p.dx = dx; p.dweight = dweight;
    p.partial = static_cast<float *>(workspace);
    return to_status(launch_norm_bwd(p, stream));
}

kda_status kda_ssm_fwd_workspace_size(const kda_ssm_desc *d, size_t *bytes) { return ssm_size(d, bytes, false); }
kda_status kda_ssm_bwd_workspace_size(const kda_ssm_desc *d, size_t *bytes) { return ssm_size(d, bytes, true); }

kda_status kda_ssm_fwd(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *Bm,
                       const void *C, const float *D, const float *dt_bias, const float *initial_state,
                       const int64_t *cu_seqlens, void *y, float *final_state, void *workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    SsmParams p;
    const kda_status st = ssm_prepare(d, p, false);
    if (st != KDA_OK) return st;
    if (p.tokens > 0 && (!x || !dt || !Bm || !C || !y)) return KDA_ERR_NULL_POINTER;
    if (!A_log) return KDA_ERR_MISSING_A_LOG;
    if ((cu_seqlens == nullptr) != (d->cu_seqlens_host == nullptr)) return KDA_ERR_VARLEN;
    if (final_state && final_state == initial_state) return KDA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ssm_workspace(p, workspace, false)) return KDA_ERR_WORKSPACE;
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.C = C; p.D = D; p.dt_bias = dt_bias; p.h0 = initial_state;
    p.cu_seqlens = cu_seqlens; p.y = y; p.ht = final_state;
    return to_status(launch_ssm_fwd(p, stream));
}

kda_status kda_ssm_bwd(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *Bm,
                       const void *C, const float *D, const float *dt_bias, const float *initial_state,
                       const int64_t *cu_seqlens, const void *dy, const float *dht, void *dx, void *ddt,
                       float *dA_log, void *dB, void *dC, float *dD, float *ddt_bias, float *dh0, void *workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    SsmParams p;
    const kda_status st = ssm_prepare(d, p, true);
    if (st != KDA_OK) return st;
    if (p.tokens > 0 && (!x || !dt || !Bm || !C || !dy || !dx || !ddt || !dB || !dC)) return KDA_ERR_NULL_POINTER;
    if (!dA_log) return KDA_ERR_NULL_POINTER;
    if (!A_log) return KDA_ERR_MISSING_A_LOG;
    if ((cu_seqlens == nullptr) != (d->cu_seqlens_host == nullptr)) return KDA_ERR_VARLEN;
    if (!workspace || workspace_bytes < ssm_workspace(p, workspace, true)) return KDA_ERR_WORKSPACE;
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.C = C; p.D = D; p.dt_bias = dt_bias; p.h0 = initial_state;
    p.cu_seqlens = cu_seqlens; p.dy = dy; p.dht = dht;
    p.dx = dx; p.ddt = ddt; p.dA_log = dA_log; p.dB = dB; p.dC = dC; p.dD = dD; p.ddt_bias = ddt_bias; p.dh0 = dh0;
    return to_status(launch_ssm_bwd(p, stream));
}

kda_status kda_ssm_step(const kda_ssm_desc *d, const void *x, const void *dt, const float *A_log, const void *Bm,
                        const void *C, const float *D, const float *dt_bias, float *state, const int32_t *slots,
                        int32_t num_slots, void *y, hipStream_t stream) {
    SsmParams p;
    const kda_status st = check_ssm(d, p);
    if (st != KDA_OK) return st;
    if (p.T != 1 || num_slots < 0 || (!slots && num_slots < p.B)) return KDA_ERR_SHAPE;
    if (d->cu_seqlens_host) return KDA_ERR_VARLEN;
    if (!x || !dt || !Bm || !C || !y || (num_slots > 0 && !state)) return KDA_ERR_NULL_POINTER;
    if (!A_log) return KDA_ERR_MISSING_A_LOG;
    p.x = x; p.dt = dt; p.A_log = A_log; p.Bm = Bm; p.C = C; p.D = D; p.dt_bias = dt_bias;
    p.state = state; p.slots = slots; p.num_slots = num_slots; p.y = y;
    return to_status(launch_ssm_step(p, stream));
}

}  // extern "C"
