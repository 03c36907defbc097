// kda_layer_abi.cpp -- the C ABI of the operators around the recurrence (short convolution,
// RMS norm) declared in include/kda.h: argument checks, workspace layout, launches.  The
// checks come before any HIP call, descriptor first, then pointers, then the workspace.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstring>

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

}  // namespace
}  // namespace kda

using namespace kda;

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

}  // extern "C"
