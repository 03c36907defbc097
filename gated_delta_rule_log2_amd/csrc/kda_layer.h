// kda_layer.h -- launch parameters of the operators that stand around the recurrence in a
// layer (short convolution, state space scan, RMS norm), shared by the C ABI's host code
// and the kernel launchers.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct ConvParams {
    int32_t B, T, D, W, N;         // N = sequences
    int64_t tokens;                // B * T
    int32_t x_bf16, w_bf16, dy_bf16, silu;
    int64_t x_stride;              // elements between two tokens of x
    int32_t num_slots;
    const void *x, *weight, *bias, *h0, *dy, *dht;
    const int64_t *cu_seqlens;     // device offsets or nullptr (then sequence n = batch row n)
    const int32_t *slots;
    void *y, *ht, *dx, *dh0, *state;
    float *dweight, *dbias;
    float *partial;                // [blocks][W + 1][D] weight and bias gradients of the backward's blocks
};

// Token runs of the backward's workgroups, one partial sum each.
int conv_bwd_blocks(const ConvParams &p);
hipError_t launch_conv_fwd(const ConvParams &p, hipStream_t s);
hipError_t launch_conv_bwd(const ConvParams &p, hipStream_t s);
hipError_t launch_conv_step(const ConvParams &p, hipStream_t s);

struct NormParams {
    int64_t rows;
    int32_t D, group;              // group: values under one scale (0: the row)
    int32_t x_bf16, w_bf16;
    float eps;
    const void *x, *residual, *weight, *dy, *dh;
    void *y, *h, *dx;
    float *scales, *dweight;
    float *partial;                // [blocks][D]
};

constexpr int kNormMaxD = 32768;
int norm_bwd_blocks(const NormParams &p);
hipError_t launch_norm_fwd(const NormParams &p, bool fp8, hipStream_t s);
hipError_t launch_norm_bwd(const NormParams &p, hipStream_t s);

// The state space scan.  L tokens make a chunk (chunks restart at every sequence), `seg`
// chunks of one sequence a segment, whose states one workgroup carries.
struct SsmParams {
    int32_t B, T, H, G, N, P, NS;  // NS = sequences
    int32_t L, total_chunks, seg, total_segs, max_segs;  // max_segs: of one sequence
    int32_t x_bf16, dt_bf16, softplus;
    int32_t num_slots;
    int32_t split;                 // backward: parts of a group's heads (one or two to a part), each with its own sums for dB, dC
    int64_t tokens;                // B * T
    int64_t x_stride, dt_stride, b_stride, c_stride;
    const void *x, *dt, *Bm, *C, *dy;
    const float *A_log, *D, *dt_bias, *h0, *dht;
    const int64_t *cu_seqlens;
    const int32_t *slots;
    void *y, *dx, *ddt, *dB, *dC;
    float *ht, *dh0, *dA_log, *dD, *ddt_bias, *state;
    // workspace
    float *d, *ch, *cl;            // [total_chunks][H][L]: see ssm_prep_kernel
    float *seg_state;              // [2][total_segs][H][N][P]: ends of segments from zero, then their starts
    float *seg_dec;                // [2][total_segs][H]
    // backward, for the gradients of steps and decays (kda_layer_ssm_bwd.hip)
    float *last_state;             // [NS][H][N][P]
    float *w_dl, *w_cols, *w_diag, *w_qdiag, *w_decay;  // [total_chunks][H][L], w_decay without [L]
    float *w_o, *w_q;              // [total_chunks][H][N / 16][L]
    float *w_dot;                  // [total_segs][H][N / 16]
    float *sums;                   // [total_chunks][H][4] terms of dA_log, ddt_bias, dD
    float *dBp, *dCp;              // [split][tokens][G][N] where split > 1
};

size_t ssm_workspace(SsmParams &p, void *ws, bool backward);  // sizes (and, with ws, binds) the workspace
hipError_t launch_ssm_fwd(const SsmParams &p, hipStream_t s);
hipError_t launch_ssm_bwd(const SsmParams &p, hipStream_t s);
hipError_t launch_ssm_step(const SsmParams &p, hipStream_t s);

}  // namespace kda
