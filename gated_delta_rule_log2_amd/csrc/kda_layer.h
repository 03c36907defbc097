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

}  // namespace kda
