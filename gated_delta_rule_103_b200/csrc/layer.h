// Launchers of the layer operators (short convolution, state-space scan,
// group norm) behind the C ABI in layer_api.cu, which has validated every
// argument.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

struct ConvArgs {
    const void* x;
    const float* weight;           // [C, W]
    const float* bias;             // [C] or nullptr
    const void* initial_state;     // [N, W-1, C] or nullptr
    const int32_t* cu_seqlens;     // nullptr: sequence n is batch row n
    void* out;
    void* final_state;             // or nullptr
    const void* d_out;             // backward
    const float* d_final_state;    // [N, W-1, C] or nullptr
    float* grad_x;
    float* grad_weight;
    float* grad_bias;              // or nullptr
    float* grad_initial_state;     // or nullptr
    void* workspace;
    int B, T, C, W, N;
    int silu;
};
cudaError_t launch_conv_fwd(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream);
cudaError_t launch_conv_step(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream);
cudaError_t launch_conv_bwd(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream);
size_t conv_bwd_workspace(int B, int T, int C, int W, int N, kda_dtype dtype);

struct ScanArgs {
    const void* u;                 // [B, T, D]
    const void* delta;             // [B, T, D]
    const float* A;                // [D, S]
    const void* Bm;                // [B, T, G, S]
    const void* Cm;                // [B, T, G, S]
    const float* skip;             // [D] or nullptr
    const void* z;                 // [B, T, D] or nullptr
    const float* delta_bias;       // [D] or nullptr
    const float* initial_state;    // [N, D, S] or nullptr
    const int32_t* cu_seqlens;
    void* out;
    float* final_state;            // or nullptr
    const void* d_out;             // backward
    const float* d_final_state;
    float *grad_u, *grad_delta, *grad_A, *grad_B, *grad_C;
    float *grad_skip, *grad_z, *grad_delta_bias, *grad_initial_state;
    void* workspace;
    int B, T, D, S, G, N;
    int softplus;
};
size_t scan_fwd_workspace(int B, int T, int D, int S, int G, int N, int packed, kda_dtype dtype);
cudaError_t launch_scan_fwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanArgs& a, kda_dtype dtype, cudaStream_t stream);
size_t scan_bwd_workspace(int B, int T, int D, int S, int G, int N, int packed, kda_dtype dtype);
cudaError_t launch_scan_bwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t stream);

struct NormArgs {
    const void* x;                 // [B, T, C]
    const float* weight;           // [C] or nullptr
    const float* bias;             // [C] or nullptr
    const int32_t* cu_seqlens;
    void* out;
    float* mean;                   // [samples, G]
    float* rstd;
    const void* d_out;             // backward
    float* grad_x;
    float* grad_weight;            // or nullptr
    float* grad_bias;              // or nullptr
    void* workspace;
    int B, T, C, G, N;
    int per_token;
    float eps;
    int silu;
};
size_t norm_fwd_workspace(int B, int T, int C, int G, int N, int per_token, int packed, kda_dtype dtype);
cudaError_t launch_norm_fwd(const NormArgs& a, kda_dtype dtype, cudaStream_t stream);
size_t norm_bwd_workspace(int B, int T, int C, int G, int N, int per_token, int packed, kda_dtype dtype);
cudaError_t launch_norm_bwd(const NormArgs& a, kda_dtype dtype, cudaStream_t stream);

}  // namespace kda
