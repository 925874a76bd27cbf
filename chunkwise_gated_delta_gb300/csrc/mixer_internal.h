// Parameter blocks and launchers of the operators declared in mixer.h.  The C-ABI layer
// (mixer_api.cu) has checked every argument and replaced row strides of 0 by the row length.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mixer {

struct NormParams {
    long long rows;
    int D;
    float eps;
    const void *x, *dy, *weight, *bias;
    long long ld_x, ld_dy, ld_y;      // ld_y: of y, or of dx in the backward
    void *y;                          // y, or dx
    float *mean, *rstd;
    void *dweight, *dbias;
    float *part;                      // [blocks][2][D]
    bool w_bf16;
};

struct ConvParams {
    int B, T, D;
    int seg;                          // tokens per unit of work
    bool silu, w_bf16;
    const void *x, *weight, *bias, *h0, *dy, *dht;
    long long ld_x, ld_y, ld_dy;      // ld_y: of y, or of dx in the backward
    void *y, *ht, *dh0, *dweight, *dbias;
    float *part;                      // [blocks of slots][D (W + 1)]
    const int32_t *cu_seqlens;
    // single tokens
    int slots;
    void *state;
    const int32_t *slot;
};

struct ScanParams {
    int B, T, D, N;
    int seg;                          // tokens per segment that the forward walks alone; >= T: whole sequences
    int lseg;                         // tokens per segment of the local pass (divides seg)
    bool softplus;
    const void *x, *delta, *Bm, *Cm, *z, *dy;
    long long ld_x, ld_delta, ld_B, ld_C, ld_z, ld_y, ld_dy;
    long long ld_dx, ld_ddelta, ld_dB, ld_dC, ld_dz;
    const float *A, *Dskip, *delta_bias, *h0, *dht;
    void *y;
    float *ht;
    void *dx, *ddelta, *dBm, *dCm, *dz;
    float *dA, *dDskip, *ddelta_bias, *dh0;
    const int32_t *cu_seqlens;
    // workspace: [slots][D][NP] states entering (and gradients leaving) each segment,
    // [slots][D] sums of dt; partial sums of the parameters' and of Bm's and Cm's gradients
    float *seg_state, *seg_grad, *seg_dt, *part_par, *part_bc;
    // single tokens
    int slots;
    float *state;
    const int32_t *slot;
};

cudaError_t launch_layer_norm_fwd(const NormParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_layer_norm_bwd(const NormParams &p, bool bf16, cudaStream_t s);
size_t layer_norm_part_floats(const NormParams &p);

cudaError_t launch_short_conv_fwd(const ConvParams &p, int W, bool bf16, cudaStream_t s);
cudaError_t launch_short_conv_bwd(const ConvParams &p, int W, bool bf16, cudaStream_t s);
cudaError_t launch_short_conv_step(const ConvParams &p, int W, bool bf16, cudaStream_t s);
size_t short_conv_part_floats(const ConvParams &p, int W);

cudaError_t launch_ssm_scan_fwd(const ScanParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_ssm_scan_step(const ScanParams &p, bool bf16, cudaStream_t s);
int ssm_scan_fwd_segment(const ScanParams &p, bool bf16);   // tokens per segment (T: unsplit)
cudaError_t launch_ssm_scan_bwd(const ScanParams &p, bool bf16, cudaStream_t s);
// Workspace floats; carve() points the parameter block into a workspace of that size.
size_t ssm_scan_fwd_floats(const ScanParams &p, bool bf16);
size_t ssm_scan_bwd_floats(const ScanParams &p);
void ssm_scan_fwd_carve(ScanParams &p, float *ws);
void ssm_scan_bwd_carve(ScanParams &p, float *ws);

}  // namespace mixer
