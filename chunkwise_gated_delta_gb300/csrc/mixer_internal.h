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

struct GatedScanParams {
    int B, T, D;
    int seg;                          // rows of a segment
    float scale;
    const void *x, *decay, *gate, *dy;
    long long ld_x, ld_decay, ld_gate, ld_y, ld_dy, ld_dx, ld_ddecay, ld_dgate;
    const float *rate, *h0, *dht;
    void *y, *dx, *ddecay, *dgate;
    float *ht, *states;               // states: [ceil(rows / 8)][D], the state that enters each 8th row
    float *drate, *dh0;
    float *ws;                        // workspace: what each segment does to a state (pairs of floats), what enters it, sums of drate
    float *seg_pair, *seg_in, *part;
    const int32_t *cu_seqlens;
    // single tokens
    int slots;
    float *state;
    const int32_t *slot;
};

struct GroupNormParams {
    long long rows;
    int G, C;                         // groups of a row, columns of a group
    float eps;
    bool center, shared, w_bf16;      // shared: one weight [C] for all groups, else [G C]
    const void *x, *gate, *dy, *weight, *bias;
    long long ld_x, ld_gate, ld_dy, ld_y, ld_dgate;   // ld_y: of y, or of dx in the backward
    void *y, *dgate;                  // y: y or dx
    float *mean, *rstd;
    void *dweight, *dbias;
    float *part;
};

struct GluParams {
    long long M;
    int D, F;
    bool gelu;
    const void *x, *wg, *wu, *dh;
    long long ld_x, ld_wg, ld_wu, ld_dh, ld_h, ld_dx, ld_dwg, ld_dwu;
    void *h, *dx, *dwg, *dwu;
    float *g, *u;                     // [M][F] the two products, or NULL
    void *dg, *du;                    // workspace [M][ld_d]: their gradients
    long long ld_d;
    void *part;                       // workspace: sums of parts of K (glu_tc_part_bytes)
    int *status;                      // status block, or NULL
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

cudaError_t launch_gated_scan_fwd(const GatedScanParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_gated_scan_bwd(const GatedScanParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_gated_scan_step(const GatedScanParams &p, bool bf16, cudaStream_t s);
size_t gated_scan_saved_rows(const GatedScanParams &p);
// Workspace floats (the backward's: the states aside, but also enough for the forward).
size_t gated_scan_fwd_floats(const GatedScanParams &p);
size_t gated_scan_bwd_floats(const GatedScanParams &p);

cudaError_t launch_group_norm_fwd(const GroupNormParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_group_norm_bwd(const GroupNormParams &p, bool bf16, cudaStream_t s);
size_t group_norm_part_floats(const GroupNormParams &p, bool bf16);

cudaError_t launch_glu_fwd(const GluParams &p, bool bf16, char *ws, cudaStream_t s);
cudaError_t launch_glu_bwd(const GluParams &p, bool bf16, char *ws, cudaStream_t s);
long long glu_grad_stride(const GluParams &p, bool bf16);
size_t glu_moved_bytes(const GluParams &p, bool bf16);       // of ws
// Forms of bfloat16 calls: the tensor cores' products, and a few rows past the weights.
size_t glu_tc_part_bytes(const GluParams &p);
cudaError_t launch_glu_tc_fwd(const GluParams &p, cudaStream_t s);
cudaError_t launch_glu_tc_grads(const GluParams &p, cudaStream_t s);
cudaError_t launch_glu_tc_dx(const GluParams &p, cudaStream_t s);
cudaError_t launch_glu_tc_dw(const GluParams &p, cudaStream_t s);
bool glu_rows_takes(const GluParams &p);
cudaError_t launch_glu_rows(const GluParams &p, cudaStream_t s);

}  // namespace mixer
