/*
 * mixer.h -- C ABI of the operators that stand around a recurrent token mixer
 * (GB300, sm_103a): layer norm, the short causal convolution, and the selective
 * state-space scan.  The pages behind kda.h do not treat them; the definitions are:
 *
 *   layer norm   y = (x - mean) rstd weight + bias,  rstd = 1 / sqrt(var + eps), per row
 *   convolution  y_t[d] = act(bias[d] + sum_j weight[d][j] x_{t-W+1+j}[d]),  act: none or SiLU
 *   scan         dt_t[d] = softplus(delta_t[d] + delta_bias[d])   (or delta + bias itself)
 *                h_t[d][n] = exp(dt_t[d] A[d][n]) h_{t-1}[d][n] + dt_t[d] x_t[d] Bm_t[n]
 *                y_t[d] = (sum_n Cm_t[n] h_t[d][n] + D[d] x_t[d]) SiLU(z_t[d])
 *
 * The scan's decay depends on channel and state together, so it has no chunkwise matrix
 * form like the one kda_chunk_fwd evaluates.
 *
 * Conventions (those of kda.h, with these differences and additions)
 *   - Sequence tensors are [B, T, C] with C fastest and a row stride in elements of their
 *     own, ld_* (0: contiguous; otherwise at least C): row t of sequence b begins at
 *     element (b T + t) ld, so the parts of a wider projection's output are used where
 *     they lie.  Every pointer is aligned to its element.  Where the base and row stride of
 *     every tensor of a call are multiples of 16 bytes and C is one of 8 elements, data moves
 *     in accesses of 8 or 16 bytes, otherwise in single elements or, where it is aligned to
 *     four of them, in fours (convolution's and scan's backward, single tokens).  The
 *     scan's forward asks for N, base and stride of Bm and Cm in multiples of four elements
 *     too, and moves everything by single elements without.  Workspaces are 16-byte aligned.
 *   - cu_seqlens as in kda_fwd_args: B sequences back to back in [1, T, C] tensors, B + 1
 *     int32 offsets on the device, clamped into [0, T]; empty sequences are allowed (their
 *     final state is their initial one).  Rows that no sequence covers are not written.
 *   - T >= 1, B >= 1 and rows (B T, in a packed batch T) at most 2^31 - 1;
 *     KDA_ERR_INVALID_ARG otherwise.
 *   - Arithmetic is float32 for both dtypes; results are rounded once on output.  Sums
 *     over tokens and channels are added in a fixed order: equal calls give equal bits.
 *   - Nothing waits on the device, so there is no status block; workspaces need no
 *     initial contents.
 *   - Outputs must not overlap inputs or each other.  Parts of one row-strided buffer do
 *     not overlap when their columns are disjoint and their strides are equal.
 */
#ifndef MIXER_H_
#define MIXER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------- layer norm */

typedef struct {
    long long rows;        /* >= 1 */
    int D;                 /* columns, >= 1 */
    kda_dtype dtype;       /* of x and y */
    kda_dtype w_dtype;     /* of weight and bias */
    float eps;             /* >= 0 */
    const void *x;         /* [rows, D] */
    long long ld_x;        /* row stride, 0 = D */
    const void *weight;    /* [D], or NULL (1) */
    const void *bias;      /* [D], or NULL (0) */
    void *y;               /* [rows, D] out */
    long long ld_y;
    float *mean, *rstd;    /* [rows] out, or NULL (not written) */
} layer_norm_fwd_args;

/* Mean and variance in two passes over the row held on chip (no cancellation). */
kda_status layer_norm_fwd(const layer_norm_fwd_args *args, kda_stream_t stream);

typedef struct {
    long long rows;
    int D;
    kda_dtype dtype;       /* of dy, x and dx */
    kda_dtype w_dtype;     /* of weight, dweight and dbias */
    const void *dy;        /* [rows, D] */
    long long ld_dy;
    const void *x;         /* [rows, D] */
    long long ld_x;
    const void *weight;    /* [D], or NULL (1) */
    const float *mean, *rstd;   /* [rows], from layer_norm_fwd */
    void *dx;              /* [rows, D] out */
    long long ld_dx;
    void *dweight;         /* [D] out, or NULL (not written) */
    void *dbias;           /* [D] out, or NULL (not written) */
    void *workspace;       /* layer_norm_bwd_workspace bytes */
    size_t workspace_bytes;
} layer_norm_bwd_args;

/* Bytes of workspace: per-block partial sums of dweight and dbias (0 on bad args, and where few rows
   take none; layer_norm_bwd tells which). */
size_t layer_norm_bwd_workspace(const layer_norm_bwd_args *args);

/*
 * With xh = (x - mean) rstd and g = dy weight:
 *     dx = rstd (g - mean_row(g) - xh mean_row(g xh)),  dweight = sum_rows dy xh,  dbias = sum_rows dy.
 */
kda_status layer_norm_bwd(const layer_norm_bwd_args *args, kda_stream_t stream);

/* --------------------------------------------------- short causal convolution */

#define SHORT_CONV_FLAG_SILU 1u

typedef struct {
    int B, T, D;           /* sequences, tokens, channels */
    int W;                 /* taps: 2, 3 or 4 (KDA_ERR_UNSUPPORTED otherwise) */
    kda_dtype dtype;       /* of x, h0, y, ht */
    kda_dtype w_dtype;     /* of weight and bias */
    unsigned flags;        /* SHORT_CONV_FLAG_* */
    const void *x;         /* [B, T, D] */
    long long ld_x;
    const void *weight;    /* [D, W], the last tap is the current token's */
    const void *bias;      /* [D], or NULL */
    const void *h0;        /* [B, W-1, D]: the inputs before the first token, oldest first; NULL: zeros */
    void *y;               /* [B, T, D] out */
    long long ld_y;
    void *ht;              /* [B, W-1, D] out: the last W-1 inputs, h0's among them when T < W-1; or NULL */
    const int32_t *cu_seqlens;
} short_conv_fwd_args;

kda_status short_conv_fwd(const short_conv_fwd_args *args, kda_stream_t stream);

typedef struct {
    int B, T, D, W;
    kda_dtype dtype;       /* of x, h0, dy, dht, dx, dh0 */
    kda_dtype w_dtype;     /* of weight, bias, dweight, dbias */
    unsigned flags;
    const void *x;
    long long ld_x;
    const void *weight, *bias, *h0;    /* as the forward's */
    const void *dy;        /* [B, T, D] */
    long long ld_dy;
    const void *dht;       /* [B, W-1, D] gradient of the final state, or NULL (zero) */
    void *dx;              /* [B, T, D] out */
    long long ld_dx;
    void *dh0;             /* [B, W-1, D] out, or NULL */
    void *dweight;         /* [D, W] out, or NULL */
    void *dbias;           /* [D] out, or NULL */
    void *workspace;       /* short_conv_bwd_workspace bytes */
    size_t workspace_bytes;
    const int32_t *cu_seqlens;
} short_conv_bwd_args;

/* Bytes of workspace (0 on bad args): per-block partial sums of dweight and dbias. */
size_t short_conv_bwd_workspace(const short_conv_bwd_args *args);
/* The values before the activation are recomputed from x. */
kda_status short_conv_bwd(const short_conv_bwd_args *args, kda_stream_t stream);

typedef struct {
    int B, D, W;           /* requests (one token each), channels, taps */
    int slots;             /* states in `state` */
    kda_dtype dtype, w_dtype;
    unsigned flags;
    const void *x;         /* [B, D] */
    long long ld_x;
    const void *weight, *bias;
    void *state;           /* [slots, W-1, D], updated in place: the oldest input leaves, x enters */
    const int32_t *slot;   /* [B] device: the state of each request, or NULL (request b has state b; slots >= B).
                              A request whose slot lies outside [0, slots) is padding: its y is 0 and no state
                              changes.  Two requests of a call must not share a slot. */
    void *y;               /* [B, D] out */
    long long ld_y;
} short_conv_step_args;

/* One token of each request. */
kda_status short_conv_step(const short_conv_step_args *args, kda_stream_t stream);

/* ---------------------------------------------------- selective state-space scan */

#define SSM_FLAG_DELTA_SOFTPLUS 1u   /* dt = softplus(delta + delta_bias); cleared: dt = delta + delta_bias */

typedef struct {
    int B, T, D;           /* sequences, tokens, channels */
    int N;                 /* states per channel, 1 to 32 (KDA_ERR_UNSUPPORTED above) */
    kda_dtype dtype;       /* of x, delta, Bm, Cm, z, y */
    unsigned flags;        /* SSM_FLAG_* */
    const void *x;         /* [B, T, D] */
    long long ld_x;
    const void *delta;     /* [B, T, D] */
    long long ld_delta;
    const void *Bm;        /* [B, T, N], shared by all channels */
    long long ld_B;
    const void *Cm;        /* [B, T, N] */
    long long ld_C;
    const void *z;         /* [B, T, D] gate, or NULL (no gate) */
    long long ld_z;
    const float *A;        /* [D, N] */
    const float *Dskip;    /* [D], or NULL (0) */
    const float *delta_bias; /* [D], or NULL (0) */
    const float *h0;       /* [B, D, N], or NULL (0) */
    void *y;               /* [B, T, D] out */
    long long ld_y;
    float *ht;             /* [B, D, N] out, or NULL */
    void *workspace;       /* ssm_scan_fwd_workspace bytes, or NULL when that is 0 */
    size_t workspace_bytes;
    const int32_t *cu_seqlens;
} ssm_scan_fwd_args;

/*
 * Bytes of workspace for the split form, which cuts long sequences into segments where whole
 * sequences would leave most of the GPU idle: 0 for the other calls and on bad args
 * (ssm_scan_fwd tells which).  With a smaller workspace the call runs unsplit.
 */
size_t ssm_scan_fwd_workspace(const ssm_scan_fwd_args *args);
kda_status ssm_scan_fwd(const ssm_scan_fwd_args *args, kda_stream_t stream);

typedef struct {
    int B, T, D, N;
    kda_dtype dtype;       /* of the sequence tensors and their gradients */
    unsigned flags;
    const void *x;
    long long ld_x;
    const void *delta;
    long long ld_delta;
    const void *Bm;
    long long ld_B;
    const void *Cm;
    long long ld_C;
    const void *z;
    long long ld_z;
    const float *A, *Dskip, *delta_bias, *h0;   /* as the forward's */
    const void *dy;        /* [B, T, D] gradient of y */
    long long ld_dy;
    const float *dht;      /* [B, D, N] gradient of the final state, or NULL (zero) */
    void *dx;              /* [B, T, D] out */
    long long ld_dx;
    void *ddelta;          /* [B, T, D] out */
    long long ld_ddelta;
    void *dBm;             /* [B, T, N] out */
    long long ld_dB;
    void *dCm;             /* [B, T, N] out */
    long long ld_dC;
    void *dz;              /* [B, T, D] out; NULL iff z is NULL */
    long long ld_dz;
    float *dA;             /* [D, N] out */
    float *dDskip;         /* [D] out, or NULL */
    float *ddelta_bias;    /* [D] out, or NULL */
    float *dh0;            /* [B, D, N] out, or NULL */
    void *workspace;       /* ssm_scan_bwd_workspace bytes */
    size_t workspace_bytes;
    const int32_t *cu_seqlens;
} ssm_scan_bwd_args;

/* Bytes of workspace (0 on bad args): boundary states and their gradients per segment of 64
   tokens, and partial sums of dBm, dCm, dA, dDskip and ddelta_bias. */
size_t ssm_scan_bwd_workspace(const ssm_scan_bwd_args *args);

/*
 * Gradients of sum(y dy) + sum(ht dht).  The forward's states are recomputed.  With
 * g_t = dy_t SiLU(z_t) and G_t the gradient of h_t,
 *     G_t = Cm_t g_t + exp(dt_{t+1} A) G_{t+1},
 *     dCm_t = sum_d g_t h_t,   dBm_t = sum_d G_t dt_t x_t,   u_t = sum_n G_t Bm_t,
 *     q_t = G_t exp(dt_t A) h_{t-1},   dA = sum_t q_t dt_t,   ddt_t = sum_n q_t A + u_t x_t,
 *     dx_t = u_t dt_t + D g_t,   ddelta = ddt sigmoid(delta + delta_bias),
 *     dz_t = dy_t (sum_n Cm_t h_t + D x_t) SiLU'(z_t).
 */
kda_status ssm_scan_bwd(const ssm_scan_bwd_args *args, kda_stream_t stream);

typedef struct {
    int B, D, N;           /* requests (one token each), channels, states per channel */
    int slots;
    kda_dtype dtype;
    unsigned flags;
    const void *x;         /* [B, D] */
    long long ld_x;
    const void *delta;     /* [B, D] */
    long long ld_delta;
    const void *Bm;        /* [B, N] */
    long long ld_B;
    const void *Cm;        /* [B, N] */
    long long ld_C;
    const void *z;         /* [B, D] or NULL */
    long long ld_z;
    const float *A, *Dskip, *delta_bias;
    float *state;          /* [slots, D, N], updated in place */
    const int32_t *slot;   /* [B] device or NULL: as short_conv_step_args */
    void *y;               /* [B, D] out */
    long long ld_y;
} ssm_scan_step_args;

/* One token of each request. */
kda_status ssm_scan_step(const ssm_scan_step_args *args, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MIXER_H_ */
