// C-ABI layer of mixer.h: argument checks, workspace queries, parameter blocks.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mixer.h"
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace {

// A block of `rows` rows of `cols` elements with a row stride of `ld`, as bytes.
struct Block {
    const void *p;
    long long rows, cols, ld;
    size_t es;
};

size_t es_of(kda_dtype d) { return d == KDA_F32 ? 4 : 2; }
bool dtype_ok(kda_dtype d) { return d == KDA_BF16 || d == KDA_F32; }

long long stride_or(long long ld, long long cols) { return ld ? ld : cols; }

bool overlap(const Block &a, const Block &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.cols < 1 || b.cols < 1) return false;
    const unsigned long long x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const unsigned long long sa = (unsigned long long)a.ld * a.es, sb = (unsigned long long)b.ld * b.es;
    const unsigned long long wa = (unsigned long long)a.cols * a.es, wb = (unsigned long long)b.cols * b.es;
    const unsigned long long ea = x + (a.rows - 1) * sa + wa, eb = y + (b.rows - 1) * sb + wb;
    if (!(x < eb && y < ea)) return false;
    if (sa != sb) return true;
    // equal strides: parts of one buffer's rows, apart when their columns are
    const unsigned long long d = (y >= x ? y - x : x - y) % sa;
    const unsigned long long first = y >= x ? wa : wb, second = y >= x ? wb : wa;
    return d < first || sa - d < second;
}

// Every output apart from every input and from the other outputs; every pointer aligned to its
// element, every stride at least the row.
template <size_t NI, size_t NO> bool blocks_ok(const Block (&in)[NI], const Block (&out)[NO]) {
    for (const Block &b : in)
        if (!mixer::aligned_to(b.p, b.es) || b.ld < b.cols || b.ld > (1LL << 40)) return false;
    for (const Block &b : out)
        if (!mixer::aligned_to(b.p, b.es) || b.ld < b.cols || b.ld > (1LL << 40)) return false;
    for (size_t i = 0; i < NO; ++i) {
        for (const Block &b : in)
            if (overlap(out[i], b)) return false;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

// A packed batch has T rows whatever B is.
bool sizes_ok(int B, int T, int D, bool packed = false) {
    return B >= 1 && T >= 1 && D >= 1 && (packed || (long long)B * T <= 0x7fffffffLL) && (long long)B * D <= (1LL << 40);
}

Block dense(const void *p, long long rows, long long cols, size_t es) { return {p, rows, cols, cols, es}; }

kda_status from(cudaError_t e) {
    if (e == cudaErrorNotSupported) return KDA_ERR_UNSUPPORTED;
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status check_space(const void *ws, size_t have, size_t need) {
    if (!ws || have < need) return KDA_ERR_WORKSPACE;
    return mixer::aligned_to(ws, 16) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

cudaStream_t stream_of(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// ------------------------------------------------------------------------------ layer norm
kda_status norm_fwd(const layer_norm_fwd_args *a, mixer::NormParams &p) {
    if (!a || a->rows < 1 || a->rows > 0x7fffffffLL || a->D < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !dtype_ok(a->w_dtype) || !(a->eps >= 0.f) || !a->x || !a->y) return KDA_ERR_INVALID_ARG;
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    p.ld_x = stride_or(a->ld_x, a->D);
    p.ld_y = stride_or(a->ld_y, a->D);
    const Block in[] = {{a->x, a->rows, a->D, p.ld_x, es}, dense(a->weight, 1, a->D, ws), dense(a->bias, 1, a->D, ws)};
    const Block out[] = {{a->y, a->rows, a->D, p.ld_y, es}, dense(a->mean, 1, a->rows, 4), dense(a->rstd, 1, a->rows, 4)};
    if (!blocks_ok(in, out)) return KDA_ERR_INVALID_ARG;
    p.rows = a->rows; p.D = a->D; p.eps = a->eps;
    p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.y = a->y; p.mean = a->mean; p.rstd = a->rstd;
    p.w_bf16 = a->w_dtype == KDA_BF16;
    return KDA_OK;
}

kda_status norm_bwd(const layer_norm_bwd_args *a, mixer::NormParams &p, size_t &need) {
    if (!a || a->rows < 1 || a->rows > 0x7fffffffLL || a->D < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !dtype_ok(a->w_dtype)) return KDA_ERR_INVALID_ARG;
    if (!a->dy || !a->x || !a->mean || !a->rstd || !a->dx) return KDA_ERR_INVALID_ARG;
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    p.ld_x = stride_or(a->ld_x, a->D);
    p.ld_dy = stride_or(a->ld_dy, a->D);
    p.ld_y = stride_or(a->ld_dx, a->D);
    p.rows = a->rows; p.D = a->D;
    p.x = a->x; p.dy = a->dy; p.weight = a->weight; p.y = a->dx;
    p.mean = const_cast<float *>(a->mean); p.rstd = const_cast<float *>(a->rstd);
    p.dweight = a->dweight; p.dbias = a->dbias; p.w_bf16 = a->w_dtype == KDA_BF16;
    need = a->dweight || a->dbias ? mixer::layer_norm_part_floats(p) * 4 : 0;
    const Block in[] = {{a->x, a->rows, a->D, p.ld_x, es}, {a->dy, a->rows, a->D, p.ld_dy, es},
                        dense(a->weight, 1, a->D, ws), dense(a->mean, 1, a->rows, 4), dense(a->rstd, 1, a->rows, 4)};
    const Block out[] = {{a->dx, a->rows, a->D, p.ld_y, es}, dense(a->dweight, 1, a->D, ws), dense(a->dbias, 1, a->D, ws),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------------------ convolution
template <class A> kda_status conv_common(const A *a) {
    if (!dtype_ok(a->dtype) || !dtype_ok(a->w_dtype) || (a->flags & ~SHORT_CONV_FLAG_SILU)) return KDA_ERR_INVALID_ARG;
    if (!a->x || !a->weight || a->W < 1) return KDA_ERR_INVALID_ARG;
    return a->W >= 2 && a->W <= 4 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
template <class A> void conv_fill(const A *a, mixer::ConvParams &p) {
    p.B = a->B; p.T = a->T; p.D = a->D;
    p.silu = a->flags & SHORT_CONV_FLAG_SILU;
    p.w_bf16 = a->w_dtype == KDA_BF16;
    p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.h0 = a->h0; p.cu_seqlens = a->cu_seqlens;
    p.ld_x = stride_or(a->ld_x, a->D);
}

kda_status conv_fwd(const short_conv_fwd_args *a, mixer::ConvParams &p) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->y) return KDA_ERR_INVALID_ARG;
    const kda_status st = conv_common(a);
    if (st != KDA_OK) return st;
    conv_fill(a, p);
    p.y = a->y; p.ht = a->ht;
    p.ld_y = stride_or(a->ld_y, a->D);
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T, hrows = (long long)a->B * (a->W - 1);
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, dense(a->weight, a->D, a->W, ws), dense(a->bias, 1, a->D, ws),
                        dense(a->h0, hrows, a->D, es), dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->y, rows, a->D, p.ld_y, es}, dense(a->ht, hrows, a->D, es)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

kda_status conv_bwd(const short_conv_bwd_args *a, mixer::ConvParams &p, size_t &need) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->dy || !a->dx) return KDA_ERR_INVALID_ARG;
    const kda_status st = conv_common(a);
    if (st != KDA_OK) return st;
    conv_fill(a, p);
    p.dy = a->dy; p.dht = a->dht; p.y = a->dx; p.dh0 = a->dh0; p.dweight = a->dweight; p.dbias = a->dbias;
    p.ld_dy = stride_or(a->ld_dy, a->D);
    p.ld_y = stride_or(a->ld_dx, a->D);
    need = a->dweight || a->dbias ? mixer::short_conv_part_floats(p, a->W) * 4 : 0;
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T, hrows = (long long)a->B * (a->W - 1);
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, {a->dy, rows, a->D, p.ld_dy, es},
                        dense(a->weight, a->D, a->W, ws), dense(a->bias, 1, a->D, ws), dense(a->h0, hrows, a->D, es),
                        dense(a->dht, hrows, a->D, es), dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->dx, rows, a->D, p.ld_y, es}, dense(a->dh0, hrows, a->D, es),
                         dense(a->dweight, a->D, a->W, ws), dense(a->dbias, 1, a->D, ws),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------------------ scan
template <class A> kda_status scan_common(const A *a) {
    if (!dtype_ok(a->dtype) || (a->flags & ~SSM_FLAG_DELTA_SOFTPLUS) || a->N < 1) return KDA_ERR_INVALID_ARG;
    if (!a->x || !a->delta || !a->Bm || !a->Cm || !a->A) return KDA_ERR_INVALID_ARG;
    return a->N <= 32 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
template <class A> void scan_fill(const A *a, mixer::ScanParams &p) {
    p.B = a->B; p.D = a->D; p.N = a->N;
    p.softplus = a->flags & SSM_FLAG_DELTA_SOFTPLUS;
    p.x = a->x; p.delta = a->delta; p.Bm = a->Bm; p.Cm = a->Cm; p.z = a->z;
    p.A = a->A; p.Dskip = a->Dskip; p.delta_bias = a->delta_bias;
    p.ld_x = stride_or(a->ld_x, a->D); p.ld_delta = stride_or(a->ld_delta, a->D); p.ld_z = stride_or(a->ld_z, a->D);
    p.ld_B = stride_or(a->ld_B, a->N); p.ld_C = stride_or(a->ld_C, a->N);
}

kda_status scan_fwd(const ssm_scan_fwd_args *a, mixer::ScanParams &p, size_t &need) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->y) return KDA_ERR_INVALID_ARG;
    const kda_status st = scan_common(a);
    if (st != KDA_OK) return st;
    scan_fill(a, p);
    p.T = a->T; p.h0 = a->h0; p.y = a->y; p.ht = a->ht; p.cu_seqlens = a->cu_seqlens;
    p.ld_y = stride_or(a->ld_y, a->D);
    need = mixer::ssm_scan_fwd_floats(p, a->dtype == KDA_BF16) * 4;
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T, hrows = (long long)a->B * a->D;
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, {a->delta, rows, a->D, p.ld_delta, es},
                        {a->Bm, rows, a->N, p.ld_B, es}, {a->Cm, rows, a->N, p.ld_C, es}, {a->z, rows, a->D, p.ld_z, es},
                        dense(a->A, a->D, a->N, 4), dense(a->Dskip, 1, a->D, 4), dense(a->delta_bias, 1, a->D, 4),
                        dense(a->h0, hrows, a->N, 4), dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->y, rows, a->D, p.ld_y, es}, dense(a->ht, hrows, a->N, 4),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

kda_status scan_bwd(const ssm_scan_bwd_args *a, mixer::ScanParams &p, size_t &need) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->dy || !a->dx || !a->ddelta || !a->dBm || !a->dCm || !a->dA)
        return KDA_ERR_INVALID_ARG;
    if ((a->z == nullptr) != (a->dz == nullptr)) return KDA_ERR_INVALID_ARG;
    const kda_status st = scan_common(a);
    if (st != KDA_OK) return st;
    scan_fill(a, p);
    p.T = a->T; p.h0 = a->h0; p.dht = a->dht; p.dy = a->dy; p.cu_seqlens = a->cu_seqlens;
    p.dx = a->dx; p.ddelta = a->ddelta; p.dBm = a->dBm; p.dCm = a->dCm; p.dz = a->dz;
    p.dA = a->dA; p.dDskip = a->dDskip; p.ddelta_bias = a->ddelta_bias; p.dh0 = a->dh0;
    p.ld_dy = stride_or(a->ld_dy, a->D); p.ld_dx = stride_or(a->ld_dx, a->D);
    p.ld_ddelta = stride_or(a->ld_ddelta, a->D); p.ld_dz = stride_or(a->ld_dz, a->D);
    p.ld_dB = stride_or(a->ld_dB, a->N); p.ld_dC = stride_or(a->ld_dC, a->N);
    need = mixer::ssm_scan_bwd_floats(p) * 4;
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T, hrows = (long long)a->B * a->D;
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, {a->delta, rows, a->D, p.ld_delta, es},
                        {a->Bm, rows, a->N, p.ld_B, es}, {a->Cm, rows, a->N, p.ld_C, es}, {a->z, rows, a->D, p.ld_z, es},
                        {a->dy, rows, a->D, p.ld_dy, es}, dense(a->A, a->D, a->N, 4), dense(a->Dskip, 1, a->D, 4),
                        dense(a->delta_bias, 1, a->D, 4), dense(a->h0, hrows, a->N, 4), dense(a->dht, hrows, a->N, 4),
                        dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->dx, rows, a->D, p.ld_dx, es}, {a->ddelta, rows, a->D, p.ld_ddelta, es},
                         {a->dBm, rows, a->N, p.ld_dB, es}, {a->dCm, rows, a->N, p.ld_dC, es},
                         {a->dz, rows, a->D, p.ld_dz, es}, dense(a->dA, a->D, a->N, 4), dense(a->dDskip, 1, a->D, 4),
                         dense(a->ddelta_bias, 1, a->D, 4), dense(a->dh0, hrows, a->N, 4),
                         dense(a->workspace, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

kda_status layer_norm_fwd(const layer_norm_fwd_args *a, kda_stream_t stream) {
    mixer::NormParams p{};
    const kda_status st = norm_fwd(a, p);
    return st != KDA_OK ? st : from(mixer::launch_layer_norm_fwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t layer_norm_bwd_workspace(const layer_norm_bwd_args *a) {
    mixer::NormParams p{};
    size_t need = 0;
    return norm_bwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status layer_norm_bwd(const layer_norm_bwd_args *a, kda_stream_t stream) {
    mixer::NormParams p{};
    size_t need = 0;
    kda_status st = norm_bwd(a, p, need);
    if (st != KDA_OK) return st;
    if (need) {
        if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
        p.part = static_cast<float *>(a->workspace);
    }
    return from(mixer::launch_layer_norm_bwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

kda_status short_conv_fwd(const short_conv_fwd_args *a, kda_stream_t stream) {
    mixer::ConvParams p{};
    const kda_status st = conv_fwd(a, p);
    return st != KDA_OK ? st : from(mixer::launch_short_conv_fwd(p, a->W, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t short_conv_bwd_workspace(const short_conv_bwd_args *a) {
    mixer::ConvParams p{};
    size_t need = 0;
    return conv_bwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status short_conv_bwd(const short_conv_bwd_args *a, kda_stream_t stream) {
    mixer::ConvParams p{};
    size_t need = 0;
    kda_status st = conv_bwd(a, p, need);
    if (st != KDA_OK) return st;
    if (need) {
        if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
        p.part = static_cast<float *>(a->workspace);
    }
    return from(mixer::launch_short_conv_bwd(p, a->W, a->dtype == KDA_BF16, stream_of(stream)));
}

kda_status short_conv_step(const short_conv_step_args *a, kda_stream_t stream) {
    if (!a || !sizes_ok(a->B, 1, a->D) || a->slots < 1 || !a->state || !a->y) return KDA_ERR_INVALID_ARG;
    if (!a->slot && a->slots < a->B) return KDA_ERR_INVALID_ARG;
    const kda_status st = conv_common(a);
    if (st != KDA_OK) return st;
    mixer::ConvParams p{};
    p.B = a->B; p.T = 1; p.D = a->D; p.slots = a->slots;
    p.silu = a->flags & SHORT_CONV_FLAG_SILU; p.w_bf16 = a->w_dtype == KDA_BF16;
    p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.state = a->state; p.slot = a->slot; p.y = a->y;
    p.ld_x = stride_or(a->ld_x, a->D);
    p.ld_y = stride_or(a->ld_y, a->D);
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    const Block in[] = {{a->x, a->B, a->D, p.ld_x, es}, dense(a->weight, a->D, a->W, ws), dense(a->bias, 1, a->D, ws),
                        dense(a->slot, 1, a->B, 4)};
    const Block out[] = {{a->y, a->B, a->D, p.ld_y, es}, dense(a->state, (long long)a->slots * (a->W - 1), a->D, es)};
    if (!blocks_ok(in, out)) return KDA_ERR_INVALID_ARG;
    return from(mixer::launch_short_conv_step(p, a->W, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t ssm_scan_fwd_workspace(const ssm_scan_fwd_args *a) {
    mixer::ScanParams p{};
    size_t need = 0;
    return scan_fwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status ssm_scan_fwd(const ssm_scan_fwd_args *a, kda_stream_t stream) {
    mixer::ScanParams p{};
    size_t need = 0;
    const kda_status st = scan_fwd(a, p, need);
    if (st != KDA_OK) return st;
    p.seg = a->T;
    if (need && a->workspace && a->workspace_bytes >= need) {
        if (!mixer::aligned_to(a->workspace, 16)) return KDA_ERR_INVALID_ARG;
        p.seg = mixer::ssm_scan_fwd_segment(p, a->dtype == KDA_BF16);
        mixer::ssm_scan_fwd_carve(p, static_cast<float *>(a->workspace));
    }
    return from(mixer::launch_ssm_scan_fwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t ssm_scan_bwd_workspace(const ssm_scan_bwd_args *a) {
    mixer::ScanParams p{};
    size_t need = 0;
    return scan_bwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status ssm_scan_bwd(const ssm_scan_bwd_args *a, kda_stream_t stream) {
    mixer::ScanParams p{};
    size_t need = 0;
    kda_status st = scan_bwd(a, p, need);
    if (st != KDA_OK) return st;
    if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
    mixer::ssm_scan_bwd_carve(p, static_cast<float *>(a->workspace));
    return from(mixer::launch_ssm_scan_bwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

kda_status ssm_scan_step(const ssm_scan_step_args *a, kda_stream_t stream) {
    if (!a || !sizes_ok(a->B, 1, a->D) || a->slots < 1 || !a->state || !a->y) return KDA_ERR_INVALID_ARG;
    if (!a->slot && a->slots < a->B) return KDA_ERR_INVALID_ARG;
    const kda_status st = scan_common(a);
    if (st != KDA_OK) return st;
    mixer::ScanParams p{};
    scan_fill(a, p);
    p.T = 1; p.slots = a->slots; p.state = a->state; p.slot = a->slot; p.y = a->y;
    p.ld_y = stride_or(a->ld_y, a->D);
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, a->B, a->D, p.ld_x, es}, {a->delta, a->B, a->D, p.ld_delta, es}, {a->Bm, a->B, a->N, p.ld_B, es},
                        {a->Cm, a->B, a->N, p.ld_C, es}, {a->z, a->B, a->D, p.ld_z, es}, dense(a->A, a->D, a->N, 4),
                        dense(a->Dskip, 1, a->D, 4), dense(a->delta_bias, 1, a->D, 4), dense(a->slot, 1, a->B, 4)};
    const Block out[] = {{a->y, a->B, a->D, p.ld_y, es}, dense(a->state, (long long)a->slots * a->D, a->N, 4)};
    if (!blocks_ok(in, out)) return KDA_ERR_INVALID_ARG;
    return from(mixer::launch_ssm_scan_step(p, a->dtype == KDA_BF16, stream_of(stream)));
}

}  // extern "C"
