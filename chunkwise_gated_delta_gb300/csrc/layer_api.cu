// C-ABI layer of mixer.h's operators behind and beside the mixer: the gated recurrence, the norm over groups
// and the gated feed-forward product.  Argument checks, workspace queries, parameter blocks.
#include "mixer_checks.h"
#include "mixer_internal.h"

namespace {

// ------------------------------------------------------------------------------ gated recurrence
template <class A> kda_status gated_common(const A *a) {
    if (!dtype_ok(a->dtype) || !a->x || !a->decay || !a->gate || !a->rate) return KDA_ERR_INVALID_ARG;
    return a->scale > 0.f && a->scale <= 3.0e38f ? KDA_OK : KDA_ERR_INVALID_ARG;
}
template <class A> void gated_fill(const A *a, mixer::GatedScanParams &p) {
    p.B = a->B; p.D = a->D; p.scale = a->scale;
    p.x = a->x; p.decay = a->decay; p.gate = a->gate; p.rate = a->rate;
    p.ld_x = stride_or(a->ld_x, a->D); p.ld_decay = stride_or(a->ld_decay, a->D); p.ld_gate = stride_or(a->ld_gate, a->D);
}

kda_status gated_fwd(const gated_scan_fwd_args *a, mixer::GatedScanParams &p, size_t &need) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->y) return KDA_ERR_INVALID_ARG;
    const kda_status st = gated_common(a);
    if (st != KDA_OK) return st;
    gated_fill(a, p);
    p.T = a->T; p.h0 = a->h0; p.y = a->y; p.ht = a->ht; p.states = a->states; p.cu_seqlens = a->cu_seqlens;
    p.ld_y = stride_or(a->ld_y, a->D);
    need = mixer::gated_scan_fwd_floats(p) * 4;
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T;
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, {a->decay, rows, a->D, p.ld_decay, es}, {a->gate, rows, a->D, p.ld_gate, es},
                        dense(a->rate, 1, a->D, 4), dense(a->h0, a->B, a->D, 4), dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->y, rows, a->D, p.ld_y, es}, dense(a->ht, a->B, a->D, 4),
                         dense(a->states, (long long)mixer::gated_scan_saved_rows(p), a->D, 4),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// need: partial sums, and the states where the caller has not kept them.
kda_status gated_bwd(const gated_scan_bwd_args *a, mixer::GatedScanParams &p, size_t &need, size_t &states) {
    if (!a || !sizes_ok(a->B, a->T, a->D, a->cu_seqlens) || !a->dy || !a->dx || !a->ddecay || !a->dgate || !a->drate)
        return KDA_ERR_INVALID_ARG;
    const kda_status st = gated_common(a);
    if (st != KDA_OK) return st;
    gated_fill(a, p);
    p.T = a->T; p.h0 = a->h0; p.dht = a->dht; p.dy = a->dy; p.cu_seqlens = a->cu_seqlens;
    p.states = const_cast<float *>(a->states);
    p.dx = a->dx; p.ddecay = a->ddecay; p.dgate = a->dgate; p.drate = a->drate; p.dh0 = a->dh0;
    p.ld_dy = stride_or(a->ld_dy, a->D); p.ld_dx = stride_or(a->ld_dx, a->D);
    p.ld_ddecay = stride_or(a->ld_ddecay, a->D); p.ld_dgate = stride_or(a->ld_dgate, a->D);
    const size_t part = mixer::gated_scan_bwd_floats(p), saved = mixer::gated_scan_saved_rows(p);
    states = a->states ? 0 : (saved * a->D + 3) / 4 * 16;
    need = states + part * 4;
    const long long rows = (long long)(a->cu_seqlens ? 1 : a->B) * a->T;
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, rows, a->D, p.ld_x, es}, {a->decay, rows, a->D, p.ld_decay, es}, {a->gate, rows, a->D, p.ld_gate, es},
                        {a->dy, rows, a->D, p.ld_dy, es}, dense(a->rate, 1, a->D, 4), dense(a->h0, a->B, a->D, 4),
                        dense(a->dht, a->B, a->D, 4), dense(a->states, (long long)saved, a->D, 4),
                        dense(a->cu_seqlens, 1, (long long)a->B + 1, 4)};
    const Block out[] = {{a->dx, rows, a->D, p.ld_dx, es}, {a->ddecay, rows, a->D, p.ld_ddecay, es},
                         {a->dgate, rows, a->D, p.ld_dgate, es}, dense(a->drate, 1, a->D, 4), dense(a->dh0, a->B, a->D, 4),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------------------ norm over groups
template <class A> kda_status group_common(const A *a, mixer::GroupNormParams &p) {
    if (a->rows < 1 || a->rows > 0x7fffffffLL || a->groups < 1 || a->C < 1 || (long long)a->groups * a->C > 0x7fffffffLL ||
        a->rows * a->groups > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !dtype_ok(a->w_dtype) || !a->x) return KDA_ERR_INVALID_ARG;
    if (a->flags & ~(GROUP_NORM_FLAG_CENTER | GROUP_NORM_FLAG_SHARED)) return KDA_ERR_INVALID_ARG;
    p.rows = a->rows; p.G = a->groups; p.C = a->C;
    p.center = a->flags & GROUP_NORM_FLAG_CENTER; p.shared = a->flags & GROUP_NORM_FLAG_SHARED;
    p.w_bf16 = a->w_dtype == KDA_BF16;
    p.x = a->x; p.gate = a->gate; p.weight = a->weight; p.bias = a->bias;
    const long long cols = (long long)a->groups * a->C;
    p.ld_x = stride_or(a->ld_x, cols); p.ld_gate = stride_or(a->ld_gate, cols);
    return KDA_OK;
}

kda_status group_fwd(const group_norm_fwd_args *a, mixer::GroupNormParams &p) {
    if (!a || !a->y || !(a->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    const kda_status st = group_common(a, p);
    if (st != KDA_OK) return st;
    const long long cols = (long long)a->groups * a->C, wc = p.shared ? a->C : cols, stats = a->rows * a->groups;
    if (a->mean && !p.center) return KDA_ERR_INVALID_ARG;
    p.eps = a->eps; p.y = a->y; p.mean = a->mean; p.rstd = a->rstd;
    p.ld_y = stride_or(a->ld_y, cols);
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    const Block in[] = {{a->x, a->rows, cols, p.ld_x, es}, {a->gate, a->rows, cols, p.ld_gate, es}, dense(a->weight, 1, wc, ws),
                        dense(a->bias, 1, wc, ws)};
    const Block out[] = {{a->y, a->rows, cols, p.ld_y, es}, dense(a->mean, 1, stats, 4), dense(a->rstd, 1, stats, 4)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

kda_status group_bwd(const group_norm_bwd_args *a, mixer::GroupNormParams &p, size_t &need) {
    if (!a || !a->dy || !a->dx || !a->rstd) return KDA_ERR_INVALID_ARG;
    const kda_status st = group_common(a, p);
    if (st != KDA_OK) return st;
    if ((a->gate == nullptr) != (a->dgate == nullptr) || p.center != (a->mean != nullptr)) return KDA_ERR_INVALID_ARG;
    const long long cols = (long long)a->groups * a->C, wc = p.shared ? a->C : cols, stats = a->rows * a->groups;
    p.dy = a->dy; p.y = a->dx; p.dgate = a->dgate;
    p.mean = const_cast<float *>(a->mean); p.rstd = const_cast<float *>(a->rstd);
    p.dweight = a->dweight; p.dbias = a->dbias;
    p.ld_dy = stride_or(a->ld_dy, cols); p.ld_y = stride_or(a->ld_dx, cols); p.ld_dgate = stride_or(a->ld_dgate, cols);
    need = a->dweight || a->dbias ? mixer::group_norm_part_floats(p, a->dtype == KDA_BF16) * 4 : 0;
    const size_t es = es_of(a->dtype), ws = es_of(a->w_dtype);
    const Block in[] = {{a->x, a->rows, cols, p.ld_x, es}, {a->gate, a->rows, cols, p.ld_gate, es},
                        {a->dy, a->rows, cols, p.ld_dy, es}, dense(a->weight, 1, wc, ws), dense(a->bias, 1, wc, ws),
                        dense(a->mean, 1, stats, 4), dense(a->rstd, 1, stats, 4)};
    const Block out[] = {{a->dx, a->rows, cols, p.ld_y, es}, {a->dgate, a->rows, cols, p.ld_dgate, es},
                         dense(a->dweight, 1, wc, ws), dense(a->dbias, 1, wc, ws),
                         dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------------------ gated feed-forward product
template <class A> kda_status glu_common(const A *a, mixer::GluParams &p) {
    if (a->rows < 1 || a->rows > 0x7fffffffLL || a->D < 1 || a->F < 1 || (long long)a->D * a->F > (1LL << 40) ||
        a->rows * a->F > (1LL << 40) || a->rows * a->D > (1LL << 40))
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || (a->flags & ~GLU_FLAG_GELU) || !a->x || !a->w_gate || !a->w_up) return KDA_ERR_INVALID_ARG;
    if ((a->g == nullptr) != (a->u == nullptr)) return KDA_ERR_INVALID_ARG;
    p.M = a->rows; p.D = a->D; p.F = a->F; p.gelu = a->flags & GLU_FLAG_GELU;
    p.x = a->x; p.wg = a->w_gate; p.wu = a->w_up;
    p.ld_x = stride_or(a->ld_x, a->D); p.ld_wg = stride_or(a->ld_w_gate, a->D); p.ld_wu = stride_or(a->ld_w_up, a->D);
    if (!mixer::aligned_to(a->status, 16)) return KDA_ERR_INVALID_ARG;
    p.status = static_cast<int *>(a->status);
    return KDA_OK;
}

kda_status glu_fwd_params(const glu_fwd_args *a, mixer::GluParams &p, size_t &need) {
    if (!a || !a->h) return KDA_ERR_INVALID_ARG;
    const kda_status st = glu_common(a, p);
    if (st != KDA_OK) return st;
    p.h = a->h; p.ld_h = stride_or(a->ld_h, a->F); p.g = a->g; p.u = a->u;
    need = mixer::glu_moved_bytes(p, a->dtype == KDA_BF16);
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, a->rows, a->D, p.ld_x, es}, {a->w_gate, a->F, a->D, p.ld_wg, es}, {a->w_up, a->F, a->D, p.ld_wu, es}};
    const Block out[] = {{a->h, a->rows, a->F, p.ld_h, es}, dense(a->g, a->rows, a->F, 4), dense(a->u, a->rows, a->F, 4),
                         dense(a->status, 1, 256, 1), dense(need ? a->workspace : nullptr, 1, (long long)a->workspace_bytes, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// need: the two products' gradients, then operands that move, then sums of parts of a product.
kda_status glu_bwd_params(const glu_bwd_args *a, mixer::GluParams &p, size_t &need, size_t &grads, size_t &moved) {
    if (!a || !a->dh || !a->dx || !a->dw_gate || !a->dw_up) return KDA_ERR_INVALID_ARG;
    const kda_status st = glu_common(a, p);
    if (st != KDA_OK) return st;
    p.dh = a->dh; p.dx = a->dx; p.dwg = a->dw_gate; p.dwu = a->dw_up;
    p.g = const_cast<float *>(a->g); p.u = const_cast<float *>(a->u);
    p.ld_dh = stride_or(a->ld_dh, a->F); p.ld_dx = stride_or(a->ld_dx, a->D);
    p.ld_dwg = stride_or(a->ld_dw_gate, a->D); p.ld_dwu = stride_or(a->ld_dw_up, a->D);
    const size_t es = es_of(a->dtype);
    p.ld_d = mixer::glu_grad_stride(p, a->dtype == KDA_BF16);
    grads = (2 * (size_t)a->rows * p.ld_d * es + 255) / 256 * 256;
    moved = mixer::glu_moved_bytes(p, a->dtype == KDA_BF16);
    need = grads + moved + (a->dtype == KDA_BF16 ? mixer::glu_tc_part_bytes(p) : 0);
    const Block in[] = {{a->x, a->rows, a->D, p.ld_x, es}, {a->w_gate, a->F, a->D, p.ld_wg, es}, {a->w_up, a->F, a->D, p.ld_wu, es},
                        {a->dh, a->rows, a->F, p.ld_dh, es}, dense(a->g, a->rows, a->F, 4), dense(a->u, a->rows, a->F, 4)};
    const Block out[] = {{a->dx, a->rows, a->D, p.ld_dx, es}, {a->dw_gate, a->F, a->D, p.ld_dwg, es},
                         {a->dw_up, a->F, a->D, p.ld_dwu, es}, dense(a->workspace, 1, (long long)a->workspace_bytes, 1),
                         dense(a->status, 1, 256, 1)};
    return blocks_ok(in, out) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

size_t gated_scan_fwd_workspace(const gated_scan_fwd_args *a) {
    mixer::GatedScanParams p{};
    size_t need = 0;
    return gated_fwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status gated_scan_fwd(const gated_scan_fwd_args *a, kda_stream_t stream) {
    mixer::GatedScanParams p{};
    size_t need = 0;
    kda_status st = gated_fwd(a, p, need);
    if (st != KDA_OK) return st;
    if (need) {
        if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
        p.ws = static_cast<float *>(a->workspace);
    }
    return from(mixer::launch_gated_scan_fwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t gated_scan_bwd_workspace(const gated_scan_bwd_args *a) {
    mixer::GatedScanParams p{};
    size_t need = 0, states = 0;
    return gated_bwd(a, p, need, states) == KDA_OK ? need : 0;
}

kda_status gated_scan_bwd(const gated_scan_bwd_args *a, kda_stream_t stream) {
    mixer::GatedScanParams p{};
    size_t need = 0, states = 0;
    kda_status st = gated_bwd(a, p, need, states);
    if (st != KDA_OK) return st;
    if (need && (st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
    char *ws = static_cast<char *>(a->workspace);
    const bool bf16 = a->dtype == KDA_BF16;
    p.ws = reinterpret_cast<float *>(ws + states);
    if (states) {                        // the forward's walk again, for the states alone
        p.states = reinterpret_cast<float *>(ws);
        const cudaError_t e = mixer::launch_gated_scan_fwd(p, bf16, stream_of(stream));
        if (e != cudaSuccess) return from(e);
    }
    return from(mixer::launch_gated_scan_bwd(p, bf16, stream_of(stream)));
}

kda_status gated_scan_step(const gated_scan_step_args *a, kda_stream_t stream) {
    if (!a || !sizes_ok(a->B, 1, a->D) || a->slots < 1 || !a->state || !a->y) return KDA_ERR_INVALID_ARG;
    if (!a->slot && a->slots < a->B) return KDA_ERR_INVALID_ARG;
    const kda_status st = gated_common(a);
    if (st != KDA_OK) return st;
    mixer::GatedScanParams p{};
    gated_fill(a, p);
    p.T = 1; p.slots = a->slots; p.state = a->state; p.slot = a->slot; p.y = a->y;
    p.ld_y = stride_or(a->ld_y, a->D);
    const size_t es = es_of(a->dtype);
    const Block in[] = {{a->x, a->B, a->D, p.ld_x, es}, {a->decay, a->B, a->D, p.ld_decay, es}, {a->gate, a->B, a->D, p.ld_gate, es},
                        dense(a->rate, 1, a->D, 4), dense(a->slot, 1, a->B, 4)};
    const Block out[] = {{a->y, a->B, a->D, p.ld_y, es}, dense(a->state, a->slots, a->D, 4)};
    if (!blocks_ok(in, out)) return KDA_ERR_INVALID_ARG;
    return from(mixer::launch_gated_scan_step(p, a->dtype == KDA_BF16, stream_of(stream)));
}

kda_status group_norm_fwd(const group_norm_fwd_args *a, kda_stream_t stream) {
    mixer::GroupNormParams p{};
    const kda_status st = group_fwd(a, p);
    return st != KDA_OK ? st : from(mixer::launch_group_norm_fwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t group_norm_bwd_workspace(const group_norm_bwd_args *a) {
    mixer::GroupNormParams p{};
    size_t need = 0;
    return group_bwd(a, p, need) == KDA_OK ? need : 0;
}

kda_status group_norm_bwd(const group_norm_bwd_args *a, kda_stream_t stream) {
    mixer::GroupNormParams p{};
    size_t need = 0;
    kda_status st = group_bwd(a, p, need);
    if (st != KDA_OK) return st;
    if (need) {
        if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
        p.part = static_cast<float *>(a->workspace);
    }
    return from(mixer::launch_group_norm_bwd(p, a->dtype == KDA_BF16, stream_of(stream)));
}

size_t glu_fwd_workspace(const glu_fwd_args *a) {
    mixer::GluParams p{};
    size_t need = 0;
    return glu_fwd_params(a, p, need) == KDA_OK ? need : 0;
}

kda_status glu_fwd(const glu_fwd_args *a, kda_stream_t stream) {
    mixer::GluParams p{};
    size_t need = 0;
    kda_status st = glu_fwd_params(a, p, need);
    if (st != KDA_OK) return st;
    if (need && (st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
    return from(mixer::launch_glu_fwd(p, a->dtype == KDA_BF16, static_cast<char *>(a->workspace), stream_of(stream)));
}

size_t glu_bwd_workspace(const glu_bwd_args *a) {
    mixer::GluParams p{};
    size_t need = 0, grads = 0, moved = 0;
    return glu_bwd_params(a, p, need, grads, moved) == KDA_OK ? need : 0;
}

kda_status glu_bwd(const glu_bwd_args *a, kda_stream_t stream) {
    mixer::GluParams p{};
    size_t need = 0, grads = 0, moved = 0;
    kda_status st = glu_bwd_params(a, p, need, grads, moved);
    if (st != KDA_OK) return st;
    if ((st = check_space(a->workspace, a->workspace_bytes, need)) != KDA_OK) return st;
    char *ws = static_cast<char *>(a->workspace);
    p.dg = ws;
    p.du = ws + (size_t)a->rows * p.ld_d * es_of(a->dtype);
    p.part = ws + grads + moved;
    return from(mixer::launch_glu_bwd(p, a->dtype == KDA_BF16, ws + grads, stream_of(stream)));
}

}  // extern "C"
