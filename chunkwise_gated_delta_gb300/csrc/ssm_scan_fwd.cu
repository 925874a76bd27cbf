// Selective state-space scan: forward and single tokens.
//
//   dt = softplus(delta + bias), h = exp(dt A) h + dt x B, y = (C . h + D x) SiLU(z)
//
// Per (token, channel, state): one exponential and four multiply-adds; per (token, channel) four
// elements of HBM traffic.  With N = 16 the exponentials (32 per clock and SM) take 1.4 times
// as long as the traffic, so the kernel is bound by the special-function and FMA pipes, and the
// states stay in registers from the first token to the last.
#include "ssm_scan.cuh"

namespace mixer {
namespace {

constexpr int TT = 32;               // tokens per staged tile

template <class T, int L>
__global__ void __launch_bounds__(kScanThreads) scan_fwd_kernel(ScanParams p, int chan_blocks, bool vec) {
    constexpr int NP = 4 * L, CW = 32 / L, K = TT / L;
    __shared__ float sB[TT][NP], sC[TT][NP];
    __shared__ float2 sd[4][TT][CW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane / L, i = lane % L;
    const long long slot = blockIdx.x / chan_blocks;
    const int d = (int)(blockIdx.x - slot * chan_blocks) * (4 * CW) + warp * CW + c;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    const bool live = d < p.D;
    const int n0 = 4 * i;
    float a2[4], h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        a2[k] = 0.f;
        h[k] = 0.f;
    }
    float skip = 0.f, dbias = 0.f;
    if (live) {
        load_states(a2, p.A + (long long)d * p.N, n0, p.N);
        if (p.seg_state) load_states(h, p.seg_state + (slot * p.D + d) * NP, n0, NP);
        else if (p.h0) load_states(h, p.h0 + ((long long)g.b * p.D + d) * p.N, n0, p.N);
        if (p.Dskip) skip = p.Dskip[d];
        if (p.delta_bias) dbias = p.delta_bias[d];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) a2[k] *= kLog2e;
    const T *x = static_cast<const T *>(p.x), *delta = static_cast<const T *>(p.delta), *z = static_cast<const T *>(p.z);
    T *y = static_cast<T *>(p.y);
    for (int t0 = 0; t0 < g.len; t0 += TT) {
        __syncthreads();
        stage_rows<T, NP, TT>(sB, p.Bm, p.ld_B, p.N, g, t0, vec);
        stage_rows<T, NP, TT>(sC, p.Cm, p.ld_C, p.N, g, t0, vec);
        float xs[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {           // lane i looks after tokens j L + i
            const int t = t0 + j * L + i;
            float dt = 0.f;
            xs[j] = 0.f;
            if (live && t < g.len) {
                const long long r = g.row0 + g.t0 + t;
                xs[j] = to_f(x[r * p.ld_x + d]);
                dt = to_f(delta[r * p.ld_delta + d]) + dbias;
                if (p.softplus) dt = softplus(dt);
            }
            sd[warp][j * L + i][c] = make_float2(dt, dt * xs[j]);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float ys[L];
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const int t = j * L + k;
                const float2 v = sd[warp][t][c];
                const float4 b = *reinterpret_cast<const float4 *>(&sB[t][n0]);
                const float4 q = *reinterpret_cast<const float4 *>(&sC[t][n0]);
                h[0] = fmaf(ex2(v.x * a2[0]), h[0], v.y * b.x);
                h[1] = fmaf(ex2(v.x * a2[1]), h[1], v.y * b.y);
                h[2] = fmaf(ex2(v.x * a2[2]), h[2], v.y * b.z);
                h[3] = fmaf(ex2(v.x * a2[3]), h[3], v.y * b.w);
                ys[k] = fmaf(h[0], q.x, h[1] * q.y) + fmaf(h[2], q.z, h[3] * q.w);
            }
            spread_sum<L, L>(ys, i);
            const int t = t0 + j * L + i;
            if (live && t < g.len) {
                const long long r = g.row0 + g.t0 + t;
                float o = fmaf(skip, xs[j], ys[0]);
                if (z) {
                    const float zv = to_f(z[r * p.ld_z + d]);
                    o *= zv * sigmoid(zv);
                }
                y[r * p.ld_y + d] = from_f<T>(o);
            }
        }
    }
    if (p.ht && live && g.i == g.n - 1) store_states(p.ht + ((long long)g.b * p.D + d) * p.N, h, n0, p.N);
}

// The same for one token of each request; the state is read, updated and written once: bound by HBM.
template <class T, int L>
__global__ void __launch_bounds__(kScanThreads) scan_step_kernel(ScanParams p, int chan_blocks) {
    constexpr int CH = kScanThreads / L;
    const int c = threadIdx.x / L, i = threadIdx.x % L, n0 = 4 * i;
    const int b = blockIdx.x / chan_blocks;
    const int d = (blockIdx.x - b * chan_blocks) * CH + c;
    const int slot = p.slot ? p.slot[b] : b;
    const bool pad = slot < 0 || slot >= p.slots, live = d < p.D && !pad;
    float y[1] = {0.f};
    float xv = 0.f;
    if (live) {
        float h[4], a[4], bv[4], cv[4];
        float *st = p.state + ((long long)slot * p.D + d) * p.N;
        load_states(h, st, n0, p.N);
        load_states(a, p.A + (long long)d * p.N, n0, p.N);
        const T *br = static_cast<const T *>(p.Bm) + b * p.ld_B, *cr = static_cast<const T *>(p.Cm) + b * p.ld_C;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bv[k] = n0 + k < p.N ? to_f(br[n0 + k]) : 0.f;
            cv[k] = n0 + k < p.N ? to_f(cr[n0 + k]) : 0.f;
        }
        xv = to_f(static_cast<const T *>(p.x)[b * p.ld_x + d]);
        float dt = to_f(static_cast<const T *>(p.delta)[b * p.ld_delta + d]) + (p.delta_bias ? p.delta_bias[d] : 0.f);
        if (p.softplus) dt = softplus(dt);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = fmaf(ex2(dt * a[k] * kLog2e), h[k], dt * xv * bv[k]);
            y[0] = fmaf(cv[k], h[k], y[0]);
        }
        store_states(st, h, n0, p.N);
    }
#pragma unroll
    for (int s = L / 2; s; s >>= 1) y[0] += __shfl_xor_sync(~0u, y[0], s);
    if (d < p.D && i == 0) {
        float o = 0.f;
        if (!pad) {
            o = fmaf(p.Dskip ? p.Dskip[d] : 0.f, xv, y[0]);
            if (p.z) {
                const float zv = to_f(static_cast<const T *>(p.z)[b * p.ld_z + d]);
                o *= zv * sigmoid(zv);
            }
        }
        static_cast<T *>(p.y)[b * p.ld_y + d] = from_f<T>(o);
    }
}

template <class T, int L> cudaError_t fwd_launch(const ScanParams &p, cudaStream_t s) {
    constexpr int CH = 4 * (32 / L);
    const int cb = (p.D + CH - 1) / CH;
    const long long blocks = scan_slots(p, p.seg) * cb;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    scan_fwd_kernel<T, L><<<(unsigned)blocks, kScanThreads, 0, s>>>(p, cb, bc_vec_ok<T>(p, 4 * L));
    return cudaGetLastError();
}

template <class T, int L> cudaError_t step_launch(const ScanParams &p, cudaStream_t s) {
    constexpr int CH = kScanThreads / L;
    const int cb = (p.D + CH - 1) / CH;
    if ((long long)p.B * cb > 0x7fffffffLL) return cudaErrorNotSupported;
    scan_step_kernel<T, L><<<(unsigned)(p.B * cb), kScanThreads, 0, s>>>(p, cb);
    return cudaGetLastError();
}

template <class T> cudaError_t fwd_type(const ScanParams &p, cudaStream_t s) {
    switch (lanes_for(p.N)) {
    case 1: return fwd_launch<T, 1>(p, s);
    case 2: return fwd_launch<T, 2>(p, s);
    case 4: return fwd_launch<T, 4>(p, s);
    default: return fwd_launch<T, 8>(p, s);
    }
}
template <class T> cudaError_t step_type(const ScanParams &p, cudaStream_t s) {
    switch (lanes_for(p.N)) {
    case 1: return step_launch<T, 1>(p, s);
    case 2: return step_launch<T, 2>(p, s);
    case 4: return step_launch<T, 4>(p, s);
    default: return step_launch<T, 8>(p, s);
    }
}

}  // namespace

int ssm_scan_fwd_segment(const ScanParams &p) { return p.T; }

size_t ssm_scan_fwd_floats(const ScanParams &p) {
    const int seg = ssm_scan_fwd_segment(p);
    if (seg >= p.T) return 0;
    return (size_t)scan_slots(p, seg) * p.D * (4 * lanes_for(p.N) + 1);
}

void ssm_scan_fwd_carve(ScanParams &p, float *ws) {
    const size_t slots = (size_t)scan_slots(p, p.seg);
    p.seg_state = ws;
    p.seg_dt = ws + slots * p.D * 4 * lanes_for(p.N);
}

cudaError_t launch_ssm_scan_fwd(const ScanParams &p, bool bf, cudaStream_t s) {
    if (p.seg_state) {
        const cudaError_t e = launch_scan_segments(p, bf, false, s);
        if (e != cudaSuccess) return e;
    }
    return bf ? fwd_type<bf16>(p, s) : fwd_type<float>(p, s);
}

cudaError_t launch_ssm_scan_step(const ScanParams &p, bool bf, cudaStream_t s) {
    return bf ? step_type<bf16>(p, s) : step_type<float>(p, s);
}

}  // namespace mixer
