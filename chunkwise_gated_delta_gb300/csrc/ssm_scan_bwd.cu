// Selective state-space scan: backward, in segments of 64 tokens that run side by side.
//
// With g_t = dy_t SiLU(z_t) and G_t the gradient of h_t:
//     G_t = C_t g_t + a_{t+1} G_{t+1},  a_t = exp(dt_t A)
//     dC_t = sum_d g_t h_t,  dB_t = sum_d G_t dt_t x_t,  u_t = sum_n G_t B_t
//     q_t = G_t a_t h_{t-1},  dA = sum_t q_t dt_t,  ddt_t = sum_n q_t A + u_t x_t
//
//  1. local pass     per segment, one forward sweep: the state it ends with from zero, the
//                    gradient of its entry state E = sum_t (a_1 ... a_t) C_t g_t, its sum of dt
//  2. boundary pass  per channel and state, over the segments: entry states forwards, exit
//                    gradients backwards (exp(A sum dt) carries both across a segment)
//  3. gradient pass  per segment and block of channels: a sweep that leaves the state before every
//                    8 tokens in shared memory, then the 8-token parts backwards, each
//                    recomputed into registers
//  4. sums           dB and dC over the channel blocks, dA, dD and dbias over the segments
//
// The gradient pass walks several groups of channels per 8-token part, so the sums of dB and dC
// over channels gather in registers and cross lanes once per part.
#include "ssm_scan.cuh"

namespace mixer {
namespace {

constexpr int SEG = kBwdSegment;

template <class T, int L, bool GRAD>
__global__ void __launch_bounds__(kScanThreads) scan_local_kernel(ScanParams p, int chan_blocks, bool vec) {
    constexpr int NP = 4 * L, CW = 32 / L, TT = L == 1 ? 16 : 32, K = TT / L;
    __shared__ float sB[TT][NP], sC[GRAD ? TT : 1][NP];
    __shared__ float4 sd[4][TT][CW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane / L, i = lane % L, n0 = 4 * i;
    const long long slot = blockIdx.x / chan_blocks;
    const int d = (int)(blockIdx.x - slot * chan_blocks) * (4 * CW) + warp * CW + c;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    const bool live = d < p.D;
    float a2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
    float m[4] = {1.f, 1.f, 1.f, 1.f};      // a_1 ... a_t
    float dbias = 0.f, sum = 0.f;
    if (live) {
        load_states(a2, p.A + (long long)d * p.N, n0, p.N);
        if (p.delta_bias) dbias = p.delta_bias[d];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) a2[k] *= kLog2e;
    const T *x = static_cast<const T *>(p.x), *delta = static_cast<const T *>(p.delta);
    const T *z = static_cast<const T *>(p.z), *dy = static_cast<const T *>(p.dy);
    for (int t0 = 0; t0 < g.len; t0 += TT) {
        __syncthreads();
        stage_rows<T, NP, TT>(sB, p.Bm, p.ld_B, p.N, g, t0, vec);
        if (GRAD) stage_rows<T, NP, TT>(reinterpret_cast<float(*)[NP]>(sC), p.Cm, p.ld_C, p.N, g, t0, vec);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int t = t0 + j * L + i;
            float dt = 0.f, xv = 0.f, gy = 0.f;
            if (live && t < g.len) {
                const long long r = g.row0 + g.t0 + t;
                xv = to_f(x[r * p.ld_x + d]);
                dt = to_f(delta[r * p.ld_delta + d]) + dbias;
                if (p.softplus) dt = softplus(dt);
                if (GRAD) {
                    gy = to_f(dy[r * p.ld_dy + d]);
                    if (z) {
                        const float zv = to_f(z[r * p.ld_z + d]);
                        gy *= zv * sigmoid(zv);
                    }
                }
            }
            sum += dt;
            sd[warp][j * L + i][c] = make_float4(dt, dt * xv, gy, 0.f);
        }
        __syncthreads();
#pragma unroll 8
        for (int t = 0; t < TT; ++t) {
            const float4 v = sd[warp][t][c];
            const float4 b = *reinterpret_cast<const float4 *>(&sB[t][n0]);
            float a[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = ex2(v.x * a2[k]);
            h[0] = fmaf(a[0], h[0], v.y * b.x);
            h[1] = fmaf(a[1], h[1], v.y * b.y);
            h[2] = fmaf(a[2], h[2], v.y * b.z);
            h[3] = fmaf(a[3], h[3], v.y * b.w);
            if (GRAD) {
                const float4 q = *reinterpret_cast<const float4 *>(&sC[t][n0]);
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] *= a[k];
                e[0] = fmaf(m[0], v.z * q.x, e[0]);
                e[1] = fmaf(m[1], v.z * q.y, e[1]);
                e[2] = fmaf(m[2], v.z * q.z, e[2]);
                e[3] = fmaf(m[3], v.z * q.w, e[3]);
            }
        }
    }
#pragma unroll
    for (int s = L / 2; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
    if (!live) return;
    const long long at = slot * p.D + d;
    *reinterpret_cast<float4 *>(p.seg_state + at * NP + n0) = make_float4(h[0], h[1], h[2], h[3]);
    if (GRAD) *reinterpret_cast<float4 *>(p.seg_grad + at * NP + n0) = make_float4(e[0], e[1], e[2], e[3]);
    if (i == 0) p.seg_dt[at] = sum;
}

// One thread per (sequence, channel, state).
template <bool GRAD> __global__ void __launch_bounds__(128) scan_boundary_kernel(ScanParams p, int NP) {
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long per = (long long)p.D * NP;
    const int b = (int)(u / per);
    if (b >= p.B) return;
    const int d = (int)((u - b * per) / NP), n = (int)(u % NP);
    long long s0;
    int count;
    if (!p.cu_seqlens) {
        count = (int)((p.T + (long long)p.seg - 1) / p.seg);
        s0 = (long long)b * count;
    } else {
        const int lo = clamped(p.cu_seqlens[b], 0, p.T), hi = clamped(p.cu_seqlens[b + 1], lo, p.T);
        count = hi > lo ? (int)((hi - lo + (long long)p.seg - 1) / p.seg) : 1;
        s0 = b + lo / p.seg;
    }
    const bool in = n < p.N;
    const float a2 = in ? p.A[(long long)d * p.N + n] * kLog2e : 0.f;
    const long long at = ((long long)b * p.D + d) * p.N + n;
    float h = in && p.h0 ? p.h0[at] : 0.f;
    for (int i = 0; i < count; ++i) {
        const long long k = (s0 + i) * p.D + d;
        const float local = p.seg_state[k * NP + n], a = ex2(a2 * p.seg_dt[k]);
        p.seg_state[k * NP + n] = h;
        h = fmaf(a, h, local);
    }
    if (!GRAD) return;
    float e = in && p.dht ? p.dht[at] : 0.f;
    for (int i = count - 1; i >= 0; --i) {
        const long long k = (s0 + i) * p.D + d;
        const float local = p.seg_grad[k * NP + n], a = ex2(a2 * p.seg_dt[k]);
        p.seg_grad[k * NP + n] = e;
        e = fmaf(a, e, local);
    }
    if (in && p.dh0) p.dh0[at] = e;
}

constexpr int TC = 8;                // tokens per part, recomputed into registers
constexpr int GROUPS = 4;            // channel groups that a block walks per part
constexpr int PARTS = SEG / TC;

// Per-thread values in shared memory, one set per channel group.
struct GradShared {
    float4 entry[GROUPS][PARTS][kScanThreads];   // states before each part
    float4 carry[GROUPS][kScanThreads];          // gradient of the state after the part at hand
    float4 dA[GROUPS][kScanThreads];
    float2 par[GROUPS][kScanThreads];            // dD, dbias
};

template <class T, int L> struct GradTiles {
    float B[SEG][4 * L], C[SEG][4 * L];
    float4 d[4][TC][32 / L];
    float red[4][TC * 2 * 4 * L];
};

template <class T, int L>
__global__ void __launch_bounds__(kScanThreads) scan_grad_kernel(ScanParams p, int chan_blocks, bool vec) {
    constexpr int NP = 4 * L, CW = 32 / L, CH = 4 * CW, TL = TC / L;
    extern __shared__ __align__(16) unsigned char raw[];
    GradShared &S = *reinterpret_cast<GradShared *>(raw);
    GradTiles<T, L> &W = *reinterpret_cast<GradTiles<T, L> *>(raw + sizeof(GradShared));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane / L, i = lane % L, n0 = 4 * i;
    const long long slot = blockIdx.x / chan_blocks;
    const int cb = (int)(blockIdx.x - slot * chan_blocks);
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    const T *x = static_cast<const T *>(p.x), *delta = static_cast<const T *>(p.delta);
    const T *z = static_cast<const T *>(p.z), *dy = static_cast<const T *>(p.dy);
    const long long row = g.row0 + g.t0;
    stage_rows<T, NP, SEG>(W.B, p.Bm, p.ld_B, p.N, g, 0, vec);
    stage_rows<T, NP, SEG>(W.C, p.Cm, p.ld_C, p.N, g, 0, vec);
    __syncthreads();
    const int parts = (g.len + TC - 1) / TC;
    // forward sweep: the state before every part
    for (int k = 0; k < GROUPS; ++k) {
        const int d = (cb * GROUPS + k) * CH + warp * CW + c;
        const bool live = d < p.D;
        float a2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
        float dbias = 0.f;
        if (live) {
            load_states(a2, p.A + (long long)d * p.N, n0, p.N);
            load_states(h, p.seg_state + (slot * p.D + d) * NP, n0, NP);
            load_states(e, p.seg_grad + (slot * p.D + d) * NP, n0, NP);
            if (p.delta_bias) dbias = p.delta_bias[d];
        }
        S.carry[k][tid] = make_float4(e[0], e[1], e[2], e[3]);
        S.dA[k][tid] = make_float4(0.f, 0.f, 0.f, 0.f);
        S.par[k][tid] = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) a2[q] *= kLog2e;
        for (int part = 0; part < parts; ++part) {
            S.entry[k][part][tid] = make_float4(h[0], h[1], h[2], h[3]);
            if (part == parts - 1) break;          // its tokens are swept below
            __syncwarp();
#pragma unroll
            for (int j = 0; j < TL; ++j) {
                const int t = part * TC + i * TL + j;
                float dt = 0.f, xv = 0.f;
                if (live && t < g.len) {
                    xv = to_f(x[(row + t) * p.ld_x + d]);
                    dt = to_f(delta[(row + t) * p.ld_delta + d]) + dbias;
                    if (p.softplus) dt = softplus(dt);
                }
                W.d[warp][i * TL + j][c] = make_float4(dt, dt * xv, 0.f, 0.f);
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                const float4 v = W.d[warp][t][c];
                const float4 b = *reinterpret_cast<const float4 *>(&W.B[part * TC + t][n0]);
                h[0] = fmaf(ex2(v.x * a2[0]), h[0], v.y * b.x);
                h[1] = fmaf(ex2(v.x * a2[1]), h[1], v.y * b.y);
                h[2] = fmaf(ex2(v.x * a2[2]), h[2], v.y * b.z);
                h[3] = fmaf(ex2(v.x * a2[3]), h[3], v.y * b.w);
            }
        }
    }
    // the parts, last to first
    for (int part = parts - 1; part >= 0; --part) {
        float acc[2][TC][4];         // dB, dC of this lane's states, over the channel groups
#pragma unroll
        for (int t = 0; t < TC; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[0][t][q] = acc[1][t][q] = 0.f;
        for (int k = 0; k < GROUPS; ++k) {
            const int d = (cb * GROUPS + k) * CH + warp * CW + c;
            const bool live = d < p.D;
            float a2[4] = {0.f, 0.f, 0.f, 0.f};
            float dbias = 0.f, skip = 0.f;
            if (live) {
                load_states(a2, p.A + (long long)d * p.N, n0, p.N);
                if (p.delta_bias) dbias = p.delta_bias[d];
                if (p.Dskip) skip = p.Dskip[d];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) a2[q] *= kLog2e;
            float dts[TL], xs[TL], zs[TL], dys[TL], sg[TL], gys[TL];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < TL; ++j) {
                const int t = part * TC + i * TL + j;
                dts[j] = xs[j] = zs[j] = dys[j] = sg[j] = gys[j] = 0.f;
                if (live && t < g.len) {
                    xs[j] = to_f(x[(row + t) * p.ld_x + d]);
                    dts[j] = to_f(delta[(row + t) * p.ld_delta + d]) + dbias;
                    sg[j] = 1.f;
                    if (p.softplus) {
                        sg[j] = sigmoid(dts[j]);
                        dts[j] = softplus(dts[j]);
                    }
                    gys[j] = dys[j] = to_f(dy[(row + t) * p.ld_dy + d]);
                    if (z) {
                        zs[j] = to_f(z[(row + t) * p.ld_z + d]);
                        gys[j] *= zs[j] * sigmoid(zs[j]);
                    }
                }
                W.d[warp][i * TL + j][c] = make_float4(dts[j], dts[j] * xs[j], gys[j], 0.f);
            }
            __syncwarp();
            float h[TC + 1][4], a[TC][4], ys[TC], us[TC], qs[TC];
            {
                const float4 v = S.entry[k][part][tid];
                h[0][0] = v.x; h[0][1] = v.y; h[0][2] = v.z; h[0][3] = v.w;
            }
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                const float4 v = W.d[warp][t][c];
                const float4 b = *reinterpret_cast<const float4 *>(&W.B[part * TC + t][n0]);
                const float4 q = *reinterpret_cast<const float4 *>(&W.C[part * TC + t][n0]);
#pragma unroll
                for (int s = 0; s < 4; ++s) a[t][s] = ex2(v.x * a2[s]);
                h[t + 1][0] = fmaf(a[t][0], h[t][0], v.y * b.x);
                h[t + 1][1] = fmaf(a[t][1], h[t][1], v.y * b.y);
                h[t + 1][2] = fmaf(a[t][2], h[t][2], v.y * b.z);
                h[t + 1][3] = fmaf(a[t][3], h[t][3], v.y * b.w);
                ys[t] = fmaf(h[t + 1][0], q.x, h[t + 1][1] * q.y) + fmaf(h[t + 1][2], q.z, h[t + 1][3] * q.w);
            }
            float G[4], dA[4];
            {
                const float4 v = S.carry[k][tid], w = S.dA[k][tid];
                G[0] = v.x; G[1] = v.y; G[2] = v.z; G[3] = v.w;
                dA[0] = w.x; dA[1] = w.y; dA[2] = w.z; dA[3] = w.w;
            }
#pragma unroll
            for (int t = TC - 1; t >= 0; --t) {
                const float4 v = W.d[warp][t][c];
                const float4 b4 = *reinterpret_cast<const float4 *>(&W.B[part * TC + t][n0]);
                const float4 c4 = *reinterpret_cast<const float4 *>(&W.C[part * TC + t][n0]);
                const float b[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                us[t] = qs[t] = 0.f;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    G[s] = fmaf(cc[s], v.z, G[s]);
                    acc[1][t][s] = fmaf(v.z, h[t + 1][s], acc[1][t][s]);
                    acc[0][t][s] = fmaf(G[s], v.y, acc[0][t][s]);
                    us[t] = fmaf(G[s], b[s], us[t]);
                    G[s] *= a[t][s];
                    const float q = G[s] * h[t][s];
                    dA[s] = fmaf(q, v.x, dA[s]);
                    qs[t] = fmaf(q, a2[s], qs[t]);
                }
            }
            S.carry[k][tid] = make_float4(G[0], G[1], G[2], G[3]);
            S.dA[k][tid] = make_float4(dA[0], dA[1], dA[2], dA[3]);
            spread_sum<TC, L>(us, i);
            spread_sum<TC, L>(qs, i);
            if (z) spread_sum<TC, L>(ys, i);
            float2 par = S.par[k][tid];
#pragma unroll
            for (int j = 0; j < TL; ++j) {
                const int t = part * TC + i * TL + j;
                if (live && t < g.len) {
                    const long long r = row + t;
                    const float dd = fmaf(us[j], xs[j], qs[j] * kLn2) * sg[j];
                    static_cast<T *>(p.dx)[r * p.ld_dx + d] = from_f<T>(fmaf(us[j], dts[j], skip * gys[j]));
                    static_cast<T *>(p.ddelta)[r * p.ld_ddelta + d] = from_f<T>(dd);
                    if (z) {
                        const float s = sigmoid(zs[j]);
                        static_cast<T *>(p.dz)[r * p.ld_dz + d] =
                            from_f<T>(dys[j] * fmaf(skip, xs[j], ys[j]) * s * fmaf(zs[j], 1.f - s, 1.f));
                    }
                    par.x = fmaf(gys[j], xs[j], par.x);
                    par.y += dd;
                }
            }
            S.par[k][tid] = par;
        }
        // dB and dC over the warp's channels, then over the four warps
        float v[2 * TC * 4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int t = 0; t < TC; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s) v[(w * TC + t) * 4 + s] = acc[w][t][s];
        int n = 2 * TC * 4, base = 0;
#pragma unroll
        for (int s = 16; s >= L; s >>= 1) {
            n /= 2;
            const bool up = lane & s;
            if (up) base += n;
#pragma unroll
            for (int k = 0; k < 2 * TC * 4; ++k)
                if (k < n) {
                    const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
                    v[k] = keep + __shfl_xor_sync(~0u, send, s);
                }
        }
        constexpr int LEFT = 2 * TC * 4 / CW;
#pragma unroll
        for (int k = 0; k < LEFT; ++k) {
            const int w = (base + k) / (TC * 4), t = (base + k) / 4 % TC, s = (base + k) % 4;
            W.red[warp][(t * 2 + w) * NP + n0 + s] = v[k];
        }
        __syncthreads();
        for (int u = tid; u < TC * 2 * NP; u += kScanThreads) {
            const int t = part * TC + u / (2 * NP);
            if (t < g.len)
                p.part_bc[((long long)cb * ((long long)(p.cu_seqlens ? 1 : p.B) * p.T) + row + t) * (2 * NP) + u % (2 * NP)] =
                    (W.red[0][u] + W.red[1][u]) + (W.red[2][u] + W.red[3][u]);
        }
        __syncthreads();
    }
    for (int k = 0; k < GROUPS; ++k) {
        const int d = (cb * GROUPS + k) * CH + warp * CW + c;
        float2 par = S.par[k][tid];
#pragma unroll
        for (int s = L / 2; s; s >>= 1) {
            par.x += __shfl_xor_sync(~0u, par.x, s);
            par.y += __shfl_xor_sync(~0u, par.y, s);
        }
        if (d >= p.D) continue;
        const float4 w = S.dA[k][tid];
        const float dA[4] = {w.x, w.y, w.z, w.w};
        float *out = p.part_par + slot * ((long long)p.D * (p.N + 2));
        store_states(out + (long long)d * p.N, dA, n0, p.N);
        if (i == 0) {
            out[(long long)p.D * p.N + d] = par.x;
            out[(long long)p.D * (p.N + 1) + d] = par.y;
        }
    }
}

// Sums dB and dC over the channel blocks and rounds them; rows outside every sequence are left alone.
template <class T> __global__ void __launch_bounds__(256) scan_bc_kernel(ScanParams p, int blocks, int NP, long long rows) {
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = u / (2 * NP);
    const int j = (int)(u - row * (2 * NP)), n = j % NP;
    if (row >= rows || n >= p.N) return;
    if (p.cu_seqlens && (row < clamped(p.cu_seqlens[0], 0, p.T) || row >= clamped(p.cu_seqlens[p.B], 0, p.T))) return;
    float s = 0.f;
    for (int k = 0; k < blocks; ++k) s += p.part_bc[(k * rows + row) * (2 * NP) + j];
    if (j < NP) static_cast<T *>(p.dBm)[row * p.ld_dB + n] = from_f<T>(s);
    else static_cast<T *>(p.dCm)[row * p.ld_dC + n] = from_f<T>(s);
}

// Slots that no sequence uses hold no partial sums: cleared, so that the sums may take all rows.
__global__ void __launch_bounds__(256) scan_clear_kernel(ScanParams p, long long per) {
    Segment g;
    if (segment_of(p.cu_seqlens, p.B, p.T, p.seg, blockIdx.x, g) && g.len > 0) return;
    for (long long k = threadIdx.x; k < per; k += 256) p.part_par[blockIdx.x * per + k] = 0.f;
}

template <class T, int L> cudaError_t segments_launch(const ScanParams &p, bool grad, cudaStream_t s) {
    constexpr int CH = 4 * (32 / L), NP = 4 * L;
    const int cb = (p.D + CH - 1) / CH;
    const long long blocks = scan_slots(p, p.seg) * cb;
    const long long bblocks = ((long long)p.B * p.D * NP + 127) / 128;
    if (blocks > 0x7fffffffLL || bblocks > 0x7fffffffLL) return cudaErrorNotSupported;
    const bool vec = bc_vec_ok<T>(p, NP);
    if (grad) scan_local_kernel<T, L, true><<<(unsigned)blocks, kScanThreads, 0, s>>>(p, cb, vec);
    else scan_local_kernel<T, L, false><<<(unsigned)blocks, kScanThreads, 0, s>>>(p, cb, vec);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (grad) scan_boundary_kernel<true><<<(unsigned)bblocks, 128, 0, s>>>(p, NP);
    else scan_boundary_kernel<false><<<(unsigned)bblocks, 128, 0, s>>>(p, NP);
    return cudaGetLastError();
}

template <class T> cudaError_t segments_type(const ScanParams &p, bool grad, cudaStream_t s) {
    switch (lanes_for(p.N)) {
    case 1: return segments_launch<T, 1>(p, grad, s);
    case 2: return segments_launch<T, 2>(p, grad, s);
    case 4: return segments_launch<T, 4>(p, grad, s);
    default: return segments_launch<T, 8>(p, grad, s);
    }
}

int grad_blocks(const ScanParams &p) {
    const int ch = GROUPS * 4 * (32 / lanes_for(p.N));
    return (p.D + ch - 1) / ch;
}

long long batch_rows(const ScanParams &p) { return (long long)(p.cu_seqlens ? 1 : p.B) * p.T; }

template <class T, int L> cudaError_t grad_launch(const ScanParams &p, cudaStream_t s) {
    const int cb = grad_blocks(p);
    const long long slots = scan_slots(p, SEG), blocks = slots * cb, rows = batch_rows(p);
    const long long out = (rows * 8 * L + 255) / 256;
    if (blocks > 0x7fffffffLL || out > 0x7fffffffLL) return cudaErrorNotSupported;
    constexpr int smem = sizeof(GradShared) + sizeof(GradTiles<T, L>);
    cudaError_t e = cudaFuncSetAttribute(scan_grad_kernel<T, L>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    scan_grad_kernel<T, L><<<(unsigned)blocks, kScanThreads, smem, s>>>(p, cb, bc_vec_ok<T>(p, 4 * L));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_bc_kernel<T><<<(unsigned)out, 256, 0, s>>>(p, cb, 4 * L, rows);
    return cudaGetLastError();
}

template <class T> cudaError_t grad_type(const ScanParams &p, cudaStream_t s) {
    switch (lanes_for(p.N)) {
    case 1: return grad_launch<T, 1>(p, s);
    case 2: return grad_launch<T, 2>(p, s);
    case 4: return grad_launch<T, 4>(p, s);
    default: return grad_launch<T, 8>(p, s);
    }
}

}  // namespace

cudaError_t launch_scan_segments(const ScanParams &p, bool bf, bool grad, cudaStream_t s) {
    return bf ? segments_type<bf16>(p, grad, s) : segments_type<float>(p, grad, s);
}

// Workspace: [slots][D][NP] x 2, [slots][D], [slots][D (N + 2)], [channel blocks][rows][2 NP].
// The first two and the last are read and written four floats at a time and lie first.
size_t ssm_scan_bwd_floats(const ScanParams &p) {
    const size_t slots = (size_t)scan_slots(p, SEG), NP = 4 * lanes_for(p.N);
    return slots * p.D * (2 * NP + 1 + p.N + 2) + (size_t)grad_blocks(p) * batch_rows(p) * 2 * NP;
}

void ssm_scan_bwd_carve(ScanParams &p, float *ws) {
    const size_t slots = (size_t)scan_slots(p, SEG), NP = 4 * lanes_for(p.N);
    p.seg_state = ws;
    p.seg_grad = p.seg_state + slots * p.D * NP;
    p.part_bc = p.seg_grad + slots * p.D * NP;
    p.seg_dt = p.part_bc + (size_t)grad_blocks(p) * batch_rows(p) * 2 * NP;
    p.part_par = p.seg_dt + slots * p.D;
}

cudaError_t launch_ssm_scan_bwd(const ScanParams &q, bool bf, cudaStream_t s) {
    ScanParams p = q;
    p.seg = SEG;
    cudaError_t e = launch_scan_segments(p, bf, true, s);
    if (e != cudaSuccess) return e;
    const long long slots = scan_slots(p, SEG), per = (long long)p.D * (p.N + 2);
    if (p.cu_seqlens) {
        scan_clear_kernel<<<(unsigned)slots, 256, 0, s>>>(p, per);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    e = bf ? grad_type<bf16>(p, s) : grad_type<float>(p, s);
    if (e != cudaSuccess) return e;
    return launch_sum_rows(p.part_par, (int)slots, {p.dA, (long long)p.D * p.N, false}, {p.dDskip, p.D, false},
                           {p.ddelta_bias, p.D, false}, s);
}

}  // namespace mixer
