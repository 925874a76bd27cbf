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
// The gradient pass walks two groups of channels per 8-token part, so the sums of dB and dC over
// channels gather in registers and cross lanes once per part.
//
// B 2, T 2048, D 2048, N 16, bfloat16: local pass 56 us, boundary 11, gradients 181, sums 12.  The gradient
// pass is bound by instructions: 26 per (token, channel, state) in half of the issue slots, 8 warps to
// an SM by registers (255) and shared memory (108 KB a block).
#include "ssm_scan.cuh"

namespace mixer {
namespace {

constexpr int SEG = kBwdSegment;

// Four neighbouring channels of one token (XV: in one access), as they lie in memory.  Channels past the
// end repeat the last ones (last: the last offset that exists).
template <class T, bool XV> struct Four {
    typename RawQuad<T>::type v;
    uint32_t e[XV ? 1 : 4];
    __device__ __forceinline__ void load(const T *p, int last) {
        if (XV) {
            v = *reinterpret_cast<const typename RawQuad<T>::type *>(p);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = load_bits(p + min(k, last));
        }
    }
    __device__ __forceinline__ void get(float (&o)[4]) const {
        if (XV) {
            const float4 q = RawQuad<T>::floats(v);
            o[0] = q.x; o[1] = q.y; o[2] = q.z; o[3] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = bits_f<T>(e[k]);
        }
    }
};
template <class T, bool XV> __device__ __forceinline__ void store_four(T *p, const float (&v)[4], int n) {
    if (XV) {
        Vec<T, 4> q;
#pragma unroll
        for (int k = 0; k < 4; ++k) q.e[k] = from_f<T>(v[k]);
        store_vec<T, 4>(p, q);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) p[k] = from_f<T>(v[k]);
    }
}

// Local pass.  A block: 128 / L channels, a lane NS states of one of them.  Per 16 tokens, first dt, dt x
// and g of all channels into shared memory (four channels per access), then the recurrences.  Five
// blocks to an SM (four in float32 and with single elements) cover each other's phases.
template <int L, int NS> struct LocalTiles {
    static constexpr int TT = 16, CH = kScanThreads / L, NP = NS * L;
    f2x2 d[TT][CH];                  // {dt, dt}, {dt x, dt x}; columns swizzled, see at()
    f2 g[TT][CH];
    float bc[128][NP];               // Bm of the segment; in the backward Bm of 64 tokens, then Cm
    float sum[TT][CH / 4][4];        // dt over a thread's tokens
    // Column of channel c: threads that write every fourth channel and threads that read neighbouring
    // ones both meet eight different 16-byte words.
    static __device__ __forceinline__ int at(int c) { return c ^ (c >> 3 & 3); }
};

template <class T, int L, int NS, bool GRAD, bool XV>
__global__ void __launch_bounds__(kScanThreads, XV && sizeof(T) == 2 ? 5 : 4) scan_local_kernel(ScanParams p, int chan_blocks, bool vec) {
    using S = LocalTiles<L, NS>;
    constexpr int TT = S::TT, CH = S::CH, NP = S::NP, H = NS / 2, Q = CH / 4, ROWS = kScanThreads / Q, K = TT / ROWS;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const long long slot = blockIdx.x / chan_blocks;
    const int d0 = (int)(blockIdx.x - slot * chan_blocks) * CH;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.lseg, slot, g)) return;
    const int tid = threadIdx.x, c = tid / L, i = tid % L, n0 = NS * i, d = d0 + c;
    const bool live = d < p.D;
    f2 a2[H], h[H], e[H], m[H];
    {
        float av[NS];
#pragma unroll
        for (int k = 0; k < NS; ++k) av[k] = 0.f;
        if (live) load_states(av, p.A + (long long)d * p.N, n0, p.N);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            a2[k] = pack2(decay_rate(av[2 * k]), decay_rate(av[2 * k + 1]));
            h[k] = e[k] = pack2(0.f, 0.f);
            m[k] = pack2(1.f, 1.f);          // a_1 ... a_t
        }
    }
    // staging: this thread's channels and first token
    const int q = tid % Q, r0 = tid / Q, ds = d0 + 4 * q, dl = XV ? min(ds, p.D - 4) : min(ds, p.D - 1), last = p.D - 1 - dl;
    const long long row = g.row0 + g.t0;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x + dl, *delta = static_cast<const T *>(p.delta) + row * p.ld_delta + dl;
    const T *dy = GRAD ? static_cast<const T *>(p.dy) + row * p.ld_dy + dl : x;
    const T *z = GRAD && p.z ? static_cast<const T *>(p.z) + row * p.ld_z + dl : x;
    const long long ldz = GRAD && p.z ? p.ld_z : p.ld_x, lddy = GRAD ? p.ld_dy : p.ld_x;
    float bias[4], sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) bias[k] = p.delta_bias && ds + k < p.D ? p.delta_bias[ds + k] : 0.f;
    static_assert(kBwdSegment <= 64 && kFwdLocal <= 128, "rows of bc");
    stage_rows<T, NP, GRAD ? 64 : 128>(sm.bc, p.Bm, p.ld_B, p.N, g, 0, vec);
    if (GRAD) stage_rows<T, NP, 64>(sm.bc + 64, p.Cm, p.ld_C, p.N, g, 0, vec);
    Four<T, XV> rx[K], rd[K], ry[GRAD ? K : 1], rz[GRAD ? K : 1];     // the next tile, on its way
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long tl = min(t0 + r0 + k * ROWS, g.len - 1);
            rx[k].load(x + tl * p.ld_x, last);
            rd[k].load(delta + tl * p.ld_delta, last);
            if (GRAD) {
                ry[k].load(dy + tl * lddy, last);
                rz[k].load(z + tl * ldz, last);
            }
        }
    };
    if (g.len > 0) fetch(0);
    for (int t0 = 0; t0 < g.len; t0 += TT) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = r0 + k * ROWS;
            const bool in = t0 + t < g.len;
            float xv[4], dv[4], yv[4], zv[4];
            rx[k].get(xv);
            rd[k].get(dv);
            if (GRAD) {
                ry[k].get(yv);
                rz[k].get(zv);
            }
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
                f2 dt = pack2(dv[s] + bias[s], dv[s + 1] + bias[s + 1]);
                if (p.softplus) dt = softplus2(dt);
                float lo, hi;
                unpack2(dt, lo, hi);
                lo = in ? lo : 0.f;
                hi = in ? hi : 0.f;
                sum[s] += lo;
                sum[s + 1] += hi;
                const float ul = in ? lo * xv[s] : 0.f, uh = in ? hi * xv[s + 1] : 0.f;
                sm.d[t][S::at(4 * q + s)] = {both(lo), both(ul)};
                sm.d[t][S::at(4 * q + s + 1)] = {both(hi), both(uh)};
                if (GRAD) {
                    f2 gy = pack2(yv[s], yv[s + 1]);
                    if (p.z) gy = mul2(gy, silu2(pack2(zv[s], zv[s + 1])));
                    unpack2(gy, lo, hi);
                    sm.g[t][S::at(4 * q + s)] = both(in ? lo : 0.f);
                    sm.g[t][S::at(4 * q + s + 1)] = both(in ? hi : 0.f);
                }
            }
        }
        fetch(t0 + TT);                  // (past the end the last row again)
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const f2x2 v = sm.d[t][S::at(c)];
            const f2 gy = GRAD ? sm.g[t][S::at(c)] : 0;
#pragma unroll
            for (int k = 0; k < H; k += 2) {
                const f2x2 b = *reinterpret_cast<const f2x2 *>(&sm.bc[t0 + t][n0 + 2 * k]);
                const f2 a0 = decay2(v.a, a2[k]), a1 = decay2(v.a, a2[k + 1]);
                h[k] = fma2(a0, h[k], mul2(v.b, b.a));
                h[k + 1] = fma2(a1, h[k + 1], mul2(v.b, b.b));
                if (GRAD) {
                    const f2x2 cq = *reinterpret_cast<const f2x2 *>(&sm.bc[64 + t0 + t][n0 + 2 * k]);
                    m[k] = mul2(m[k], a0);
                    m[k + 1] = mul2(m[k + 1], a1);
                    e[k] = fma2(m[k], mul2(gy, cq.a), e[k]);
                    e[k + 1] = fma2(m[k + 1], mul2(gy, cq.b), e[k + 1]);
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) sm.sum[r0][q][k] = sum[k];
    __syncthreads();
    const long long at = slot * p.D + d;
    if (tid < CH && d0 + tid < p.D) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) s += sm.sum[k][tid / 4][tid % 4];
        p.seg_dt[slot * p.D + d0 + tid] = s;
    }
    if (!live) return;
#pragma unroll
    for (int k = 0; k < H; k += 2) {
        *reinterpret_cast<f2x2 *>(p.seg_state + at * NP + n0 + 2 * k) = {h[k], h[k + 1]};
        if (GRAD) *reinterpret_cast<f2x2 *>(p.seg_grad + at * NP + n0 + 2 * k) = {e[k], e[k + 1]};
    }
}

// One thread per (sequence, channel, state) and direction: entry states forwards (blockIdx.y = 0), exit
// gradients backwards (1), eight segments' values on their way at a time.
__global__ void __launch_bounds__(128) scan_boundary_kernel(ScanParams p, int NP) {
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long per = (long long)p.D * NP;
    const long long b = u / per;
    if (b >= p.B) return;
    const int d = (int)((u - b * per) / NP), n = (int)(u % NP);
    const bool back = blockIdx.y;
    long long s0;
    int count;
    if (!p.cu_seqlens) {
        count = (int)((p.T + (long long)p.lseg - 1) / p.lseg);
        s0 = b * count;
    } else {
        const int lo = clamped(p.cu_seqlens[b], 0, p.T), hi = clamped(p.cu_seqlens[b + 1], lo, p.T);
        count = hi > lo ? (int)((hi - lo + (long long)p.lseg - 1) / p.lseg) : 1;
        s0 = b + lo / p.lseg;
    }
    const bool in = n < p.N;
    const float a2 = in ? decay_rate(p.A[(long long)d * p.N + n]) : 0.f;
    const long long at = (b * p.D + d) * p.N + n;
    const float *first = back ? p.dht : p.h0;
    float v = in && first ? first[at] : 0.f;
    const long long step = back ? -(long long)p.D : p.D;
    const long long k0 = (back ? s0 + count - 1 : s0) * p.D + d;
    float *vals = (back ? p.seg_grad : p.seg_state) + n;
    constexpr int K = 8;
    float local[K], dt[K];
    auto fetch = [&](int i) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const long long k = k0 + (long long)min(i + j, count - 1) * step;
            local[j] = vals[k * NP];
            dt[j] = p.seg_dt[k];
        }
    };
    fetch(0);
    for (int i = 0; i < count; i += K) {
        float now[K], a[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            now[j] = local[j];
            a[j] = ex2(a2 * dt[j]);
        }
        if (i + K < count) fetch(i + K);       // before this batch is stored: nothing of it is read again
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (i + j < count) {
                vals[(k0 + (i + j) * step) * NP] = v;
                v = fmaf(a[j], v, now[j]);
            }
    }
    if (back && in && p.dh0) p.dh0[at] = v;
}

constexpr int TC = 8;                // tokens per part, recomputed into registers
constexpr int GROUPS = 2;            // channel groups that a block walks per part
constexpr int PARTS = SEG / TC;
constexpr int kGradThreads = 128;   // two blocks to an SM: one loads or stores while the other computes
constexpr int kGradWarps = kGradThreads / 32;

template <int L> struct GradTiles {
    static constexpr int NP = 4 * L, CW = 32 / L, CG = kGradWarps * CW, CH = GROUPS * CG;   // channels of a warp, group, block
    static constexpr int XS = CH + 4;
    f2x2 entry[GROUPS][PARTS][kGradThreads];     // states before each part
    float2 du[SEG][XS];                          // dt, dt x; after a part: dt, sum_n G B
    float g[SEG][XS];                            // g; after a part: sum_n q A / ln 2
    float y[SEG][XS];                            // sum_n C h
    float B[SEG][NP], C[SEG][NP];
    float red[kGradWarps][TC * 2 * NP];
};

// A block: 64 tokens, 8 CW channels, 4 warps.  All inputs go through shared memory once, four channels
// per access; the parts leave their sums over states there, and a last sweep over (token, channel) turns
// them into dx, ddelta and dz, again four channels per access.
template <class T, int L, bool XV>
__global__ void __launch_bounds__(kGradThreads, 2) scan_grad_kernel(ScanParams p, int chan_blocks, bool vec) {
    using S = GradTiles<L>;
    constexpr int NP = S::NP, CW = S::CW, CH = S::CH, TL = TC / L, Q = CH / 4, ROWS = kGradThreads / Q, K = SEG / ROWS;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane / L, i = lane % L, n0 = 4 * i;
    const long long slot = blockIdx.x / chan_blocks;
    const int cb = (int)(blockIdx.x - slot * chan_blocks), d0 = cb * CH;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, SEG, slot, g)) {
        // a slot that no sequence uses: its partial sums are zeros, so that the sums may take all slots
        float *out = p.part_par + slot * ((long long)p.D * (p.N + 2));
        const int end = min(d0 + CH, p.D);
        for (long long u = (long long)d0 * p.N + tid; u < (long long)end * p.N; u += kGradThreads) out[u] = 0.f;
        for (int d = d0 + tid; d < end; d += kGradThreads)
            out[(long long)p.D * p.N + d] = out[(long long)p.D * (p.N + 1) + d] = 0.f;
        return;
    }
    const long long row = g.row0 + g.t0;

    // ---- inputs to shared memory
    const int q = tid % Q, r0 = tid / Q, ds = d0 + 4 * q, dl = XV ? min(ds, p.D - 4) : min(ds, p.D - 1), last = p.D - 1 - dl;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x + dl, *delta = static_cast<const T *>(p.delta) + row * p.ld_delta + dl;
    const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy + dl;
    const T *z = p.z ? static_cast<const T *>(p.z) + row * p.ld_z + dl : x;
    const long long ldz = p.z ? p.ld_z : p.ld_x;
    float bias[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) bias[k] = p.delta_bias && ds + k < p.D ? p.delta_bias[ds + k] : 0.f;
    constexpr int KB = K < 4 ? K : 4;            // tokens per thread whose loads are in flight together
    Four<T, XV> rx[KB], rd[KB], ry[KB], rz[KB];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const long long tl = min(r0 + (k0 + k) * ROWS, g.len - 1);
            rx[k].load(x + tl * p.ld_x, last);
            rd[k].load(delta + tl * p.ld_delta, last);
            ry[k].load(dy + tl * p.ld_dy, last);
            rz[k].load(z + tl * ldz, last);
        }
    };
    for (int k0 = 0; k0 < K && g.len > 0; k0 += KB) {
        fetch(k0);
        if (k0 == 0) {
            stage_rows<T, NP, SEG, kGradThreads>(sm.B, p.Bm, p.ld_B, p.N, g, 0, vec);
            stage_rows<T, NP, SEG, kGradThreads>(sm.C, p.Cm, p.ld_C, p.N, g, 0, vec);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int t = r0 + (k0 + k) * ROWS;
            const bool in = t < g.len;
            float xv[4], dv[4], yv[4], zv[4];
            rx[k].get(xv);
            rd[k].get(dv);
            ry[k].get(yv);
            rz[k].get(zv);
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
                f2 dt = pack2(dv[s] + bias[s], dv[s + 1] + bias[s + 1]), gy = pack2(yv[s], yv[s + 1]);
                if (p.softplus) dt = softplus2(dt);
                if (p.z) gy = mul2(gy, silu2(pack2(zv[s], zv[s + 1])));
                float lo, hi, gl, gh;
                unpack2(dt, lo, hi);
                unpack2(gy, gl, gh);
                // tokens past the end leave the state as it is, channels past the end add nothing to dB and dC
                const bool il = in && ds + s < p.D, ih = in && ds + s + 1 < p.D;
                *reinterpret_cast<float4 *>(&sm.du[t][4 * q + s]) =
                    make_float4(il ? lo : 0.f, il ? lo * xv[s] : 0.f, ih ? hi : 0.f, ih ? hi * xv[s + 1] : 0.f);
                *reinterpret_cast<float2 *>(&sm.g[t][4 * q + s]) = make_float2(il ? gl : 0.f, ih ? gh : 0.f);
            }
        }
    }
    __syncthreads();
    const int parts = (g.len + TC - 1) / TC;

    f2 a2[GROUPS][2], carry[GROUPS][2], dA[GROUPS][2];   // per channel group: A log2 e, gradient of the state after the part
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        const int d = d0 + k * S::CG + warp * CW + c;
        float av[4] = {0.f, 0.f, 0.f, 0.f}, hv[4] = {0.f, 0.f, 0.f, 0.f}, ev[4] = {0.f, 0.f, 0.f, 0.f};
        if (d < p.D) {
            load_states(av, p.A + (long long)d * p.N, n0, p.N);
            load_states(hv, p.seg_state + (slot * p.D + d) * NP, n0, NP);
            load_states(ev, p.seg_grad + (slot * p.D + d) * NP, n0, NP);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            a2[k][s] = pack2(decay_rate(av[2 * s]), decay_rate(av[2 * s + 1]));
            carry[k][s] = pack2(ev[2 * s], ev[2 * s + 1]);
            dA[k][s] = pack2(0.f, 0.f);
        }
        // ---- forward sweep: the state before every part (the last part's tokens are swept below)
        f2 h0 = pack2(hv[0], hv[1]), h1 = pack2(hv[2], hv[3]);
        const int cc = k * S::CG + warp * CW + c;
        for (int part = 0; part < parts; ++part) {
            sm.entry[k][part][tid] = {h0, h1};
            if (part == parts - 1) break;
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                const float2 v = sm.du[part * TC + t][cc];
                const f2x2 b = *reinterpret_cast<const f2x2 *>(&sm.B[part * TC + t][n0]);
                const f2 dt = both(v.x), u = both(v.y);
                h0 = fma2(decay2(dt, a2[k][0]), h0, mul2(u, b.a));
                h1 = fma2(decay2(dt, a2[k][1]), h1, mul2(u, b.b));
            }
        }
    }

    // ---- the parts, last to first
    for (int part = parts - 1; part >= 0; --part) {
        f2 accB[TC][2], accC[TC][2];     // dB, dC of this lane's states, over the channel groups
        const int real = g.len - part * TC;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
            const int cc = k * S::CG + warp * CW + c;
            float ys[TC], us[TC], qs[TC];
            f2 h[TC + 1][2], a[TC][2];
            {
                const f2x2 v = sm.entry[k][part][tid];
                h[0][0] = v.a;
                h[0][1] = v.b;
            }
#pragma unroll
            for (int t = 0; t < TC; ++t) {
                const float2 v = sm.du[part * TC + t][cc];
                const f2x2 b = *reinterpret_cast<const f2x2 *>(&sm.B[part * TC + t][n0]);
                const f2x2 cq = *reinterpret_cast<const f2x2 *>(&sm.C[part * TC + t][n0]);
                const f2 dt = both(v.x), u = both(v.y);
                a[t][0] = decay2(dt, a2[k][0]);
                a[t][1] = decay2(dt, a2[k][1]);
                h[t + 1][0] = fma2(a[t][0], h[t][0], mul2(u, b.a));
                h[t + 1][1] = fma2(a[t][1], h[t][1], mul2(u, b.b));
                float lo, hi;
                unpack2(fma2(h[t + 1][0], cq.a, mul2(h[t + 1][1], cq.b)), lo, hi);
                ys[t] = lo + hi;
            }
            f2 G0 = carry[k][0], G1 = carry[k][1];
#pragma unroll
            for (int t = TC - 1; t >= 0; --t) {
                const float2 v = sm.du[part * TC + t][cc];
                const f2 dt = both(v.x), u = both(v.y), gy = both(sm.g[part * TC + t][cc]);
                const f2x2 b = *reinterpret_cast<const f2x2 *>(&sm.B[part * TC + t][n0]);
                const f2x2 cq = *reinterpret_cast<const f2x2 *>(&sm.C[part * TC + t][n0]);
                G0 = fma2(cq.a, gy, G0);
                G1 = fma2(cq.b, gy, G1);
                accC[t][0] = k ? fma2(gy, h[t + 1][0], accC[t][0]) : mul2(gy, h[t + 1][0]);
                accC[t][1] = k ? fma2(gy, h[t + 1][1], accC[t][1]) : mul2(gy, h[t + 1][1]);
                accB[t][0] = k ? fma2(u, G0, accB[t][0]) : mul2(u, G0);
                accB[t][1] = k ? fma2(u, G1, accB[t][1]) : mul2(u, G1);
                float lo, hi;
                unpack2(fma2(G0, b.a, mul2(G1, b.b)), lo, hi);
                us[t] = lo + hi;
                G0 = mul2(G0, a[t][0]);
                G1 = mul2(G1, a[t][1]);
                const f2 q0 = mul2(G0, h[t][0]), q1 = mul2(G1, h[t][1]);
                if (t < real) {          // past the end q may be infinite, and dt is 0
                    dA[k][0] = fma2(q0, dt, dA[k][0]);
                    dA[k][1] = fma2(q1, dt, dA[k][1]);
                }
                unpack2(fma2(q0, a2[k][0], mul2(q1, a2[k][1])), lo, hi);
                qs[t] = lo + hi;
            }
            carry[k][0] = G0;
            carry[k][1] = G1;
            spread_sum<TC, L>(us, i);
            spread_sum<TC, L>(qs, i);
            spread_sum<TC, L>(ys, i);
            __syncwarp();                // du and g of these tokens have been read by the channel's lanes
#pragma unroll
            for (int j = 0; j < TL; ++j) {
                const int t = part * TC + i * TL + j;
                sm.du[t][cc].y = us[j];
                sm.g[t][cc] = qs[j];
                sm.y[t][cc] = ys[j];
            }
        }
        // dB and dC over the warp's channels, then over the warps
        float v[2 * TC * 4];
#pragma unroll
        for (int t = 0; t < TC; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                unpack2(accB[t][s], v[t * 4 + 2 * s], v[t * 4 + 2 * s + 1]);
                unpack2(accC[t][s], v[(TC + t) * 4 + 2 * s], v[(TC + t) * 4 + 2 * s + 1]);
            }
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
            sm.red[warp][(t * 2 + w) * NP + n0 + s] = v[k];
        }
        __syncthreads();
        for (int u = tid; u < TC * 2 * NP; u += kGradThreads) {
            const int t = part * TC + u / (2 * NP);
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kGradWarps; ++w) s += sm.red[w][u];
            if (t < g.len)
                p.part_bc[((long long)cb * ((long long)(p.cu_seqlens ? 1 : p.B) * p.T) + row + t) * (2 * NP) + u % (2 * NP)] = s;
        }
        __syncthreads();
    }
    float *out = p.part_par + slot * ((long long)p.D * (p.N + 2));
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        const int d = d0 + k * S::CG + warp * CW + c;
        float w[4];
        unpack2(dA[k][0], w[0], w[1]);
        unpack2(dA[k][1], w[2], w[3]);
        if (d < p.D) store_states(out + (long long)d * p.N, w, n0, p.N);
    }

    // ---- outputs, token by token of this thread's four channels
    __syncthreads();
    const int nl = p.D - ds;
    float pd[4] = {0.f, 0.f, 0.f, 0.f}, pb[4] = {0.f, 0.f, 0.f, 0.f}, skip[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) skip[k] = p.Dskip && ds + k < p.D ? p.Dskip[ds + k] : 0.f;
    T *dx = static_cast<T *>(p.dx) + row * p.ld_dx + ds, *dd = static_cast<T *>(p.ddelta) + row * p.ld_ddelta + ds;
    T *dz = static_cast<T *>(p.dz) + row * p.ld_dz + ds;
    for (int k0 = 0; k0 < K && g.len > 0 && nl > 0; k0 += KB) {
        fetch(k0);                               // (from L2)
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int t = r0 + (k0 + k) * ROWS;
            const bool in = t < g.len;
            const long long tl = t;
            float xv[4], dv[4], yv[4], zv[4], ox[4], od[4], oz[4];
            rx[k].get(xv);
            rd[k].get(dv);
            ry[k].get(yv);
            rz[k].get(zv);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 w = sm.du[t][4 * q + s];
                const float sz = sigmoid(zv[s]), gy = p.z ? yv[s] * zv[s] * sz : yv[s];
                const float sd = p.softplus ? sigmoid(dv[s] + bias[s]) : 1.f;
                ox[s] = fmaf(w.y, w.x, skip[s] * gy);
                od[s] = fmaf(w.y, xv[s], sm.g[t][4 * q + s] * kLn2) * sd;
                oz[s] = yv[s] * fmaf(skip[s], xv[s], sm.y[t][4 * q + s]) * sz * fmaf(zv[s], 1.f - sz, 1.f);
                pd[s] = in ? fmaf(gy, xv[s], pd[s]) : pd[s];
                pb[s] = in ? pb[s] + od[s] : pb[s];
            }
            if (in) {
                store_four<T, XV>(dx + tl * p.ld_dx, ox, nl);
                store_four<T, XV>(dd + tl * p.ld_ddelta, od, nl);
                if (p.z) store_four<T, XV>(dz + tl * p.ld_dz, oz, nl);
            }
        }
    }
    // dD and dbias over the block's tokens
    float *part = &sm.red[0][0];                 // [ROWS][CH][2]
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        part[(r0 * CH + 4 * q + s) * 2] = pd[s];
        part[(r0 * CH + 4 * q + s) * 2 + 1] = pb[s];
    }
    __syncthreads();
    for (int u = tid; u < 2 * CH; u += kGradThreads) {
        const int d = d0 + u / 2;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s += part[r * CH * 2 + u];
        if (d < p.D) out[(long long)p.D * (p.N + (u & 1)) + d] = s;
    }
}

// The sums, in a fixed order: blocks 0 .. bc_blocks - 1 add dB and dC over the channel blocks and round them
// (rows outside every sequence are left alone), the others dA, dD and dbias over the segments, 32
// columns of [D N + 2 D] each.
template <class T>
__global__ void __launch_bounds__(256) scan_sums_kernel(ScanParams p, int blocks, int NP, long long rows, unsigned bc_blocks, int slots) {
    if (blockIdx.x < bc_blocks) {
        const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
        const long long row = u / (2 * NP);
        const int j = (int)(u - row * (2 * NP)), n = j % NP;
        if (row >= rows || n >= p.N) return;
        if (p.cu_seqlens && (row < clamped(p.cu_seqlens[0], 0, p.T) || row >= clamped(p.cu_seqlens[p.B], 0, p.T))) return;
        float s = 0.f;
#pragma unroll 4
        for (int k = 0; k < blocks; ++k) s += p.part_bc[(k * rows + row) * (2 * NP) + j];
        if (j < NP) static_cast<T *>(p.dBm)[row * p.ld_dB + n] = from_f<T>(s);
        else static_cast<T *>(p.dCm)[row * p.ld_dC + n] = from_f<T>(s);
        return;
    }
    __shared__ float sm[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long par = (long long)p.D * p.N, cols = par + 2LL * p.D;
    const long long c = (long long)(blockIdx.x - bc_blocks) * 32 + tx;
    float s = 0.f;
    if (c < cols) {
        const float *q = p.part_par + c;
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        int r = ty;
        for (; r + 24 < slots; r += 32) {
            a0 += q[(long long)r * cols];
            a1 += q[(long long)(r + 8) * cols];
            a2 += q[(long long)(r + 16) * cols];
            a3 += q[(long long)(r + 24) * cols];
        }
        for (; r < slots; r += 8) a0 += q[(long long)r * cols];
        s = (a0 + a1) + (a2 + a3);
    }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty || c >= cols) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sm[k][tx];
    if (c < par) p.dA[c] = s;
    else if (c < par + p.D) {
        if (p.dDskip) p.dDskip[c - par] = s;
    } else if (p.ddelta_bias) {
        p.ddelta_bias[c - par - p.D] = s;
    }
}

// Four channels per access where every array that is read or written allows it.
template <class T> bool local_xv(const ScanParams &p) {
    const size_t es = sizeof(T), n = 4 * es;
    return p.D % 4 == 0 && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.delta, p.ld_delta, es, n) &&
           rows_aligned(p.z, p.ld_z, es, n) && rows_aligned(p.dy, p.ld_dy, es, n);
}
template <class T> bool grad_xv(const ScanParams &p) {
    const size_t es = sizeof(T), n = 4 * es;
    return local_xv<T>(p) && rows_aligned(p.dx, p.ld_dx, es, n) && rows_aligned(p.ddelta, p.ld_ddelta, es, n) &&
           rows_aligned(p.dz, p.ld_dz, es, n);
}

template <class T, int L, int NS, bool GRAD, bool XV> cudaError_t local_start(const ScanParams &p, cudaStream_t s) {
    using S = LocalTiles<L, NS>;
    const int cb = (p.D + S::CH - 1) / S::CH;
    const long long blocks = scan_slots(p, p.lseg) * cb;
    const long long bblocks = ((long long)p.B * p.D * S::NP + 127) / 128;
    if (blocks > 0x7fffffffLL || bblocks > 0x7fffffffLL) return cudaErrorNotSupported;
    cudaError_t e = cudaFuncSetAttribute(scan_local_kernel<T, L, NS, GRAD, XV>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(S));
    if (e != cudaSuccess) return e;
    scan_local_kernel<T, L, NS, GRAD, XV><<<(unsigned)blocks, kScanThreads, sizeof(S), s>>>(p, cb, bc_vec_ok<T>(p, S::NP));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_boundary_kernel<<<dim3((unsigned)bblocks, GRAD ? 2 : 1), 128, 0, s>>>(p, S::NP);
    return cudaGetLastError();
}
template <class T, int L, int NS, bool GRAD> cudaError_t local_launch(const ScanParams &p, cudaStream_t s) {
    return local_xv<T>(p) ? local_start<T, L, NS, GRAD, true>(p, s) : local_start<T, L, NS, GRAD, false>(p, s);
}

// The states' layout in the workspace, [slots][D][padded states]: the forward takes its own padding, the
// backward's two passes share theirs (16 or 32).
template <class T> cudaError_t segments_type(const ScanParams &p, bool grad, cudaStream_t s) {
    if (grad) return p.N <= 16 ? local_launch<T, 2, 8, true>(p, s) : local_launch<T, 4, 8, true>(p, s);
    if (p.N <= 4) return local_launch<T, 1, 4, false>(p, s);
    if (p.N <= 8) return local_launch<T, 1, 8, false>(p, s);
    return p.N <= 16 ? local_launch<T, 2, 8, false>(p, s) : local_launch<T, 4, 8, false>(p, s);
}

int grad_states(int N) { return N <= 16 ? 16 : 32; }
int grad_blocks(const ScanParams &p) {
    const int ch = p.N <= 16 ? GradTiles<4>::CH : GradTiles<8>::CH;
    return (p.D + ch - 1) / ch;
}

long long batch_rows(const ScanParams &p) { return (long long)(p.cu_seqlens ? 1 : p.B) * p.T; }

template <class T, int L, bool XV> cudaError_t grad_start(const ScanParams &p, cudaStream_t s) {
    const int cb = grad_blocks(p);
    const long long slots = scan_slots(p, SEG), blocks = slots * cb, rows = batch_rows(p);
    const long long bc = (rows * 8 * L + 255) / 256, par = ((long long)p.D * (p.N + 2) + 31) / 32;
    if (blocks > 0x7fffffffLL || bc + par > 0x7fffffffLL) return cudaErrorNotSupported;
    constexpr int smem = sizeof(GradTiles<L>);
    cudaError_t e = cudaFuncSetAttribute(scan_grad_kernel<T, L, XV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    scan_grad_kernel<T, L, XV><<<(unsigned)blocks, kGradThreads, smem, s>>>(p, cb, bc_vec_ok<T>(p, 4 * L));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_sums_kernel<T><<<(unsigned)(bc + par), 256, 0, s>>>(p, cb, 4 * L, rows, (unsigned)bc, (int)slots);
    return cudaGetLastError();
}
template <class T> cudaError_t grad_type(const ScanParams &p, cudaStream_t s) {
    if (p.N <= 16) return grad_xv<T>(p) ? grad_start<T, 4, true>(p, s) : grad_start<T, 4, false>(p, s);
    return grad_xv<T>(p) ? grad_start<T, 8, true>(p, s) : grad_start<T, 8, false>(p, s);
}

}  // namespace

cudaError_t launch_scan_segments(const ScanParams &p, bool bf, bool grad, cudaStream_t s) {
    return bf ? segments_type<bf16>(p, grad, s) : segments_type<float>(p, grad, s);
}

// Workspace: [slots][D][NP] x 2, [slots][D], [slots][D (N + 2)], [channel blocks][rows][2 NP].
// The first two and the last are read and written four floats at a time and lie first.
size_t ssm_scan_bwd_floats(const ScanParams &p) {
    const size_t slots = (size_t)scan_slots(p, SEG), NP = grad_states(p.N);
    return slots * p.D * (2 * NP + 1 + p.N + 2) + (size_t)grad_blocks(p) * batch_rows(p) * 2 * NP;
}

void ssm_scan_bwd_carve(ScanParams &p, float *ws) {
    const size_t slots = (size_t)scan_slots(p, SEG), NP = grad_states(p.N);
    p.seg_state = ws;
    p.seg_grad = p.seg_state + slots * p.D * NP;
    p.part_bc = p.seg_grad + slots * p.D * NP;
    p.seg_dt = p.part_bc + (size_t)grad_blocks(p) * batch_rows(p) * 2 * NP;
    p.part_par = p.seg_dt + slots * p.D;
}

cudaError_t launch_ssm_scan_bwd(const ScanParams &q, bool bf, cudaStream_t s) {
    ScanParams p = q;
    p.seg = p.lseg = SEG;
    const cudaError_t e = launch_scan_segments(p, bf, true, s);
    if (e != cudaSuccess) return e;
    return bf ? grad_type<bf16>(p, s) : grad_type<float>(p, s);
}

}  // namespace mixer
