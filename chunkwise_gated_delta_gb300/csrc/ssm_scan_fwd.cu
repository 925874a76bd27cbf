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

// A block: 128 / L channels, four warps that carry the states (32 / L channels each) and four that
// feed them.  Per tile of 8 L tokens
//   the feeders   bring x, delta, z (8 neighbouring channels of one token per thread) and Bm, Cm of
//                 the tile after the next into registers, turn the next tile's delta into dt and
//                 leave {dt, dt, dt x, dt x} and float32 Bm, Cm in shared memory, and finish the
//                 last tile's outputs: + D x, gate, rounding, store;
//   the carriers  run the recurrence over the tile, four states of a channel per lane, and leave
//                 sum_n C h in shared memory.
// Both sides work on double buffers and meet once per tile.  Alone, a carrier warp waits for its
// own shared-memory loads and exponentials two cycles of three, and one block of 32 channels per
// 1.7 warps and scheduler is all that B 4, D 2048 has: the feeders fill those slots.
constexpr int kFwdThreads = 2 * kScanThreads;
constexpr int KT = 8;                      // tokens of a tile per lane

template <int L> struct FwdTiles {
    static constexpr int NP = 4 * L, CW = 32 / L, CH = 4 * CW, TT = KT * L, YS = CH + CW;
    f2x2 d[2][TT * CH];                    // {dt, dt}, {dt x, dt x}; 16-byte words swizzled, see at()
    float B[2][TT][NP], C[2][TT][NP];
    float y[2][TT][YS];                    // row stride: the tokens of a channel's lanes in different banks
    // Word of token t, channel c.  A feeder writes 8 neighbouring channels one after the other, a
    // carrier warp reads 8 of one token at once: the exclusive or keeps both free of bank conflicts.
    static __device__ __forceinline__ int at(int s) { return s ^ (s >> 3 & 7); }
};

__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(kFwdThreads) : "memory"); }

// Eight neighbouring channels of one token, as they lie in memory (XV: two or one 16-byte accesses).
template <class T, bool XV> struct Eight {
    static constexpr int W = 8 * sizeof(T) / 16;
    uint4 v[XV ? W : 1];
    T e[XV ? 1 : 8];
    __device__ __forceinline__ void load(const T *p, int n) {        // n: channels that exist
        if (XV) {
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] = reinterpret_cast<const uint4 *>(p)[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) e[k] = p[k];
        }
    }
    __device__ __forceinline__ void zero() {
        if (XV) {
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = from_f<T>(0.f);
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if (!XV) return to_f(e[k]);
        const uint4 &q = v[k * sizeof(T) / 16];
        const int w = k * sizeof(T) / 4 % 4;
        const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
        if (sizeof(T) == 4) return __uint_as_float(u);
        return __uint_as_float(k & 1 ? u & 0xffff0000u : u << 16);
    }
};

template <class T, int L, bool XV>
__global__ void __launch_bounds__(kFwdThreads) scan_fwd_kernel(ScanParams p, int chan_blocks) {
    using S = FwdTiles<L>;
    constexpr int NP = S::NP, CW = S::CW, CH = S::CH, TT = S::TT;
    extern __shared__ __align__(16) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const long long slot = blockIdx.x / chan_blocks;
    const int d0 = (int)(blockIdx.x - slot * chan_blocks) * CH;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    const int tiles = (g.len + TT - 1) / TT;
    const long long row0 = g.row0 + g.t0;

    if (threadIdx.x >= kScanThreads) {
        // ------------------------------------------------------------------ feeders
        const int tid = threadIdx.x - kScanThreads;
        const int t = tid / (CH / 8), c0 = tid % (CH / 8) * 8;       // this thread's token and channels
        const int d = d0 + c0, n = p.D - d;                          // n <= 0: none of them exist
        const bool some = n > 0;
        const long long r = row0 + t;
        const T *x = static_cast<const T *>(p.x) + r * p.ld_x + d, *delta = static_cast<const T *>(p.delta) + r * p.ld_delta + d;
        const T *z = p.z ? static_cast<const T *>(p.z) + r * p.ld_z + d : nullptr;
        T *y = static_cast<T *>(p.y) + r * p.ld_y + d;
        float dbias[8], skip[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dbias[k] = k < n && p.delta_bias ? p.delta_bias[d + k] : 0.f;
            skip[k] = k < n && p.Dskip ? p.Dskip[d + k] : 0.f;
        }
        // Bm and Cm of a tile: elements tid, tid + 128, ...
        constexpr int E = TT * NP < kScanThreads ? 1 : TT * NP / kScanThreads;
        const int bt = tid / NP, bn = tid % NP;                      // NP divides 128
        const bool bs = TT * NP >= kScanThreads || bt < TT;          // (L = 1: 32 elements)
        const T *Bp = static_cast<const T *>(p.Bm) + (row0 + bt) * p.ld_B + bn;
        const T *Cp = static_cast<const T *>(p.Cm) + (row0 + bt) * p.ld_C + bn;
        constexpr int BT = kScanThreads / NP;                        // tokens between a thread's elements
        Eight<T, XV> xn, dn, zn, xc, zc, xo, zo;                     // next, current, last tile
        T be[E], ce[E];
        auto fetch = [&](int tile) {
            const int t0 = tile * TT;
            xn.zero();
            dn.zero();
            zn.zero();
            if (some && t0 + t < g.len) {
                xn.load(x + t0 * p.ld_x, n);
                dn.load(delta + t0 * p.ld_delta, n);
                if (z) zn.load(z + t0 * p.ld_z, n);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                be[k] = ce[k] = from_f<T>(0.f);
                if (bs && bn < p.N && t0 + bt + k * BT < g.len) {
                    be[k] = Bp[(t0 + k * BT) * p.ld_B];
                    ce[k] = Cp[(t0 + k * BT) * p.ld_C];
                }
            }
        };
        auto stage = [&](int tile) {
            const int b = tile & 1;
            const bool in = tile * TT + t < g.len;                   // behind the end the state stays as it is
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                float lo = dn.get(k) + dbias[k], hi = dn.get(k + 1) + dbias[k + 1];
                if (p.softplus) unpack2(softplus2(lo, hi), lo, hi);
                lo = in ? lo : 0.f;
                hi = in ? hi : 0.f;
                const float ul = lo * xn.get(k), uh = hi * xn.get(k + 1);
                sm.d[b][S::at(tid * 8 + k)] = {pack2(lo, lo), pack2(ul, ul)};
                sm.d[b][S::at(tid * 8 + k + 1)] = {pack2(hi, hi), pack2(uh, uh)};
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                if (!bs) break;
                sm.B[b][bt + k * BT][bn] = to_f(be[k]);
                sm.C[b][bt + k * BT][bn] = to_f(ce[k]);
            }
            xc = xn;
            zc = zn;
        };
        auto finish = [&](int tile) {
            if (!some || tile * TT + t >= g.len) return;
            const float *src = &sm.y[tile & 1][t][c0];
            const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
            float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = fmaf(skip[k], xo.get(k), o[k]);
            if (z)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float zv = zo.get(k);
                    o[k] *= zv * sigmoid(zv);
                }
            T *out = y + (long long)tile * TT * p.ld_y;
            if (XV) {
#pragma unroll
                for (int k = 0; k < 8; k += 16 / (int)sizeof(T)) {
                    Vec<T, 16 / sizeof(T)> q;
#pragma unroll
                    for (int e = 0; e < 16 / (int)sizeof(T); ++e) q.e[e] = from_f<T>(o[k + e]);
                    store_vec<T, 16 / sizeof(T)>(out + k, q);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < n) out[k] = from_f<T>(o[k]);
            }
        };
        if (tiles > 0) {
            fetch(0);
            stage(0);
            if (tiles > 1) fetch(1);
        }
        for (int tile = 0; tile < tiles; ++tile) {
            meet();                              // tile staged; tile - 1 carried
            if (tile > 0) finish(tile - 1);
            xo = xc;
            zo = zc;
            if (tile + 1 < tiles) stage(tile + 1);
            if (tile + 2 < tiles) fetch(tile + 2);
        }
        meet();
        if (tiles > 0) finish(tiles - 1);
        return;
    }
    // ---------------------------------------------------------------------- carriers
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane / L, i = lane % L, n0 = 4 * i;
    const int d = d0 + warp * CW + c;
    const bool live = d < p.D;
    float a2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        load_states(a2, p.A + (long long)d * p.N, n0, p.N);
        if (p.seg_state) load_states(h, p.seg_state + (slot * p.D + d) * NP, n0, NP);
        else if (p.h0) load_states(h, p.h0 + ((long long)g.b * p.D + d) * p.N, n0, p.N);
    }
    const f2 a01 = pack2(a2[0] * kLog2e, a2[1] * kLog2e), a23 = pack2(a2[2] * kLog2e, a2[3] * kLog2e);
    f2 h01 = pack2(h[0], h[1]), h23 = pack2(h[2], h[3]);
    // the swizzle's period in tokens: at() sees t CH / 8 modulo 8
    constexpr int P = L <= 2 ? 1 : L / 2;
    int off[P];
#pragma unroll
    for (int k = 0; k < P; ++k) off[k] = S::at(k * CH + warp * CW + c) - k * CH;
    for (int tile = 0; tile < tiles; ++tile) {
        meet();
        const int b = tile & 1;
        const f2x2 *sd = sm.d[b];
        // L tokens at a time: their decays and inputs do not wait for the state, so they are
        // prepared one group ahead.  No branch in here: the whole tile is one block to schedule.
        f2 da[2][L][2], du[2][L][2];
        auto prepare = [&](int j) {
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const int t = j * L + k;
                const f2x2 v = sd[t * CH + off[t % P]];
                const f2x2 bq = *reinterpret_cast<const f2x2 *>(&sm.B[b][t][n0]);
                da[j & 1][k][0] = ex2_2(mul2(v.a, a01));
                da[j & 1][k][1] = ex2_2(mul2(v.a, a23));
                du[j & 1][k][0] = mul2(v.b, bq.a);
                du[j & 1][k][1] = mul2(v.b, bq.b);
            }
        };
        prepare(0);
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            if (j + 1 < KT) prepare(j + 1);
            float ys[L];
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const f2x2 q = *reinterpret_cast<const f2x2 *>(&sm.C[b][j * L + k][n0]);
                h01 = fma2(da[j & 1][k][0], h01, du[j & 1][k][0]);
                h23 = fma2(da[j & 1][k][1], h23, du[j & 1][k][1]);
                float lo, hi;
                unpack2(fma2(h01, q.a, mul2(h23, q.b)), lo, hi);
                ys[k] = lo + hi;
            }
            spread_sum<L, L>(ys, i);
            sm.y[b][j * L + i][warp * CW + c] = ys[0];
        }
    }
    meet();
    if (p.ht && live && g.i == g.n - 1) {
        unpack2(h01, h[0], h[1]);
        unpack2(h23, h[2], h[3]);
        store_states(p.ht + ((long long)g.b * p.D + d) * p.N, h, n0, p.N);
    }
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

template <class T, int L, bool XV> cudaError_t fwd_start(const ScanParams &p, cudaStream_t s) {
    const int cb = (p.D + FwdTiles<L>::CH - 1) / FwdTiles<L>::CH;
    const long long blocks = scan_slots(p, p.seg) * cb;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    constexpr int smem = sizeof(FwdTiles<L>);
    const cudaError_t e = cudaFuncSetAttribute(scan_fwd_kernel<T, L, XV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    scan_fwd_kernel<T, L, XV><<<(unsigned)blocks, kFwdThreads, smem, s>>>(p, cb);
    return cudaGetLastError();
}

// 16-byte accesses to x, delta, z and y where all of them allow it.
template <class T, int L> cudaError_t fwd_launch(const ScanParams &p, cudaStream_t s) {
    const bool xv = p.D % 8 == 0 && rows_aligned(p.x, p.ld_x, sizeof(T), 16) && rows_aligned(p.delta, p.ld_delta, sizeof(T), 16) &&
                    rows_aligned(p.z, p.ld_z, sizeof(T), 16) && rows_aligned(p.y, p.ld_y, sizeof(T), 16);
    return xv ? fwd_start<T, L, true>(p, s) : fwd_start<T, L, false>(p, s);
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
