// Selective state-space scan: forward and single tokens.
//
//   dt = softplus(delta + bias), h = exp(dt A) h + dt x B, y = (C . h + D x) SiLU(z)
//
// Per (token, channel, state): one exponential and four multiply-adds; per (token, channel) four more
// special functions (softplus, gate) and four elements of HBM traffic.  With N = 16 the special functions
// (32 per clock and SM) take 1.8 times as long as the traffic, so the states stay in registers from
// the first token to the last and everything else is arranged around that pipe and the FMA pipe.
// B 4, T 4096, D 2048, N 16, bfloat16: 182 us (special functions 73, traffic 40).
#include <type_traits>

#include "ssm_scan.cuh"

namespace mixer {
namespace {

// A block: WN warps that carry the states (32 / L channels each, NS states of a channel per lane) and
// KT / 8 times as many that feed them (twice, with four of 16 states per lane as many).  Per tile of KT L tokens
//   the feeders   bring x, delta, z (8 neighbouring channels of one token per thread, three tiles ahead) and
//                 Bm, Cm into shared memory or registers, turn the next tile's delta into dt and leave
//                 {dt, dt, dt x, dt x} and float32 Bm, Cm in shared memory, and finish the last tile's
//                 outputs: + D x, gate, rounding, store;
//   the carriers  run the recurrence over the tile and leave sum_n C h in shared memory.
// Both sides work on double buffers and meet once per tile.  With one kind of warp doing both, 8 warps to
// an SM at B 4, D 2048 waited for their own loads and chains two cycles of three (382 us against 248
// with four states per lane).  Eight states per lane amortise the loads and the sum over lanes: one
// carrier warp per scheduler then issues near what the half-rate packed and quarter-rate exponential
// instructions of one warp allow, 70 cycles a token, 85 with the feeders in the other slots.  Two carrier
// warps of four states per scheduler take 242 us, 512 feeders of four channels 217.
// L lanes of NS states per channel, WN carrier warps; a tile has KT tokens per lane.
template <int L, int NS, int KT, int WN> struct FwdTiles {
    static constexpr int kFeeders = 4 * WN * KT, kCarriers = 32 * WN, kThreads = kCarriers + kFeeders;   // one feeder per 8 channels of a token
    static_assert(NS % 4 == 0 && 32 % L == 0, "16-byte shared-memory accesses take four states");
    static constexpr int NP = NS * L, CW = 32 / L, CH = WN * CW, TT = KT * L, YS = CH + CW;
    f2x2 d[2][TT * CH];                    // {dt, dt}, {dt x, dt x}; 16-byte words swizzled, see at()
    float B[2][TT][NP], C[2][TT][NP];
    float y[2][TT][YS];                    // row stride: the tokens of a channel's lanes in different banks
    // Word of token t, channel c.  A feeder writes 8 neighbouring channels one after the other, a
    // carrier warp reads 8 of one token at once: the exclusive or keeps both free of bank conflicts.
    static __device__ __forceinline__ int at(int s) { return s ^ (s >> 3 & 7); }
};

template <int N> __device__ __forceinline__ void meet_all() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void store_pairs(uint32_t to, f2 a, f2 b) {
    asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(to), "l"(a), "l"(b) : "memory");
}
// Eight neighbouring channels of one token, as they lie in memory (XV: two or one 16-byte accesses).
template <class T, bool XV> struct Eight {
    static constexpr int W = 8 * sizeof(T) / 16;
    uint4 v[XV ? W : 1];
    uint32_t e[XV ? 1 : 8];
    __device__ __forceinline__ void load(const T *p, int last) {     // element k past `last` repeats it
        if (XV) {
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] = reinterpret_cast<const uint4 *>(p)[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = load_bits(p + min(k, last));
        }
    }
    // elements k and k + 1, k even
    __device__ __forceinline__ f2 pair(int k) const {
        if (!XV) return pack2(bits_f<T>(e[k]), bits_f<T>(e[k + 1]));
        if (sizeof(T) == 4) return k & 2 ? reinterpret_cast<const f2x2 &>(v[k / 4]).b : reinterpret_cast<const f2x2 &>(v[k / 4]).a;
        const uint32_t u = k == 0 ? v[0].x : k == 2 ? v[0].y : k == 4 ? v[0].z : v[0].w;
        return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};

template <class T, int L, int NS, int KT, int WN, bool XV>
__global__ void __launch_bounds__(4 * WN * KT + 32 * WN) scan_fwd_kernel(ScanParams p, int chan_blocks) {
    using S = FwdTiles<L, NS, KT, WN>;
    constexpr int kFeeders = S::kFeeders;
    auto meet = [] { meet_all<S::kThreads>(); };
    constexpr int NP = S::NP, CW = S::CW, CH = S::CH, TT = S::TT;
    extern __shared__ __align__(128) unsigned char raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const long long slot = blockIdx.x / chan_blocks;
    const int d0 = (int)(blockIdx.x - slot * chan_blocks) * CH;
    Segment g;
    if (!segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    const int tiles = tiles_of(g.len, TT);
    const long long row0 = g.row0 + g.t0;

    if (threadIdx.x >= S::kCarriers) {
        // ------------------------------------------------------------------ feeders
        const int tid = threadIdx.x - S::kCarriers;
        const int t = tid / (CH / 8), c0 = tid % (CH / 8) * 8;       // this thread's token and channels
        const int d = d0 + c0, n = p.D - d;                          // n <= 0: none of them exist
        const bool some = n > 0;
        // Loads into registers take no branch: tokens past the end repeat the last one and channels past
        // the end the last ones, and what comes of them is set to 0 or not stored.  (Where two branches
        // meet, a loaded value is waited for on the spot: 1000 cycles a tile.)
        const int dl = XV ? min(d, p.D - 8) : min(d, p.D - 1), last = p.D - 1 - dl;
        const T *x = static_cast<const T *>(p.x) + row0 * p.ld_x + dl, *delta = static_cast<const T *>(p.delta) + row0 * p.ld_delta + dl;
        const T *z = p.z ? static_cast<const T *>(p.z) + row0 * p.ld_z + dl : nullptr;
        T *y = static_cast<T *>(p.y) + (row0 + t) * p.ld_y + d;
        f2 dbias[4], skip[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = 2 * k;
            dbias[k] = pack2(e < n && p.delta_bias ? p.delta_bias[d + e] : 0.f, e + 1 < n && p.delta_bias ? p.delta_bias[d + e + 1] : 0.f);
            skip[k] = pack2(e < n && p.Dskip ? p.Dskip[d + e] : 0.f, e + 1 < n && p.Dskip ? p.Dskip[d + e + 1] : 0.f);
        }
        // Bm and Cm of a tile: four neighbouring states per access (XV), or elements tid, tid + feeders, ...
        constexpr int EV = (2 * TT * NP / 4 + kFeeders - 1) / kFeeders;
        constexpr int E = TT * NP < kFeeders ? 1 : TT * NP / kFeeders;
        const int bt = tid / NP, bn = tid % NP;                      // NP divides the feeders
        const bool bs = TT * NP >= kFeeders || bt < TT;              // (N <= 8: more threads than elements)
        const int bl = min(bn, p.N - 1);
        const T *const Bp = static_cast<const T *>(p.Bm) + row0 * p.ld_B, *const Cp = static_cast<const T *>(p.Cm) + row0 * p.ld_C;
        constexpr int BT = kFeeders / NP;                            // tokens between a thread's elements
        using Quad = RawQuad<T>;
        // x, delta and z on their way.  XV: asynchronous copies of three tiles, each thread its own
        // eight channels into words of its own, so nobody else waits for them.  Otherwise one tile in registers.
        using Data = Eight<T, XV>;
        constexpr int RING = XV ? 3 : 0;
        uint4 *const ring = reinterpret_cast<uint4 *>(raw + sizeof(S)) + tid;      // [RING][3][W][feeders]
        Data f[XV ? 1 : 3] = {};
        Data xc{}, zc{}, xo{}, zo{};                                 // x and z of the current and the last tile
        uint32_t be[XV ? 1 : E], ce[XV ? 1 : E];                     // the next tile's Bm and Cm
        typename Quad::type bq[XV ? EV : 1];
        const T *const pz = z ? z : x;                               // (no gate: loaded all the same, not used)
        const long long ldz = z ? p.ld_z : p.ld_x, sy = TT * p.ld_y;
        unsigned row = t;                                            // of the next fetch
        int slot3 = 0;                                               // its place in the ring
        auto fetch = [&] {                                           // tile by tile; past the end the last row again
            const long long r = row_or_last(row, g.len);
            const T *px = x + r * p.ld_x, *pd = delta + r * p.ld_delta, *pg = pz + r * ldz;
            if (XV) {
                if (inside(row - t, g.len)) {
                    uint4 *to = ring + slot3 * (3 * Data::W * kFeeders);
#pragma unroll
                    for (int k = 0; k < Data::W; ++k) {
                        copy_async<16>(to + k * kFeeders, px + k * (16 / sizeof(T)));
                        copy_async<16>(to + (Data::W + k) * kFeeders, pd + k * (16 / sizeof(T)));
                        if (z) copy_async<16>(to + (2 * Data::W + k) * kFeeders, pg + k * (16 / sizeof(T)));
                    }
                }
                copies_end();
                slot3 = slot3 == RING - 1 ? 0 : slot3 + 1;
            } else {
                f[0].load(px, last);
                f[XV ? 0 : 1].load(pd, last);
                f[XV ? 0 : 2].load(pg, last);
            }
            row += TT;
        };
        unsigned rowb = 0;
        auto fetch_bc = [&] {
            if constexpr (XV) {
#pragma unroll
                for (int k = 0; k < EV; ++k) {
                    constexpr int PER = TT * NP / 4;                 // quads of Bm, then as many of Cm
                    const int u = min(tid + k * kFeeders, 2 * PER - 1), w = u % PER;
                    const long long r = row_or_last(rowb + w / (NP / 4), g.len);
                    const int n = min(w % (NP / 4) * 4, p.N - 4);
                    bq[k] = *reinterpret_cast<const typename Quad::type *>((u < PER ? Bp + r * p.ld_B : Cp + r * p.ld_C) + n);
                }
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const long long r = row_or_last(rowb + bt + k * BT, g.len);
                    be[k] = load_bits(Bp + r * p.ld_B + bl);
                    ce[k] = load_bits(Cp + r * p.ld_C + bl);
                }
            }
            rowb += TT;
        };
        // Tokens past the end are staged as zeros: their dt x is 0, and an infinity of the last row times 0
        // would turn the final state into NaN.
        auto stage_bc = [&](int tile) {
            const int b = tile & 1;
            if constexpr (XV) {
#pragma unroll
                for (int k = 0; k < EV; ++k) {
                    constexpr int PER = TT * NP / 4;
                    const int u = tid + k * kFeeders, w = u % PER, n = w % (NP / 4) * 4;
                    float4 v = Quad::floats(bq[k]);
                    if (n >= p.N || !inside(tile_token(tile, TT, w / (NP / 4)), g.len)) v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (u < 2 * PER) *reinterpret_cast<float4 *>(&(u < PER ? sm.B : sm.C)[b][w / (NP / 4)][n]) = v;
                }
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    if (!bs) break;
                    const bool real = bn < p.N && inside(tile_token(tile, TT, bt + k * BT), g.len);
                    sm.B[b][bt + k * BT][bn] = real ? bits_f<T>(be[k]) : 0.f;
                    sm.C[b][bt + k * BT][bn] = real ? bits_f<T>(ce[k]) : 0.f;
                }
            }
        };
        // word at(tid 8 + k) = tid 8 + (k ^ (tid & 7)): the address is that of k = 0, exclusive or 16 k
        const uint32_t sd0 = (uint32_t)__cvta_generic_to_shared(&sm.d[0][tid * 8 + (tid & 7)]);
        const uint32_t sd1 = (uint32_t)__cvta_generic_to_shared(&sm.d[1][tid * 8 + (tid & 7)]);
        int from = 0;
        // Stage one tile and finish another.  The two have nothing to do with each other, and there is no
        // branch in either, so their long dependent chains (exponential, sum, reciprocal, ...) overlap.
        // PLAIN: a gate, a softplus and a whole tile, which take no selections.
        auto work_on = [&](auto plain, int staged, int finished, bool store) {
            constexpr bool PLAIN = decltype(plain)::value;
            const uint32_t sd = staged & 1 ? sd1 : sd0;
            Data dc{}, xn{}, zn{};
            if (XV) {
                copies_wait<2>();
                const uint4 *src = ring + from * (3 * Data::W * kFeeders);
#pragma unroll
                for (int k = 0; k < Data::W; ++k) {
                    xn.v[k] = src[k * kFeeders];
                    dc.v[k] = src[(Data::W + k) * kFeeders];
                    zn.v[k] = src[(2 * Data::W + k) * kFeeders];
                }
                from = from == RING - 1 ? 0 : from + 1;
            } else {
                xn = f[0];
                dc = f[XV ? 0 : 1];
                zn = f[XV ? 0 : 2];
            }
            const f2x2 *src = reinterpret_cast<const f2x2 *>(&sm.y[finished & 1][t][c0]);
            const f2x2 ya = src[0], yb = src[1];
            f2 o[4] = {ya.a, ya.b, yb.a, yb.b};
            const bool in = inside(tile_token(staged, TT, t), g.len);                 // behind the end the state stays as it is
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                f2 dt = add2(dc.pair(k), dbias[k / 2]);
                const f2 sp = softplus2(dt);
                dt = PLAIN || p.softplus ? sp : dt;
                o[k / 2] = fma2(skip[k / 2], xo.pair(k), o[k / 2]);
                const f2 gated = mul2(o[k / 2], silu2(zo.pair(k)));
                o[k / 2] = PLAIN || z ? gated : o[k / 2];
                float lo, hi, ul, uh;
                unpack2(dt, lo, hi);
                unpack2(mul2(dt, xn.pair(k)), ul, uh);
                if (!PLAIN) {
                    lo = in ? lo : 0.f;
                    hi = in ? hi : 0.f;
                    ul = in ? ul : 0.f;
                    uh = in ? uh : 0.f;
                }
                store_pairs(sd ^ 16 * k, both(lo), both(ul));
                store_pairs(sd ^ 16 * (k + 1), both(hi), both(uh));
            }
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) unpack2(o[k], v[2 * k], v[2 * k + 1]);
            if (XV) {
#pragma unroll
                for (int k = 0; k < 8; k += 16 / (int)sizeof(T)) {
                    Vec<T, 16 / sizeof(T)> q;
#pragma unroll
                    for (int e = 0; e < 16 / (int)sizeof(T); ++e) q.e[e] = from_f<T>(v[k + e]);
                    if (store) store_vec<T, 16 / sizeof(T)>(y + k, q);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (store && k < n) y[k] = from_f<T>(v[k]);
            }
            xo = xc;
            zo = zc;
            xc = xn;
            zc = zn;
        };
        auto work = [&](int staged, int finished, bool store) {
            if (z && p.softplus && inside(tile_token(staged, TT, TT - 1), g.len)) work_on(std::true_type{}, staged, finished, store);
            else work_on(std::false_type{}, staged, finished, store);
        };
        if (tiles > 0) {
            fetch_bc();
            fetch();
            if (XV) {
                fetch();
                fetch();
            }
            stage_bc(0);
            fetch_bc();
            work(0, 0, false);
            fetch();
        }
        for (int tile = 0; tile < tiles; ++tile) {
            meet();                              // tile staged; tile - 1 carried
            stage_bc(tile + 1);                  // (past the last tile: read by nobody)
            fetch_bc();
            work(tile + 1, tile - 1, tile > 0 && some && inside(tile_token(tile - 1, TT, t), g.len));
            fetch();
            if (tile > 0) y += sy;
        }
        meet();
        if (tiles > 0) work(tiles + 1, tiles - 1, some && inside(tile_token(tiles - 1, TT, t), g.len));
        if (XV) copies_wait<0>();
        return;
    }
    // ---------------------------------------------------------------------- carriers
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane / L, i = lane % L, n0 = NS * i;
    const int d = d0 + warp * CW + c;
    const bool live = d < p.D;
    constexpr int H = NS / 2;
    f2 a2[H], h[H];
    {
        float av[NS], hv[NS];
#pragma unroll
        for (int k = 0; k < NS; ++k) av[k] = hv[k] = 0.f;
        if (live) {
            load_states(av, p.A + (long long)d * p.N, n0, p.N);
            if (p.seg_state)
                load_states(hv, p.seg_state + (slot_at(p.cu_seqlens, p.T, p.lseg, g.b, g.t0) * p.D + d) * NP, n0, NP);
            else if (p.h0) load_states(hv, p.h0 + ((long long)g.b * p.D + d) * p.N, n0, p.N);
        }
#pragma unroll
        for (int k = 0; k < H; ++k) {
            a2[k] = pack2(decay_rate(av[2 * k]), decay_rate(av[2 * k + 1]));
            h[k] = pack2(hv[2 * k], hv[2 * k + 1]);
        }
    }
    // the swizzle's period in tokens: at() sees t CH / 8 modulo 8
    constexpr int P = CH >= 64 ? 1 : 64 / CH;
    int off[P];
#pragma unroll
    for (int k = 0; k < P; ++k) off[k] = S::at(k * CH + warp * CW + c) - k * CH;
    for (int tile = 0; tile < tiles; ++tile) {
        meet();
        const int b = tile & 1;
        const f2x2 *sd = sm.d[b];
        // L tokens at a time, in three stages that overlap: the shared-memory loads of group j + 2, the
        // decays and inputs of group j + 1 (which do not wait for the state), the recurrence of group j.
        // A pair of states costs two exponentials (8 cycles of the special-function pipe) and four packed
        // FMAs (8 cycles of theirs); they are written, and kept by `volatile`, in the order that feeds both
        // pipes at once.  No branch in here: the whole tile is one block to schedule.
        constexpr int G = KT;                  // groups of L tokens
        f2x2 sv[L], bv[L][H / 2], cv[2][L][H / 2];
        f2 e[2][L][H], u[2][L][H];
        auto load = [&](int j) {               // raw operands of group j
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const int t = j * L + k;
                sv[k] = sd[t * CH + off[t % P]];
#pragma unroll
                for (int q = 0; q < H / 2; ++q) {
                    bv[k][q] = *reinterpret_cast<const f2x2 *>(&sm.B[b][t][n0 + 4 * q]);
                    cv[j & 1][k][q] = *reinterpret_cast<const f2x2 *>(&sm.C[b][t][n0 + 4 * q]);
                }
            }
        };
        auto half = [](const f2x2 &v, int q) { return q & 1 ? v.b : v.a; };
        load(0);
#pragma unroll
        for (int k = 0; k < L; ++k)
#pragma unroll
            for (int q = 0; q < H; ++q) {
                e[0][k][q] = decay2(sv[k].a, a2[q]);
                u[0][k][q] = mul2(sv[k].b, half(bv[k][q / 2], q));
            }
        load(1);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int x = j & 1, y = x ^ 1;
            if (j + 1 < G)
#pragma unroll
                for (int k = 0; k < L; ++k)
#pragma unroll
                    for (int q = 0; q < H; ++q) {
                        e[y][k][q] = fma2v(sv[k].a, a2[q], both(kDecayBias));
                        u[y][k][q] = mul2v(sv[k].b, half(bv[k][q / 2], q));
                    }
            float ys[L];
            f2x2 cj[L][H / 2];
#pragma unroll
            for (int k = 0; k < L; ++k)
#pragma unroll
                for (int q = 0; q < H / 2; ++q) cj[k][q] = cv[x][k][q];
            if (j + 2 < G) load(j + 2);
#pragma unroll
            for (int k = 0; k < L; ++k) {
                f2 acc;
#pragma unroll
                for (int q = 0; q < H; ++q) {
                    if (j + 1 < G) e[y][k][q] = ex2_2v(e[y][k][q]);
                    h[q] = fma2v(e[x][k][q], h[q], u[x][k][q]);
                    acc = q ? fma2v(h[q], half(cj[k][q / 2], q), acc) : mul2v(h[q], half(cj[k][q / 2], q));
                }
                float lo, hi;
                unpack2(acc, lo, hi);
                ys[k] = lo + hi;
            }
            spread_sum<L, L>(ys, i);
            sm.y[b][j * L + i][warp * CW + c] = ys[0];
        }
    }
    meet();
    if (p.ht && live && g.i == g.n - 1) {
        float hv[NS];
#pragma unroll
        for (int k = 0; k < H; ++k) unpack2(h[k], hv[2 * k], hv[2 * k + 1]);
        store_states(p.ht + ((long long)g.b * p.D + d) * p.N, hv, n0, p.N);
    }
}

// The same for one token of each request; the state is read, updated and written once: bound by HBM.
// VEC: N = 4 L, state, A, Bm and Cm in accesses of four.
template <class T, int L, bool VEC>
__global__ void __launch_bounds__(kScanThreads) scan_step_kernel(ScanParams p) {
    constexpr int CH = kScanThreads / L;
    const int c = threadIdx.x / L, i = threadIdx.x % L, n0 = 4 * i;
    const int b = blockIdx.x, d = blockIdx.y * CH + c;
    const int slot = p.slot ? p.slot[b] : b;
    const bool pad = slot < 0 || slot >= p.slots, live = d < p.D && !pad;
    float y = 0.f, xv = 0.f, zv = 0.f, skip = 0.f;
    if (live) {
        float h[4], a[4], bv[4], cv[4];
        float *st = p.state + ((long long)slot * p.D + d) * p.N;
        const float *ar = p.A + (long long)d * p.N;
        const T *br = static_cast<const T *>(p.Bm) + b * p.ld_B, *cr = static_cast<const T *>(p.Cm) + b * p.ld_C;
        if (VEC) {
            const float4 hq = *reinterpret_cast<const float4 *>(st + n0), aq = __ldg(reinterpret_cast<const float4 *>(ar + n0));
            const float4 bq = RawQuad<T>::floats(__ldg(reinterpret_cast<const typename RawQuad<T>::type *>(br + n0)));
            const float4 cq = RawQuad<T>::floats(__ldg(reinterpret_cast<const typename RawQuad<T>::type *>(cr + n0)));
            h[0] = hq.x; h[1] = hq.y; h[2] = hq.z; h[3] = hq.w;
            a[0] = aq.x; a[1] = aq.y; a[2] = aq.z; a[3] = aq.w;
            bv[0] = bq.x; bv[1] = bq.y; bv[2] = bq.z; bv[3] = bq.w;
            cv[0] = cq.x; cv[1] = cq.y; cv[2] = cq.z; cv[3] = cq.w;
        } else {
            load_states(h, st, n0, p.N);
            load_states(a, ar, n0, p.N);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bv[k] = n0 + k < p.N ? to_f(br[n0 + k]) : 0.f;
                cv[k] = n0 + k < p.N ? to_f(cr[n0 + k]) : 0.f;
            }
        }
        xv = bits_f<T>(load_bits(static_cast<const T *>(p.x) + b * p.ld_x + d));
        if (p.z) zv = bits_f<T>(load_bits(static_cast<const T *>(p.z) + b * p.ld_z + d));
        if (p.Dskip) skip = __ldg(p.Dskip + d);
        float dt = bits_f<T>(load_bits(static_cast<const T *>(p.delta) + b * p.ld_delta + d));
        if (p.delta_bias) dt += __ldg(p.delta_bias + d);
        if (p.softplus) dt = softplus(dt);
        const float e = dt * kLog2e, u = dt * xv;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = fmaf(ex2(fmaf(e, a[k], kDecayBias)), h[k], u * bv[k]);
            y = fmaf(cv[k], h[k], y);
        }
        if (VEC) *reinterpret_cast<float4 *>(st + n0) = make_float4(h[0], h[1], h[2], h[3]);
        else store_states(st, h, n0, p.N);
    }
#pragma unroll
    for (int s = L / 2; s; s >>= 1) y += __shfl_xor_sync(~0u, y, s);
    if (d < p.D && i == 0) {
        y = fmaf(skip, xv, y);
        if (p.z) y *= zv * sigmoid(zv);
        static_cast<T *>(p.y)[b * p.ld_y + d] = from_f<T>(pad ? 0.f : y);
    }
}

template <class T, int L, int NS, int KT, int WN, bool XV> cudaError_t fwd_start(const ScanParams &p, cudaStream_t s) {
    using S = FwdTiles<L, NS, KT, WN>;
    const int cb = (p.D + S::CH - 1) / S::CH;
    const long long blocks = scan_slots(p, p.seg) * cb;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    constexpr int smem = sizeof(S) + (XV ? 3 * 3 * Eight<T, XV>::W * 16 * S::kFeeders : 0);
    const cudaError_t e =
        cudaFuncSetAttribute(scan_fwd_kernel<T, L, NS, KT, WN, XV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    scan_fwd_kernel<T, L, NS, KT, WN, XV><<<(unsigned)blocks, S::kThreads, smem, s>>>(p, cb);
    return cudaGetLastError();
}

// 16-byte accesses to x, delta, z and y, and four states of Bm and Cm at a time, where all of them allow it.
bool fwd_xv(const ScanParams &p, size_t es) {
    return p.D % 8 == 0 && rows_aligned(p.x, p.ld_x, es, 16) && rows_aligned(p.delta, p.ld_delta, es, 16) &&
           rows_aligned(p.z, p.ld_z, es, 16) && rows_aligned(p.y, p.ld_y, es, 16) && p.N % 4 == 0 &&
           rows_aligned(p.Bm, p.ld_B, es, 4 * es) && rows_aligned(p.Cm, p.ld_C, es, 4 * es);
}
template <class T, int L, int NS, int KT, int WN> cudaError_t fwd_warps(const ScanParams &p, cudaStream_t s) {
    return fwd_xv(p, sizeof(T)) ? fwd_start<T, L, NS, KT, WN, true>(p, s) : fwd_start<T, L, NS, KT, WN, false>(p, s);
}
// Half as many carrier warps to a block where full blocks would leave half of the SMs without one: the same
// work on twice the SMs (training step B 2, T 2048, D 2048, both with eight states per lane: 382 -> 368 us).
template <class T, int L, int NS, int KT, int WN> cudaError_t fwd_launch(const ScanParams &p, cudaStream_t s) {
    constexpr int CH = WN * 32 / L;
    const long long full = scan_slots(p, p.seg) * ((p.D + CH - 1) / CH);
    return 2 * full <= sm_count() ? fwd_warps<T, L, NS, KT, WN / 2>(p, s) : fwd_warps<T, L, NS, KT, WN>(p, s);
}

template <class T, int L> cudaError_t step_launch(const ScanParams &p, cudaStream_t s) {
    constexpr int CH = kScanThreads / L;
    const int cb = (p.D + CH - 1) / CH;
    if (cb > 65535) return cudaErrorNotSupported;
    const dim3 grid(p.B, cb);
    if (bc_vec_ok<T>(p, 4 * L) && aligned_to(p.state, 16) && aligned_to(p.A, 16))
        scan_step_kernel<T, L, true><<<grid, kScanThreads, 0, s>>>(p);
    else
        scan_step_kernel<T, L, false><<<grid, kScanThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T> cudaError_t fwd_type(const ScanParams &p, cudaStream_t s) {
    if (p.N <= 4) return fwd_launch<T, 1, 4, 16, 4>(p, s);
    if (p.N <= 8) return fwd_launch<T, 1, 8, 16, 4>(p, s);
    if (p.N <= 16) {
        // Where half-sized blocks are taken (fwd_launch), four states per lane in twice as many carrier warps are
        // shorter per token in bfloat16 with vector accesses: 12.6 us for 14.6 at T 256, 70 for 82 at T 2048, 528 for 619 at
        // T 16384, from D 64 to B 4, D 1216.  Single elements (N 9: 109 for 99 at T 2048, 1037 for 877 at T 16384) and
        // float32 (14.6 for 15.5 at T 256, 81 for 82, 616 for 615; D 1000: 86 for 84) are not, and do not take them.
        const long long full = scan_slots(p, p.seg) * ((p.D + 63) / 64);
        if constexpr (sizeof(T) == 2)
            if (2 * full <= sm_count() && fwd_xv(p, sizeof(T))) return fwd_start<T, 4, 4, 8, 4, true>(p, s);
        return fwd_launch<T, 2, 8, 16, 4>(p, s);
    }
    return fwd_launch<T, 4, 8, 16, 4>(p, s);
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

// Whole sequences, or segments of them side by side where that is sooner done.  Measured, by type and states of a
// channel (up to 4, 8, 16, 32): ns that a token takes a block where half-sized (or four-state) blocks are taken and
// where full ones are (fwd_launch, fwd_type), and ps that the local pass over all tokens takes per token and channel
// with every SM busy.  Two more launches and the latencies of the local and boundary passes come to 18 us, 4 of
// which a whole sequence has too.  Both forms, us, at the sizes where two or four segments fit:
//                     bfloat16                              float32
//   N 8    B 2 D 2048 T 4096    whole 179, split 127    whole 185, split 158
//          B 4 D 2048 T 16384   whole 698, split 896    whole 732, split 1100
//   N 16   B 1 D 2048 T 4096    whole 135, split  88    whole 158, split 111
//          B 2 D 2048 T 4096    whole 136, split 162    whole 160, split 205
//   N 32   B 1 D 1024 T 2048    whole 101, split  60    whole 102, split  64
//          B 1 D 2048 T 16384   whole 866, split 672    whole 851, split 756
// Over 168 such sizes of each type the choice takes 0.2 % more than the better form of each on average and at
// most 14 % (of 30 us); over 108 of each with accesses of single elements 0.7 % and at most 13 %.  The lengths of packed sequences are not known here: one of them may have nearly all tokens.
struct ScanCost {
    double half, full, local;
};
constexpr ScanCost kScanCost[2][4] = {{{42.5, 67, 1.9}, {43, 69, 2.35}, {32.5, 44.5, 3.35}, {55, 52, 6.7}},
                                      {{68, 95, 2.1}, {44.5, 93.5, 2.4}, {38, 61, 3.5}, {55, 63, 6.9}}};

int ssm_scan_fwd_segment(const ScanParams &p, bool bf) {
    const int ch = p.N <= 8 ? 128 : p.N <= 16 ? 64 : 32;
    const long long cb = (p.D + ch - 1) / ch, batch = p.cu_seqlens ? 1 : p.B, sms = sm_count();
    const long long cuts = sms / (cb * batch);
    if (cuts < 2) return p.T;
    long long seg = (p.T + cuts - 1) / cuts;
    seg = (seg + kFwdLocal - 1) / kFwdLocal * kFwdLocal;
    if (seg < 256) seg = 256;
    if (seg >= p.T) return p.T;
    const ScanCost &c = kScanCost[bf ? 0 : 1][p.N <= 4 ? 0 : p.N <= 8 ? 1 : p.N <= 16 ? 2 : 3];
    auto walk = [&](int tokens) { return (2 * scan_slots(p, tokens) * cb <= sms ? c.half : c.full) * tokens; };
    const double whole = 4000.0 + walk(p.T), split = 18000.0 + walk((int)seg) + 1e-3 * c.local * (double)batch * p.T * p.D;
    return split < whole ? (int)seg : p.T;
}

size_t ssm_scan_fwd_floats(const ScanParams &p, bool bf) {
    if (ssm_scan_fwd_segment(p, bf) >= p.T) return 0;
    return (size_t)scan_slots(p, kFwdLocal) * p.D * (padded_states(p.N) + 1);
}

void ssm_scan_fwd_carve(ScanParams &p, float *ws) {
    p.lseg = kFwdLocal;
    p.seg_state = ws;
    p.seg_dt = ws + (size_t)scan_slots(p, kFwdLocal) * p.D * padded_states(p.N);
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
