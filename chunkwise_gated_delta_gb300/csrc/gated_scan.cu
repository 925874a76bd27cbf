// Gated recurrence (one state per channel), forward, backward and single tokens.
//
// All rows of a chain of sequences form one axis.  Tiles of it, 64 rows by 64 channels, go to the blocks of a cluster in
// turn; the next tile is on its way to shared memory while one is worked on.  Of a tile every warp has 8 neighbouring
// rows and a lane two channels.  A warp reduces its rows to h_out = h + A h_in, the block's warps and then the cluster's
// blocks exchange these pairs through shared memory, and each warp walks its rows again from the state that enters them.
// So every tensor is read once and written once, whatever the sequences' lengths, and the order of the sums is
// fixed.  Where a sequence begins inside a tile the link is cut by selection (never by a product with 0: a state
// of an earlier sequence may be an infinity).
//
// The backward runs the same walk from the end, with G_t = dy_t + a_{t+1} G_{t+1}; the states that enter its
// tiles are the forward's, saved every 64 rows in float32 (3 % of one bfloat16 tensor), so that it too reads each tensor once.
#include "gated_scan.cuh"
#include "tc_common.cuh"

namespace mixer {
namespace {

using namespace gs;

constexpr int MAX_CLUSTER = 8;

// ------------------------------------------------------------------------------------------ exchange
// 16 bytes, and a word, into the same place of another block's shared memory.
__device__ __forceinline__ void store_remote(const float4 *at, unsigned rank, float4 v) {
    const uint32_t a = kda::tc::map_to_rank((uint32_t)__cvta_generic_to_shared(at), rank);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void store_remote(const int *at, unsigned rank, int v) {
    const uint32_t a = kda::tc::map_to_rank((uint32_t)__cvta_generic_to_shared(at), rank);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive_release() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void sync_rows() { asm volatile("bar.sync 1, %0;" ::"n"(LANES) : "memory"); }
// All N threads of the block; whether the predicate holds in any of them.
template <int N> __device__ __forceinline__ bool sync_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "n"(N) : "memory");
    return r != 0;
}
__device__ __forceinline__ float4 quad(f2 a, f2 b) {
    float4 r;
    unpack2(a, r.x, r.y);
    unpack2(b, r.z, r.w);
    return r;
}

// What the warps of a block and the blocks of a cluster tell each other of a tile, in two sets that take turns:
// h_out = h + A h_in of their rows (A, h), or h_out = h alone where the link is cut (a sequence begins; ends, in the backward).
struct Exchange {
    float4 warp[2][WARPS][32];
    float4 block[2][MAX_CLUSTER][32];
    int warp_cut[2][WARPS], block_cut[2][MAX_CLUSTER];
};
// h_out of the rows that (A, h) stand for.
__device__ __forceinline__ f2 through(float4 g, f2 h) { return fma2(pack2(g.x, g.y), h, pack2(g.z, g.w)); }
__device__ __forceinline__ f2 through(float4 g, bool cut, f2 h) { return cut ? pack2(g.z, g.w) : through(g, h); }

// The state (or its gradient) that enters this warp's rows, and the one that leaves the cluster's tiles (carry).
// REV: warps and blocks count from the last row.  prod, out: this warp's pair.
template <bool REV, bool CLUSTER>
__device__ __forceinline__ f2 enter(Exchange &ex, int buf, int warp, int lane, unsigned rank, int blocks, f2 prod, f2 out, bool cut,
                                    f2 &carry) {
    ex.warp[buf][warp][lane] = quad(prod, out);
    if (lane == 0) ex.warp_cut[buf][warp] = cut;
    const bool any = sync_any<LANES + (CLUSTER ? 32 : 0)>(cut);
    if constexpr (!CLUSTER) {
        f2 mine = carry;
        if (!any) {
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const int k = REV ? WARPS - 1 - i : i;
                if (k == warp) mine = carry;
                carry = through(ex.warp[buf][k][lane], carry);
            }
        } else {
            for (int i = 0; i < WARPS; ++i) {
                const int k = REV ? WARPS - 1 - i : i;
                if (k == warp) mine = carry;
                carry = through(ex.warp[buf][k][lane], ex.warp_cut[buf][k], carry);
            }
        }
        return mine;
    }
    cluster_arrive_relaxed();            // (the warp that writes to other blocks releases)
    // the pair of the warps before this one
    f2 ma = both(1.f), mh = both(0.f);
    bool mc = false;
    const int before = REV ? WARPS - 1 - warp : warp;
    for (int i = 0; i < before; ++i) {
        const int k = REV ? WARPS - 1 - i : i;
        const float4 g = ex.warp[buf][k][lane];
        const bool c = any && ex.warp_cut[buf][k];
        mh = i == 0 ? pack2(g.z, g.w) : through(g, c, mh);
        ma = mul2(ma, pack2(g.x, g.y));
        mc |= c;
    }
    cluster_wait();
    f2 into = carry;
    for (int i = 0; i < blocks; ++i) {
        const int k = REV ? blocks - 1 - i : i;
        if (k == (int)rank) into = carry;
        carry = through(ex.block[buf][k][lane], ex.block_cut[buf][k], carry);
    }
    return before == 0 ? into : mc ? mh : fma2(ma, into, mh);
}

// The warp that tells the other blocks of a cluster what a tile of this one does to a state.  A warp of its own, for its release
// must not wait for rows that the others are still storing.
template <bool REV> __device__ __forceinline__ void exchange_warp(Exchange &ex, int turns, int lane, unsigned rank, int blocks) {
    for (int i = 0; i < turns; ++i) {
        const int buf = i & 1;
        const bool any = sync_any<LANES + 32>(false);
        f2 pa = both(1.f), ph = both(0.f);
        bool pc = false;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int k = REV ? WARPS - 1 - w : w;
            const float4 g = ex.warp[buf][k][lane];
            const bool c = any && ex.warp_cut[buf][k];
            ph = w == 0 ? pack2(g.z, g.w) : through(g, c, ph);
            pa = mul2(pa, pack2(g.x, g.y));
            pc |= c;
        }
        for (int b = 0; b < blocks; ++b) store_remote(&ex.block[buf][rank][lane], b, quad(pa, ph));
        if (lane < blocks) store_remote(&ex.block_cut[buf][rank], lane, (int)pc);
        cluster_arrive_release();
        cluster_wait();
    }
}

// Where a block works.
struct Where {
    int warp, lane, blocks, c0, c, cl;   // c: this lane's first channel, cl: the same or, of idle lanes, one inside
    unsigned rank;
    bool on;
    Chain k;
    long long tile0;
    int turns;
};
__device__ __forceinline__ Where where(const GatedScanParams &p) {
    Where w;
    w.warp = threadIdx.x >> 5;
    w.lane = threadIdx.x & 31;
    w.blocks = p.cluster;
    w.rank = blockIdx.x % (unsigned)p.cluster;
    w.c0 = (int)(blockIdx.x / (unsigned)p.cluster) * COLS;
    w.c = w.c0 + w.lane * 2;
    w.on = w.c < p.D;
    w.cl = w.on ? w.c : w.c0;
    w.k = chain_of(p.cu_seqlens, p.B, p.T, p.chains, blockIdx.y);
    w.tile0 = w.k.c0 / TILE;
    const long long tiles = ((long long)w.k.c1 + TILE - 1) / TILE - w.tile0;
    w.turns = (int)((tiles + w.blocks - 1) / w.blocks);
    return w;
}

// ------------------------------------------------------------------------------------------ forward
template <class T, int CP, bool CLUSTER>
__global__ void __launch_bounds__(LANES + (CLUSTER ? 32 : 0), sizeof(T) == 2 ? 3 : 2) gated_scan_fwd_kernel(GatedScanParams p) {
    using S = Stage<T, CP>;
    constexpr bool VEC = CP > (int)sizeof(T);
    extern __shared__ __align__(16) char stages[];   // [2][3][S::BYTES]
    __shared__ Exchange ex;
    const Where w = where(p);
    const Chain &k = w.k;
    const int warp = w.warp, lane = w.lane, c = w.c, D = p.D;
    if (p.cu_seqlens && p.ht && w.rank == 0 && w.on && warp < WARPS)   // empty sequences: the state passes through
        for (int s = k.s0 + warp; s < k.s1; s += WARPS) {
            const int lo = clamped(p.cu_seqlens[s], 0, p.T), hi = clamped(p.cu_seqlens[s + 1], lo, p.T);
            if (lo == hi) store_state(p.ht + (long long)s * D, c, D, p.h0 ? load_state(p.h0 + (long long)s * D, c, D) : both(0.f));
        }
    if (k.c0 >= k.c1) return;                        // (the whole cluster)
    if constexpr (CLUSTER) {
        kda::tc::cluster_sync_all();                 // every block has begun: its shared memory may be written
        if (warp == WARPS) {
            exchange_warp<false>(ex, w.turns, lane, w.rank, w.blocks);
            return;
        }
    }
    const f2 coef = coefficients(p, w.cl);
    auto bring = [&](int buf, long long r0) {
        char *to = stages + buf * 3 * S::BYTES;
        S::bring(to, static_cast<const T *>(p.x), p.ld_x, w.c0, D, r0, k.c0, k.c1);
        S::bring(to + S::BYTES, static_cast<const T *>(p.decay), p.ld_decay, w.c0, D, r0, k.c0, k.c1);
        S::bring(to + 2 * S::BYTES, static_cast<const T *>(p.gate), p.ld_gate, w.c0, D, r0, k.c0, k.c1);
        copies_end();
    };
    long long t0 = (w.tile0 + w.rank) * TILE;        // the tile's first row
    bring(0, t0);
    Marks marks;
    f2 carry = both(0.f);
    for (int i = 0; i < w.turns; ++i, t0 += (long long)w.blocks * TILE) {
        copies_wait<0>();
        sync_rows();                                 // the tile is there, the one before has been read
        if (i + 1 < w.turns) bring(i + 1 & 1, t0 + (long long)w.blocks * TILE);
        const char *sx = stages + (i & 1) * 3 * S::BYTES + warp * ROWS * S::ROW, *sd = sx + S::BYTES, *sg = sd + S::BYTES;
        const long long r0 = t0 + warp * ROWS;
        f2 a[ROWS], v[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) a[j] = mul2(coef, sigmoid2(S::pair(sd, j, lane)));
        one_less_exps(a);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const f2 q = a[j];
            a[j] = decay_of(q);
            v[j] = mul2(mul2(sqrt2(rest_of(q, a[j])), sigmoid2(S::pair(sg, j, lane))), S::pair(sx, j, lane));
        }
        marks.find(p, k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        f2 h = v[0], prod = a[0];
        if (starts == 0) {
#pragma unroll
            for (int j = 1; j < ROWS; ++j) {
                h = fma2(a[j], h, v[j]);
                prod = mul2(prod, a[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (starts >> j & 1) {
                    h = p.h0 ? fma2(a[j], load_state(p.h0 + (long long)marks.sequence(j) * D, w.cl, D), v[j]) : v[j];
                    v[j] = h;                        // the walk below begins here anew
                } else if (j) {
                    h = fma2(a[j], h, v[j]);
                }
                if (j) prod = mul2(prod, a[j]);
            }
        }
        h = enter<false, CLUSTER>(ex, i & 1, warp, lane, w.rank, w.blocks, prod, h, starts != 0, carry);
        if (p.states && warp == 0 && r0 >= k.c0 && r0 < k.c1 && w.on) store_state(p.states + r0 / SAVE * D, c, D, h);
        if ((starts | ends) == 0 && r0 >= k.c0 && r0 + ROWS <= k.c1) {
            if (p.y == nullptr) continue;            // (the states alone)
            T *y = static_cast<T *>(p.y) + r0 * p.ld_y;
#pragma unroll
            for (int j = 0; j < ROWS; ++j, y += p.ld_y) {
                h = fma2(a[j], h, v[j]);
                if (w.on) store_pair<T, VEC>(y, c, D, h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                h = starts >> j & 1 ? v[j] : fma2(a[j], h, v[j]);
                const long long r = r0 + j;
                if (w.on && r >= k.c0 && r < k.c1 && p.y) store_pair<T, VEC>(static_cast<T *>(p.y) + r * p.ld_y, c, D, h);
                if (ends >> j & 1) {
                    const int s = marks.sequence(j);
                    if (p.ht && w.on) store_state(p.ht + (long long)s * D, c, D, h);
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------------ backward
// With q the exponent, s and u the two sigmoids, v = u x and G_t the gradient of h_t:
//     dq = G (v a^2 / m - a h_{t-1}),  ddecay = dq q (1 - s),  drate = scale sigmoid(rate) sum dq s,
//     dx = G m u,  dgate = G m x u (1 - u),  dh0 = a G of the first token.
// The first walk keeps 1 - a, m v and dy in registers; the second takes the inputs from shared memory once more.
template <class T, int CP, bool CLUSTER>
__global__ void __launch_bounds__(LANES + (CLUSTER ? 32 : 0), sizeof(T) == 2 ? 2 : 1) gated_scan_bwd_kernel(GatedScanParams p) {
    using S = Stage<T, CP>;
    constexpr bool VEC = CP > (int)sizeof(T);
    extern __shared__ __align__(16) char stages[];   // [2][4][S::BYTES]
    __shared__ Exchange ex;
    __shared__ float4 fwd[2][WARPS][32];             // (A, h) of the warps' rows, first to last
    __shared__ int fwd_cut[2][WARPS];
    const Where w = where(p);
    const Chain &k = w.k;
    const int warp = w.warp, lane = w.lane, c = w.c, D = p.D;
    float *part = p.part + ((long long)blockIdx.y * w.blocks + w.rank) * D;
    if (p.cu_seqlens && p.dh0 && w.rank == 0 && w.on && warp < WARPS)  // empty sequences hand the gradient through
        for (int s = k.s0 + warp; s < k.s1; s += WARPS) {
            const int lo = clamped(p.cu_seqlens[s], 0, p.T), hi = clamped(p.cu_seqlens[s + 1], lo, p.T);
            if (lo == hi) store_state(p.dh0 + (long long)s * D, c, D, p.dht ? load_state(p.dht + (long long)s * D, c, D) : both(0.f));
        }
    if (k.c0 >= k.c1) {                              // (the whole cluster)
        if (warp == 0 && w.on) store_state(part, c, D, both(0.f));
        return;
    }
    if constexpr (CLUSTER) {
        kda::tc::cluster_sync_all();                 // every block has begun: its shared memory may be written
        if (warp == WARPS) {
            exchange_warp<true>(ex, w.turns, lane, w.rank, w.blocks);
            return;
        }
    }
    const f2 coef = coefficients(p, w.cl), minus = both(-1.f), one = both(1.f);
    auto bring = [&](int buf, long long r0) {
        char *to = stages + buf * 4 * S::BYTES;
        S::bring(to, static_cast<const T *>(p.x), p.ld_x, w.c0, D, r0, k.c0, k.c1);
        S::bring(to + S::BYTES, static_cast<const T *>(p.decay), p.ld_decay, w.c0, D, r0, k.c0, k.c1);
        S::bring(to + 2 * S::BYTES, static_cast<const T *>(p.gate), p.ld_gate, w.c0, D, r0, k.c0, k.c1);
        S::bring(to + 3 * S::BYTES, static_cast<const T *>(p.dy), p.ld_dy, w.c0, D, r0, k.c0, k.c1);
        copies_end();
    };
    // The state that enters a tile (one that begins outside the chain has none and needs none).
    auto saved_at = [&](long long top) {
        return top >= k.c0 && top < k.c1 ? load_state(p.states + top / SAVE * D, w.cl, D) : both(0.f);
    };
    // The cluster's tiles of a turn are neighbours, the last block's the last; turns go from the end.
    const long long step = (long long)w.blocks * TILE;
    long long t0 = (w.tile0 + (long long)(w.turns - 1) * w.blocks + w.rank) * TILE;
    bring(0, t0);
    f2 saved = saved_at(t0);
    Marks marks;
    f2 carry = both(0.f), sum = both(0.f);
    for (int i = 0; i < w.turns; ++i, t0 -= step) {
        copies_wait<0>();
        sync_rows();                                 // the tile is there, the one before has been read
        f2 h = saved;
        if (i + 1 < w.turns) {
            bring(i + 1 & 1, t0 - step);
            saved = saved_at(t0 - step);
        }
        const char *sx = stages + (i & 1) * 4 * S::BYTES + warp * ROWS * S::ROW, *sd = sx + S::BYTES, *sg = sd + S::BYTES, *sy = sg + S::BYTES;
        const long long r0 = t0 + warp * ROWS;
        f2 q[ROWS], v[ROWS], gy[ROWS];               // 1 - a; m u x, then the state before each row; dy
#pragma unroll
        for (int j = 0; j < ROWS; ++j) q[j] = mul2(coef, sigmoid2(S::pair(sd, j, lane)));
        one_less_exps(q);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            v[j] = mul2(mul2(sqrt2(rest_of(q[j], decay_of(q[j]))), sigmoid2(S::pair(sg, j, lane))), S::pair(sx, j, lane));
            gy[j] = S::pair(sy, j, lane);
        }
        marks.find(p, k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        // both walks over this warp's rows alone: the states from 0, the gradients from 0
        f2 hw = v[0], prod = decay_of(q[0]), gw = mul2(decay_of(q[ROWS - 1]), gy[ROWS - 1]);
        if ((starts | ends) == 0) {
#pragma unroll
            for (int j = 1; j < ROWS; ++j) {
                const f2 a = decay_of(q[j]);
                hw = fma2(a, hw, v[j]);
                prod = mul2(prod, a);
            }
#pragma unroll
            for (int j = ROWS - 2; j >= 0; --j) gw = mul2(decay_of(q[j]), add2(gy[j], gw));
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const f2 a = decay_of(q[j]);
                if (starts >> j & 1) hw = p.h0 ? fma2(a, load_state(p.h0 + (long long)marks.sequence(j) * D, w.cl, D), v[j]) : v[j];
                else if (j) hw = fma2(a, hw, v[j]);
                if (j) prod = mul2(prod, a);
            }
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j) {
                const f2 a = decay_of(q[j]);
                if (ends >> j & 1) {
                    const f2 g = p.dht ? load_state(p.dht + (long long)marks.sequence(j) * D, w.cl, D) : both(0.f);
                    gy[j] = add2(gy[j], g);          // the walk below begins here anew
                    gw = mul2(a, gy[j]);
                } else if (j < ROWS - 1) {
                    gw = mul2(a, add2(gy[j], gw));
                }
            }
        }
        fwd[i & 1][warp][lane] = quad(prod, hw);
        if (lane == 0) fwd_cut[i & 1][warp] = starts != 0;
        f2 grad = enter<true, CLUSTER>(ex, i & 1, warp, lane, w.rank, w.blocks, prod, gw, ends != 0, carry);
        for (int b = 0; b < warp; ++b) h = through(fwd[i & 1][b][lane], fwd_cut[i & 1][b], h);
        // the state before each row takes the place of its input
        if (starts == 0) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const f2 t = v[j];
                v[j] = h;
                h = fma2(decay_of(q[j]), h, t);
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (starts >> j & 1) h = p.h0 ? load_state(p.h0 + (long long)marks.sequence(j) * D, w.cl, D) : both(0.f);
                const f2 t = v[j];
                v[j] = h;
                h = fma2(decay_of(q[j]), h, t);
            }
        }
        auto row = [&](int j, f2 G, f2 aG, T *pd, T *px, T *pg) {
            const f2 s = sigmoid2(S::pair(sd, j, lane)), u = sigmoid2(S::pair(sg, j, lane)), a = decay_of(q[j]), r = rest_of(q[j], a);
            float w0, w1;
            unpack2(r, w0, w1);      // 1 - a^2 of 0 (no decay at all): its root's reciprocal stays finite, so that times q = 0 it is 0
            const f2 rm = pack2(rsqrt_fast(fmaxf(w0, 1e-36f)), rsqrt_fast(fmaxf(w1, 1e-36f)));
            const f2 vx = mul2(u, S::pair(sx, j, lane)), gm = mul2(G, mul2(r, rm));
            const f2 ds = mul2(mul2(aG, fma2(mul2(vx, a), rm, mul2(v[j], minus))), s);      // a G (v a / m - h) s
            sum = add2(sum, ds);
            if (!w.on) return;
            store_pair<T, VEC>(pd, c, D, mul2(mul2(ds, coef), fma2(s, minus, one)));
            store_pair<T, VEC>(px, c, D, mul2(gm, u));
            store_pair<T, VEC>(pg, c, D, mul2(mul2(gm, vx), fma2(u, minus, one)));
        };
        T *od = static_cast<T *>(p.ddecay) + (r0 + ROWS - 1) * p.ld_ddecay, *ox = static_cast<T *>(p.dx) + (r0 + ROWS - 1) * p.ld_dx,
          *og = static_cast<T *>(p.dgate) + (r0 + ROWS - 1) * p.ld_dgate;
        if ((starts | ends) == 0 && r0 >= k.c0 && r0 + ROWS <= k.c1) {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j) {
                const f2 G = add2(gy[j], grad);
                grad = mul2(decay_of(q[j]), G);
                row(j, G, grad, od, ox, og);
                od -= p.ld_ddecay;
                ox -= p.ld_dx;
                og -= p.ld_dgate;
            }
        } else {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j) {
                const long long r = r0 + j;
                const f2 G = ends >> j & 1 ? gy[j] : add2(gy[j], grad);
                grad = mul2(decay_of(q[j]), G);
                if (starts >> j & 1) {
                    const int b = marks.sequence(j);
                    if (p.dh0 && w.on) store_state(p.dh0 + (long long)b * D, c, D, grad);
                }
                if (r >= k.c0 && r < k.c1) row(j, G, grad, od, ox, og);      // (the same for all lanes of a warp)
                od -= p.ld_ddecay;
                ox -= p.ld_dx;
                og -= p.ld_dgate;
            }
        }
    }
    sync_rows();                                     // the exchange's last set has been read
    ex.warp[0][warp][lane] = quad(sum, sum);
    sync_rows();
    if (warp == 0 && w.on) {
        f2 t = both(0.f);
#pragma unroll
        for (int b = 0; b < WARPS; ++b) t = add2(t, pack2(ex.warp[0][b][lane].x, ex.warp[0][b][lane].y));
        const float e0 = p.rate[c], e1 = p.rate[min(c + 1, D - 1)];
        store_state(part, c, D, mul2(t, pack2(p.scale * sigmoid(e0), p.scale * sigmoid(e1))));
    }
}

// ------------------------------------------------------------------------------------------ single tokens
template <class T, bool VEC> __global__ void __launch_bounds__(128) gated_scan_step_kernel(GatedScanParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int pairs = (p.D - 1) / 2 + 1, D = p.D;
    const long long b = i / pairs;
    if (b >= p.B) return;
    const int c = (int)(i - b * pairs) * 2;
    const int slot = p.slot ? p.slot[b] : (int)b;
    T *y = static_cast<T *>(p.y) + b * p.ld_y;
    if (slot < 0 || slot >= p.slots) {
        store_pair<T, VEC>(y, c, D, both(0.f));
        return;
    }
    const f2 x = load_pair(static_cast<const T *>(p.x) + b * p.ld_x, c, D), d = load_pair(static_cast<const T *>(p.decay) + b * p.ld_decay, c, D),
             g = load_pair(static_cast<const T *>(p.gate) + b * p.ld_gate, c, D);
    float *state = p.state + (long long)slot * D;
    const f2 old = load_state(state, c, D);
    const f2 q = one_less_exp(mul2(coefficients(p, c), sigmoid2(d))), a = decay_of(q);
    const f2 h = fma2(a, old, mul2(mul2(sqrt2(rest_of(q, a)), sigmoid2(g)), x));
    store_state(state, c, D, h);
    store_pair<T, VEC>(y, c, D, h);
}

// The largest access (16, 4 bytes, or an element) that the bases, the rows and D of a call's tensors allow.
int access_of(const GatedScanParams &p, bool bf16) {
    const size_t es = bf16 ? 2 : 4;
    for (int n = 16; n > (int)es; n = n == 16 ? 4 : 0)
        if (p.D * es % n == 0 && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.decay, p.ld_decay, es, n) &&
            rows_aligned(p.gate, p.ld_gate, es, n) && rows_aligned(p.y, p.ld_y, es, n) && rows_aligned(p.dy, p.ld_dy, es, n) &&
            rows_aligned(p.dx, p.ld_dx, es, n) && rows_aligned(p.ddecay, p.ld_ddecay, es, n) && rows_aligned(p.dgate, p.ld_dgate, es, n))
            return n;
    return (int)es;
}

template <class T, int CP, bool CLUSTER, bool BWD> cudaError_t launch(const GatedScanParams &p, cudaStream_t s) {
    const auto kernel = BWD ? gated_scan_bwd_kernel<T, CP, CLUSTER> : gated_scan_fwd_kernel<T, CP, CLUSTER>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.D - 1) / COLS + 1) * p.cluster, p.chains);
    cfg.blockDim = dim3(LANES + (CLUSTER ? 32 : 0));
    cfg.dynamicSmemBytes = 2 * (BWD ? 4 : 3) * Stage<T, CP>::BYTES;
    cfg.stream = s;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CLUSTER ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <class T, int CP, bool BWD> cudaError_t launch(const GatedScanParams &p, cudaStream_t s) {
    return p.cluster > 1 ? launch<T, CP, true, BWD>(p, s) : launch<T, CP, false, BWD>(p, s);
}
template <bool BWD> cudaError_t launch(const GatedScanParams &p, bool bf16_, cudaStream_t s) {
    const int n = access_of(p, bf16_);
    if (bf16_) return n == 16 ? launch<bf16, 16, BWD>(p, s) : n == 4 ? launch<bf16, 4, BWD>(p, s) : launch<bf16, 2, BWD>(p, s);
    return n == 16 ? launch<float, 16, BWD>(p, s) : launch<float, 4, BWD>(p, s);
}

long long rows_of(const GatedScanParams &p) { return (long long)(p.cu_seqlens ? 1 : p.B) * p.T; }

// Chains side by side cost nothing, so there are as many as fill the GPU, up to one per sequence; what they leave idle,
// clusters of up to eight blocks fill by sharing a chain's tiles.  All blocks run at once: a few more than fit would run alone
// after the others.
void split(GatedScanParams &p, int per_sm) {
    const long long cols = (p.D - 1) / COLS + 1, room = (long long)per_sm * sm_count(), rows = rows_of(p);
    long long each = (cols * p.B + room - 1) / room;             // sequences of a chain
    if (each < 1) each = 1;
    p.chains = (int)((p.B + each - 1) / each);
    p.cluster = 1;
    // (a cluster's blocks need a place in one group of SMs: of these up to a seventh stays empty)
    while (p.cluster < MAX_CLUSTER && cols * p.chains * p.cluster * 2 <= room * 6 / 7 && rows > (long long)TILE * p.chains * p.cluster)
        p.cluster *= 2;
}
void split_fwd(GatedScanParams &p, bool bf16_) { split(p, bf16_ ? 3 : 2); }
void split_bwd(GatedScanParams &p, bool bf16_) { split(p, bf16_ ? 2 : 1); }

}  // namespace

size_t gated_scan_saved_rows(const GatedScanParams &p) { return (size_t)((rows_of(p) + SAVE - 1) / SAVE); }

size_t gated_scan_part_floats(const GatedScanParams &p, bool bf16_) {
    GatedScanParams q = p;
    split_bwd(q, bf16_);
    return (size_t)q.chains * q.cluster * p.D;
}

cudaError_t launch_gated_scan_fwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    split_fwd(p, bf16_);
    return launch<false>(p, bf16_, s);
}

cudaError_t launch_gated_scan_bwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    split_bwd(p, bf16_);
    const cudaError_t e = launch<true>(p, bf16_, s);
    if (e != cudaSuccess) return e;
    return launch_sum_rows(p.part, p.chains * p.cluster, SumOut{p.drate, p.D, false}, SumOut{nullptr, 0, false}, s);
}

cudaError_t launch_gated_scan_step(const GatedScanParams &p, bool bf16_, cudaStream_t s) {
    const long long n = (long long)p.B * ((p.D - 1) / 2 + 1);
    const unsigned grid = (unsigned)((n + 127) / 128);
    const bool v = access_of(p, bf16_) > (bf16_ ? 2 : 4);
    if (bf16_) {
        if (v) gated_scan_step_kernel<bf16, true><<<grid, 128, 0, s>>>(p);
        else gated_scan_step_kernel<bf16, false><<<grid, 128, 0, s>>>(p);
    } else {
        if (v) gated_scan_step_kernel<float, true><<<grid, 128, 0, s>>>(p);
        else gated_scan_step_kernel<float, false><<<grid, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace mixer
