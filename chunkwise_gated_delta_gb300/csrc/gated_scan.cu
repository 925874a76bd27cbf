// Gated recurrence (one state per channel), forward, backward and single tokens.
//
// All rows of a call form one axis, cut where a sequence begins, in segments whatever the sequences' lengths: of 16 to 96 rows where
// there are places for all their warps, up to 192 where the channels alone take most of them, and a call of up to 128 rows is one.
// A warp has a segment's rows and 64 channels, a lane two of them, eight rows in registers and the next eight on their way:
//
//   local pass      what a segment does to a state: h_out = h + A h_in (A, h), or h alone where a sequence begins in it
//   boundary pass   the states that enter the segments, in order
//   walk            the segment again from the state that enters it; y, final states, the states before every 8th row
//
// Warps wait for no other, and every pass is as parallel as the call has rows and channels.  The walk goes through the segments
// from the last, whose inputs the local pass has left in L2.
// Gates are computed twice, and the passes are bound by instructions and their latency (57 and 63 per row and pair of channels, 66 %
// of the issue slots at 20 warps to an SM; four channels to a lane, a seventh fewer instructions at 12 or 16 warps, takes as long):
// 4 sequences of 4096 x 2048 bfloat16 take 88 us, of which local pass 42, boundary 5, walk 44 (traffic of one pass: 39); one of
// 16384 x 1024 takes 51 to 54.  Those are channels that remember long.  A warp with one whose exponent may reach 1/4 takes the general
// form of a decay, ten instructions more: 97 us (local pass 48, walk 49) and 58.  One pass was slower: clusters of blocks that carry the state through shared memory took 104 and 109 us,
// tiles that take what enters from the tiles before by flags in memory 154 and 93, both waiting for each other most of the time.
// Where a sequence begins the link is cut by selection (never by a product with 0: a state of an earlier sequence
// may be an infinity).
//
// The backward does the same from the end, with G_t = dy_t + a_{t+1} G_{t+1}: its local pass takes decay and dy alone, and its walk
// has the state before every eighth row from the forward.  4 x 4096 x 2048 takes 134 us, 147 in the general form (139 and 160
// instructions per row and pair in the walk).
#include "gated_scan.cuh"
#include "tc_common.cuh"

namespace mixer {
namespace {

using namespace gs;

__host__ __device__ __forceinline__ long long rows_of(const GatedScanParams &p) { return (long long)(p.cu_seqlens ? 1 : p.B) * p.T; }

// Where a warp works: segment, channels.
struct Where {
    int lane, c, cl;             // c: this lane's first channel; cl: the same or, of idle lanes, one inside
    long long seg, segs, r0;     // the segment, their number, the segment's first row
    bool any, on;
    Extent k;
};
template <bool BACK> __device__ __forceinline__ Where where(const GatedScanParams &p) {
    Where w;
    w.lane = threadIdx.x & 31;
    const long long cols = (p.D - 1) / COLS + 1;
    w.segs = (rows_of(p) + p.seg - 1) / p.seg;
    long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    w.any = unit < cols * w.segs;
    if (BACK) unit = cols * w.segs - 1 - unit;
    w.seg = unit / cols;
    w.r0 = w.seg * p.seg;
    const int c0 = (int)(unit - w.seg * cols) * COLS;
    w.c = c0 + w.lane * 2;
    w.on = w.c < p.D;
    w.cl = w.on ? w.c : c0;
    w.k = extent_of(p.cu_seqlens, p.B, p.T);
    return w;
}

// The gates of a row: the decay's exponent, and m u x.
__device__ __forceinline__ f2 exponent(f2 coef, f2 d) { return mul2(coef, sigmoid2(d)); }
__device__ __forceinline__ f2 input_v(const Decay &d, f2 g, f2 x) { return mul2(mul2(sqrt2(rest_of(d)), sigmoid2(g)), x); }

// Rows on their way: a ring of this warp's in shared memory, eight rows of N tensors per stage, STAGES - 1 of them in flight.
// BACK: from the last rows to the first.
constexpr int STAGES = 3;
template <class T, int CP, int N, bool BACK> struct Ring {
    using S = Stage<T, CP>;
    static constexpr int SIZE = N * S::BYTES, BYTES = STAGES * SIZE;
    char *base;
    int to, read;                        // byte offsets of the stage that is filled next, and of the one that is read
    const T *at[N];                      // this lane's access of the rows that come next
    long long ld[N];
    long long next, last;                // those rows' first, and the first of the last ones
    int left;
    Extent k;

    __device__ __forceinline__ void begin(char *all, const GatedScanParams &p, const Where &w, const void *const (&from)[N],
                                          const long long (&stride)[N]) {
        base = all + (threadIdx.x >> 5) * BYTES;
        to = 0;
        read = -SIZE;
        k = w.k;
        const long long end = min((long long)k.hi, w.r0 + p.seg), behind = w.r0 + (end - 1 - w.r0) / ROWS * ROWS;
        next = BACK ? behind : w.r0;
        last = BACK ? w.r0 : behind;
        const int c = w.c - w.lane * 2 + S::col();
        left = p.D - c;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            ld[n] = stride[n];
            at[n] = static_cast<const T *>(from[n]) + (next + S::row()) * ld[n] + c;
        }
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) bring();
    }
    __device__ __forceinline__ void bring() {
        if (BACK ? next >= last : next <= last) {
            if (next >= k.lo && next + ROWS <= k.hi) {
#pragma unroll
                for (int n = 0; n < N; ++n) S::bring(base + to + n * S::BYTES, at[n], ld[n], left);
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n)
                    S::bring_clamped(base + to + n * S::BYTES, at[n] - (next + S::row()) * ld[n], ld[n], left, next, k);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) at[n] += (BACK ? -ROWS : ROWS) * ld[n];
            next += BACK ? -ROWS : ROWS;
            to = to == (STAGES - 1) * SIZE ? 0 : to + SIZE;
        }
        copies_end();
    }
    // The next stage is there, and the one before it has been read by all lanes and is filled again.
    __device__ __forceinline__ const char *step() {
        copies_wait<STAGES - 2>();
        __syncwarp();
        bring();
        read = read == (STAGES - 1) * SIZE ? 0 : read + SIZE;
        return base + read;
    }
    static __device__ __forceinline__ f2 pair(const char *st, int n, int row, int lane) { return S::pair(st + n * S::BYTES, row, lane); }
};

// ------------------------------------------------------------------------------------------ forward
// A segment's effect is kept as A >= 0 and h; A = -1 says that the link is cut and h alone counts.  (A, h) of a pair of channels
// lie together, rows of pairs are as wide as D rounded up to even.  A product of positive decays that underflows is kept at the smallest
// positive number: an infinity that enters then leaves as one, not as 0 times infinity.  (Of a finite state that is 2^-149 of itself, where
// a test for infinities in the chain of segments would take 2 us of the 51 of the long prompt.)
constexpr float LEAST = 1.40129846e-45f;
__device__ __forceinline__ void store_segment(const GatedScanParams &p, const Where &w, f2 a, f2 h, bool cut) {
    float4 q;
    unpack2(a, q.x, q.z);
    q.x = cut ? -1.f : fmaxf(q.x, LEAST);
    q.z = cut ? -1.f : fmaxf(q.z, LEAST);
    unpack2(h, q.y, q.w);
    reinterpret_cast<float4 *>(p.seg_pair)[(w.seg * ((p.D + 1) & ~1) + w.c) / 2] = q;
}
template <class T, int CP, bool WALK, bool SMALL_Q>
__device__ __forceinline__ void forward_rows(const GatedScanParams &p, const Where &w, f2 coef, Ring<T, CP, 3, false> &ring) {
    constexpr bool VEC = CP > (int)sizeof(T);
    const int D = p.D, lane = w.lane;
    const long long end = min((long long)w.k.hi, w.r0 + p.seg);
    f2 h = both(0.f), prod = both(1.f);
    bool cut = false;
    if (WALK && p.seg_in) h = load_state(p.seg_in + w.seg * D, w.cl, D);      // (the boundary pass leaves there what enters)
    Marks marks;
    for (long long r0 = w.r0; r0 < end; r0 += ROWS) {
        const char *st = ring.step();
        f2 a[ROWS], v[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const Decay d = decay_at<SMALL_Q>(exponent(coef, ring.pair(st, 1, j, lane)));
            a[j] = d.a;
            v[j] = input_v(d, ring.pair(st, 2, j, lane), ring.pair(st, 0, j, lane));
        }
        marks.find(p, w.k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        if (WALK && p.states && r0 >= w.k.lo && w.on) store_state(p.states + r0 / ROWS * D, w.c, D, h);
        if ((starts | ends) == 0 && r0 >= w.k.lo && r0 + ROWS <= w.k.hi) {
            T *y = static_cast<T *>(p.y) + r0 * p.ld_y + w.c;
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                h = fma2(a[j], h, v[j]);
                if (WALK) v[j] = h;
                else prod = mul2(prod, a[j]);
            }
            if (WALK && p.y && w.on)
#pragma unroll
                for (int j = 0; j < ROWS; ++j, y += p.ld_y) store_pair<T, VEC>(y, 0, D - w.c, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const long long r = r0 + j;
                if (r < w.k.lo || r >= w.k.hi) continue;         // (the same for all lanes)
                if (starts >> j & 1) {
                    h = p.h0 ? fma2(a[j], load_state(p.h0 + (long long)marks.sequence(j) * D, w.cl, D), v[j]) : v[j];
                    cut = true;
                } else {
                    h = fma2(a[j], h, v[j]);
                }
                if (!WALK) {
                    prod = mul2(prod, a[j]);
                    continue;
                }
                if (w.on && p.y) store_pair<T, VEC>(static_cast<T *>(p.y) + r * p.ld_y, w.c, D, h);
                if (ends >> j & 1) {
                    const int s = marks.sequence(j);
                    if (p.ht && w.on) store_state(p.ht + (long long)s * D, w.c, D, h);
                }
            }
        }
    }
    if (!WALK && w.on) {
        store_segment(p, w, prod, h, cut);
    }
}

template <class T, int CP, bool WALK> __global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 6 : 3) gated_scan_fwd_kernel(GatedScanParams p) {
    extern __shared__ __align__(16) char rings[];        // [WARPS][Ring::BYTES]
    const Where w = where<WALK>(p);
    kda::tc::grid_dep_launch();
    if (!w.any) return;
    const bool some = covers(w.k, w.r0, p.seg);
    Ring<T, CP, 3, false> ring;
    if (some) ring.begin(rings, p, w, {p.x, p.decay, p.gate}, {p.ld_x, p.ld_decay, p.ld_gate});      // (the inputs wait for no pass)
    const f2 coef = coefficients(p, w.cl);
    float lo, hi;
    unpack2(coef, lo, hi);
    const bool small = __all_sync(~0u, lo < SMALL && hi < SMALL);        // exponents are at most their coefficients
    if (WALK) kda::tc::grid_dep_wait();
    if (WALK && p.cu_seqlens && p.ht && w.on)        // empty sequences: the state passes through
        for (long long s = w.seg; s < p.B; s += w.segs) {
            const int a = clamped(p.cu_seqlens[s], 0, p.T), b = clamped(p.cu_seqlens[s + 1], a, p.T);
            if (a == b) store_state(p.ht + s * p.D, w.c, p.D, p.h0 ? load_state(p.h0 + s * p.D, w.c, p.D) : both(0.f));
        }
    if (!some) return;
    if (small) forward_rows<T, CP, WALK, true>(p, w, coef, ring);
    else forward_rows<T, CP, WALK, false>(p, w, coef, ring);
}

// What enters each segment.  32 channels to a block, its warps 8 segments each at a time; BACK: from the last segment to the first.
constexpr int BWARPS = 16, BEACH = 8;
template <bool BACK> __global__ void __launch_bounds__(32 * BWARPS) gated_scan_boundary_kernel(GatedScanParams p) {
    __shared__ float2 sm[BWARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = p.D, pitch = (D + 1) & ~1;
    const int c = min((int)blockIdx.x * 32 + lane, D - 1);               // (lanes past the end repeat the last channel)
    const int segs = (int)((rows_of(p) + p.seg - 1) / p.seg);
    const Extent k = extent_of(p.cu_seqlens, p.B, p.T);
    const int s0 = k.lo / p.seg, s1 = min(segs, (int)(((long long)k.hi + p.seg - 1) / p.seg)), n = k.lo < k.hi ? s1 - s0 : 0;
    kda::tc::grid_dep_launch();
    kda::tc::grid_dep_wait();
    float carry = 0.f;
    for (int base = 0; base < n; base += BWARPS * BEACH) {
        const int i0 = base + warp * BEACH, at = BACK ? s1 - 1 - i0 : s0 + i0;
        const float2 *from = reinterpret_cast<const float2 *>(p.seg_pair) + (long long)at * pitch + c;
        float2 g[BEACH];
#pragma unroll
        for (int j = 0; j < BEACH; ++j) g[j] = i0 + j < n ? from[(BACK ? -j : j) * (long long)pitch] : make_float2(1.f, 0.f);
        float pa = 1.f, ph = 0.f;
        bool cut = false;
#pragma unroll
        for (int j = 0; j < BEACH; ++j) {
            const bool here = g[j].x == -1.f;
            ph = here || j == 0 ? g[j].y : fmaf(g[j].x, ph, g[j].y);
            cut |= here;
            pa *= g[j].x;
        }
        __syncthreads();                             // the last round's pairs have been read
        sm[warp][lane] = make_float2(cut ? -1.f : fmaxf(pa, LEAST), ph);
        __syncthreads();
        float in = carry;
#pragma unroll
        for (int q = 0; q < BWARPS; ++q) {
            if (q == warp) in = carry;
            const float2 t = sm[q][lane];
            carry = t.x == -1.f ? t.y : fmaf(t.x, carry, t.y);
        }
        float *to = p.seg_in + (long long)at * D + c;
#pragma unroll
        for (int j = 0; j < BEACH; ++j) {
            if (i0 + j < n) to[(BACK ? -j : j) * (long long)D] = in;
            in = g[j].x == -1.f ? g[j].y : fmaf(g[j].x, in, g[j].y);
        }
    }
}

// ------------------------------------------------------------------------------------------ backward
// The first row of a segment's last eight.
__device__ __forceinline__ long long last_rows(const GatedScanParams &p, const Where &w) {
    const long long end = min((long long)w.k.hi, w.r0 + p.seg);
    return w.r0 + (end - 1 - w.r0) / ROWS * ROWS;
}
// The local pass: what a segment does to the gradient that comes from behind it, a_t G_t of its first token.
template <class T, int CP, bool SMALL_Q>
__device__ __forceinline__ void backward_local(const GatedScanParams &p, const Where &w, f2 coef, Ring<T, CP, 2, true> &ring) {
    const int D = p.D, lane = w.lane;
    f2 g = both(0.f), prod = both(1.f);
    bool cut = false;
    Marks marks;
    for (long long r0 = last_rows(p, w); r0 >= w.r0; r0 -= ROWS) {
        const char *st = ring.step();
        f2 a[ROWS], gy[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            a[j] = decay_at<SMALL_Q>(exponent(coef, ring.pair(st, 0, j, lane))).a;
            gy[j] = ring.pair(st, 1, j, lane);
        }
        marks.find(p, w.k, r0);
        const unsigned ends = marks.ends;
        if (ends == 0 && r0 >= w.k.lo && r0 + ROWS <= w.k.hi) {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j) {
                g = mul2(a[j], add2(gy[j], g));
                prod = mul2(prod, a[j]);
            }
        } else {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j) {
                const long long r = r0 + j;
                if (r < w.k.lo || r >= w.k.hi) continue;
                if (ends >> j & 1) {
                    g = p.dht ? load_state(p.dht + (long long)marks.sequence(j) * D, w.cl, D) : both(0.f);
                    cut = true;
                }
                g = mul2(a[j], add2(gy[j], g));
                prod = mul2(prod, a[j]);
            }
        }
    }
    if (w.on) {
        store_segment(p, w, prod, g, cut);
    }
}
template <class T, int CP> __global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 6 : 4) gated_scan_bwd_local_kernel(GatedScanParams p) {
    extern __shared__ __align__(16) char rings[];        // [WARPS][Ring::BYTES]
    const Where w = where<false>(p);
    kda::tc::grid_dep_launch();
    if (!w.any || !covers(w.k, w.r0, p.seg)) return;
    Ring<T, CP, 2, true> ring;
    ring.begin(rings, p, w, {p.decay, p.dy}, {p.ld_decay, p.ld_dy});
    const f2 coef = coefficients(p, w.cl);
    float lo, hi;
    unpack2(coef, lo, hi);
    if (__all_sync(~0u, lo < SMALL && hi < SMALL)) backward_local<T, CP, true>(p, w, coef, ring);
    else backward_local<T, CP, false>(p, w, coef, ring);
}

// With q the exponent, s and u the two sigmoids, v = u x and G_t the gradient of h_t:
//     dq = G (v a^2 / m - a h_{t-1}),  ddecay = dq q (1 - s),  drate = scale sigmoid(rate) sum dq s,
//     dx = G m u,  dgate = G m x u (1 - u),  dh0 = a G of the first token.
// Eight rows at a time from the last: forward through them from the saved state, then back.  Their inputs wait in a ring
// of this warp's in shared memory, for both ways take them.
template <class T, int CP, bool SMALL_Q>
__device__ __forceinline__ f2 backward_rows(const GatedScanParams &p, const Where &w, f2 coef, Ring<T, CP, 4, true> &ring) {
    using S = Stage<T, CP>;
    constexpr bool VEC = CP > (int)sizeof(T);
    const int D = p.D, lane = w.lane;
    const f2 minus = both(-1.f), one = both(1.f);
    // (eight rows of which the first lie outside have no saved state and need none)
    auto saved_at = [&](long long r0) { return r0 >= w.k.lo ? load_state(p.states + r0 / ROWS * D, w.cl, D) : both(0.f); };
    f2 sum = both(0.f);
    Marks marks;
    long long r0 = last_rows(p, w);
    f2 saved = saved_at(r0);
    f2 grad = p.seg_in ? load_state(p.seg_in + w.seg * D, w.cl, D) : both(0.f);
    for (; r0 >= w.r0; r0 -= ROWS) {
        const char *sx = ring.step();
        f2 h = saved;
        if (r0 > w.r0) saved = saved_at(r0 - ROWS);
        const char *sd = sx + S::BYTES, *sg = sd + S::BYTES, *sy = sg + S::BYTES;
        marks.find(p, w.k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        f2 q[ROWS], before[ROWS];        // the decay, kept in one number; the state before each row
        if (starts == 0) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                q[j] = kept_decay<SMALL_Q>(exponent(coef, S::pair(sd, j, lane)));
                before[j] = h;
                if (j + 1 < ROWS) {
                    const Decay d = decay_of<SMALL_Q>(q[j]);
                    h = fma2(d.a, h, input_v(d, S::pair(sg, j, lane), S::pair(sx, j, lane)));
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                q[j] = kept_decay<SMALL_Q>(exponent(coef, S::pair(sd, j, lane)));
                if (starts >> j & 1) h = p.h0 ? load_state(p.h0 + (long long)marks.sequence(j) * D, w.cl, D) : both(0.f);
                before[j] = h;
                const Decay d = decay_of<SMALL_Q>(q[j]);
                h = fma2(d.a, h, input_v(d, S::pair(sg, j, lane), S::pair(sx, j, lane)));
            }
        }
        // a row's outputs from G; leaves a G in grad
        auto row = [&](int j, f2 G, T *pd, T *px, T *pg) {
            const f2 s = sigmoid2(S::pair(sd, j, lane)), u = sigmoid2(S::pair(sg, j, lane));
            const Decay d = decay_of<SMALL_Q>(q[j]);
            const f2 a = d.a, r = rest_of(d);
            float w0, w1;
            unpack2(r, w0, w1);          // 1 - a^2 of 0 (no decay at all): its root's reciprocal stays finite, so that times q = 0 it is 0
            const f2 rm = pack2(rsqrt_fast(fmaxf(w0, 1e-36f)), rsqrt_fast(fmaxf(w1, 1e-36f)));
            const f2 v = mul2(u, S::pair(sx, j, lane)), gm = mul2(G, mul2(r, rm));
            grad = mul2(a, G);
            const f2 ds = mul2(mul2(grad, fma2(mul2(v, a), rm, mul2(before[j], minus))), s);     // a G (v a / m - h) s
            sum = add2(sum, ds);
            if (!w.on) return;
            store_pair<T, VEC>(pd, w.c, D, mul2(mul2(ds, coef), fma2(s, minus, one)));
            store_pair<T, VEC>(px, w.c, D, mul2(gm, u));
            store_pair<T, VEC>(pg, w.c, D, mul2(mul2(gm, v), fma2(u, minus, one)));
        };
        T *od = static_cast<T *>(p.ddecay) + (r0 + ROWS - 1) * p.ld_ddecay, *ox = static_cast<T *>(p.dx) + (r0 + ROWS - 1) * p.ld_dx,
          *og = static_cast<T *>(p.dgate) + (r0 + ROWS - 1) * p.ld_dgate;
        if ((starts | ends) == 0 && r0 >= w.k.lo && r0 + ROWS <= w.k.hi) {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j, od -= p.ld_ddecay, ox -= p.ld_dx, og -= p.ld_dgate)
                row(j, add2(S::pair(sy, j, lane), grad), od, ox, og);
        } else {
#pragma unroll
            for (int j = ROWS - 1; j >= 0; --j, od -= p.ld_ddecay, ox -= p.ld_dx, og -= p.ld_dgate) {
                const long long r = r0 + j;
                if (r < w.k.lo || r >= w.k.hi) continue;         // (the same for all lanes)
                if (ends >> j & 1) grad = p.dht ? load_state(p.dht + (long long)marks.sequence(j) * D, w.cl, D) : both(0.f);
                row(j, add2(S::pair(sy, j, lane), grad), od, ox, og);
                if (starts >> j & 1) {
                    const int b = marks.sequence(j);
                    if (p.dh0 && w.on) store_state(p.dh0 + (long long)b * D, w.c, D, grad);
                }
            }
        }
    }
    return sum;
}
template <class T, int CP> __global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 4 : 2) gated_scan_bwd_kernel(GatedScanParams p) {
    extern __shared__ __align__(16) char rings[];        // [WARPS][Ring::BYTES]
    const Where w = where<false>(p);
    kda::tc::grid_dep_launch();
    if (!w.any) return;
    const bool some = covers(w.k, w.r0, p.seg);
    Ring<T, CP, 4, true> ring;
    if (some) ring.begin(rings, p, w, {p.x, p.decay, p.gate, p.dy}, {p.ld_x, p.ld_decay, p.ld_gate, p.ld_dy});   // (the inputs wait for no pass)
    kda::tc::grid_dep_wait();
    const int D = p.D;
    if (p.cu_seqlens && p.dh0 && w.on)                   // empty sequences hand the gradient through
        for (long long s = w.seg; s < p.B; s += w.segs) {
            const int a = clamped(p.cu_seqlens[s], 0, p.T), b = clamped(p.cu_seqlens[s + 1], a, p.T);
            if (a == b) store_state(p.dh0 + s * D, w.c, D, p.dht ? load_state(p.dht + s * D, w.c, D) : both(0.f));
        }
    f2 sum = both(0.f);
    if (some) {
        const f2 coef = coefficients(p, w.cl);
        float lo, hi;
        unpack2(coef, lo, hi);
        if (__all_sync(~0u, lo < SMALL && hi < SMALL)) sum = backward_rows<T, CP, true>(p, w, coef, ring);
        else sum = backward_rows<T, CP, false>(p, w, coef, ring);
    }
    if (w.on) {
        const float e0 = p.rate[w.c], e1 = p.rate[min(w.c + 1, D - 1)];
        store_state(p.part + w.seg * D, w.c, D, mul2(sum, pack2(p.scale * sigmoid(e0), p.scale * sigmoid(e1))));
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
    const Decay q = decay_at<false>(exponent(coefficients(p, c), d));
    const f2 h = fma2(q.a, old, input_v(q, g, x));
    store_state(state, c, D, h);
    store_pair<T, VEC>(y, c, D, h);
}

// The largest access (16, 4 bytes, or an element) that the bases, the rows and D of a call's tensors allow.
int access_of(const GatedScanParams &p, bool bf16) {
    const size_t es = bf16 ? 2 : 4;
    for (int n = 16; n > (int)es; n = n == 16 ? (bf16 ? 4 : 8) : 0)
        if (p.D * es % n == 0 && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.decay, p.ld_decay, es, n) &&
            rows_aligned(p.gate, p.ld_gate, es, n) && rows_aligned(p.y, p.ld_y, es, n) && rows_aligned(p.dy, p.ld_dy, es, n) &&
            rows_aligned(p.dx, p.ld_dx, es, n) && rows_aligned(p.ddecay, p.ld_ddecay, es, n) && rows_aligned(p.dgate, p.ld_dgate, es, n))
            return n;
    return (int)es;
}

// Rows of a segment, such that the warps of a pass (`warps` to an SM) all run at once, or in as few rounds as make segments of about
// MOST rows (their number is rounded down, so where fewer than two or three fit beside one another a segment has up to 192 or 144):
// a last round that is not full costs as much as a full one (B4 T4096 D2048: 90 us in segments of 64, 88 so).  Up to FEW
// rows are one segment, a launch instead of three: calls of 128 x 512 back to back take 22 us for 30 (with gradients 58 for 77),
// waited for one by one 43 for 40.
constexpr int MOST = 96, FEW = 128;
int segment_of(const GatedScanParams &p, int warps) {
    const long long cols = (p.D - 1) / COLS + 1, rows = rows_of(p), places = (long long)warps * sm_count();
    if (rows <= FEW) return (int)((rows + ROWS - 1) / ROWS * ROWS);
    const long long rounds = (cols * rows + places * MOST - 1) / (places * MOST), segs = max(1LL, places * rounds / cols);
    const long long seg = ((rows + segs - 1) / segs + ROWS - 1) / ROWS * ROWS;
    return (int)max(seg, 16LL);
}
int fwd_segment(const GatedScanParams &p) { return segment_of(p, 24); }
int bwd_segment(const GatedScanParams &p) { return segment_of(p, 16); }
long long segments_of(const GatedScanParams &p, int seg) { return (rows_of(p) + seg - 1) / seg; }
unsigned blocks_of(const GatedScanParams &p) {
    const long long cols = (p.D - 1) / COLS + 1;
    return (unsigned)((cols * segments_of(p, p.seg) + WARPS - 1) / WARPS);
}

// A kernel whose blocks may set up while the one before it ends; they wait for it themselves.
template <auto KERNEL> cudaError_t launch(unsigned grid, int threads, size_t smem, bool after, const GatedScanParams &p, cudaStream_t s) {
    const cudaError_t e = allow_shared<KERNEL>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <class T, int CP> cudaError_t forward(GatedScanParams &p, cudaStream_t s) {
    constexpr size_t smem = WARPS * Ring<T, CP, 3, false>::BYTES;
    const unsigned n = blocks_of(p);
    if (segments_of(p, p.seg) == 1) return launch<gated_scan_fwd_kernel<T, CP, true>>(n, THREADS, smem, false, p, s);
    cudaError_t e = launch<gated_scan_fwd_kernel<T, CP, false>>(n, THREADS, smem, false, p, s);
    if (e == cudaSuccess) e = launch<gated_scan_boundary_kernel<false>>((unsigned)((p.D - 1) / 32 + 1), 32 * BWARPS, 0, true, p, s);
    if (e == cudaSuccess) e = launch<gated_scan_fwd_kernel<T, CP, true>>(n, THREADS, smem, true, p, s);
    return e;
}
template <class T, int CP> cudaError_t backward(GatedScanParams &p, cudaStream_t s) {
    const unsigned n = blocks_of(p);
    const bool one = segments_of(p, p.seg) == 1;
    cudaError_t e = cudaSuccess;
    if (!one) {
        e = launch<gated_scan_bwd_local_kernel<T, CP>>(n, THREADS, WARPS * Ring<T, CP, 2, true>::BYTES, false, p, s);
        if (e == cudaSuccess) e = launch<gated_scan_boundary_kernel<true>>((unsigned)((p.D - 1) / 32 + 1), 32 * BWARPS, 0, true, p, s);
    }
    if (e == cudaSuccess) e = launch<gated_scan_bwd_kernel<T, CP>>(n, THREADS, WARPS * Ring<T, CP, 4, true>::BYTES, !one, p, s);
    return e;
}
template <bool BWD, class T, int CP> cudaError_t run(GatedScanParams &p, cudaStream_t s) {
    if constexpr (BWD) return backward<T, CP>(p, s);
    else return forward<T, CP>(p, s);
}
size_t pair_floats(const GatedScanParams &p, size_t segs) { return 2 * segs * ((p.D + 1) & ~1); }
// Points the parameter block into its workspace (the forward has no `part`).  One segment takes none: nothing enters it.
void carve(GatedScanParams &p) {
    const size_t n = (size_t)segments_of(p, p.seg);
    if (n == 1) {
        p.seg_pair = p.seg_in = nullptr;
        p.part = p.drate;
        return;
    }
    p.seg_pair = p.ws;                   // (16-byte aligned)
    p.seg_in = p.ws + pair_floats(p, n);
    p.part = p.seg_in + n * p.D;
}

template <bool BWD> cudaError_t run(GatedScanParams &p, bool bf16_, cudaStream_t s) {
    p.seg = BWD ? bwd_segment(p) : fwd_segment(p);
    carve(p);
    const int n = access_of(p, bf16_);
    if (bf16_) return n == 16 ? run<BWD, bf16, 16>(p, s) : n == 4 ? run<BWD, bf16, 4>(p, s) : run<BWD, bf16, 2>(p, s);
    return n == 16 ? run<BWD, float, 16>(p, s) : n == 8 ? run<BWD, float, 8>(p, s) : run<BWD, float, 4>(p, s);
}

}  // namespace

size_t gated_scan_saved_rows(const GatedScanParams &p) { return (size_t)((rows_of(p) + ROWS - 1) / ROWS); }

size_t gated_scan_fwd_floats(const GatedScanParams &p) {
    const size_t n = (size_t)segments_of(p, fwd_segment(p));
    return n > 1 ? pair_floats(p, n) + n * p.D : 0;
}
// Without the forward's states its walk runs here first, in segments of its own: it may take space where the backward takes none.
size_t gated_scan_bwd_floats(const GatedScanParams &p) {
    const size_t n = (size_t)segments_of(p, bwd_segment(p)), own = n > 1 ? pair_floats(p, n) + 2 * n * p.D : 0;
    return p.states ? own : max(own, gated_scan_fwd_floats(p));
}
cudaError_t launch_gated_scan_fwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    return run<false>(p, bf16_, s);
}

cudaError_t launch_gated_scan_bwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    const cudaError_t e = run<true>(p, bf16_, s);
    const int segs = (int)segments_of(p, p.seg);
    if (e != cudaSuccess || segs == 1) return e;             // (one segment's sums are drate)
    return launch_sum_rows(p.part, segs, SumOut{p.drate, p.D, false}, SumOut{nullptr, 0, false}, s);
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
