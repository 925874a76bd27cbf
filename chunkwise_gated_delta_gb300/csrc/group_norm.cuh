// Norm over each group of neighbouring channels of a row (a mixer's heads), with a gate, forward and backward.
//
//   forward   n = (x - mean) rstd w + b over a group's C columns (uncentred: x rstd w + b), y = n z sigmoid(z)
//   backward  d = dy z sigmoid(z), dz = dy n (sigmoid(z) (1 + z (1 - sigmoid(z)))), g = d w,
//             dx = rstd (g - [mean(g)] - xh mean(g xh)); dweight = sum d xh and dbias = sum d per thread over
//             the rows that a block visits, then over its groups where they share a weight, then over blocks.
//
// A group of up to 32 vectors of 16 bytes takes a part of a warp (a power of two of lanes), one of up to 128 a whole warp with
// up to four vectors per lane, and a longer one up to eight warps, whose sums cross in shared memory (a warp for each row as long as that
// fits: with two warps to 8192 x 8 x 512, or one vector per lane, the barriers cost a tenth).  A thread keeps its group, and with
// it the weights and their sums, and goes down the rows.
//
// Bound by HBM and, not far behind, by instructions (66 % of the issue slots): 16384 rows of 16 groups of 128 bfloat16 with a gate
// take 32 us forward (6.2 TB/s), 8192 rows of 32 groups 33 forward and 51 to 58 backward (6.6 to 5.8 TB/s), the sums over blocks 3 more.
// With the next row in registers, and the bias' sums always kept, they took 39 and 86: too few bytes on their way.  8192 rows of one group
// of 2048: 23 forward, 39 backward with its sums (a block for each group in three passes took 60 and 180).
#pragma once

#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace {

constexpr int TPB = 256;

// Sums over the L lanes of a group, N values at a time: within a warp, then (L > 32) over its warps through shared memory.  Every
// thread of the block takes part.  Two places take turns, so that one barrier parts a sum's reads from the next but one's writes.
template <int L> struct Sums {
    float (*sm)[2][TPB / 32];            // [2]
    int turn = 0;
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int s = (L < 32 ? L : 32) / 2; s; s >>= 1) v[n] += __shfl_xor_sync(~0u, v[n], s);
        if constexpr (L > 32) {
            constexpr int WARPS = L / 32;
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int n = 0; n < N; ++n) sm[turn][n][warp] = v[n];
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; ++n) {
                v[n] = 0.f;
#pragma unroll
                for (int k = 0; k < WARPS; ++k) v[n] += sm[turn][n][warp / WARPS * WARPS + k];
            }
            turn ^= 1;
        }
    }
};

// Where a thread works: groups count in slots of L lanes, `per` (a power of two) of them to a row.  `part`: which `per` groups.
struct Place {
    int group, row, rows;       // group, first row and rows of a block's visit
    bool on;
};
template <int L> __device__ __forceinline__ Place place_of(const GroupNormParams &p, int per, unsigned part) {
    constexpr int SLOTS = TPB / L;
    const int slot = threadIdx.x / L;
    Place q;
    const unsigned group = part * per + slot % per;          // (without a sign: slots past 2^31 - 1 groups do not wrap)
    q.row = slot / per;
    q.rows = SLOTS / per;
    q.on = group < (unsigned)p.G;
    q.group = q.on ? (int)group : p.G - 1;
    return q;
}
int slots_per_row(int G, int slots) {
    int n = 1;
    while (n < G && n < slots) n *= 2;
    return n;
}

// Rows on their way: every thread copies its own vectors of N tensors into its own places of shared memory, DEPTH rows ahead,
// and reads them back, so nobody waits for anybody.  (Single bfloat16 elements are too short for asynchronous copies.)
template <class T, int V, int ITEMS, int N> struct Ahead {
    static constexpr int DEPTH = ITEMS == 1 ? 4 : 2, BYTES = V * (int)sizeof(T) < 4 ? 4 : V * (int)sizeof(T);
    static constexpr int STAGE = N * ITEMS * TPB * BYTES, SMEM = DEPTH * STAGE;
    static __device__ __forceinline__ char *place(char *sm, int stage, int n, int k) {
        return sm + stage * STAGE + ((n * ITEMS + k) * TPB + threadIdx.x) * BYTES;
    }
    static __device__ __forceinline__ void bring(char *sm, int stage, int n, int k, const T *from) {
        char *to = place(sm, stage, n, k);
        if constexpr (V * sizeof(T) < 4) *reinterpret_cast<uint32_t *>(to) = load_bits(from);
        else copy_async<BYTES>(to, from);
    }
    static __device__ __forceinline__ Lanes<T, V> take(char *sm, int stage, int n, int k) {
        Lanes<T, V> v;
        v.load_shared(place(sm, stage, n, k));
        return v;
    }
};

template <class T, int V, int ITEMS, int L, bool GATE>
__global__ void __launch_bounds__(TPB) group_norm_fwd_kernel(GroupNormParams p, int per, unsigned first) {
    constexpr int P = (V + 1) / 2;
    const Place q = place_of<L>(p, per, first + blockIdx.y);
    const int lane = threadIdx.x % L, nv = p.C / V;
    const float inv = 1.f / (float)p.C;
    const long long col = (long long)q.group * p.C;
    f2 w[ITEMS][P], b[ITEMS][P];
    int at[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        at[k] = min(lane + k * L, nv - 1) * V;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            w[k][e] = both(1.f);
            b[k][e] = both(0.f);
        }
        const long long c = p.shared ? at[k] : col + at[k];
        if (p.weight) load_param_pairs<V>(w[k], p.weight, c, p.w_bf16);
        if (p.bias) load_param_pairs<V>(b[k], p.bias, c, p.w_bf16);
    }
    using A = Ahead<T, V, ITEMS, GATE ? 2 : 1>;
    extern __shared__ __align__(16) char sm[];
    __shared__ float cross[2][2][TPB / 32];
    Sums<L> sum{cross};
    const long long step = (long long)gridDim.x * q.rows;
    long long row = (long long)blockIdx.x * q.rows + q.row, next = row;
    auto bring = [&](int stage) {                    // rows past the end: the last
        const long long r = next < p.rows ? next : p.rows - 1;
        const T *x = static_cast<const T *>(p.x) + r * p.ld_x + col;
        const T *g = static_cast<const T *>(p.gate) + r * p.ld_gate + col;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (lane + k * L >= nv) break;
            A::bring(sm, stage, 0, k, x + at[k]);
            if (GATE) A::bring(sm, stage, 1, k, g + at[k]);
        }
        copies_end();
        next += step;
    };
#pragma unroll
    for (int d = 0; d < A::DEPTH; ++d) bring(d);
    // every lane goes through as many visits as the block's first row takes: their sums are taken together
    int stage = 0;
    for (long long base = (long long)blockIdx.x * q.rows; base < p.rows; base += step, row += step) {
        copies_wait<A::DEPTH - 1>();
        f2 v[ITEMS][P], z[ITEMS][P];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const Lanes<T, V> x = A::take(sm, stage, 0, k);
#pragma unroll
            for (int e = 0; e < P; ++e) v[k][e] = x.pair(e);
            if (GATE) {
                const Lanes<T, V> g = A::take(sm, stage, 1, k);
#pragma unroll
                for (int e = 0; e < P; ++e) z[k][e] = g.pair(e);
            }
        }
        bring(stage);
        stage = stage + 1 == A::DEPTH ? 0 : stage + 1;
        float mean = 0.f;
        if (p.center) {
            f2 acc = both(0.f);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (lane + k * L < nv)
#pragma unroll
                    for (int e = 0; e < P; ++e) acc = add2(acc, v[k][e]);
            float t[1] = {pair_sum<V>(acc)};
            sum(t);
            mean = t[0] * inv;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                for (int e = 0; e < P; ++e) v[k][e] = add2(v[k][e], both(-mean));
        }
        f2 acc = both(0.f);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (lane + k * L < nv)
#pragma unroll
                for (int e = 0; e < P; ++e) acc = fma2(v[k][e], v[k][e], acc);
        float t[1] = {pair_sum<V>(acc)};
        sum(t);
        const float rstd = inv_sqrt(t[0] * inv + p.eps);
        if (!q.on || row >= p.rows) continue;
        if (lane == 0) {
            if (p.mean) p.mean[row * p.G + q.group] = mean;
            if (p.rstd) p.rstd[row * p.G + q.group] = rstd;
        }
        T *y = static_cast<T *>(p.y) + row * p.ld_y + col;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (lane + k * L < nv) {
                f2 o[P];
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    o[e] = fma2(mul2(v[k][e], both(rstd)), w[k][e], b[k][e]);
                    if (GATE) o[e] = mul2(o[e], silu2(z[k][e]));
                }
                store_lanes<T, V>(y + at[k], o);
            }
    }
    copies_wait<0>();                                        // (rows past the end were on their way too)
}

// BIAS: the call has a bias or wants its gradient.
template <class T, int V, int ITEMS, int L, bool GATE, bool BIAS>
__global__ void __launch_bounds__(TPB, ITEMS == 1 ? (V == 1 ? 4 : 2) : V == 1 && ITEMS < 8 ? 2 : 1) group_norm_bwd_kernel(GroupNormParams p, int per, unsigned first) {
    constexpr int P = (V + 1) / 2, SLOTS = TPB / L;
    const Place q = place_of<L>(p, per, first + blockIdx.y);
    const int lane = threadIdx.x % L, nv = p.C / V;
    const float inv = 1.f / (float)p.C;
    const long long col = (long long)q.group * p.C;
    f2 w[ITEMS][P], b[ITEMS][P], aw[ITEMS][P], ab[ITEMS][P];
    int at[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        at[k] = min(lane + k * L, nv - 1) * V;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            w[k][e] = both(1.f);
            b[k][e] = aw[k][e] = ab[k][e] = both(0.f);
        }
        const long long c = p.shared ? at[k] : col + at[k];
        if (p.weight) load_param_pairs<V>(w[k], p.weight, c, p.w_bf16);
        if (GATE && BIAS && p.bias) load_param_pairs<V>(b[k], p.bias, c, p.w_bf16);
    }
    using A = Ahead<T, V, ITEMS, GATE ? 3 : 2>;
    extern __shared__ __align__(16) char sm[];
    float2 *stats = reinterpret_cast<float2 *>(sm + A::SMEM);        // [DEPTH][TPB] mean and rstd
    __shared__ float cross[2][2][TPB / 32];
    Sums<L> sum{cross};
    const long long step = (long long)gridDim.x * q.rows;
    long long row = (long long)blockIdx.x * q.rows + q.row, next = row;
    auto bring = [&](int stage) {
        const long long r = next < p.rows ? next : p.rows - 1;
        const T *x = static_cast<const T *>(p.x) + r * p.ld_x + col;
        const T *d = static_cast<const T *>(p.dy) + r * p.ld_dy + col;
        const T *g = static_cast<const T *>(p.gate) + r * p.ld_gate + col;
        float2 *to = stats + stage * TPB + threadIdx.x;
        if (p.center) copy_async<4>(&to->x, p.mean + r * p.G + q.group);
        copy_async<4>(&to->y, p.rstd + r * p.G + q.group);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (lane + k * L >= nv) break;
            A::bring(sm, stage, 0, k, x + at[k]);
            A::bring(sm, stage, 1, k, d + at[k]);
            if (GATE) A::bring(sm, stage, 2, k, g + at[k]);
        }
        copies_end();
        next += step;
    };
#pragma unroll
    for (int d = 0; d < A::DEPTH; ++d) bring(d);
    int stage = 0;
    for (long long base = (long long)blockIdx.x * q.rows; base < p.rows; base += step, row += step) {
        copies_wait<A::DEPTH - 1>();
        const bool live = q.on && row < p.rows;
        f2 xh[ITEMS][P], g[ITEMS][P], s0 = both(0.f), s1 = both(0.f);
        const float2 stat = stats[stage * TPB + threadIdx.x];
        const float nm = p.center ? stat.x : 0.f, rstd = stat.y;
        T *dgate = static_cast<T *>(p.dgate) + row * p.ld_dgate + col;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const bool in = live && lane + k * L < nv;
            f2 dz[P];
            const Lanes<T, V> vx = A::take(sm, stage, 0, k), vd = A::take(sm, stage, 1, k);
            Lanes<T, V> vg;
            if (GATE) vg = A::take(sm, stage, 2, k);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                f2 d = vd.pair(e);
                xh[k][e] = mul2(add2(vx.pair(e), both(-nm)), both(rstd));
                if (GATE) {
                    const f2 z = vg.pair(e), sg = sigmoid2(z), sz = mul2(sg, z);
                    // d silu / dz = sg + sz - sz sg
                    dz[e] = mul2(mul2(d, BIAS ? fma2(xh[k][e], w[k][e], b[k][e]) : mul2(xh[k][e], w[k][e])), fma2(sz, mul2(sg, both(-1.f)), add2(sg, sz)));
                    d = mul2(d, sz);
                }
                g[k][e] = mul2(d, w[k][e]);
                if (in) {                        // (what stands in for a row past the end is not counted: by selection)
                    aw[k][e] = fma2(d, xh[k][e], aw[k][e]);
                    if (BIAS) ab[k][e] = add2(ab[k][e], d);
                    s0 = add2(s0, g[k][e]);
                    s1 = fma2(g[k][e], xh[k][e], s1);
                }
            }
            if (GATE && in) store_lanes<T, V>(dgate + at[k], dz);
        }
        bring(stage);
        stage = stage + 1 == A::DEPTH ? 0 : stage + 1;
        float t[2] = {pair_sum<V>(s1), pair_sum<V>(s0)};
        sum(t);
        const float mgx = t[0] * -inv, mg = p.center ? t[1] * -inv : 0.f;
        if (!live) continue;
        T *dx = static_cast<T *>(p.y) + row * p.ld_y + col;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (lane + k * L < nv) {
                f2 o[P];
#pragma unroll
                for (int e = 0; e < P; ++e) o[e] = mul2(fma2(xh[k][e], both(mgx), add2(g[k][e], both(mg))), both(rstd));
                store_lanes<T, V>(dx + at[k], o);
            }
    }
    copies_wait<0>();                                        // (rows past the end were on their way too)
    if (!p.part) return;
    // the block's sums, over the slots that have the same weight, in their order
    auto sums = reinterpret_cast<float (*)[L][2 * V]>(sm);     // [SLOTS]
    const int keys = p.shared ? 1 : per, key = threadIdx.x / L, cols = p.shared ? p.C : p.G * p.C;
    const long long rowp = p.shared ? (long long)blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x;
    const unsigned kg = (first + blockIdx.y) * per + key;    // (unshared: the key's group)
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float lo, hi;
            unpack2(aw[k][e / 2], lo, hi);
            sums[threadIdx.x / L][lane][e] = e & 1 ? hi : lo;
            unpack2(ab[k][e / 2], lo, hi);
            sums[threadIdx.x / L][lane][V + e] = e & 1 ? hi : lo;
        }
        __syncthreads();
        if (key < keys && (p.shared || kg < (unsigned)p.G) && lane + k * L < nv) {
            float t[2 * V];
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) t[e] = 0.f;
            for (int s = key; s < SLOTS; s += keys)
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) t[e] += sums[s][lane][e];
            float *out = p.part + rowp * 2 * cols + (p.shared ? 0 : (long long)kg * p.C) + at[k];
            if (p.shared && first)                           // the sums of the launch before, of other groups
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    t[e] += out[e];
                    t[V + e] += out[cols + e];
                }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                out[e] = t[e];
                out[cols + e] = t[V + e];
            }
        }
    }
}

// Groups too long for a warp's registers: a block for each, its columns in several passes (the later ones from L2).
template <int N> __device__ __forceinline__ float block_sum(float v, float *sm) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.f;
#pragma unroll
    for (int k = 0; k < N / 32; ++k) r += sm[k];
    return r;
}

template <class T> __global__ void __launch_bounds__(512) group_norm_fwd_long_kernel(GroupNormParams p) {
    __shared__ float sm[16];
    const long long row = blockIdx.x / (unsigned)p.G;
    const int g = (int)(blockIdx.x % (unsigned)p.G);
    const long long col = (long long)g * p.C;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x + col, *z = static_cast<const T *>(p.gate) + row * p.ld_gate + col;
    T *y = static_cast<T *>(p.y) + row * p.ld_y + col;
    const float inv = 1.f / (float)p.C;
    float mean = 0.f;
    if (p.center) {
        float s = 0.f;
        for (unsigned c = threadIdx.x; c < (unsigned)p.C; c += 512) s += to_f(x[c]);
        mean = block_sum<512>(s, sm) * inv;
    }
    float s = 0.f;
    for (unsigned c = threadIdx.x; c < (unsigned)p.C; c += 512) {
        const float d = to_f(x[c]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = inv_sqrt(block_sum<512>(s, sm) * inv + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row * p.G + g] = mean;
        if (p.rstd) p.rstd[row * p.G + g] = rstd;
    }
    for (unsigned c = threadIdx.x; c < (unsigned)p.C; c += 512) {
        const long long k = p.shared ? c : col + c;
        const float w = p.weight ? load_w(p.weight, k, p.w_bf16) : 1.f, b = p.bias ? load_w(p.bias, k, p.w_bf16) : 0.f;
        float v = fmaf((to_f(x[c]) - mean) * rstd, w, b);
        if (p.gate) v *= to_f(z[c]) * sigmoid(to_f(z[c]));
        y[c] = from_f<T>(v);
    }
}

// dy of a column with its gate, and the gate's gradient.
template <class T> __device__ __forceinline__ float gated(const GroupNormParams &p, float dy, float n, const T *z, float &dz) {
    dz = 0.f;
    if (!p.gate) return dy;
    const float v = to_f(*z), sg = sigmoid(v), sz = v * sg;
    dz = dy * n * (sg + sz - sz * sg);
    return dy * sz;
}

template <class T> __global__ void __launch_bounds__(512) group_norm_bwd_long_kernel(GroupNormParams p) {
    __shared__ float sm[16];
    const long long row = blockIdx.x / (unsigned)p.G;
    const int g = (int)(blockIdx.x % (unsigned)p.G);
    const long long col = (long long)g * p.C;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x + col, *z = static_cast<const T *>(p.gate) + row * p.ld_gate + col;
    const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy + col;
    T *dx = static_cast<T *>(p.y) + row * p.ld_y + col, *dgate = static_cast<T *>(p.dgate) + row * p.ld_dgate + col;
    const float mean = p.mean ? p.mean[row * p.G + g] : 0.f, rstd = p.rstd[row * p.G + g], inv = 1.f / (float)p.C;
    float s0 = 0.f, s1 = 0.f;
    auto column = [&](unsigned c, float &xh, float &dz) {
        const long long k = p.shared ? c : col + c;
        const float w = p.weight ? load_w(p.weight, k, p.w_bf16) : 1.f, b = p.bias ? load_w(p.bias, k, p.w_bf16) : 0.f;
        xh = (to_f(x[c]) - mean) * rstd;
        return gated(p, to_f(dy[c]), fmaf(xh, w, b), z + c, dz) * w;
    };
    for (unsigned c = threadIdx.x; c < (unsigned)p.C; c += 512) {
        float xh, dz;
        const float v = column(c, xh, dz);
        s0 += v;
        s1 = fmaf(v, xh, s1);
    }
    const float mg = p.center ? block_sum<512>(s0, sm) * inv : 0.f, mgx = block_sum<512>(s1, sm) * inv;
    for (unsigned c = threadIdx.x; c < (unsigned)p.C; c += 512) {
        float xh, dz;
        const float v = column(c, xh, dz);
        dx[c] = from_f<T>(rstd * (v - mg - xh * mgx));
        if (p.gate) dgate[c] = from_f<T>(dz);
    }
}

// The sums over rows for these: a thread per column of the weight, a part of the rows (of few rows whose groups share a weight: of the
// groups too) per block.  Sums of up to 256 terms at a time, and of up to 256 of those, so that one of many like terms keeps growing by them.
template <class T> __global__ void __launch_bounds__(256) group_norm_sums_kernel(GroupNormParams p, int row_parts, long long each_rows, int each_groups) {
    const long long cols = p.shared ? p.C : (long long)p.G * p.C, c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    const int gpart = blockIdx.y / row_parts;
    const long long r0 = (blockIdx.y % row_parts) * each_rows, r1 = min(r0 + each_rows, p.rows);
    const int g0 = p.shared ? gpart * each_groups : (int)(c / p.C), g1 = p.shared ? min(g0 + each_groups, p.G) : g0 + 1;
    const int in = (int)(p.shared ? c : c % p.C);
    const float w = p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f, b = p.bias ? load_w(p.bias, c, p.w_bf16) : 0.f;
    float aw = 0.f, ab = 0.f, mw = 0.f, mb = 0.f;
    for (long long row = r0; row < r1; ++row) {
        for (int from = g0; from < g1; from += 256) {
            float sw = 0.f, sb = 0.f;
            for (int g = from; g < min(from + 256, g1); ++g) {
                const long long k = (long long)g * p.C + in;
                const float mean = p.mean ? p.mean[row * p.G + g] : 0.f;
                const float xh = (to_f(static_cast<const T *>(p.x)[row * p.ld_x + k]) - mean) * p.rstd[row * p.G + g];
                float dz;
                const float d = gated(p, to_f(static_cast<const T *>(p.dy)[row * p.ld_dy + k]), fmaf(xh, w, b),
                                      static_cast<const T *>(p.gate) + row * p.ld_gate + k, dz);
                sw = fmaf(d, xh, sw);
                sb += d;
            }
            mw += sw;
            mb += sb;
        }
        if (row % 256 == 255 || row + 1 == r1 || g1 - g0 > 256) {
            aw += mw;
            ab += mb;
            mw = mb = 0.f;
        }
    }
    p.part[blockIdx.y * 2 * cols + c] = aw;
    p.part[blockIdx.y * 2 * cols + cols + c] = ab;
}

// The kernel form of a call: vectors, lanes and vectors per lane of a group, and the grid.
struct Plan {
    int V, L, items;            // items 0: the long form
    int per;
    unsigned gx, gy;            // blocks down the rows, and over the parts of the groups
    int parts;                  // rows of partial sums (the long form: row_parts times parts of the groups)
    int row_parts, each_groups;
    long long each_rows;
};
constexpr unsigned GRID_Y = 65535;       // what a grid's second axis takes: more parts take several launches, whose sums add up
Plan plan_of(const GroupNormParams &p, bool bf16_, bool bwd) {
    const size_t es = bf16_ ? 2 : 4;
    Plan q{};
    q.V = bf16_ ? 8 : 4;
    const bool wide = p.C % q.V == 0 && rows_aligned(p.x, p.ld_x, es, 16) && rows_aligned(p.gate, p.ld_gate, es, 16) &&
                      rows_aligned(p.y, p.ld_y, es, 16) && rows_aligned(p.dy, p.ld_dy, es, 16) &&
                      rows_aligned(p.dgate, p.ld_dgate, es, 16) && aligned_to(p.weight, 16) && aligned_to(p.bias, 16);
    if (!wide) q.V = 1;
    const int nv = p.C / q.V;
    q.L = 4;
    while (q.L < nv && q.L < 32) q.L *= 2;
    q.items = 1;
    while (q.L * q.items < nv && q.items < 4) q.items *= 2;
    while (q.L * q.items < nv && q.L < TPB) q.L *= 2;
    while (q.L * q.items < nv) q.items *= 2;
    const int sms = sm_count();
    if (q.items > (q.V == 8 ? 4 : 8)) {       // (eight vectors of eight and their sums do not fit the registers)
        q.items = 0;
        q.each_rows = (p.rows + 63) / 64;
        q.row_parts = (int)((p.rows + q.each_rows - 1) / q.each_rows);
        const int most = p.shared ? 64 / q.row_parts : 1;
        q.each_groups = (p.G - 1) / most + 1;
        q.parts = q.row_parts * (p.shared ? (p.G - 1) / q.each_groups + 1 : 1);
        return q;
    }
    q.per = slots_per_row(p.G, TPB / q.L);
    q.gy = (unsigned)((p.G - 1) / q.per + 1);
    const int rows = TPB / q.L / q.per;                      // rows of a block's visit
    const long long visits = (p.rows + rows - 1) / rows;
    // Blocks to an SM.  Vectors: as few as keep enough rows on their way (16384 x 16 x 128 bfloat16, L2 flushed: two take 41 us forward
    // and 76 backward, four 43 and 86; 8192 x 8 x 512: one backward 72, three 87).  Single elements are bound by instructions: as many as
    // an SM holds (8192 x 16 x 131: four 105 us forward, two 184).
    const int held = q.V == 1 ? (bwd ? (q.items == 1 ? 4 : q.items < 8 ? 2 : 1) : q.items < 8 ? 4 : 2)
                              : bwd ? (q.items == 1 && q.V == 8 ? 2 : 1) : q.items < 4 ? 2 : 1;
    long long gx = (long long)sms * held / q.gy;
    if (gx < 1) gx = 1;
    q.gx = (unsigned)(visits < gx ? visits : gx);
    q.parts = (int)(p.shared ? q.gx * (q.gy < GRID_Y ? q.gy : GRID_Y) : q.gx);
    return q;
}

template <auto KERNEL> cudaError_t launch(const GroupNormParams &p, const Plan &q, size_t smem, cudaStream_t s) {
    const cudaError_t e = allow_shared<KERNEL>(smem);
    if (e != cudaSuccess) return e;
    for (unsigned first = 0; first < q.gy; first += GRID_Y) {
        KERNEL<<<dim3(q.gx, q.gy - first < GRID_Y ? q.gy - first : GRID_Y), TPB, smem, s>>>(p, q.per, first);
        const cudaError_t l = cudaGetLastError();
        if (l != cudaSuccess) return l;
    }
    return cudaSuccess;
}
template <class T, int V, int ITEMS, int L, bool GATE, bool BIAS> cudaError_t run_bwd(const GroupNormParams &p, const Plan &q, cudaStream_t s) {
    using A = Ahead<T, V, ITEMS, GATE ? 3 : 2>;
    const size_t smem = A::SMEM + A::DEPTH * TPB * sizeof(float2), sums = TPB * 2 * V * sizeof(float);
    return launch<group_norm_bwd_kernel<T, V, ITEMS, L, GATE, BIAS>>(p, q, smem > sums ? smem : sums, s);
}
template <class T, int V, int ITEMS, int L>
cudaError_t run_one(const GroupNormParams &p, const Plan &q, bool bwd, cudaStream_t s) {
    if (bwd) {
        const bool bias = p.bias || p.dbias;
        if (p.gate) return bias ? run_bwd<T, V, ITEMS, L, true, true>(p, q, s) : run_bwd<T, V, ITEMS, L, true, false>(p, q, s);
        return bias ? run_bwd<T, V, ITEMS, L, false, true>(p, q, s) : run_bwd<T, V, ITEMS, L, false, false>(p, q, s);
    }
    if (p.gate) return launch<group_norm_fwd_kernel<T, V, ITEMS, L, true>>(p, q, Ahead<T, V, ITEMS, 2>::SMEM, s);
    return launch<group_norm_fwd_kernel<T, V, ITEMS, L, false>>(p, q, Ahead<T, V, ITEMS, 1>::SMEM, s);
}
template <class T, int V> cudaError_t run_v(const GroupNormParams &p, const Plan &q, bool bwd, cudaStream_t s) {
    switch (q.L * q.items) {
        case 4: return run_one<T, V, 1, 4>(p, q, bwd, s);
        case 8: return run_one<T, V, 1, 8>(p, q, bwd, s);
        case 16: return run_one<T, V, 1, 16>(p, q, bwd, s);
        case 32: return run_one<T, V, 1, 32>(p, q, bwd, s);
        case 64: return run_one<T, V, 2, 32>(p, q, bwd, s);
        case 128: return run_one<T, V, 4, 32>(p, q, bwd, s);
        case 256: return run_one<T, V, 4, 64>(p, q, bwd, s);
        case 512: return run_one<T, V, 4, 128>(p, q, bwd, s);
        case 1024: return run_one<T, V, 4, 256>(p, q, bwd, s);
    }
    if constexpr (V < 8) return run_one<T, V, 8, 256>(p, q, bwd, s);
    return cudaErrorInvalidValue;
}
template <class T> cudaError_t run_t(const GroupNormParams &p, const Plan &q, bool bwd, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T);
    if (q.items) return q.V == 1 ? run_v<T, 1>(p, q, bwd, s) : run_v<T, W>(p, q, bwd, s);
    const unsigned units = (unsigned)(p.rows * p.G);
    if (!bwd) {
        group_norm_fwd_long_kernel<T><<<units, 512, 0, s>>>(p);
        return cudaGetLastError();
    }
    group_norm_bwd_long_kernel<T><<<units, 512, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    const long long cols = p.shared ? p.C : (long long)p.G * p.C;
    group_norm_sums_kernel<T><<<dim3((unsigned)((cols + 255) / 256), q.parts), 256, 0, s>>>(p, q.row_parts, q.each_rows, q.each_groups);
    return cudaGetLastError();
}

}  // namespace

// Launches a call's kernels up to the partial sums of the parameters' gradients; one source file each, which compile side by side.
cudaError_t run_group_norm_bf16(const GroupNormParams &p, bool bwd, cudaStream_t s);
cudaError_t run_group_norm_f32(const GroupNormParams &p, bool bwd, cudaStream_t s);

}  // namespace mixer
