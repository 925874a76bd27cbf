// What the forward, backward and single-token kernels of the gated recurrence share.
//
//   q = scale softplus(rate) sigmoid(decay),  a = exp(-q),  m = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(gate_t) x_t
//
// a is close to 1 for channels that remember long, and 1 - a^2 then loses its digits.  Both come from
// p = 1 - exp(-q), a series where q < 1/4: a = 1 - p and 1 - a^2 = p (1 + a).  The difference 1 - p is
// rounded without a bias, which a long product of decays would multiply.
#pragma once

#include "mixer.h"
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace gs {

constexpr int WARPS = 8, LANES = 32 * WARPS;     // warps that walk rows, their threads
constexpr int ROWS = 8, TILE = ROWS * WARPS;      // rows of a warp and of a block's tile
constexpr int COLS = 64;                          // channels of a block, two per lane
constexpr int SAVE = GATED_SCAN_STATE_ROWS;       // rows from one saved state to the next
static_assert(SAVE == TILE, "a saved state enters every tile of the backward");

// A tile's rows of one tensor in shared memory, and how they get there: accesses of CP bytes, asynchronous ones of 16 or
// 4 bytes, or single bfloat16 elements (CP = 2).  Rows past the chain are its first or last, channels past D are
// left out (their lanes write nothing).
template <class T, int CP> struct Stage {
    static constexpr int ROW = COLS * (int)sizeof(T), BYTES = TILE * ROW;
    static constexpr int PER = ROW / CP, STEP = LANES / PER < 1 ? 1 : LANES / PER;    // accesses of a row, rows at a time
    static constexpr int E = CP / (int)sizeof(T) < 1 ? 1 : CP / (int)sizeof(T);       // elements of an access
    static __device__ __forceinline__ void bring(char *to, const T *from, long long ld, int c0, int D, long long r0, int lo, int hi) {
        const int t = threadIdx.x, at = t % PER * E, row = t / PER;
        if (c0 + at >= D) return;
        const T *p = from + c0 + at;
        char *q = to + row * ROW + at * (int)sizeof(T);
        if (r0 >= lo && r0 + TILE <= hi) {               // a tile inside: one stride
            const T *s = p + (r0 + row) * ld;
#pragma unroll
            for (int k = 0; k < TILE / STEP; ++k, s += STEP * ld) one(q + k * STEP * ROW, s);
        } else {
#pragma unroll
            for (int k = 0; k < TILE / STEP; ++k) {
                const long long r = r0 + row + k * STEP;
                one(q + k * STEP * ROW, p + (r < lo ? lo : r >= hi ? hi - 1 : r) * ld);
            }
        }
    }
    static __device__ __forceinline__ void one(char *to, const T *from) {
        if constexpr (CP == 2) *reinterpret_cast<unsigned short *>(to) = __ldg(reinterpret_cast<const unsigned short *>(from));
        else copy_async<CP>(to, from);
    }
    static __device__ __forceinline__ f2 pair(const char *tile, int row, int lane) {
        Lanes<T, 2> v;
        v.load_shared(tile + row * ROW + lane * 2 * (int)sizeof(T));
        return v.pair(0);
    }
};
// Two neighbouring channels: one access, or two with the channel past an odd end left out.
template <class T, bool VEC> __device__ __forceinline__ void store_pair(T *row, int c, int D, f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    if constexpr (VEC) {
        store_vec<T, 2>(row + c, Vec<T, 2>{{from_f<T>(lo), from_f<T>(hi)}});
    } else {
        row[c] = from_f<T>(lo);
        if (c + 1 < D) row[c + 1] = from_f<T>(hi);
    }
}
template <class T> __device__ __forceinline__ f2 load_pair(const T *row, int c, int D) {
    return pack2(bits_f<T>(load_bits(row + c)), bits_f<T>(load_bits(row + min(c + 1, D - 1))));
}
// The float32 vectors of D channels (states) have no row stride: pairs are aligned where D is even.
__device__ __forceinline__ f2 load_state(const float *row, int c, int D) { return pack2(row[c], row[min(c + 1, D - 1)]); }
__device__ __forceinline__ void store_state(float *row, int c, int D, f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    row[c] = lo;
    if (c + 1 < D) row[c + 1] = hi;
}

// scale softplus(rate) of two channels.
__device__ __forceinline__ float softplus_of(float v) { return v > 20.f ? v : log1pf(expf(v)); }
__device__ __forceinline__ f2 coefficients(const GatedScanParams &p, int c) {
    return pack2(p.scale * softplus_of(p.rate[c]), p.scale * softplus_of(p.rate[min(c + 1, p.D - 1)]));
}

// p = 1 - exp(-q) for 0 <= q < 1/4: six terms of the series, the seventh is below 5e-8 of the first; and for any q >= 0.
constexpr float SMALL = 0.25f;
__device__ __forceinline__ f2 one_less_exp_small(f2 q) {
    f2 s = fma2(q, both(-1.f / 720.f), both(1.f / 120.f));
    s = fma2(s, q, both(-1.f / 24.f));
    s = fma2(s, q, both(1.f / 6.f));
    s = fma2(s, q, both(-0.5f));
    s = fma2(s, q, both(1.f));
    return mul2(s, q);
}
__device__ __forceinline__ f2 one_less_exp(f2 q) {
    float s0, s1, q0, q1, e0, e1;
    unpack2(one_less_exp_small(q), s0, s1);
    unpack2(q, q0, q1);
    unpack2(mul2(q, both(-kLog2e)), e0, e1);
    return pack2(q0 < SMALL ? s0 : 1.f - ex2(e0), q1 < SMALL ? s1 : 1.f - ex2(e1));
}
// Of several at once: a warp whose exponents are all small leaves the exponential out (the same values).
template <int N> __device__ __forceinline__ void one_less_exps(f2 (&q)[N]) {
    bool large = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float lo, hi;
        unpack2(q[j], lo, hi);
        large |= !(lo < SMALL && hi < SMALL);
    }
    if (__any_sync(~0u, large)) {
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = one_less_exp(q[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = one_less_exp_small(q[j]);
    }
}
__device__ __forceinline__ float sqrt_fast(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsqrt_fast(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// From p: the decay a = 1 - p, and 1 - a^2 = p (1 + a).
__device__ __forceinline__ f2 decay_of(f2 p) { return fma2(p, both(-1.f), both(1.f)); }
__device__ __forceinline__ f2 rest_of(f2 p, f2 a) { return fma2(p, a, p); }
__device__ __forceinline__ f2 sqrt2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(sqrt_fast(lo), sqrt_fast(hi));
}

// The rows and sequences of one chain: neighbouring sequences that blocks walk one after the other, as one
// axis that is cut at every sequence's first row.  Dense batches: B / P sequences each.  Packed ones: the
// sequences that begin in the p-th of P equal parts of the T rows.
struct Chain {
    int s0, s1;         // sequences
    int c0, c1;         // rows
};
__device__ __forceinline__ int first_at(const int32_t *cu, int B, long long row) {
    int lo = 0, hi = B;                  // the first sequence that begins at or behind the row
    while (lo < hi) {
        const int mid = (int)(((long long)lo + hi) >> 1);
        if (cu[mid] >= row) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ Chain chain_of(const int32_t *cu, int B, int T, int P, int p) {
    Chain k;
    if (!cu) {
        k.s0 = (int)((long long)p * B / P);
        k.s1 = (int)((long long)(p + 1) * B / P);
        k.c0 = k.s0 * T;
        k.c1 = k.s1 * T;
    } else {
        k.s0 = p ? first_at(cu, B, (long long)p * T / P) : 0;
        k.s1 = p + 1 < P ? first_at(cu, B, (long long)(p + 1) * T / P) : B;
        k.c0 = clamped(cu[k.s0], 0, T);
        k.c1 = k.s1 > k.s0 ? clamped(cu[k.s1], k.c0, T) : k.c0;
    }
    return k;
}

// Where sequences begin and end among the rows from r0 that a warp holds (bit j: row r0 + j), and the
// sequence of row r0 + lane.  The warp keeps the sequence of its last row: rows inside it take no search.
struct Marks {
    static constexpr int N = ROWS;
    int lo = 1, hi = 0;                  // the kept sequence's rows
    unsigned starts, ends;
    int seq;
    __device__ __forceinline__ void find(const GatedScanParams &p, const Chain &k, long long r0) {
        starts = ends = 0;
        if (r0 > lo && r0 + N < hi) return;
        const int lane = threadIdx.x & 31;
        const long long row = r0 + lane;
        bool first = false, last = false;
        int a = 1, b = 0;
        if (lane < N && row >= k.c0 && row < k.c1) {
            if (!p.cu_seqlens) {
                seq = (int)((unsigned)row / (unsigned)p.T);
                a = seq * p.T;
                b = a + p.T;
            } else {
                int x = k.s0, y = k.s1 - 1;          // the last sequence that begins at or before the row
                while (x < y) {
                    const int mid = (int)(((long long)x + y + 1) >> 1);
                    if (p.cu_seqlens[mid] <= row) x = mid;
                    else y = mid - 1;
                }
                seq = x;
                a = clamped(p.cu_seqlens[x], 0, p.T);
                b = clamped(p.cu_seqlens[x + 1], a, p.T);
            }
            first = row == a;
            last = row == b - 1;
        }
        starts = __ballot_sync(~0u, first);
        ends = __ballot_sync(~0u, last);
        lo = __shfl_sync(~0u, a, N - 1);
        hi = __shfl_sync(~0u, b, N - 1);
    }
    __device__ __forceinline__ int sequence(int j) const { return __shfl_sync(~0u, seq, j); }
};

}  // namespace gs
}  // namespace mixer
