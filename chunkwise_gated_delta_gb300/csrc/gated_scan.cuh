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

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int COLS = 64;            // channels of a block, two per lane
constexpr int SAVE = GATED_SCAN_STATE_ROWS;  // rows from one saved state to the next (a tile of the backward)

// Two neighbouring channels of a row as they lie in memory: one access, or two with the channel past an odd
// end replaced by the last.
template <class T, bool VEC> struct Raw {
    Lanes<T, 2> v;
    __device__ __forceinline__ void load(const T *row, int c, int) { v.load(row + c); }
    __device__ __forceinline__ f2 pair() const { return v.pair(0); }
};
template <class T> struct Raw<T, false> {
    uint32_t w[2];
    __device__ __forceinline__ void load(const T *row, int c, int D) {
        w[0] = load_bits(row + c);
        w[1] = load_bits(row + min(c + 1, D - 1));
    }
    __device__ __forceinline__ f2 pair() const { return pack2(bits_f<T>(w[0]), bits_f<T>(w[1])); }
};
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

// p = 1 - exp(-q), q >= 0.  Below 1/4 six terms of the series: the seventh is below 5e-8 of the first.
__device__ __forceinline__ f2 one_less_exp(f2 q) {
    f2 s = fma2(q, both(-1.f / 720.f), both(1.f / 120.f));
    s = fma2(s, q, both(-1.f / 24.f));
    s = fma2(s, q, both(1.f / 6.f));
    s = fma2(s, q, both(-0.5f));
    s = fma2(s, q, both(1.f));
    s = mul2(s, q);
    float s0, s1, q0, q1, e0, e1;
    unpack2(s, s0, s1);
    unpack2(q, q0, q1);
    unpack2(mul2(q, both(-kLog2e)), e0, e1);
    return pack2(q0 < 0.25f ? s0 : 1.f - ex2(e0), q1 < 0.25f ? s1 : 1.f - ex2(e1));
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
// The decay and the input's weight without its gate: a and 1 - a^2.
__device__ __forceinline__ void decay_of(f2 q, f2 &a, f2 &w) {
    const f2 p = one_less_exp(q);
    a = fma2(p, both(-1.f), both(1.f));
    w = fma2(p, a, p);
}
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

// Where sequences begin and end among the N rows from r0 that a warp holds (bit j: row r0 + j), and the
// sequence of row r0 + lane.  The warp keeps the sequence of its last row: rows inside it take no search.
template <int N> struct Marks {
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
