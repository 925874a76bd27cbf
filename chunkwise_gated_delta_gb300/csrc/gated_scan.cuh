// What the forward, backward and single-token kernels of the gated recurrence share.
//
//   q = scale softplus(rate) sigmoid(decay),  a = exp(-q),  m = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(gate_t) x_t
//
// a is close to 1 for channels that remember long, and 1 - a^2 then loses its digits.  Where q < 1/4 both come from
// p = 1 - exp(-q), a series: a = 1 - p and 1 - a^2 = p (1 + a).  The difference 1 - p is rounded without a bias, which a
// long product of decays would multiply.  From 1/4 on a = exp(-q) is what has the digits, and p = 1 - a: gradients are products with
// a, and 1 - p would leave an error of 2^-25 where a may be 2^-25 itself (q = 17).
#pragma once

#include "mixer.h"
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace gs {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int COLS = 64;                          // channels of a warp, two per lane
constexpr int ROWS = GATED_SCAN_STATE_ROWS;       // rows that a warp has in hand at a time

// ROWS rows of a warp's channels in shared memory, and how they get there: accesses of CP bytes, asynchronous ones of 16
// or 4 bytes, or single bfloat16 elements (CP = 2).  Rows past the call's are its first or last, channels past D are
// left out (their lanes write nothing).
template <class T, int CP> struct Stage {
    static constexpr int ROW = COLS * (int)sizeof(T), BYTES = ROWS * ROW;
    static constexpr int PER = ROW / CP, STEP = PER < 32 ? 32 / PER : 1, PARTS = PER > 32 ? PER / 32 : 1;
    static constexpr int E = CP / (int)sizeof(T);        // elements of an access
    // This lane's first access of a row: its row of the first STEP, its channel of COLS.
    static __device__ __forceinline__ int row() { return (int)(threadIdx.x & 31) / PER; }
    static __device__ __forceinline__ int col() { return (int)(threadIdx.x & 31) % PER * E; }
    // Rows that lie inside; at: this lane's access of the first ones.  left: channels from this lane's to D.
    static __device__ __forceinline__ void bring(char *to, const T *at, long long ld, int left) {
        to += row() * ROW + col() * (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < ROWS / STEP; ++k, at += STEP * ld)
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
                if (part * 32 * E < left) one(to + k * STEP * ROW + part * 32 * CP, at + part * 32 * E);
    }
    static __device__ __forceinline__ void bring_clamped(char *to, const T *from, long long ld, int left, long long r0, const Extent &k) {
        to += row() * ROW + col() * (int)sizeof(T);
#pragma unroll 1
        for (int i = 0; i < ROWS / STEP; ++i) {
            const T *at = from + nearest_row(k, r0 + row() + i * STEP) * ld;
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
                if (part * 32 * E < left) one(to + i * STEP * ROW + part * 32 * CP, at + part * 32 * E);
        }
    }
    static __device__ __forceinline__ void one(char *to, const T *from) {
        if constexpr (CP == 2) *reinterpret_cast<unsigned short *>(to) = __ldg(reinterpret_cast<const unsigned short *>(from));
        else copy_async<CP>(to, from);
    }
    static __device__ __forceinline__ f2 pair(const char *rows, int row, int lane) {
        Lanes<T, 2> v;
        v.load_shared(rows + row * ROW + lane * 2 * (int)sizeof(T));
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

// A row's decay a, and p = 1 - a.
struct Decay {
    f2 p, a;
};
// p for 0 <= q < 1/4: six terms of the series, the seventh is below 5e-8 of the first.
constexpr float SMALL = 0.25f;
__device__ __forceinline__ f2 one_less_exp_small(f2 q) {
    f2 s = fma2(q, both(-1.f / 720.f), both(1.f / 120.f));
    s = fma2(s, q, both(-1.f / 24.f));
    s = fma2(s, q, both(1.f / 6.f));
    s = fma2(s, q, both(-0.5f));
    s = fma2(s, q, both(1.f));
    return mul2(s, q);
}
__device__ __forceinline__ f2 one_less(f2 v) { return fma2(v, both(-1.f), both(1.f)); }
// From one number per channel, which is what a pass keeps that takes a row's decay twice: p, or -a (a sign bit, also of 0) from 1/4 on.
// ALL_SMALL: no channel's exponent reaches 1/4.
template <bool ALL_SMALL> __device__ __forceinline__ f2 kept_decay(f2 q) {
    const f2 s = one_less_exp_small(q);
    if constexpr (ALL_SMALL) return s;
    float s0, s1, q0, q1, e0, e1;
    unpack2(s, s0, s1);
    unpack2(q, q0, q1);
    unpack2(mul2(q, both(-kLog2e)), e0, e1);
    return pack2(q0 < SMALL ? s0 : -ex2(e0), q1 < SMALL ? s1 : -ex2(e1));
}
template <bool ALL_SMALL> __device__ __forceinline__ Decay decay_of(f2 kept) {
    if constexpr (ALL_SMALL) return {kept, one_less(kept)};
    float k0, k1;
    unpack2(kept, k0, k1);
    const float t0 = fabsf(k0), t1 = fabsf(k1), o0 = 1.f - t0, o1 = 1.f - t1;
    const bool n0 = __float_as_int(k0) < 0, n1 = __float_as_int(k1) < 0;
    return {pack2(n0 ? o0 : t0, n1 ? o1 : t1), pack2(n0 ? t0 : o0, n1 ? t1 : o1)};
}
// Both at once, of exponents q >= 0.
template <bool ALL_SMALL> __device__ __forceinline__ Decay decay_at(f2 q) {
    const f2 s = one_less_exp_small(q);
    if constexpr (ALL_SMALL) return {s, one_less(s)};
    float s0, s1, o0, o1, q0, q1, e0, e1;
    unpack2(s, s0, s1);
    unpack2(one_less(s), o0, o1);
    unpack2(q, q0, q1);
    unpack2(mul2(q, both(-kLog2e)), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    float c0, c1;
    unpack2(one_less(pack2(e0, e1)), c0, c1);
    const bool b0 = q0 < SMALL, b1 = q1 < SMALL;
    return {pack2(b0 ? s0 : c0, b1 ? s1 : c1), pack2(b0 ? o0 : e0, b1 ? o1 : e1)};
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
// 1 - a^2 = p (1 + a).
__device__ __forceinline__ f2 rest_of(const Decay &d) { return fma2(d.p, d.a, d.p); }
__device__ __forceinline__ f2 sqrt2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(sqrt_fast(lo), sqrt_fast(hi));
}

// Where sequences begin and end among the rows from r0 that a warp holds (bit j: row r0 + j), and the
// sequence of row r0 + lane.  The warp keeps the sequence of its last row: rows inside it take no search.
struct Marks {
    static constexpr int N = ROWS;
    int lo = 1, hi = 0;                  // the kept sequence's rows
    unsigned starts, ends;
    int seq;
    __device__ __forceinline__ void find(const GatedScanParams &p, const Extent &k, long long r0) {
        starts = ends = 0;
        if (r0 > lo && r0 + N < hi) return;
        const int lane = threadIdx.x & 31;
        const long long row = r0 + lane;
        bool first = false, last = false;
        int a = 1, b = 0;
        if (lane < N && row >= k.lo && row < k.hi) {
            if (!p.cu_seqlens) {
                seq = (int)((unsigned)row / (unsigned)p.T);
                a = seq * p.T;
                b = a + p.T;
            } else {
                int x = 0, y = p.B - 1;          // the last sequence that begins at or before the row
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
