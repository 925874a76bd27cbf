// Pieces shared by the scan's forward, backward and single-token kernels.
//
// A channel's N states are spread over L lanes, a warp holds 32 / L channels; absent states have A = B = C = 0 and
// stay 0.  Single tokens and the gradient pass have four states per lane (L = 1, 2, 4 or 8 for N up to
// 4, 8, 16 or 32; the gradient pass 4 or 8), the forward and the local pass eight (four for N up to 4, and
// in the forward of few bfloat16 blocks).
#pragma once

#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {

constexpr int kScanThreads = 128;
constexpr int kBwdSegment = 64;      // tokens between boundary states in the backward
constexpr int kFwdLocal = 128;       // and in the split forward

// Added to the exponent of a decay, 2^(dt A log2 e): the special-function unit's results lie 0.5e-8 to 2.6e-8
// (relative) below the exact ones on average for exponents between -1 and 0 (measured), and a state
// multiplies as many of them as it remembers tokens.  With this the averages are within 1.2e-8 of 0 on
// all of that range, like expf's; at dt = 0 the decay is exactly 1.
constexpr float kDecayBias = 2.5e-8f;

// A log2 e.  An infinity (minus infinity: a state without memory) becomes the largest value of its sign: the
// tokens that fill the end of a tile have dt = 0 and leave the state as it is, but 0 times infinity is NaN.
__device__ __forceinline__ float decay_rate(float a) {
    const float v = a * kLog2e;
    return isinf(v) ? copysignf(3.402823466e38f, v) : v;
}

// log(1 + u) for u in [0, 1]: 2 atanh(s) with s = u / (2 + u) <= 1/3, atanh(s) = s + s^3 P(s^2) with P
// fitted for the smallest relative error of atanh on that interval (Lawson's reweighted least
// squares): 5.4e-9 with these four coefficients, below the rounding of one operation.  Relative
// accuracy holds down to u = 0, where steps of the order of 1e-3 and less come from.
constexpr float kAtanh[4] = {0.3333320915699005f, 0.2001076340675354f, 0.14000900089740753f, 0.14006005227565765f};
__device__ __forceinline__ float log1p_unit(float u) {
    const float s = u * rcp(2.f + u), q = s * s;
    const float r = fmaf(fmaf(fmaf(kAtanh[3], q, kAtanh[2]), q, kAtanh[1]), q, kAtanh[0]);
    return 2.f * fmaf(s * q, r, s);
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1p_unit(ex2(-kLog2e * fabsf(v))); }

// The same, kept in the order in which they are written.
__device__ __forceinline__ f2 mul2v(f2 a, f2 b) {
    f2 r;
    asm volatile("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2v(f2 a, f2 b, f2 c) {
    f2 r;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 ex2_2v(f2 v) {
    float a, b;
    unpack2(v, a, b);
    asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack2(a, b);
}
struct alignas(16) f2x2 {
    f2 a, b;
};

// softplus of two values at once.
__device__ __forceinline__ f2 softplus2(f2 v) {
    float a, b, lo, hi;
    unpack2(v, a, b);
    unpack2(mul2(pack2(fabsf(a), fabsf(b)), both(-kLog2e)), lo, hi);
    const f2 u = pack2(ex2(lo), ex2(hi));
    unpack2(add2(u, both(2.f)), lo, hi);
    const f2 s = mul2(u, pack2(rcp(lo), rcp(hi))), q = mul2(s, s);
    const f2 r = fma2(fma2(fma2(both(kAtanh[3]), q, both(kAtanh[2])), q, both(kAtanh[1])), q, both(kAtanh[0]));
    return fma2(fma2(mul2(s, q), r, s), both(2.f), pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
// The decays of two states.
__device__ __forceinline__ f2 decay2(f2 dt, f2 a2) { return ex2_2(fma2(dt, a2, both(kDecayBias))); }

// Sums v[k] over the L lanes of a channel; lane i ends with the sums of k = i K / L ... in v[0 ..].
// K is a multiple of L.
template <int K, int L> __device__ __forceinline__ void spread_sum(float (&v)[K], int i) {
    int n = K;
#pragma unroll
    for (int s = L / 2; s; s >>= 1) {
        n /= 2;
        const bool up = i & s;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < n) {
                const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
                v[k] = keep + __shfl_xor_sync(~0u, send, s);
            }
    }
}

// Rows t0 .. t0 + TT - 1 of Bm or Cm into shared memory as float32 [TT][NP], zero behind the
// segment's end and past N.  One thread per group of four states.
template <class T, int NP, int TT, int THREADS = kScanThreads>
__device__ __forceinline__ void stage_rows(float (*dst)[NP], const void *src, long long ld, int N, const Segment &g, int t0,
                                           bool vec) {
    constexpr int Q = NP / 4;
    for (int u = threadIdx.x; u < TT * Q; u += THREADS) {
        const int t = u / Q, n = u % Q * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + t < g.len) {
            const T *r = static_cast<const T *>(src) + (g.row0 + g.t0 + t0 + t) * ld + n;
            if (vec) {       // N = NP and rows aligned to four elements
                const Vec<T, 4> q = load_vec<T, 4>(r);
                v = make_float4(to_f(q.e[0]), to_f(q.e[1]), to_f(q.e[2]), to_f(q.e[3]));
            } else {
                if (n < N) v.x = to_f(r[0]);
                if (n + 1 < N) v.y = to_f(r[1]);
                if (n + 2 < N) v.z = to_f(r[2]);
                if (n + 3 < N) v.w = to_f(r[3]);
            }
        }
        *reinterpret_cast<float4 *>(&dst[t][n]) = v;
    }
}

// K states n0, n0 + 1, ... of a row of N into registers, and back.
template <int K> __device__ __forceinline__ void load_states(float (&h)[K], const float *row, int n0, int N) {
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = n0 + k < N ? row[n0 + k] : 0.f;
}
template <int K> __device__ __forceinline__ void store_states(float *row, const float (&h)[K], int n0, int N) {
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (n0 + k < N) row[n0 + k] = h[k];
}

template <class T> inline bool bc_vec_ok(const ScanParams &p, int NP) {
    return p.N == NP && rows_aligned(p.Bm, p.ld_B, sizeof(T), 4 * sizeof(T)) &&
           rows_aligned(p.Cm, p.ld_C, sizeof(T), 4 * sizeof(T));
}

// Lanes (of four states) per channel of the single-token kernel, and the forward's padded states.
inline int lanes_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }
inline int padded_states(int N) { return 4 * lanes_for(N); }

inline long long scan_slots(const ScanParams &p, int seg) { return segment_slots(p.B, p.T, seg, p.cu_seqlens != nullptr); }

// Local pass over every segment of p.lseg tokens: the state it ends with when it starts from zero
// (seg_state), its sum of dt (seg_dt) and, where grad is set, the gradient of the state entering
// it when none comes from behind (seg_grad).  Then the boundary pass turns them into the state
// entering and the gradient leaving each segment, in place.
cudaError_t launch_scan_segments(const ScanParams &p, bool bf16, bool grad, cudaStream_t s);

}  // namespace mixer
