// Pieces shared by the scan's forward, backward and single-token kernels.
//
// A channel's N states are spread over L lanes, four states each (L = 1, 2, 4 or 8 for N up to
// 4, 8, 16 or 32; absent states have A = B = C = 0 and stay 0).  A warp holds 32 / L channels.
#pragma once

#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {

constexpr int kScanThreads = 128;
constexpr int kBwdSegment = 64;      // tokens between boundary states in the backward

// log(1 + u) for u in [0, 1]: 2 atanh(u / (2 + u)) by its series, whose argument is at most 1/3
// (the first term left out is below 2^-26 of the sum).  Relative accuracy holds down to u = 0,
// where steps of the order of 1e-3 and less come from.
__device__ __forceinline__ float log1p_unit(float u) {
    const float s = u * rcp(2.f + u), q = s * s;
    float r = 1.f / 15.f;
    r = fmaf(r, q, 1.f / 13.f);
    r = fmaf(r, q, 1.f / 11.f);
    r = fmaf(r, q, 1.f / 9.f);
    r = fmaf(r, q, 1.f / 7.f);
    r = fmaf(r, q, 1.f / 5.f);
    r = fmaf(r, q, 1.f / 3.f);
    return 2.f * fmaf(s * q, r, s);
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1p_unit(ex2(-kLog2e * fabsf(v))); }

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
template <class T, int NP, int TT>
__device__ __forceinline__ void stage_rows(float (*dst)[NP], const void *src, long long ld, int N, const Segment &g, int t0,
                                           bool vec) {
    constexpr int Q = NP / 4;
    for (int u = threadIdx.x; u < TT * Q; u += kScanThreads) {
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

// Four states of row `base` (of N) into registers, and back.
__device__ __forceinline__ void load_states(float (&h)[4], const float *row, int n0, int N) {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = n0 + k < N ? row[n0 + k] : 0.f;
}
__device__ __forceinline__ void store_states(float *row, const float (&h)[4], int n0, int N) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (n0 + k < N) row[n0 + k] = h[k];
}

template <class T> inline bool bc_vec_ok(const ScanParams &p, int NP) {
    return p.N == NP && rows_aligned(p.Bm, p.ld_B, sizeof(T), 4 * sizeof(T)) &&
           rows_aligned(p.Cm, p.ld_C, sizeof(T), 4 * sizeof(T));
}

inline int lanes_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }

inline long long scan_slots(const ScanParams &p, int seg) { return segment_slots(p.B, p.T, seg, p.cu_seqlens != nullptr); }

// Local pass over every segment of p.seg tokens: the state it ends with when it starts from zero
// (seg_state), its sum of dt (seg_dt) and, where grad is set, the gradient of the state entering
// it when none comes from behind (seg_grad).  Then the boundary pass turns them into the state
// entering and the gradient leaving each segment, in place.
cudaError_t launch_scan_segments(const ScanParams &p, bool bf16, bool grad, cudaStream_t s);

}  // namespace mixer
