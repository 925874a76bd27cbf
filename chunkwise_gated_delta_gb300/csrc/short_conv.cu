// Short causal convolution per channel, with an optional SiLU: forward, backward, single tokens.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y_t = act(pre_t)
//   dpre_t = dy_t act'(pre_t),  dx_p = sum_j w_j dpre_{p+W-1-j},
//   dw_j = sum_t dpre_t x_{t-W+1+j},  dbias = sum_t dpre_t
//
// A unit of work is V neighbouring channels of one segment of a sequence; a thread walks its
// tokens with the last W - 1 inputs in registers, so every row is read once (and the W - 1 rows
// before a segment once more).  Bound by HBM.
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace {

template <class T, int V> __device__ __forceinline__ void load_f(float (&o)[V], const T *p) {
    const Vec<T, V> v = load_vec<T, V>(p);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = to_f(v.e[e]);
}
template <class T, int V> __device__ __forceinline__ void store_f(T *p, const float (&o)[V]) {
    Vec<T, V> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = from_f<T>(o[e]);
    store_vec<T, V>(p, v);
}

// Input at position t of a sequence: its tokens, then (t < 0) the initial state, then zeros.
template <class T, int W, int V>
__device__ __forceinline__ void load_input(float (&o)[V], const ConvParams &p, const Segment &g, int t, int c) {
    if (t >= 0)
        load_f<T, V>(o, static_cast<const T *>(p.x) + (g.row0 + t) * p.ld_x + c);
    else if (p.h0)
        load_f<T, V>(o, static_cast<const T *>(p.h0) + ((long long)g.b * (W - 1) + t + W - 1) * p.D + c);
    else
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
}

template <int W, int V>
__device__ __forceinline__ void load_taps(float (&w)[W][V], float (&b)[V], const ConvParams &p, int c) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = load_w(p.weight, (long long)(c + e) * W + j, p.w_bf16);
        b[e] = p.bias ? load_w(p.bias, c + e, p.w_bf16) : 0.f;
    }
}

template <class T, int W, int V>
__global__ void __launch_bounds__(128) conv_fwd_kernel(ConvParams p, long long slots) {
    const int groups = p.D / V;
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long slot = u / groups;
    const int c = (int)(u - slot * groups) * V;
    Segment g;
    if (slot >= slots || !segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    float w[W][V], bias[V], win[W][V];
    load_taps<W, V>(w, bias, p, c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_input<T, W, V>(win[j], p, g, g.t0 - (W - 1) + j, c);
    const T *x = static_cast<const T *>(p.x) + (g.row0 + g.t0) * p.ld_x + c;
    T *y = static_cast<T *>(p.y) + (g.row0 + g.t0) * p.ld_y + c;
    for (int t0 = 0; t0 < g.len; t0 += 4) {
        Vec<T, V> in[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t0 + k < g.len) in[k] = load_vec<T, V>(x + (t0 + k) * p.ld_x);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t0 + k < g.len) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    win[W - 1][e] = to_f(in[k].e[e]);
                    float pre = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) pre = fmaf(w[j][e], win[j][e], pre);
                    o[e] = p.silu ? pre * sigmoid(pre) : pre;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j][e] = win[j + 1][e];
                }
                store_f<T, V>(y + (t0 + k) * p.ld_y, o);
            }
    }
    if (p.ht && g.i == g.n - 1)     // the last inputs, the state's among them after a short sequence
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_f<T, V>(static_cast<T *>(p.ht) + ((long long)g.b * (W - 1) + j) * p.D + c, win[j]);
}

// Backward of V channels of one segment: tokens t0 .. t0 + len + W - 2, the last W - 1 of which
// belong to the next segment (their dpre is computed there again for dw and dbias).
// blockDim = (32 channel groups, 4 segments); the four partial sums are joined in shared memory.
template <class T, int W, int V>
__global__ void __launch_bounds__(128) conv_bwd_kernel(ConvParams p, long long slots) {
    __shared__ float sm[3][(W + 1) * V][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int groups = p.D / V, gx = (groups + 31) / 32;
    const long long by = blockIdx.x / gx;
    const int grp = (int)(blockIdx.x - by * gx) * 32 + lane;
    const int c = grp * V;
    const long long slot = by * 4 + row;
    float dw[W][V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    Segment g;
    if (grp < groups && slot < slots && segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) {
        float w[W][V], bias[V], win[W][V], dp[W][V];     // dp[i]: dpre of token t - (W - 1) + i
        load_taps<W, V>(w, bias, p, c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_input<T, W, V>(win[j], p, g, g.t0 - (W - 1) + j, c);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) dp[j][e] = 0.f;
        const int end = g.t0 + g.len + W - 1;
        for (int t = g.t0; t < end; ++t) {
            if (t < g.total) {
                float dy[V];
                load_f<T, V>(win[W - 1], static_cast<const T *>(p.x) + (g.row0 + t) * p.ld_x + c);
                load_f<T, V>(dy, static_cast<const T *>(p.dy) + (g.row0 + t) * p.ld_dy + c);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float d = dy[e];
                    if (p.silu) {
                        float pre = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) pre = fmaf(w[j][e], win[j][e], pre);
                        const float sg = sigmoid(pre);
                        d *= sg * fmaf(pre, 1.f - sg, 1.f);
                    }
                    dp[W - 1][e] = d;
                    if (t < g.t0 + g.len) {
                        db[e] += d;
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][e] = fmaf(d, win[j][e], dw[j][e]);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) dp[W - 1][e] = win[W - 1][e] = 0.f;
            }
            const int q = t - (W - 1);                   // its gradient is complete now
            if (q >= g.t0 || (g.i == 0 && q < 0 && p.dh0)) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    o[e] = 0.f;
#pragma unroll
                    for (int i = 0; i < W; ++i) o[e] = fmaf(w[W - 1 - i][e], dp[i][e], o[e]);
                }
                const int k = q - (g.total - (W - 1));   // its place in the final state
                if (p.dht && k >= 0) {
                    float h[V];
                    load_f<T, V>(h, static_cast<const T *>(p.dht) + ((long long)g.b * (W - 1) + k) * p.D + c);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += h[e];
                }
                if (q >= 0)
                    store_f<T, V>(static_cast<T *>(p.y) + (g.row0 + q) * p.ld_y + c, o);
                else
                    store_f<T, V>(static_cast<T *>(p.dh0) + ((long long)g.b * (W - 1) + q + W - 1) * p.D + c, o);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    win[j][e] = win[j + 1][e];
                    dp[j][e] = dp[j + 1][e];
                }
        }
    }
    if (!p.part) return;
    if (row)
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) sm[row - 1][e * W + j][lane] = dw[j][e];
            sm[row - 1][W * V + e][lane] = db[e];
        }
    __syncthreads();
    if (row == 0 && grp < groups) {
        float *out = p.part + by * (long long)p.D * (W + 1);
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                out[(long long)(c + e) * W + j] =
                    dw[j][e] + sm[0][e * W + j][lane] + sm[1][e * W + j][lane] + sm[2][e * W + j][lane];
            out[(long long)p.D * W + c + e] =
                db[e] + sm[0][W * V + e][lane] + sm[1][W * V + e][lane] + sm[2][W * V + e][lane];
        }
    }
}

template <class T, int W, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvParams p) {
    const int groups = p.D / V;
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const int b = (int)(u / groups), c = (int)(u - (long long)b * groups) * V;
    if (b >= p.B) return;
    const int slot = p.slot ? p.slot[b] : b;
    T *y = static_cast<T *>(p.y) + (long long)b * p.ld_y + c;
    float o[V];
    if (slot < 0 || slot >= p.slots) {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
        store_f<T, V>(y, o);
        return;
    }
    T *st = static_cast<T *>(p.state) + (long long)slot * (W - 1) * p.D + c;
    Vec<T, V> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = load_vec<T, V>(st + (long long)j * p.D);
    in[W - 1] = load_vec<T, V>(static_cast<const T *>(p.x) + (long long)b * p.ld_x + c);
    float w[W][V], bias[V];
    load_taps<W, V>(w, bias, p, c);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float pre = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) pre = fmaf(w[j][e], to_f(in[j].e[e]), pre);
        o[e] = p.silu ? pre * sigmoid(pre) : pre;
    }
    store_f<T, V>(y, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_vec<T, V>(st + (long long)j * p.D, in[j + 1]);
}

template <class T, int V> bool conv_vec_ok(const ConvParams &p) {
    const size_t es = sizeof(T), n = V * es;
    return p.D % V == 0 && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.y, p.ld_y, es, n) &&
           rows_aligned(p.dy, p.ld_dy, es, n) && rows_aligned(p.h0, p.D, es, n) && rows_aligned(p.ht, p.D, es, n) &&
           rows_aligned(p.dht, p.D, es, n) && rows_aligned(p.dh0, p.D, es, n) && rows_aligned(p.state, p.D, es, n);
}

enum Way { kFwd, kBwd, kStep };

template <class T, int W, int V> cudaError_t conv_launch(const ConvParams &p, Way way, cudaStream_t s) {
    const int groups = p.D / V;
    if (way == kStep) {
        const long long blocks = ((long long)p.B * groups + 127) / 128;
        if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
        conv_step_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p);
        return cudaGetLastError();
    }
    const long long slots = segment_slots(p.B, p.T, p.seg, p.cu_seqlens != nullptr);
    const long long blocks = way == kFwd ? (slots * groups + 127) / 128 : (slots + 3) / 4 * ((groups + 31) / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    if (way == kFwd) conv_fwd_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p, slots);
    else conv_bwd_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p, slots);
    return cudaGetLastError();
}

template <class T, int W> cudaError_t conv_width(const ConvParams &p, Way way, cudaStream_t s) {
    return conv_vec_ok<T, 4>(p) ? conv_launch<T, W, 4>(p, way, s) : conv_launch<T, W, 1>(p, way, s);
}

template <class T> cudaError_t conv_type(const ConvParams &p, int W, Way way, cudaStream_t s) {
    switch (W) {
    case 2: return conv_width<T, 2>(p, way, s);
    case 3: return conv_width<T, 3>(p, way, s);
    default: return conv_width<T, 4>(p, way, s);
    }
}

}  // namespace

cudaError_t launch_short_conv_fwd(const ConvParams &q, int W, bool bf, cudaStream_t s) {
    ConvParams p = q;
    p.seg = 16;
    return bf ? conv_type<bf16>(p, W, kFwd, s) : conv_type<float>(p, W, kFwd, s);
}

constexpr int kBwdSeg = 32;

size_t short_conv_part_floats(const ConvParams &p, int W) {
    const long long slots = segment_slots(p.B, p.T, kBwdSeg, p.cu_seqlens != nullptr);
    return (size_t)((slots + 3) / 4) * p.D * (W + 1);
}

cudaError_t launch_short_conv_bwd(const ConvParams &q, int W, bool bf, cudaStream_t s) {
    ConvParams p = q;
    p.seg = kBwdSeg;
    const cudaError_t e = bf ? conv_type<bf16>(p, W, kBwd, s) : conv_type<float>(p, W, kBwd, s);
    if (e != cudaSuccess || !p.part) return e;
    const long long slots = segment_slots(p.B, p.T, kBwdSeg, p.cu_seqlens != nullptr);
    return launch_sum_rows(p.part, (int)((slots + 3) / 4), {p.dweight, (long long)p.D * W, p.w_bf16},
                           {p.dbias, p.D, p.w_bf16}, {nullptr, 0, false}, s);
}

cudaError_t launch_short_conv_step(const ConvParams &p, int W, bool bf, cudaStream_t s) {
    return bf ? conv_type<bf16>(p, W, kStep, s) : conv_type<float>(p, W, kStep, s);
}

}  // namespace mixer
