// Short causal convolution per channel, with an optional SiLU: forward, backward, single tokens.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y_t = act(pre_t)
//   dpre_t = dy_t act'(pre_t),  dx_p = sum_j w_j dpre_{p+W-1-j},
//   dw_j = sum_t dpre_t x_{t-W+1+j},  dbias = sum_t dpre_t
//
// A unit of work is V neighbouring channels of one segment of a sequence; a thread walks its
// tokens with the last W - 1 inputs in registers, so every row is read once (and the W - 1 rows
// before a segment once more).  The forward is bound by HBM (B 8, T 2048, D 4096, four taps, bfloat16:
// 47 us, 5.7 TB/s), the backward by instructions and the loads' latency: its taps, window and sums leave
// 16 warps to an SM, their rows on the way in shared memory (8191 x 2048: 29 us, 3.5 TB/s).
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace {

// Input at position t of a sequence as pairs: its tokens, then (t < 0) the initial state, then zeros.
template <class T, int W, int V>
__device__ __forceinline__ void load_input(f2 (&o)[(V + 1) / 2], const ConvParams &p, const Segment &g, int t, int c) {
    Lanes<T, V> v;
    if (t >= 0) v.load(static_cast<const T *>(p.x) + (g.row0 + t) * p.ld_x + c);
    else if (p.h0) v.load(static_cast<const T *>(p.h0) + ((long long)g.b * (W - 1) + t + W - 1) * p.D + c);
#pragma unroll
    for (int e = 0; e < (V + 1) / 2; ++e) o[e] = t >= 0 || p.h0 ? v.pair(e) : both(0.f);
}

// The taps and bias of V channels as pairs: V W neighbouring parameters, in accesses of V.
template <int W, int V>
__device__ __forceinline__ void load_taps(f2 (&w)[W][(V + 1) / 2], f2 (&b)[(V + 1) / 2], const ConvParams &p, int c) {
    float q[W][V];
#pragma unroll
    for (int j = 0; j < W; ++j) load_params<V>(q[j], p.weight, (long long)c * W + j * V, p.w_bf16);
#pragma unroll
    for (int e = 0; e < (V + 1) / 2; ++e) {
        const int lo = 2 * e, hi = V == 1 ? 0 : 2 * e + 1;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = pack2(q[(lo * W + j) / V][(lo * W + j) % V], q[(hi * W + j) / V][(hi * W + j) % V]);
        b[e] = both(0.f);
    }
    if (p.bias) load_param_pairs<V>(b, p.bias, c, p.w_bf16);
}

template <class T, int W, int V>
__global__ void __launch_bounds__(128, 4) conv_fwd_kernel(ConvParams p, long long slots) {
    constexpr int P = (V + 1) / 2;
    const int groups = p.D / V;
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long slot = u / groups;
    const int c = (int)(u - slot * groups) * V;
    Segment g;
    if (slot >= slots || !segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) return;
    f2 w[W][P], bias[P], win[W][P];
    load_taps<W, V>(w, bias, p, c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_input<T, W, V>(win[j], p, g, g.t0 - (W - 1) + j, c);
    const T *x = static_cast<const T *>(p.x) + (g.row0 + g.t0) * p.ld_x + c;
    T *y = static_cast<T *>(p.y) + (g.row0 + g.t0) * p.ld_y + c;
    // four rows at a time, the next four on their way (past the end the last row again, without a branch)
    Lanes<T, V> in[4], next[4];
    auto fetch = [&](int last) {               // rows 0 .. 3 from x, at most up to row `last`
#pragma unroll
        for (int k = 0; k < 4; ++k) next[k].load(x + min(k, last) * p.ld_x);
        x += 4 * p.ld_x;
    };
    auto token = [&](const Lanes<T, V> &v) {
        f2 o[P];
#pragma unroll
        for (int e = 0; e < P; ++e) {
            win[W - 1][e] = v.pair(e);
            f2 pre = bias[e];
#pragma unroll
            for (int j = 0; j < W; ++j) pre = fma2(w[j][e], win[j][e], pre);
            o[e] = p.silu ? silu2(pre) : pre;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j][e] = win[j + 1][e];
        }
        store_lanes<T, V>(y, o);
        y += p.ld_y;
    };
    int left = g.len;
    if (left > 0) fetch(left - 1);
    for (; left >= 4; left -= 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) in[k] = next[k];
        fetch(left - 5);                       // (at or before the last row)
#pragma unroll
        for (int k = 0; k < 4; ++k) token(in[k]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < left) token(next[k]);
    if (p.ht && g.i == g.n - 1)     // the last inputs, the state's among them after a short sequence
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_lanes<T, V>(static_cast<T *>(p.ht) + ((long long)g.b * (W - 1) + j) * p.D + c, win[j]);
}

// Backward of V channels of one segment: tokens t0 .. t0 + len + W - 2, the last W - 1 of which
// belong to the next segment (their dpre is computed there again for dw and dbias).
// A block: 32 channel groups, 4 segments; the four partial sums are joined in shared memory.
constexpr int kBwdBlocks = 4;        // to an SM
template <class T, int W, int V>
__global__ void __launch_bounds__(128, kBwdBlocks) conv_bwd_kernel(ConvParams p, long long slots) {
    constexpr int P = (V + 1) / 2, BYTES = V * sizeof(T);
    // Rows on their way: groups of four, asynchronous copies into words of the thread's own (a register
    // ring of one group leaves too few bytes in flight); single bfloat16 elements, which are too small
    // for that, one group ahead in registers.
    constexpr bool RING = BYTES >= 4;
    constexpr int GROUPS = BYTES == 16 ? 2 : 3;
    __shared__ __align__(16) unsigned char ring[RING ? GROUPS * 8 * 128 * BYTES : 16];
    __shared__ f2 sm[3][(W + 1) * P][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int groups = p.D / V, gx = (groups + 31) / 32;
    const long long by = blockIdx.x / gx;
    const int grp = (int)(blockIdx.x - by * gx) * 32 + lane;
    const int c = grp * V;
    const long long slot = by * 4 + row;
    f2 dw[W][P], db[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
        db[e] = both(0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = both(0.f);
    }
    Segment g;
    if (grp < groups && slot < slots && segment_of(p.cu_seqlens, p.B, p.T, p.seg, slot, g)) {
        f2 w[W][P], bias[P], win[W][P], dp[W][P];     // dp[i]: dpre of token t - (W - 1) + i
        load_taps<W, V>(w, bias, p, c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_input<T, W, V>(win[j], p, g, g.t0 - (W - 1) + j, c);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) dp[j][e] = both(0.f);
        const T *x = static_cast<const T *>(p.x) + (g.row0 + g.t0) * p.ld_x + c;
        const T *gy = static_cast<const T *>(p.dy) + (g.row0 + g.t0) * p.ld_dy + c;
        T *dx = static_cast<T *>(p.y) + (g.row0 + g.t0) * p.ld_y + c;
        // dpre of token t from its input and dy
        auto dpre = [&](const Lanes<T, V> &xi, const Lanes<T, V> &di, bool mine) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                win[W - 1][e] = xi.pair(e);
                f2 d = di.pair(e);
                if (p.silu) {
                    f2 pre = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) pre = fma2(w[j][e], win[j][e], pre);
                    const f2 sg = sigmoid2(pre);      // SiLU' = sg (1 + pre (1 - sg))
                    d = mul2(mul2(d, sg), fma2(pre, fma2(sg, both(-1.f), both(1.f)), both(1.f)));
                }
                dp[W - 1][e] = d;
                if (mine) {
                    db[e] = add2(db[e], d);
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][e] = fma2(d, win[j][e], dw[j][e]);
                }
            }
        };
        // the gradient of position t - (W - 1), complete now
        auto gradient = [&](f2 (&o)[P]) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                o[e] = mul2(w[W - 1][e], dp[0][e]);
#pragma unroll
                for (int i = 1; i < W; ++i) o[e] = fma2(w[W - 1 - i][e], dp[i][e], o[e]);
            }
        };
        auto shift = [&] {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    win[j][e] = win[j + 1][e];
                    dp[j][e] = dp[j + 1][e];
                }
        };
        // where the gradient of position q goes: its row, or the initial state's (nowhere before another segment)
        auto put = [&](int q, f2 (&o)[P]) {
            const int h = q - (g.total - (W - 1));       // its place in the final state
            if (p.dht && h >= 0) {
                Lanes<T, V> v;
                v.load(static_cast<const T *>(p.dht) + ((long long)g.b * (W - 1) + h) * p.D + c);
#pragma unroll
                for (int e = 0; e < P; ++e) o[e] = add2(o[e], v.pair(e));
            }
            if (q >= g.t0) store_lanes<T, V>(dx + (q - g.t0) * p.ld_y, o);
            else if (q < 0 && p.dh0) store_lanes<T, V>(static_cast<T *>(p.dh0) + ((long long)g.b * (W - 1) + q + W - 1) * p.D + c, o);
        };
        Lanes<T, V> xi[4], di[4], xn[RING ? 1 : 4], dn[RING ? 1 : 4];
        const int last = g.total - 1 - g.t0;             // the sequence's last row from here
        int ahead = 0, at = 0;                           // first row of the next copy; the ring's next group
        auto word = [&](int group, int k) { return ring + (((group * 4 + k) * 2) * 128 + threadIdx.x) * BYTES; };
        auto copy = [&](int group) {                     // past the sequence's end its last row again
            if (last >= 0)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const long long r = min(ahead + k, last);
                    copy_async<RING ? BYTES : 4>(word(group, k), x + r * p.ld_x);
                    copy_async<RING ? BYTES : 4>(word(group, k) + 128 * BYTES, gy + r * p.ld_dy);
                }
            copies_end();
            ahead += 4;
        };
        auto next = [&] {
            if (last >= 0)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const long long r = min(ahead + k, last);
                    xn[RING ? 0 : k].load(x + r * p.ld_x);
                    dn[RING ? 0 : k].load(gy + r * p.ld_dy);
                }
            ahead += 4;
        };
        if constexpr (RING) {
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) copy(k);
        } else {
            next();
        }
        T *out = dx - (W - 1) * p.ld_y;                  // of position t - (W - 1)
        auto four = [&] {                                // the next four rows to work on
            if constexpr (RING) {
                copies_wait<GROUPS - 1>();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xi[k].load_shared(word(at, k));
                    di[k].load_shared(word(at, k) + 128 * BYTES);
                }
                copy(at);
                at = at == GROUPS - 1 ? 0 : at + 1;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xi[k] = xn[RING ? 0 : k];
                    di[k] = dn[RING ? 0 : k];
                }
                next();
            }
        };
        auto edge = [&](int t) {                         // near the ends of the segment or of the sequence
            four();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t + k < g.len) {
                    f2 o[P];
                    dpre(xi[k], di[k], true);
                    gradient(o);
                    put(g.t0 + t + k - (W - 1), o);
                    shift();
                }
            out += 4 * p.ld_y;
        };
        int t = 0;
        if (g.len > 0) edge(0);
        // inside, with nothing to ask for: positions t - (W - 1) .. are this segment's, and before the final state's
        for (t = 4; t + 4 <= g.len; t += 4) {
            four();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f2 o[P];
                dpre(xi[k], di[k], true);
                gradient(o);
                store_lanes<T, V>(out, o);
                out += p.ld_y;
                shift();
            }
        }
        for (; t < g.len; t += 4) edge(t);
        if constexpr (RING) copies_wait<0>();
        // the W - 1 tokens behind the segment: the next segment's, or none (dpre = 0)
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = g.len + k;
            f2 o[P];
            if (t <= last) {
                Lanes<T, V> a, b;
                a.load(x + (long long)t * p.ld_x);
                b.load(gy + (long long)t * p.ld_dy);
                dpre(a, b, false);
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e) dp[W - 1][e] = win[W - 1][e] = both(0.f);
            }
            gradient(o);
            put(g.t0 + t - (W - 1), o);
            shift();
        }
    }
    if (!p.part) return;
    if (row)
#pragma unroll
        for (int e = 0; e < P; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) sm[row - 1][e * W + j][lane] = dw[j][e];
            sm[row - 1][W * P + e][lane] = db[e];
        }
    __syncthreads();
    if (row == 0 && grp < groups) {
        float *out = p.part + by * (long long)p.D * (W + 1);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float lo, hi;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                unpack2(add2(add2(dw[j][e], sm[0][e * W + j][lane]), add2(sm[1][e * W + j][lane], sm[2][e * W + j][lane])), lo, hi);
                out[(long long)(c + 2 * e) * W + j] = lo;
                if (V > 1) out[(long long)(c + 2 * e + 1) * W + j] = hi;
            }
            unpack2(add2(add2(db[e], sm[0][W * P + e][lane]), add2(sm[1][W * P + e][lane], sm[2][W * P + e][lane])), lo, hi);
            out[(long long)p.D * W + c + 2 * e] = lo;
            if (V > 1) out[(long long)p.D * W + c + 2 * e + 1] = hi;
        }
    }
}

template <class T, int W, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvParams p) {
    const int groups = p.D / V;
    const long long u = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long b = u / groups;                // (the last block's threads may pass 2^31 requests)
    const int c = (int)(u - b * groups) * V;
    if (b >= p.B) return;
    const int slot = p.slot ? p.slot[b] : (int)b;
    T *y = static_cast<T *>(p.y) + b * p.ld_y + c;
    constexpr int P = (V + 1) / 2;
    f2 o[P];
    if (slot < 0 || slot >= p.slots) {
#pragma unroll
        for (int e = 0; e < P; ++e) o[e] = both(0.f);
        store_lanes<T, V>(y, o);
        return;
    }
    T *st = static_cast<T *>(p.state) + (long long)slot * (W - 1) * p.D + c;
    Vec<T, V> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = load_vec<T, V>(st + (long long)j * p.D);
    in[W - 1] = load_vec<T, V>(static_cast<const T *>(p.x) + b * p.ld_x + c);
    f2 w[W][P], bias[P];
    load_taps<W, V>(w, bias, p, c);
#pragma unroll
    for (int e = 0; e < P; ++e) {
        f2 pre = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j)
            pre = fma2(w[j][e], pack2(to_f(in[j].e[2 * e]), V == 1 ? 0.f : to_f(in[j].e[V == 1 ? 0 : 2 * e + 1])), pre);
        o[e] = p.silu ? silu2(pre) : pre;
    }
    store_lanes<T, V>(y, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_vec<T, V>(st + (long long)j * p.D, in[j + 1]);
}

template <class T, int V> bool conv_vec_ok(const ConvParams &p) {
    const size_t es = sizeof(T), n = V * es;
    return p.D % V == 0 && aligned_to(p.weight, 16) && aligned_to(p.bias, 16) && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.y, p.ld_y, es, n) &&
           rows_aligned(p.dy, p.ld_dy, es, n) && rows_aligned(p.h0, p.D, es, n) && rows_aligned(p.ht, p.D, es, n) &&
           rows_aligned(p.dht, p.D, es, n) && rows_aligned(p.dh0, p.D, es, n) && rows_aligned(p.state, p.D, es, n);
}

enum Way { kFwd, kBwd, kStep };

template <class T, int W, int V> cudaError_t fwd_start(const ConvParams &p, cudaStream_t s) {
    const long long slots = segment_slots(p.B, p.T, p.seg, p.cu_seqlens != nullptr), blocks = (slots * (p.D / V) + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    conv_fwd_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p, slots);
    return cudaGetLastError();
}
template <class T, int W, int V> cudaError_t other_start(const ConvParams &p, Way way, cudaStream_t s) {
    const int groups = p.D / V;
    const long long slots = segment_slots(p.B, p.T, p.seg, p.cu_seqlens != nullptr);
    const long long blocks = way == kStep ? ((long long)p.B * groups + 127) / 128 : (slots + 3) / 4 * ((groups + 31) / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    if (way == kStep) conv_step_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p);
    else conv_bwd_kernel<T, W, V><<<(unsigned)blocks, 128, 0, s>>>(p, slots);
    return cudaGetLastError();
}

// Channels per access: 16 bytes in the forward, four channels in the backward (whose taps, window and
// sums are four times V values per tap) and for single tokens (whose threads are few); else one.
template <class T, int W> cudaError_t conv_width(const ConvParams &p, Way way, cudaStream_t s) {
    constexpr int F = 16 / sizeof(T);
    const bool four = conv_vec_ok<T, 4>(p);
    if (way != kFwd) return four ? other_start<T, W, 4>(p, way, s) : other_start<T, W, 1>(p, way, s);
    if (conv_vec_ok<T, F>(p)) return fwd_start<T, W, F>(p, s);
    return fwd_start<T, W, 1>(p, s);
}

template <class T> cudaError_t conv_type(const ConvParams &p, int W, Way way, cudaStream_t s) {
    switch (W) {
    case 2: return conv_width<T, 2>(p, way, s);
    case 3: return conv_width<T, 3>(p, way, s);
    default: return conv_width<T, 4>(p, way, s);
    }
}

}  // namespace

namespace {
// Tokens per thread.  Each segment costs its tokens plus about eight for the taps and the rows before
// it, and the last wave of blocks should be full: the length with the smallest number of waves times
// cost, `resident` blocks of 128 threads to an SM.
int segment_length(const ConvParams &p, int V, int resident) {
    const long long tokens = (long long)(p.cu_seqlens ? 1 : p.B) * p.T, groups = (p.D + V - 1) / V;
    const long long room = 128LL * resident * sm_count();
    long long best = 0;
    int seg = 4;
    for (int s = 4; s <= 64; s += 4) {
        const long long threads = ((tokens + s - 1) / s + (p.cu_seqlens ? p.B : 0)) * groups, cost = (threads + room - 1) / room * (s + 8);
        if (!best || cost <= best) {
            best = cost;
            seg = s;
        }
    }
    return seg;
}
int bwd_segment(const ConvParams &p) { return segment_length(p, 4, kBwdBlocks); }
}  // namespace

cudaError_t launch_short_conv_fwd(const ConvParams &q, int W, bool bf, cudaStream_t s) {
    ConvParams p = q;
    p.seg = segment_length(p, bf ? 8 : 4, 4);
    return bf ? conv_type<bf16>(p, W, kFwd, s) : conv_type<float>(p, W, kFwd, s);
}

size_t short_conv_part_floats(const ConvParams &p, int W) {
    const long long slots = segment_slots(p.B, p.T, bwd_segment(p), p.cu_seqlens != nullptr);
    return (size_t)((slots + 3) / 4) * p.D * (W + 1);
}

cudaError_t launch_short_conv_bwd(const ConvParams &q, int W, bool bf, cudaStream_t s) {
    ConvParams p = q;
    p.seg = bwd_segment(p);
    const cudaError_t e = bf ? conv_type<bf16>(p, W, kBwd, s) : conv_type<float>(p, W, kBwd, s);
    if (e != cudaSuccess || !p.part) return e;
    const long long slots = segment_slots(p.B, p.T, p.seg, p.cu_seqlens != nullptr);
    return launch_sum_rows(p.part, (int)((slots + 3) / 4), {p.dweight, (long long)p.D * W, p.w_bf16},
                           {p.dbias, p.D, p.w_bf16}, s);
}

cudaError_t launch_short_conv_step(const ConvParams &q, int W, bool bf, cudaStream_t s) {
    ConvParams p = q;
    p.seg = 1;
    return bf ? conv_type<bf16>(p, W, kStep, s) : conv_type<float>(p, W, kStep, s);
}

}  // namespace mixer
