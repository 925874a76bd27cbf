// Layer norm over the last axis, forward and backward.
//
//   forward   mean = sum x / D, var = sum (x - mean)^2 / D over the row held in registers (two
//             passes over registers, so a large common offset cancels nothing), y = xh w + b,
//             xh = (x - mean) rstd.  2 elements of traffic per element.
//   backward  g = dy w, dx = rstd (g - mean(g) - xh mean(g xh)); dweight = sum_rows dy xh and
//             dbias = sum_rows dy are summed per thread over the rows that a block visits, then
//             over blocks by sum_rows_kernel: a fixed order, no atomics.  3 elements of traffic.
//
// Both are bound by HBM: 16384 rows of 2048 bfloat16 elements take 25 us (5.3 TB/s) and 36 us (5.5 TB/s),
// the sums over blocks 5 more.
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace {

// Sum of two values over a block of TPR threads.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *sm) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();                       // the previous sum has been read
    if (lane == 0) sm[warp] = v;
    __syncthreads();
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < TPR / 32; ++k) {
        r.x += sm[k].x;
        r.y += sm[k].y;
    }
    return r;
}

// Sums of N values (a power of two, at most 8) over a block of TPR threads: every thread ends with all of
// them.  A warp folds the values and its lanes into each other (half as many values at each step), so
// several rows cost hardly more than one.
template <int N, int TPR>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*sm)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int n = N, base = 0;
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        if (n > 1) {
            n /= 2;
            const bool up = lane & s;
            if (up) base += n;
#pragma unroll
            for (int k = 0; k < N / 2; ++k)
                if (k < n) {
                    const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
                    v[k] = keep + __shfl_xor_sync(~0u, send, s);
                }
        } else {
            v[0] += __shfl_xor_sync(~0u, v[0], s);
        }
    }
    __syncthreads();                       // the previous sums have been read
    if ((lane & (32 / N - 1)) == 0) sm[warp][base] = v[0];
    __syncthreads();
    // N times warps values, one per lane (the lanes beyond repeat them): over the warps, then to everyone
    constexpr int M = TPR / 32 * N;
    static_assert(M <= 32, "one value per lane");
    float t = (&sm[0][0])[lane % M];
#pragma unroll
    for (int s = N; s < M; s <<= 1) t += __shfl_xor_sync(~0u, t, s);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(~0u, t, k);
}

// Short rows: one per warp, lane i with vectors i and i + 32.
template <class T, int V, int ITEMS>
__global__ void __launch_bounds__(128) norm_fwd_warp_kernel(NormParams p) {
    constexpr int P = (V + 1) / 2;
    const int lane = threadIdx.x & 31, nv = p.D / V;       // V divides D
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    T *y = static_cast<T *>(p.y) + row * p.ld_y;
    Lanes<T, V> in[ITEMS];
    f2 v[ITEMS][P], acc = both(0.f);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) in[k].load(x + (size_t)min(lane + k * 32, nv - 1) * V);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            v[k][e] = in[k].pair(e);
            if (lane + k * 32 < nv) acc = add2(acc, v[k][e]);
        }
    const float mean = warp_sum(pair_sum<V>(acc)) / (float)p.D;
    acc = both(0.f);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            v[k][e] = add2(v[k][e], both(-mean));
            if (lane + k * 32 < nv) acc = fma2(v[k][e], v[k][e], acc);
        }
    const float rstd = inv_sqrt(warp_sum(pair_sum<V>(acc)) / (float)p.D + p.eps);
    if (lane == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (lane + k * 32 < nv) {
            const int c0 = (lane + k * 32) * V;
            f2 w[P], b[P], o[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                w[e] = both(1.f);
                b[e] = both(0.f);
            }
            if (p.weight) load_param_pairs<V>(w, p.weight, c0, p.w_bf16);
            if (p.bias) load_param_pairs<V>(b, p.bias, c0, p.w_bf16);
#pragma unroll
            for (int e = 0; e < P; ++e) o[e] = fma2(mul2(v[k][e], both(rstd)), w[e], b[e]);
            store_lanes<T, V>(y + c0, o);
        }
}

// Longer rows: a block owns all columns (and keeps their weights) and visits R neighbouring rows at a time,
// their sums taken together and the next R rows on their way.  A warp per row of 2048 bfloat16 elements,
// with the weights fetched for every row, took 33 to 56 us for 16384 rows; this takes 25 (traffic 20).
template <class T, int V, int ITEMS, int TPR, int R>
__global__ void __launch_bounds__(TPR, 512 / TPR) norm_fwd_kernel(NormParams p) {
    __shared__ float sm[TPR / 32][R];
    constexpr int P = (V + 1) / 2;
    const int tid = threadIdx.x, nv = p.D / V;
    const float inv = 1.f / (float)p.D;
    f2 w[ITEMS][P], b[ITEMS][P];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            w[k][e] = both(1.f);
            b[k][e] = both(0.f);
        }
        const long long c = (long long)min(tid + k * TPR, nv - 1) * V;
        if (p.weight) load_param_pairs<V>(w[k], p.weight, c, p.w_bf16);
        if (p.bias) load_param_pairs<V>(b[k], p.bias, c, p.w_bf16);
    }
    Lanes<T, V> in[R][ITEMS];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int r = 0; r < R; ++r) {      // past the end the last row and vector again, not counted
            const T *x = static_cast<const T *>(p.x) + (row + r < p.rows ? row + r : p.rows - 1) * p.ld_x;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) in[r][k].load(x + (size_t)min(tid + k * TPR, nv - 1) * V);
        }
    };
    const long long step = (long long)gridDim.x * R;
    fetch((long long)blockIdx.x * R);
    for (long long row = (long long)blockIdx.x * R; row < p.rows; row += step) {
        f2 v[R][ITEMS][P];
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f2 acc = both(0.f);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    v[r][k][e] = in[r][k].pair(e);
                    if (tid + k * TPR < nv) acc = add2(acc, v[r][k][e]);
                }
            s[r] = pair_sum<V>(acc);
        }
        fetch(row + step);
        block_sums<R, TPR>(s, sm);
        float mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = s[r] * inv;
            f2 acc = both(0.f);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    v[r][k][e] = add2(v[r][k][e], both(-mean[r]));
                    if (tid + k * TPR < nv) acc = fma2(v[r][k][e], v[r][k][e], acc);
                }
            s[r] = pair_sum<V>(acc);
        }
        block_sums<R, TPR>(s, sm);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row + r >= p.rows) break;
            const float rstd = inv_sqrt(s[r] * inv + p.eps);
            if (tid == 0) {
                if (p.mean) p.mean[row + r] = mean[r];
                if (p.rstd) p.rstd[row + r] = rstd;
            }
            T *y = static_cast<T *>(p.y) + (row + r) * p.ld_y;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (tid + k * TPR < nv) {
                    f2 o[P];
#pragma unroll
                    for (int e = 0; e < P; ++e) o[e] = fma2(mul2(v[r][k][e], both(rstd)), w[k][e], b[k][e]);
                    store_lanes<T, V>(y + (size_t)(tid + k * TPR) * V, o);
                }
        }
    }
}

// Rows too long for registers: three passes over the row (the later ones from L2), 1024 threads.  Columns
// are counted without a sign: a step past a width near 2^31 does not wrap below 0.
template <class T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormParams p) {
    __shared__ float2 sm[32];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    T *y = static_cast<T *>(p.y) + row * p.ld_y;
    float s = 0.f;
    for (unsigned c = threadIdx.x; c < (unsigned)p.D; c += 1024) s += to_f(x[c]);
    const float mean = row_sum2<1024>(make_float2(s, 0.f), sm).x / (float)p.D;
    float q = 0.f;
    for (unsigned c = threadIdx.x; c < (unsigned)p.D; c += 1024) {
        const float d = to_f(x[c]) - mean;
        q = fmaf(d, d, q);
    }
    const float rstd = inv_sqrt(row_sum2<1024>(make_float2(q, 0.f), sm).x / (float)p.D + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    for (unsigned c = threadIdx.x; c < (unsigned)p.D; c += 1024) {
        const float w = p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f;
        const float b = p.bias ? load_w(p.bias, c, p.w_bf16) : 0.f;
        y[c] = from_f<T>(fmaf((to_f(x[c]) - mean) * rstd, w, b));
    }
}

// Backward: a block owns all columns and visits R neighbouring rows at a time, their sums taken together
// and the next R rows on their way.
template <class T, int V, int ITEMS, int TPR, int R>
__global__ void __launch_bounds__(TPR, 512 / TPR) norm_bwd_kernel(NormParams p) {
    __shared__ float sm[TPR / 32][2 * R];
    constexpr int P = (V + 1) / 2;
    const int tid = threadIdx.x, nv = p.D / V;
    const float inv = 1.f / (float)p.D;
    f2 aw[ITEMS][P], ab[ITEMS][P], w[ITEMS][P];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            aw[k][e] = ab[k][e] = both(0.f);
            w[k][e] = both(1.f);
        }
        if (p.weight && tid + k * TPR < nv) load_param_pairs<V>(w[k], p.weight, (long long)(tid + k * TPR) * V, p.w_bf16);
    }
    Lanes<T, V> nx[R][ITEMS], nd[R][ITEMS];
    float nm[R], nr[R];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long q = row + r < p.rows ? row + r : p.rows - 1;     // past the end: the last row, not counted
            const T *x = static_cast<const T *>(p.x) + q * p.ld_x;
            const T *dy = static_cast<const T *>(p.dy) + q * p.ld_dy;
            nm[r] = p.mean[q];
            nr[r] = p.rstd[q];
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const size_t at = (size_t)min(tid + k * TPR, nv - 1) * V;
                nx[r][k].load(x + at);
                nd[r][k].load(dy + at);
            }
        }
    };
    const long long step = (long long)gridDim.x * R;
    fetch((long long)blockIdx.x * R);
    for (long long row = (long long)blockIdx.x * R; row < p.rows; row += step) {
        Lanes<T, V> vx[R][ITEMS], vd[R][ITEMS];
        float mean[R], rstd[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // The dy of a row past the end becomes zeros by its bits: times 0 an infinity of the last row, which
            // stands in for it, would turn the sums into NaN.
            const bool on = r == 0 || row + r < p.rows;
            mean[r] = nm[r];
            rstd[r] = nr[r];
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                vx[r][k] = nx[r][k];
                vd[r][k] = nd[r][k].kept(on);
            }
        }
        fetch(row + step);
        f2 xh[R][ITEMS][P], g[R][ITEMS][P];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (tid + k * TPR < nv)
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const f2 d = vd[r][k].pair(e);
                        xh[r][k][e] = mul2(add2(vx[r][k].pair(e), both(-mean[r])), both(rstd[r]));
                        g[r][k][e] = mul2(d, w[k][e]);
                        s0 = add2(s0, g[r][k][e]);
                        s1 = fma2(g[r][k][e], xh[r][k][e], s1);
                        aw[k][e] = fma2(d, xh[r][k][e], aw[k][e]);
                        ab[k][e] = add2(ab[k][e], d);
                    }
            s[2 * r] = pair_sum<V>(s0);
            s[2 * r + 1] = pair_sum<V>(s1);
        }
        block_sums<2 * R, TPR>(s, sm);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row + r >= p.rows) break;
            T *dx = static_cast<T *>(p.y) + (row + r) * p.ld_y;
            const f2 mg = both(-s[2 * r] * inv), mgx = both(-s[2 * r + 1] * inv);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (tid + k * TPR < nv) {
                    f2 o[P];
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        o[e] = mul2(fma2(xh[r][k][e], mgx, add2(g[r][k][e], mg)), both(rstd[r]));
                    store_lanes<T, V>(dx + (size_t)(tid + k * TPR) * V, o);
                }
        }
    }
    if (!p.part) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv) {
            const int c = (tid + k * TPR) * V;
            store_lanes<float, V>(part + c, aw[k]);
            store_lanes<float, V>(part + p.D + c, ab[k]);
        }
}

// Long rows: dx in two passes over the row, and the partial sums of a block of columns over a
// range of rows by a second kernel.
template <class T>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(NormParams p) {
    __shared__ float2 sm[32];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
    T *dx = static_cast<T *>(p.y) + row * p.ld_y;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (unsigned c = threadIdx.x; c < (unsigned)p.D; c += 1024) {
        const float g = to_f(dy[c]) * (p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f);
        s.x += g;
        s.y = fmaf(g, (to_f(x[c]) - mean) * rstd, s.y);
    }
    s = row_sum2<1024>(s, sm);
    const float mg = s.x / (float)p.D, mgx = s.y / (float)p.D;
    for (unsigned c = threadIdx.x; c < (unsigned)p.D; c += 1024) {
        const float g = to_f(dy[c]) * (p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f);
        dx[c] = from_f<T>(rstd * (g - mg - (to_f(x[c]) - mean) * rstd * mgx));
    }
}
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(NormParams p) {
    const unsigned c = blockIdx.x * 256 + threadIdx.x;      // (columns in x: y ends at 65535 blocks)
    if (c >= (unsigned)p.D) return;
    float aw = 0.f, ab = 0.f;
    for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float d = to_f(static_cast<const T *>(p.dy)[row * p.ld_dy + c]);
        const float xh = (to_f(static_cast<const T *>(p.x)[row * p.ld_x + c]) - p.mean[row]) * p.rstd[row];
        aw = fmaf(d, xh, aw);
        ab += d;
    }
    p.part[(size_t)blockIdx.y * 2 * p.D + c] = aw;
    p.part[(size_t)blockIdx.y * 2 * p.D + p.D + c] = ab;
}

// Blocks of the backward: two of 256 threads per SM (128 registers each) visit the rows, at least four
// each where there are that many.
int bwd_blocks(long long rows) {
    const long long most = 2LL * sm_count(), want = rows <= 256 ? rows : (rows + 3) / 4;
    return (int)(want < most ? want : most);
}

// Few rows: dx by one block per row and dweight, dbias by blocks of 32 columns that read all rows once more
// (from L2), in one launch and without partial sums.
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_few_kernel(NormParams p, int col_blocks) {
    __shared__ float2 sm[8][33];
    const int tid = threadIdx.x;
    if ((int)blockIdx.x < col_blocks) {
        const int tx = tid & 31, ty = tid >> 5, c = blockIdx.x * 32 + tx;
        float aw = 0.f, ab = 0.f;
        if (c < p.D)
#pragma unroll 4
            for (int row = ty; row < (int)p.rows; row += 8) {
                const float d = bits_f<T>(load_bits(static_cast<const T *>(p.dy) + row * p.ld_dy + c));
                const float x = bits_f<T>(load_bits(static_cast<const T *>(p.x) + row * p.ld_x + c));
                aw = fmaf(d, (x - __ldg(p.mean + row)) * __ldg(p.rstd + row), aw);
                ab += d;
            }
        sm[ty][tx] = make_float2(aw, ab);
        __syncthreads();
        if (ty == 0 && c < p.D) {
#pragma unroll
            for (int k = 1; k < 8; ++k) {
                aw += sm[k][tx].x;
                ab += sm[k][tx].y;
            }
            if (p.dweight) store_w(p.dweight, c, p.w_bf16, aw);
            if (p.dbias) store_w(p.dbias, c, p.w_bf16, ab);
        }
        return;
    }
    const long long row = blockIdx.x - col_blocks;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x, *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
    T *dx = static_cast<T *>(p.y) + row * p.ld_y;
    const float mean = p.mean[row], rstd = p.rstd[row];
    constexpr int K = 16;                        // D <= 256 K
    float g[K], xh[K];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = tid + 256 * k, cl = min(c, p.D - 1);
        g[k] = bits_f<T>(load_bits(dy + cl)) * (p.weight ? load_w(p.weight, cl, p.w_bf16) : 1.f);
        xh[k] = (bits_f<T>(load_bits(x + cl)) - mean) * rstd;
        if (c < p.D) {
            s.x += g[k];
            s.y = fmaf(g[k], xh[k], s.y);
        }
    }
    s = row_sum2<256>(s, &sm[0][0]);
    const float mg = s.x / (float)p.D, mgx = s.y / (float)p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (tid + 256 * k < p.D) dx[tid + 256 * k] = from_f<T>(rstd * (g[k] - mg - xh[k] * mgx));
}
// where the second reading costs less than a second launch
bool few_rows(const NormParams &p) { return p.rows <= 256 && p.D <= 4096; }

template <class T> constexpr int kVec = 16 / sizeof(T);

template <class T> bool vec_ok(const NormParams &p) {
    return p.D % kVec<T> == 0 && rows_aligned(p.x, p.ld_x, sizeof(T), 16) && rows_aligned(p.y, p.ld_y, sizeof(T), 16) &&
           rows_aligned(p.dy, p.ld_dy, sizeof(T), 16) &&
           aligned_to(p.weight, 16) && aligned_to(p.bias, 16);
}

template <class T, int V> cudaError_t fwd_vec(const NormParams &p, cudaStream_t s) {
    const int nv = p.D / V;
    if (nv <= 64) {
        const unsigned grid = (unsigned)((p.rows + 3) / 4);
        if (nv <= 32) norm_fwd_warp_kernel<T, V, 1><<<grid, 128, 0, s>>>(p);
        else norm_fwd_warp_kernel<T, V, 2><<<grid, 128, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (nv > (V == 1 ? 8 : 4) * 512) {
        norm_fwd_long_kernel<T><<<(unsigned)p.rows, 1024, 0, s>>>(p);
        return cudaGetLastError();
    }
    // two blocks of 256 threads (or one of 512) per SM; four rows at a time where there are rows enough
    const long long most = (nv <= 512 ? 2LL : 1LL) * sm_count();
    const unsigned blocks = (unsigned)(p.rows < most ? p.rows : most);
    if (nv <= 256 && p.rows >= 4 * most) norm_fwd_kernel<T, V, 1, 256, 4><<<blocks, 256, 0, s>>>(p);
    else if (nv <= 256) norm_fwd_kernel<T, V, 1, 256, 1><<<blocks, 256, 0, s>>>(p);
    else if (nv <= 512) norm_fwd_kernel<T, V, 2, 256, 1><<<blocks, 256, 0, s>>>(p);
    else if (nv <= 1024) norm_fwd_kernel<T, V, 2, 512, 1><<<blocks, 512, 0, s>>>(p);
    else if (nv <= 2048) norm_fwd_kernel<T, V, 4, 512, 1><<<blocks, 512, 0, s>>>(p);
    else if constexpr (V == 1) norm_fwd_kernel<T, V, 8, 512, 1><<<blocks, 512, 0, s>>>(p);
    return cudaGetLastError();
}

// Rows at a time: two while a thread has one vector of each; 512 threads where 256 would run out of
// registers.
template <class T, int V> cudaError_t bwd_vec(const NormParams &p, cudaStream_t s) {
    const int nv = p.D / V, blocks = bwd_blocks(p.rows);
    if (nv <= (V == 1 ? 8 : 2) * 512) {
        if (nv <= 256 && p.rows > blocks) norm_bwd_kernel<T, V, 1, 256, 2><<<blocks, 256, 0, s>>>(p);
        else if (nv <= 256) norm_bwd_kernel<T, V, 1, 256, 1><<<blocks, 256, 0, s>>>(p);
        else if (nv <= 512) norm_bwd_kernel<T, V, 2, 256, 1><<<blocks, 256, 0, s>>>(p);
        else if (nv <= 1024) norm_bwd_kernel<T, V, 2, 512, 1><<<blocks, 512, 0, s>>>(p);
        else if constexpr (V == 1) norm_bwd_kernel<T, V, 8, 512, 1><<<blocks, 512, 0, s>>>(p);
    } else {
        norm_bwd_long_kernel<T><<<(unsigned)p.rows, 1024, 0, s>>>(p);
        if (p.part) norm_bwd_cols_kernel<T><<<dim3(((unsigned)p.D + 255) / 256, blocks), 256, 0, s>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    return launch_sum_rows(p.part, blocks, {p.dweight, p.D, p.w_bf16}, {p.dbias, p.D, p.w_bf16}, s);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const NormParams &p, bool bf, cudaStream_t s) {
    if (bf) return vec_ok<bf16>(p) ? fwd_vec<bf16, 8>(p, s) : fwd_vec<bf16, 1>(p, s);
    return vec_ok<float>(p) ? fwd_vec<float, 4>(p, s) : fwd_vec<float, 1>(p, s);
}

cudaError_t launch_layer_norm_bwd(const NormParams &p, bool bf, cudaStream_t s) {
    if (few_rows(p)) {
        const int cols = p.dweight || p.dbias ? (p.D + 31) / 32 : 0;
        const unsigned grid = (unsigned)(cols + p.rows);
        if (bf) norm_bwd_few_kernel<bf16><<<grid, 256, 0, s>>>(p, cols);
        else norm_bwd_few_kernel<float><<<grid, 256, 0, s>>>(p, cols);
        return cudaGetLastError();
    }
    if (bf) return vec_ok<bf16>(p) ? bwd_vec<bf16, 8>(p, s) : bwd_vec<bf16, 1>(p, s);
    return vec_ok<float>(p) ? bwd_vec<float, 4>(p, s) : bwd_vec<float, 1>(p, s);
}

size_t layer_norm_part_floats(const NormParams &p) {
    return few_rows(p) ? 0 : (size_t)bwd_blocks(p.rows) * 2 * p.D;
}

}  // namespace mixer
