// Layer norm over the last axis, forward and backward.
//
//   forward   mean = sum x / D, var = sum (x - mean)^2 / D over the row held in registers (two
//             passes over registers, so a large common offset cancels nothing), y = xh w + b,
//             xh = (x - mean) rstd.  2 elements of traffic per element.
//   backward  g = dy w, dx = rstd (g - mean(g) - xh mean(g xh)); dweight = sum_rows dy xh and
//             dbias = sum_rows dy are summed per thread over the rows that a block visits, then
//             over blocks by sum_rows_kernel: a fixed order, no atomics.  3 elements of traffic.
//
// Both are bound by HBM.
#include "mixer_common.cuh"
#include "mixer_internal.h"

namespace mixer {
namespace {

// Sum over the TPR threads of a row of two values.  TPR = 32: one warp; otherwise the whole block.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *sm) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (TPR == 32) return v;
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

// One row per TPR threads, the row packed in registers: thread i holds vectors i, i + TPR, ...
template <class T, int V, int ITEMS, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) norm_fwd_kernel(NormParams p) {
    __shared__ float2 sm[TPR / 32];
    constexpr int ROWS = TPR == 32 ? 4 : 1;
    const int tid = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long row = (long long)blockIdx.x * ROWS + (TPR == 32 ? threadIdx.x >> 5 : 0);
    if (row >= p.rows) return;             // whole warps (TPR = 32) or the whole block
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    T *y = static_cast<T *>(p.y) + row * p.ld_y;
    const int nv = p.D / V;                // V divides D
    Vec<T, V> v[ITEMS];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv) v[k] = load_vec<T, V>(x + (size_t)(tid + k * TPR) * V);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv)
#pragma unroll
            for (int e = 0; e < V; ++e) s += to_f(v[k].e[e]);
    const float mean = row_sum2<TPR>(make_float2(s, 0.f), sm).x / (float)p.D;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float c = to_f(v[k].e[e]) - mean;
                q = fmaf(c, c, q);
            }
    const float rstd = 1.f / sqrtf(row_sum2<TPR>(make_float2(q, 0.f), sm).x / (float)p.D + p.eps);
    if (tid == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv) {
            const int c0 = (tid + k * TPR) * V;
            Vec<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float w = p.weight ? load_w(p.weight, c0 + e, p.w_bf16) : 1.f;
                const float b = p.bias ? load_w(p.bias, c0 + e, p.w_bf16) : 0.f;
                o.e[e] = from_f<T>(fmaf((to_f(v[k].e[e]) - mean) * rstd, w, b));
            }
            store_vec<T, V>(y + c0, o);
        }
}

// Rows too long for registers: three passes over the row (the later ones from L2), 1024 threads.
template <class T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormParams p) {
    __shared__ float2 sm[32];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    T *y = static_cast<T *>(p.y) + row * p.ld_y;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.D; c += 1024) s += to_f(x[c]);
    const float mean = row_sum2<1024>(make_float2(s, 0.f), sm).x / (float)p.D;
    float q = 0.f;
    for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float d = to_f(x[c]) - mean;
        q = fmaf(d, d, q);
    }
    const float rstd = 1.f / sqrtf(row_sum2<1024>(make_float2(q, 0.f), sm).x / (float)p.D + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float w = p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f;
        const float b = p.bias ? load_w(p.bias, c, p.w_bf16) : 0.f;
        y[c] = from_f<T>(fmaf((to_f(x[c]) - mean) * rstd, w, b));
    }
}

// Backward: a block owns all columns and visits every gridDim.x-th row.
template <class T, int V, int ITEMS, int TPR>
__global__ void __launch_bounds__(TPR) norm_bwd_kernel(NormParams p) {
    __shared__ float2 sm[TPR / 32];
    const int tid = threadIdx.x, nv = p.D / V;
    float aw[ITEMS][V], ab[ITEMS][V];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) aw[k][e] = ab[k][e] = 0.f;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
        const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
        T *dx = static_cast<T *>(p.y) + row * p.ld_y;
        const float mean = p.mean[row], rstd = p.rstd[row];
        Vec<T, V> vx[ITEMS], vd[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (tid + k * TPR < nv) {
                vx[k] = load_vec<T, V>(x + (size_t)(tid + k * TPR) * V);
                vd[k] = load_vec<T, V>(dy + (size_t)(tid + k * TPR) * V);
            }
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (tid + k * TPR < nv)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = (tid + k * TPR) * V + e;
                    const float d = to_f(vd[k].e[e]), xh = (to_f(vx[k].e[e]) - mean) * rstd;
                    const float g = p.weight ? d * load_w(p.weight, c, p.w_bf16) : d;
                    s.x += g;
                    s.y = fmaf(g, xh, s.y);
                    aw[k][e] = fmaf(d, xh, aw[k][e]);
                    ab[k][e] += d;
                }
        s = row_sum2<TPR>(s, sm);
        const float mg = s.x / (float)p.D, mgx = s.y / (float)p.D;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (tid + k * TPR < nv) {
                Vec<T, V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int c = (tid + k * TPR) * V + e;
                    const float d = to_f(vd[k].e[e]), xh = (to_f(vx[k].e[e]) - mean) * rstd;
                    const float g = p.weight ? d * load_w(p.weight, c, p.w_bf16) : d;
                    o.e[e] = from_f<T>(rstd * (g - mg - xh * mgx));
                }
                store_vec<T, V>(dx + (size_t)(tid + k * TPR) * V, o);
            }
    }
    if (!p.part) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (tid + k * TPR < nv)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = (tid + k * TPR) * V + e;
                part[c] = aw[k][e];
                part[p.D + c] = ab[k][e];
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
    for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float g = to_f(dy[c]) * (p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f);
        s.x += g;
        s.y = fmaf(g, (to_f(x[c]) - mean) * rstd, s.y);
    }
    s = row_sum2<1024>(s, sm);
    const float mg = s.x / (float)p.D, mgx = s.y / (float)p.D;
    for (int c = threadIdx.x; c < p.D; c += 1024) {
        const float g = to_f(dy[c]) * (p.weight ? load_w(p.weight, c, p.w_bf16) : 1.f);
        dx[c] = from_f<T>(rstd * (g - mg - (to_f(x[c]) - mean) * rstd * mgx));
    }
}
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(NormParams p) {
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= p.D) return;
    float aw = 0.f, ab = 0.f;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float d = to_f(static_cast<const T *>(p.dy)[row * p.ld_dy + c]);
        const float xh = (to_f(static_cast<const T *>(p.x)[row * p.ld_x + c]) - p.mean[row]) * p.rstd[row];
        aw = fmaf(d, xh, aw);
        ab += d;
    }
    p.part[(size_t)blockIdx.x * 2 * p.D + c] = aw;
    p.part[(size_t)blockIdx.x * 2 * p.D + p.D + c] = ab;
}

constexpr int kBwdBlocks = 2 * 152;    // two blocks of 256 threads per SM visit the rows

int bwd_blocks(long long rows) { return (int)(rows < kBwdBlocks ? rows : kBwdBlocks); }

template <class T> constexpr int kVec = 16 / sizeof(T);

template <class T> bool vec_ok(const NormParams &p) {
    return p.D % kVec<T> == 0 && rows_aligned(p.x, p.ld_x, sizeof(T), 16) && rows_aligned(p.y, p.ld_y, sizeof(T), 16) &&
           rows_aligned(p.dy, p.ld_dy, sizeof(T), 16);
}

template <class T, int V, int TPR>
cudaError_t fwd_items(const NormParams &p, int items, cudaStream_t s) {
    const unsigned grid = (unsigned)(TPR == 32 ? (p.rows + 3) / 4 : p.rows);
    const int threads = TPR == 32 ? 128 : TPR;
    if (items <= 1) norm_fwd_kernel<T, V, 1, TPR><<<grid, threads, 0, s>>>(p);
    else if (items <= 2) norm_fwd_kernel<T, V, 2, TPR><<<grid, threads, 0, s>>>(p);
    else if (items <= 4) norm_fwd_kernel<T, V, 4, TPR><<<grid, threads, 0, s>>>(p);
    else norm_fwd_kernel<T, V, 8, TPR><<<grid, threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T, int V> cudaError_t fwd_vec(const NormParams &p, cudaStream_t s) {
    const int nv = p.D / V;
    if (nv <= 8 * 32) return fwd_items<T, V, 32>(p, (nv + 31) / 32, s);
    if (nv <= 8 * 256) return fwd_items<T, V, 256>(p, (nv + 255) / 256, s);
    norm_fwd_long_kernel<T><<<(unsigned)p.rows, 1024, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T, int V, int TPR>
void bwd_items(const NormParams &p, int items, int blocks, cudaStream_t s) {
    if (items <= 1) norm_bwd_kernel<T, V, 1, TPR><<<blocks, TPR, 0, s>>>(p);
    else if (items <= 2) norm_bwd_kernel<T, V, 2, TPR><<<blocks, TPR, 0, s>>>(p);
    else norm_bwd_kernel<T, V, 4, TPR><<<blocks, TPR, 0, s>>>(p);
}

template <class T, int V> cudaError_t bwd_vec(const NormParams &p, cudaStream_t s) {
    const int nv = p.D / V, blocks = bwd_blocks(p.rows);
    if (nv <= 4 * 256) {
        bwd_items<T, V, 256>(p, (nv + 255) / 256, blocks, s);
    } else {
        norm_bwd_long_kernel<T><<<(unsigned)p.rows, 1024, 0, s>>>(p);
        if (p.part) norm_bwd_cols_kernel<T><<<dim3(blocks, (p.D + 255) / 256), 256, 0, s>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    return launch_sum_rows(p.part, blocks, {p.dweight, p.D, p.w_bf16}, {p.dbias, p.D, p.w_bf16}, {nullptr, 0, false}, s);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const NormParams &p, bool bf, cudaStream_t s) {
    if (bf) return vec_ok<bf16>(p) ? fwd_vec<bf16, 8>(p, s) : fwd_vec<bf16, 1>(p, s);
    return vec_ok<float>(p) ? fwd_vec<float, 4>(p, s) : fwd_vec<float, 1>(p, s);
}

cudaError_t launch_layer_norm_bwd(const NormParams &p, bool bf, cudaStream_t s) {
    if (bf) return vec_ok<bf16>(p) ? bwd_vec<bf16, 8>(p, s) : bwd_vec<bf16, 1>(p, s);
    return vec_ok<float>(p) ? bwd_vec<float, 4>(p, s) : bwd_vec<float, 1>(p, s);
}

size_t layer_norm_part_floats(const NormParams &p, bool) { return (size_t)bwd_blocks(p.rows) * 2 * p.D; }

}  // namespace mixer
