// Gated feed-forward product on the CUDA cores, in float32: the form of float32 calls (whose products the tensor
// cores would round).
//
//   forward   h = act(x Wg^T) (x Wu^T), both products in one tile
//   backward  dg = dh u act'(g), du = dh act(g); dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x
//
// A block of 256 threads has a tile of 128 x 128 products, a thread 8 x 8 of them in two quads per axis; in the
// forward the left half of the columns is Wg's and the right half Wu's, so a thread has both of its outputs' products.
#include "glu.cuh"

namespace mixer {
namespace {

using namespace glu;

constexpr int TILE = 128, KT = 16, PITCH = TILE + 4;

// 8 elements of an operand's tile [KT][TILE] per thread: along k, or along the rows, whichever lies contiguous.
template <class T, bool KMAJOR> struct Stage {
    float v[8];
    // row0, k0: the tile's corner; rows, ks: the operand's extent; ld: stride between the non-contiguous axis' elements.
    __device__ __forceinline__ void load(const T *p, long long ld, long long row0, long long rows, long long k0, long long ks) {
        const int t = threadIdx.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const long long r = row0 + (KMAJOR ? t / 2 : t % 16 * 8 + e), k = k0 + (KMAJOR ? t % 2 * 8 + e : t / 16);
            v[e] = r < rows && k < ks ? to_f(p[KMAJOR ? r * ld + k : k * ld + r]) : 0.f;
        }
    }
    __device__ __forceinline__ void store(float (*sm)[PITCH], int at) const {
        const int t = threadIdx.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (KMAJOR) sm[t % 2 * 8 + e][at + t / 2] = v[e];
            else sm[t / 16][at + t % 16 * 8 + e] = v[e];
        }
    }
};

enum Mode { FWD, RECOMPUTE, DX, DW };

template <class T, Mode MODE> __global__ void __launch_bounds__(256, 2) glu_simt_kernel(GluParams p) {
    __shared__ __align__(16) float sa[2][KT][PITCH], sb[2][KT][PITCH];
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE, AK = MODE != DW, BK = DUAL;
    const int t = threadIdx.x, tx = t % 16, ty = t / 16;
    constexpr int TN = DUAL ? TILE / 2 : TILE;
    const bool up = MODE == DW && blockIdx.y;
    const long long ms = MODE == DW ? p.F : p.M, ns = DUAL ? p.F : p.D, ks = MODE == DW ? p.M : MODE == DX ? p.F : p.D;
    const unsigned cols = (unsigned)((ns + TN - 1) / TN);    // tiles of a row of tiles
    const long long m0 = (long long)(blockIdx.x / cols) * TILE, n0 = (long long)(blockIdx.x % cols) * TN;
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    Stage<T, AK> a;
    Stage<T, BK> b;
    const long long per = (ks + KT - 1) / KT, steps = MODE == DX ? 2 * per : per;
    auto fetch = [&](long long i) {
        if constexpr (DUAL) {
            a.load(static_cast<const T *>(p.x), p.ld_x, m0, ms, i * KT, ks);
            // rows 0 .. 63 of the tile from Wg, 64 .. 127 from Wu (threads 0 .. 127 and 128 .. 255)
            const bool right = t >= 128;
            const T *w = static_cast<const T *>(right ? p.wu : p.wg);
            b.load(w, right ? p.ld_wu : p.ld_wg, right ? n0 - TILE / 2 : n0, ns, i * KT, ks);
        } else if constexpr (MODE == DX) {
            const bool second = i >= per;
            const long long k0 = (second ? i - per : i) * KT;
            a.load(static_cast<const T *>(second ? p.du : p.dg), p.ld_d, m0, ms, k0, ks);
            b.load(static_cast<const T *>(second ? p.wu : p.wg), second ? p.ld_wu : p.ld_wg, n0, ns, k0, ks);
        } else {
            a.load(static_cast<const T *>(up ? p.du : p.dg), p.ld_d, m0, ms, i * KT, ks);
            b.load(static_cast<const T *>(p.x), p.ld_x, n0, ns, i * KT, ks);
        }
    };
    fetch(0);
    a.store(sa[0], 0);
    b.store(sb[0], 0);
    __syncthreads();
    for (long long i = 0; i < steps; ++i) {
        const int cur = i & 1;
        if (i + 1 < steps) fetch(i + 1);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float av[8], bv[8];
            *reinterpret_cast<float4 *>(av) = *reinterpret_cast<const float4 *>(&sa[cur][k][ty * 4]);
            *reinterpret_cast<float4 *>(av + 4) = *reinterpret_cast<const float4 *>(&sa[cur][k][64 + ty * 4]);
            *reinterpret_cast<float4 *>(bv) = *reinterpret_cast<const float4 *>(&sb[cur][k][tx * 4]);
            *reinterpret_cast<float4 *>(bv + 4) = *reinterpret_cast<const float4 *>(&sb[cur][k][64 + tx * 4]);
#pragma unroll
            for (int y = 0; y < 8; ++y)
#pragma unroll
                for (int x = 0; x < 8; ++x) acc[y][x] = fmaf(av[y], bv[x], acc[y][x]);
        }
        if (i + 1 < steps) {
            a.store(sa[cur ^ 1], 0);
            b.store(sb[cur ^ 1], 0);
        }
        __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < 8; ++y) {
        const long long m = m0 + (y < 4 ? ty * 4 + y : 60 + ty * 4 + y);
        if (m >= ms) continue;
        if constexpr (DUAL) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const long long n = n0 + tx * 4 + x;
                if (n >= ns) continue;
                const float g = acc[y][x], u = acc[y][x + 4];
                if constexpr (MODE == FWD) {
                    static_cast<T *>(p.h)[m * p.ld_h + n] = from_f<T>(act(g, p.gelu) * u);
                    if (p.g) {
                        p.g[m * p.F + n] = g;
                        p.u[m * p.F + n] = u;
                    }
                } else {
                    const Act f = act_and_slope(g, p.gelu);
                    const float d = to_f(static_cast<const T *>(p.dh)[m * p.ld_dh + n]);
                    static_cast<T *>(p.dg)[m * p.ld_d + n] = from_f<T>(d * u * f.d);
                    static_cast<T *>(p.du)[m * p.ld_d + n] = from_f<T>(d * f.v);
                }
            }
        } else {
            T *out = static_cast<T *>(MODE == DX ? p.dx : up ? p.dwu : p.dwg) + m * (MODE == DX ? p.ld_dx : up ? p.ld_dwu : p.ld_dwg);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const long long n = n0 + (x < 4 ? tx * 4 + x : 60 + tx * 4 + x);
                if (n < ns) out[n] = from_f<T>(acc[y][x]);
            }
        }
    }
}

// dg and du of saved products: V columns per thread.
template <class T, int V> __global__ void __launch_bounds__(256) glu_slope_kernel(GluParams p) {
    const long long per = (p.F + V - 1) / V, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * p.M) return;
    const long long m = i / per, n = (i - m * per) * V;
    float g[V], u[V];
    load_params<V>(g, p.g, m * p.F + n, false);
    load_params<V>(u, p.u, m * p.F + n, false);
    const Vec<T, V> d = load_const<T, V>(static_cast<const T *>(p.dh) + m * p.ld_dh + n);
    Vec<T, V> dg, du;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const Act f = act_and_slope(g[e], p.gelu);
        dg.e[e] = from_f<T>(to_f(d.e[e]) * u[e] * f.d);
        du.e[e] = from_f<T>(to_f(d.e[e]) * f.v);
    }
    store_vec<T, V>(static_cast<T *>(p.dg) + m * p.ld_d + n, dg);
    store_vec<T, V>(static_cast<T *>(p.du) + m * p.ld_d + n, du);
}

template <class T, Mode MODE> cudaError_t run_simt(const GluParams &p, cudaStream_t s) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE;
    const long long ms = MODE == DW ? p.F : p.M, ns = DUAL ? p.F : p.D, tn = DUAL ? TILE / 2 : TILE;
    const long long gy = (ms + TILE - 1) / TILE;
    const long long tiles = gy * ((ns + tn - 1) / tn);
    glu_simt_kernel<T, MODE><<<dim3((unsigned)tiles, MODE == DW ? 2 : 1), 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T> cudaError_t slopes(const GluParams &p, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T);
    const bool wide = p.F % W == 0 && rows_aligned(p.dh, p.ld_dh, sizeof(T), 16) && rows_aligned(p.dg, p.ld_d, sizeof(T), 16) &&
                      aligned_to(p.du, 16) && aligned_to(p.g, 16) && aligned_to(p.u, 16);
    const int v = wide ? W : 1;
    const long long n = (p.F + v - 1) / v * p.M;
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (wide) glu_slope_kernel<T, W><<<grid, 256, 0, s>>>(p);
    else glu_slope_kernel<T, 1><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T> cudaError_t bwd(const GluParams &p, cudaStream_t s) {
    cudaError_t e = p.g ? slopes<T>(p, s) : run_simt<T, RECOMPUTE>(p, s);
    if (e == cudaSuccess) e = run_simt<T, DX>(p, s);
    if (e == cudaSuccess) e = run_simt<T, DW>(p, s);
    return e;
}

}  // namespace

long long glu_grad_stride(const GluParams &p, bool bf16_) {
    const long long n = bf16_ ? 16 : 4;                      // rows of 32-byte sectors, of 16-byte accesses
    return (p.F + n - 1) / n * n;
}

cudaError_t launch_glu_fwd(const GluParams &p, bool bf16_, cudaStream_t s) {
    if (!bf16_) return run_simt<float, FWD>(p, s);
    if (glu_rows_takes(p)) return launch_glu_rows(p, s);
    return glu_tc_takes(p) ? launch_glu_tc_fwd(p, s) : run_simt<bf16, FWD>(p, s);
}
cudaError_t launch_glu_bwd(const GluParams &p, bool bf16_, cudaStream_t s) {
    if (!bf16_ || !glu_tc_takes(p)) return bf16_ ? bwd<bf16>(p, s) : bwd<float>(p, s);
    cudaError_t e = p.g ? slopes<bf16>(p, s) : launch_glu_tc_grads(p, s);
    if (e == cudaSuccess) e = launch_glu_tc_dx(p, s);
    if (e == cudaSuccess) e = launch_glu_tc_dw(p, s);
    return e;
}

}  // namespace mixer
