// Gated feed-forward product: choice of form, float32 calls, and what surrounds the tensor cores' products.
//
//   forward   h = act(x Wg^T) (x Wu^T), both products in one tile
//   backward  dg = dh u act'(g), du = dh act(g); dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x
//
// float32 products run on the CUDA cores, which do not round their operands.  A block has a tile of SIDE x SIDE products, a thread
// two quads of them per axis, two columns to a packed multiplication; in the forward the left half of the columns is Wg's and the
// right half Wu's.  Where tiles of 128 leave the GPU idle, tiles of 64 are used, and a cluster of up to sixteen blocks shares the
// sum of a tile, joined in the blocks' order through shared memory.  Bound by the multiplications: 2048 x 1024 x 2048 takes 359 us,
// 48 TFLOP/s (with one multiplication per instruction and 4-byte loads 431).
#include <type_traits>

#include "glu.cuh"
#include "tc_common.cuh"

namespace mixer {
namespace {

using namespace glu;

enum Mode { FWD, RECOMPUTE, DX, DW };

template <int SIDE> struct Tiles {
    static constexpr int THREADS = SIDE * SIDE / 64, KT = 16, PITCH = SIDE + 4, E = SIDE * KT / THREADS;
    static constexpr int STAGE = KT * PITCH;                 // floats of an operand's tile
    static constexpr int SUMS = SIDE == 64 ? SIDE * (SIDE + 1) : 0, FLOATS = 4 * STAGE > SUMS ? 4 * STAGE : SUMS;
    static_assert(FLOATS * 4 <= 48 * 1024, "no more than every kernel may have");
};

// E elements of an operand's tile [KT][SIDE] per thread, V (1 or 4) per access, neighbouring threads along the axis that lies
// contiguous (k, or the rows).  With V = 4 that axis' extent is a multiple of 4.
template <int SIDE, bool KMAJOR, int V> struct Operand {
    using S = Tiles<SIDE>;
    static constexpr int LEN = (KMAJOR ? S::KT : SIDE) / V, STEP = S::THREADS / LEN, N = S::E / V;   // accesses of a stretch; stretches at a time
    Vec<float, V> v[N];
    // p: the tile's first element; left_r, left_k: the operand's extent from there; ld: stride of the axis that is not contiguous.
    __device__ __forceinline__ void load(const float *p, long long ld, long long left_r, long long left_k) {
        const int in = threadIdx.x % LEN * V, out = threadIdx.x / LEN;
        p += out * ld + in;
        const bool inside = in < (KMAJOR ? left_k : left_r);
#pragma unroll
        for (int e = 0; e < N; ++e, p += STEP * ld) one(e, p, inside && out + e * STEP < (KMAJOR ? left_r : left_k));
    }
    __device__ __forceinline__ void one(int e, const float *p, bool on) {
        if (on) v[e] = load_const<float, V>(p);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) v[e].e[i] = 0.f;
    }
    __device__ __forceinline__ void store(float *sm) const {
        const int in = threadIdx.x % LEN * V, out = threadIdx.x / LEN;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (KMAJOR)
#pragma unroll
                for (int i = 0; i < V; ++i) sm[(in + i) * S::PITCH + out + e * STEP] = v[e].e[i];
            else store_vec<float, V>(sm + (out + e * STEP) * S::PITCH + in, v[e]);
        }
    }
};
// The forward's tile of weights: its first half of rows from Wg, its second from Wu, k contiguous.
template <int SIDE, int V> struct Weights : Operand<SIDE, true, V> {
    using O = Operand<SIDE, true, V>;
    static constexpr int TN = SIDE / 2;
    __device__ __forceinline__ void load(const float *g, long long ldg, const float *u, long long ldu, long long left_r, long long left_k) {
        const int in = threadIdx.x % O::LEN * V, out = threadIdx.x / O::LEN;
#pragma unroll
        for (int e = 0; e < O::N; ++e) {
            const int row = out + e * O::STEP, r = row % TN;
            this->one(e, (row < TN ? g + r * ldg : u + r * ldu) + in, in < left_k && r < left_r);
        }
    }
};

// One element's outputs from its sums (second: u, in the forward's modes).
template <Mode MODE> __device__ __forceinline__ void finish(const GluParams &p, bool up, long long m, long long n, float first, float second) {
    if constexpr (MODE == FWD) {
        static_cast<float *>(p.h)[m * p.ld_h + n] = act(first, p.gelu) * second;
        if (p.g) {
            p.g[m * p.F + n] = first;
            p.u[m * p.F + n] = second;
        }
    } else if constexpr (MODE == RECOMPUTE) {
        const Act f = act_and_slope(first, p.gelu);
        const float d = static_cast<const float *>(p.dh)[m * p.ld_dh + n];
        static_cast<float *>(p.dg)[m * p.ld_d + n] = d * second * f.d;
        static_cast<float *>(p.du)[m * p.ld_d + n] = d * f.v;
    } else if constexpr (MODE == DX) {
        static_cast<float *>(p.dx)[m * p.ld_dx + n] = first;
    } else {
        if (up) static_cast<float *>(p.dwu)[m * p.ld_dwu + n] = first;
        else static_cast<float *>(p.dwg)[m * p.ld_dwg + n] = first;
    }
}

template <int SIDE, Mode MODE, int V> __global__ void __launch_bounds__(Tiles<SIDE>::THREADS, SIDE == 128 ? 2 : 8) glu_f32_kernel(GluParams p, int blocks) {
    using S = Tiles<SIDE>;
    extern __shared__ __align__(16) float sm[];              // operands' tiles [2][2][STAGE], then (tiles of 64) the block's sums [SIDE][SIDE + 1]
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE, AK = MODE != DW, BK = DUAL;
    constexpr int TN = DUAL ? SIDE / 2 : SIDE, HALF = SIDE / 2, SPAN = SIDE / 8;     // a thread's quads: columns tx 4 and HALF + tx 4
    const int t = threadIdx.x, tx = t % SPAN, ty = t / SPAN;
    const bool up = MODE == DW && blockIdx.y;
    const long long ms = MODE == DW ? p.F : p.M, ns = DUAL ? p.F : p.D, ks = MODE == DW ? p.M : MODE == DX ? p.F : p.D;
    const unsigned cols = (unsigned)((ns + TN - 1) / TN), tile = blockIdx.x / blocks;
    const int rank = (int)(blockIdx.x % blocks);
    const long long m0 = (long long)(tile / cols) * SIDE, n0 = (long long)(tile % cols) * TN;
    f2 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
    Operand<SIDE, AK, V> a;
    std::conditional_t<DUAL, Weights<SIDE, V>, Operand<SIDE, BK, V>> b;
    const long long per = (ks + S::KT - 1) / S::KT, steps = MODE == DX ? 2 * per : per;
    const long long first = steps * rank / blocks, end = steps * (rank + 1) / blocks;
    auto fetch = [&](long long i) {
        const long long k0 = (MODE == DX && i >= per ? i - per : i) * S::KT;
        if constexpr (DUAL) {
            a.load(static_cast<const float *>(p.x) + m0 * p.ld_x + k0, p.ld_x, ms - m0, ks - k0);
            b.load(static_cast<const float *>(p.wg) + n0 * p.ld_wg + k0, p.ld_wg, static_cast<const float *>(p.wu) + n0 * p.ld_wu + k0, p.ld_wu,
                   ns - n0, ks - k0);
        } else if constexpr (MODE == DX) {
            const bool second = i >= per;
            a.load(static_cast<const float *>(second ? p.du : p.dg) + m0 * p.ld_d + k0, p.ld_d, ms - m0, ks - k0);
            const long long ld = second ? p.ld_wu : p.ld_wg;
            b.load(static_cast<const float *>(second ? p.wu : p.wg) + k0 * ld + n0, ld, ns - n0, ks - k0);
        } else {
            a.load(static_cast<const float *>(up ? p.du : p.dg) + k0 * p.ld_d + m0, p.ld_d, ms - m0, ks - k0);
            b.load(static_cast<const float *>(p.x) + k0 * p.ld_x + n0, p.ld_x, ns - n0, ks - k0);
        }
    };
    float *sa = sm, *sb = sm + 2 * S::STAGE;
    if (first < end) {
        fetch(first);
        a.store(sa);
        b.store(sb);
    }
    __syncthreads();
    for (long long i = first; i < end; ++i) {
        const int cur = (int)(i - first) & 1;
        if (i + 1 < end) fetch(i + 1);
        const float *pa = sa + cur * S::STAGE + ty * 4, *pb = sb + cur * S::STAGE + tx * 4;
#pragma unroll
        for (int k = 0; k < S::KT; ++k) {
            float av[8];
            f2 bv[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                *reinterpret_cast<float4 *>(av + 4 * q) = *reinterpret_cast<const float4 *>(pa + k * S::PITCH + HALF * q);
                const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(pb + k * S::PITCH + HALF * q);
                bv[2 * q] = w.x;
                bv[2 * q + 1] = w.y;
            }
#pragma unroll
            for (int y = 0; y < 8; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[y][x] = fma2(both(av[y]), bv[x], acc[y][x]);
        }
        if (i + 1 < end) {
            a.store(sa + (cur ^ 1) * S::STAGE);
            b.store(sb + (cur ^ 1) * S::STAGE);
        }
        __syncthreads();
    }
    auto row_of = [&](int y) { return (y < 4 ? 0 : HALF - 4) + ty * 4 + y; };
    auto col_of = [&](int x) { return (x < 4 ? 0 : HALF - 4) + tx * 4 + x; };
    auto value = [&](int y, int x) {
        float lo, hi;
        unpack2(acc[y][x / 2], lo, hi);
        return x & 1 ? hi : lo;
    };
    if constexpr (SIDE == 128) {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const long long m = m0 + row_of(y);
            if (m >= ms) continue;
#pragma unroll
            for (int x = 0; x < (DUAL ? 4 : 8); ++x) {
                const long long n = n0 + col_of(x);
                if (n < ns) finish<MODE>(p, up, m, n, value(y, x), DUAL ? value(y, x + 4) : 0.f);
            }
        }
    } else {
        // the block's sums where the others of its cluster can read them; each finishes a part of the tile's rows
#pragma unroll
        for (int y = 0; y < 8; ++y)
#pragma unroll
            for (int x = 0; x < 8; ++x) sm[row_of(y) * (SIDE + 1) + col_of(x)] = value(y, x);
        if (blocks > 1) kda::tc::cluster_sync_all();
        else __syncthreads();
        const uint32_t local = kda::tc::smem_u32(sm);
        const int rows = SIDE / blocks;
        for (int i = t; i < rows * TN; i += S::THREADS) {
            const int y = rank * rows + i / TN, x = i % TN;
            const long long m = m0 + y, n = n0 + x;
            if (m >= ms || n >= ns) continue;
            float v = 0.f, u = 0.f;
            for (int r = 0; r < blocks; ++r) {
                const uint32_t at = kda::tc::map_to_rank(local + (y * (SIDE + 1) + x) * 4, r);
                float g;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(g) : "r"(at) : "memory");
                v += g;
                if (DUAL) {
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(g) : "r"(at + TN * 4) : "memory");
                    u += g;
                }
            }
            finish<MODE>(p, up, m, n, v, u);
        }
        if (blocks > 1) kda::tc::cluster_sync_all();         // nobody leaves while others read its sums
    }
}

// dg and du of saved products: V columns per thread.  They are rounded to T, as operands of products on the tensor cores have to be: the
// weights' gradients are then 2.3e-3 off in bfloat16, where one rounding of the exact result is 1.7e-3.  (What the rounding drops,
// carried as a second operand, would double those products' work.)
template <class T, int V> __global__ void __launch_bounds__(256) glu_slope_kernel(GluParams p) {
    const long long per = (p.F - 1) / V + 1, i = (long long)blockIdx.x * 256 + threadIdx.x;
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

// A matrix's rows to where they are 16-byte aligned: as T, one or two elements, 16 of them on their way per thread (four columns of four
// rows; `cols`, `ld` and `pitch` count them).
template <class T> __global__ void __launch_bounds__(256) glu_align_kernel(const T *__restrict__ from, long long ld, T *__restrict__ to, long long pitch, long long rows, unsigned cols) {
    const unsigned c = blockIdx.x * 1024 + threadIdx.x;          // (without a sign: a step past a width near 2^31 does not wrap)
    for (long long r = blockIdx.y * 4LL; r < rows; r += gridDim.y * 4LL) {
        T v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r + j < rows && c + k * 256 < cols) v[j][k] = from[(r + j) * ld + c + k * 256];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r + j < rows && c + k * 256 < cols) to[(r + j) * pitch + c + k * 256] = v[j][k];
    }
}

template <int SIDE, Mode MODE, int V> cudaError_t run_side(const GluParams &p, long long tiles, int blocks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * blocks), MODE == DW ? 2 : 1);
    cfg.blockDim = dim3(Tiles<SIDE>::THREADS);
    cfg.dynamicSmemBytes = Tiles<SIDE>::FLOATS * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    if (blocks > 8) {
        const cudaError_t e = allow_large_clusters<glu_f32_kernel<SIDE, MODE, V>>();
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, glu_f32_kernel<SIDE, MODE, V>, p, blocks);
}
// Tiles of 128 where they fill the SMs' places (two to an SM) twice over, else tiles of 64 (eight), and a cluster of up to sixteen
// blocks to each where those leave half of the places empty and every block has eight steps.
template <Mode MODE> cudaError_t run_f32(const GluParams &p, cudaStream_t s) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE;
    const long long ms = MODE == DW ? p.F : p.M, ns = DUAL ? p.F : p.D, ks = MODE == DW ? p.M : MODE == DX ? 2LL * p.F : p.D;
    auto tiles = [&](int side) {
        const int tn = DUAL ? side / 2 : side;
        return ((ms + side - 1) / side) * ((ns + tn - 1) / tn);
    };
    bool wide = p.D % 4 == 0 && rows_aligned(p.x, p.ld_x, 4, 16) && rows_aligned(p.wg, p.ld_wg, 4, 16) && rows_aligned(p.wu, p.ld_wu, 4, 16);
    if (!DUAL) wide = wide && p.F % 4 == 0 && rows_aligned(p.dg, p.ld_d, 4, 16) && aligned_to(p.du, 16);
    const long long z = MODE == DW ? 2 : 1, sms = sm_count();
    if (tiles(64) * z * 8 > 0x7fffffffLL) return cudaErrorNotSupported;
    if (tiles(128) * z >= 4 * sms) return wide ? run_side<128, MODE, 4>(p, tiles(128), 1, s) : run_side<128, MODE, 1>(p, tiles(128), 1, s);
    int blocks = 1;
    while (blocks < 16 && tiles(64) * z * blocks * 2 <= 8 * sms && ks >= 256LL * blocks) blocks *= 2;
    return wide ? run_side<64, MODE, 4>(p, tiles(64), blocks, s) : run_side<64, MODE, 1>(p, tiles(64), blocks, s);
}

template <class T> cudaError_t slopes(const GluParams &p, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T);
    auto fits = [&](int v) {
        const size_t n = v * sizeof(T), m = v < 4 ? v * 4 : 16;
        return p.F % v == 0 && rows_aligned(p.dh, p.ld_dh, sizeof(T), n) && rows_aligned(p.dg, p.ld_d, sizeof(T), n) && aligned_to(p.du, n) &&
               aligned_to(p.g, m) && aligned_to(p.u, m);
    };
    const int v = fits(W) ? W : fits(2) ? 2 : 1;             // (3770 x 9058 bfloat16: pairs 88 us, single elements 147)
    const unsigned grid = (unsigned)((((p.F - 1) / v + 1) * p.M + 255) / 256);
    if (v == W) glu_slope_kernel<T, W><<<grid, 256, 0, s>>>(p);
    else if (v == 2) glu_slope_kernel<T, 2><<<grid, 256, 0, s>>>(p);
    else glu_slope_kernel<T, 1><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

// Operands of bfloat16 products that TMA could not read where they are (bases or rows off 16 bytes) move into the workspace.
struct Moved {
    const void **p;
    long long *ld, rows;
};
long long moved_pitch(int D) { return (D + 7LL) / 8 * 8; }
size_t moved_bytes(const Moved &m, int D) { return ((size_t)m.rows * moved_pitch(D) * 2 + 255) / 256 * 256; }
template <class F> cudaError_t each_moved(GluParams &p, F f) {
    const Moved all[] = {{&p.x, &p.ld_x, p.M}, {&p.wg, &p.ld_wg, p.F}, {&p.wu, &p.ld_wu, p.F}};
    for (const Moved &m : all)
        if (!rows_aligned(*m.p, *m.ld, 2, 16)) {
            const cudaError_t e = f(m);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}
cudaError_t align(GluParams &p, char *ws, cudaStream_t s) {
    return each_moved(p, [&](const Moved &m) {
        const long long pitch = moved_pitch(p.D);
        const bool two = p.D % 2 == 0 && rows_aligned(*m.p, *m.ld, 2, 4);
        const unsigned cols = (unsigned)p.D / (two ? 2 : 1), gx = (cols - 1) / 1024 + 1, gy = (unsigned)(m.rows < 131072 ? (m.rows + 3) / 4 : 32768);
        if (two) glu_align_kernel<<<dim3(gx, gy), 256, 0, s>>>(static_cast<const uint32_t *>(*m.p), *m.ld / 2, reinterpret_cast<uint32_t *>(ws), pitch / 2, m.rows, cols);
        else glu_align_kernel<<<dim3(gx, gy), 256, 0, s>>>(static_cast<const unsigned short *>(*m.p), *m.ld, reinterpret_cast<unsigned short *>(ws), pitch, m.rows, cols);
        *m.p = ws;
        *m.ld = pitch;
        ws += moved_bytes(m, p.D);
        return cudaGetLastError();
    });
}

}  // namespace

size_t glu_moved_bytes(const GluParams &q, bool bf16_) {
    GluParams p = q;
    size_t n = 0;
    if (bf16_)
        each_moved(p, [&](const Moved &m) {
            n += moved_bytes(m, p.D);
            return cudaSuccess;
        });
    return n;
}

long long glu_grad_stride(const GluParams &p, bool bf16_) {
    const long long n = bf16_ ? 16 : 4;                      // rows of 32-byte sectors, of 16-byte accesses
    return (p.F + n - 1) / n * n;
}

cudaError_t launch_glu_fwd(const GluParams &q, bool bf16_, char *ws, cudaStream_t s) {
    if (!bf16_) return run_f32<FWD>(q, s);
    if (glu_rows_takes(q)) return launch_glu_rows(q, s);
    GluParams p = q;
    const cudaError_t e = align(p, ws, s);
    return e == cudaSuccess ? launch_glu_tc_fwd(p, s) : e;
}

cudaError_t launch_glu_bwd(const GluParams &q, bool bf16_, char *ws, cudaStream_t s) {
    cudaError_t e;
    if (!bf16_) {
        e = q.g ? slopes<float>(q, s) : run_f32<RECOMPUTE>(q, s);
        if (e == cudaSuccess) e = run_f32<DX>(q, s);
        if (e == cudaSuccess) e = run_f32<DW>(q, s);
        return e;
    }
    GluParams p = q;
    e = align(p, ws, s);
    if (e == cudaSuccess) e = p.g ? slopes<bf16>(p, s) : launch_glu_tc_grads(p, s);
    if (e == cudaSuccess) e = launch_glu_tc_dx(p, s);
    if (e == cudaSuccess) e = launch_glu_tc_dw(p, s);
    return e;
}

}  // namespace mixer
