// Gated feed-forward product of a few rows (bfloat16): a decoding step.  The weights pass by once, 4 D F bytes, which
// bounds it.  A block takes 16 rows of both weights, its warps a part of the columns each; a lane reads 16 bytes of a
// row at a time, straight into the operands of mma.m16n8k16 (weights as A, x as B: the eight elements of a lane
// stand for other positions along K than the instruction's, the same ones in both operands, so their sum is the same).
// 4096 x 11008: 31 us, 5.8 TB/s.
#include "glu.cuh"

namespace mixer {
namespace {

using namespace glu;

constexpr int WARPS = 8, THREADS = 32 * WARPS, ROWS = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes that pass by once.
__device__ __forceinline__ uint4 load_stream(const bf16 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// NT groups of 8 rows of x; U steps of 32 columns in flight.
template <int NT, int U> __global__ void __launch_bounds__(THREADS) glu_rows_kernel(GluParams p) {
    __shared__ float sm[WARPS][2][8 * NT][ROWS + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const long long f0 = (long long)blockIdx.x * ROWS;
    const bf16 *w[4];                                        // Wg and Wu, rows g and g + 8 (past the end: the last)
    const long long fa = min(f0 + g, (long long)p.F - 1), fb = min(f0 + g + 8, (long long)p.F - 1);
    w[0] = static_cast<const bf16 *>(p.wg) + fa * p.ld_wg + q * 8;
    w[1] = static_cast<const bf16 *>(p.wg) + fb * p.ld_wg + q * 8;
    w[2] = static_cast<const bf16 *>(p.wu) + fa * p.ld_wu + q * 8;
    w[3] = static_cast<const bf16 *>(p.wu) + fb * p.ld_wu + q * 8;
    const bf16 *x = static_cast<const bf16 *>(p.x) + q * 8;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
    // the warps' steps take turns, so that together they read whole stretches of a row
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const unsigned D = (unsigned)p.D;                        // (columns without a sign: a step past a width near 2^31 does not wrap)
    for (unsigned k0 = warp * 32 * U; k0 < D; k0 += WARPS * 32 * U) {
        uint4 a[U][4], b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned k = k0 + u * 32;
            const bool in = k + q * 8 < D;                 // (D is a multiple of 8: all of a lane's elements or none)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[u][i] = in ? load_stream(w[i] + k) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const long long m = n * 8 + g;
                b[u][n] = in && m < p.M ? __ldg(reinterpret_cast<const uint4 *>(x + m * p.ld_x + k)) : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma16816(acc[i][n], a[u][2 * i].x, a[u][2 * i + 1].x, a[u][2 * i].y, a[u][2 * i + 1].y, b[u][n].x, b[u][n].y);
                    mma16816(acc[i][n], a[u][2 * i].z, a[u][2 * i + 1].z, a[u][2 * i].w, a[u][2 * i + 1].w, b[u][n].z, b[u][n].w);
                }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sm[warp][i][n * 8 + q * 2 + (e & 1)][g + (e >> 1) * 8] = acc[i][n][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 8 * NT * ROWS; o += THREADS) {
        const int m = o / ROWS, r = o % ROWS;
        const long long f = f0 + r;
        if (m >= p.M || f >= p.F) continue;
        float gv = 0.f, uv = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            gv += sm[k][0][m][r];
            uv += sm[k][1][m][r];
        }
        static_cast<bf16 *>(p.h)[m * p.ld_h + f] = from_f<bf16>(act(gv, p.gelu) * uv);
        if (p.g) {
            p.g[m * (long long)p.F + f] = gv;
            p.u[m * (long long)p.F + f] = uv;
        }
    }
}

}  // namespace

// Up to 16 rows (of 4096 x 11008: 31 us up to 8, 38 up to 16, as the tensor cores' form takes from 1 to 128; 24 rows here 57), and
// reads of 16 bytes.
bool glu_rows_takes(const GluParams &p) {
    return p.M <= 16 && p.D % 8 == 0 && rows_aligned(p.x, p.ld_x, 2, 16) && rows_aligned(p.wg, p.ld_wg, 2, 16) &&
           rows_aligned(p.wu, p.ld_wu, 2, 16);
}
cudaError_t launch_glu_rows(const GluParams &p, cudaStream_t s) {
    const unsigned grid = (unsigned)((p.F - 1) / ROWS + 1);
    if (p.M <= 8) glu_rows_kernel<1, 4><<<grid, THREADS, 0, s>>>(p);
    else glu_rows_kernel<2, 2><<<grid, THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mixer
