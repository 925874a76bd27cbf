// Gated feed-forward product on the tensor cores (bfloat16): forward, and the products of its backward.
//
//   FWD        h = act(g) u, g = x Wg^T, u = x Wu^T in float32 accumulators side by side     4 M D F operations
//   RECOMPUTE  the same products, then dg = dh u act'(g), du = dh act(g)
//   DX         dx = dg Wg + du Wu, one sum over both                                         4 M D F
//   DW         dWg = dg^T x, dWu = du^T x                                                    4 M D F
//
// A pair of CTAs (PAIR; or one alone) makes tiles of 256 (128) rows by 256 columns, persistent over the tiles: one
// thread of each CTA brings the operands' tiles by TMA, one thread of the pair issues tcgen05.mma on both SMs (each holds
// half of the rows of A and half of the columns of B, and gets the accumulators of its rows), four warps empty one
// of two accumulators in TMEM while the other fills.  In FWD the accumulator's left half is Wg's and its right half Wu's, so
// a thread of the epilogue has both products of its row.  Operands lie as they are: K-major (x, the weights in FWD)
// or with K outermost (weights in DX, dg, du and x in DW), which the matrix descriptors express; TMA fills what lies past an
// extent with zeros.
//
// Bound by the tensor cores and, in a run of such products, by the power limit: 8192 x 2048 x 8192 takes 305 us (1.80 PFLOP/s) after a
// pause and 350 (1.57) back to back, where 8192^3 of cuBLAS reach 1.90 and 1.71.  Six stages of 32 KB are what shared memory
// holds; a pair needs half of a lone CTA's reads of B.  4096 x 2048 x 5632 with its saved products (230 MB out) takes 128 us: stores of whole
// 32-byte sectors, of 16 bytes 153.  DX and DW of that size take 119 and 112, in one launch with a balanced schedule as long.
//
// Waits are bounded.  Where one runs out the kernel stops its work, lets what is in flight arrive, frees TMEM, leaves NaN in
// the outputs of tiles that it did not finish, and records the timeout in the caller's status block if there is one.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "glu.cuh"
#include "kda_internal.h"
#include "tc_common.cuh"

namespace mixer {
namespace {

using namespace glu;
using namespace kda::tc;

constexpr int BK = 64;                      // K of a stage: one 128-byte row of bfloat16
constexpr int HALF = 128;                   // rows of A, and rows (columns) of B, in units that CTAs load
constexpr int UNIT = HALF * BK * 2;         // bytes of one such operand tile
constexpr int COLS = 256;                   // accumulator columns of a tile
constexpr int EPI_WARPS = 4, THREADS = 64 + 32 * EPI_WARPS;

enum Mode { FWD, RECOMPUTE, DX, DW };

template <bool PAIR> struct Cfg {
    static constexpr int B_UNITS = PAIR ? 1 : 2;             // of B, per CTA and stage
    static constexpr int STAGE = UNIT * (1 + B_UNITS);
    static constexpr int STAGES = PAIR ? 6 : 4;
    static constexpr int SMEM = STAGES * STAGE + 1024;       // (the tiles begin on a multiple of 1024 bytes)
    static constexpr int ROWS = PAIR ? 2 * HALF : HALF;
};

struct TcArgs {
    CUtensorMap a0, a1, b0, b1;
    GluParams p;
    int tiles_m, tiles_n, tiles;            // tiles: over both outputs in DW
    int kb, segments;                       // K blocks of a segment, and segments (DX: dg Wg, then du Wu)
    int splits;                             // parts of K, each a unit of work with its own sums (DX, DW)
    float *part;                            // [splits][outputs][rows][pitch] those sums, where there are several parts
    long long pitch;
    int *status;
};

struct Shared {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    unsigned issued[2];                     // stages that each CTA of the pair began to load
    float turn[EPI_WARPS][32][33];
};

// ------------------------------------------------------------------------------------- pair forms
__device__ __forceinline__ uint32_t leader_bar(uint64_t *bar) { return map_to_rank(smem_u32(bar), 0); }

template <bool PAIR> __device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                     : "memory");
}
template <bool PAIR> __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc)
                     : "memory");
    else
        mma_bf16(d, a, b, idesc, acc);
}
// Arrive on `bar` of each CTA of the pair when the products issued so far are done.
template <bool PAIR> __device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                     "h"((unsigned short)3)
                     : "memory");
    else
        mma_commit(bar);
}
template <bool PAIR> __device__ __forceinline__ void alloc(uint32_t *dst) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(2 * COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, 2 * COLS);
        tmem_relinquish();
    }
}
template <bool PAIR> __device__ __forceinline__ void dealloc(uint32_t t) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(2 * COLS) : "memory");
    else tmem_dealloc(t, 2 * COLS);
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------------------------- bounded waits
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort, int *status, uint32_t bound) {
    for (uint32_t i = 0; i < bound; ++i) {
        if (*abort) return false;
        if (mbar_try_wait_cluster(bar, parity)) return true;
    }
    *abort = 1;
    if (status) atomicExch(status, kda::kDevTimeout);
    return false;
}
struct Waits {
    volatile int *abort;
    int *status;
    uint32_t bound;         // polls; the caller's budget, or the library's
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (bound == kWaitBound ? mbar_try_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
        return wait_slow(bar, parity, abort, status, bound);
    }
};
// For what completes by itself (copies, products): the library's bound whatever the caller's budget.
__device__ __noinline__ void drain(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitBound; ++i)
        if (mbar_try_wait_cluster(bar, parity)) return;
}

// ------------------------------------------------------------------------------------- tiles
struct Tile {
    int z, m, n;            // output (DW), row and column of tiles
    int split, k0, k1;      // part of K, its blocks
};
// Bands of 8 rows of tiles, column by column: the blocks that run together share rows of A and columns of B.
__device__ __forceinline__ Tile tile_of(const TcArgs &t, int i) {
    Tile q;
    q.split = i % t.splits;
    i /= t.splits;
    const int kbs = t.kb * t.segments;
    q.k0 = (int)((long long)kbs * q.split / t.splits);
    q.k1 = (int)((long long)kbs * (q.split + 1) / t.splits);
    const int per = t.tiles_m * t.tiles_n;
    q.z = i / per;
    i -= q.z * per;
    const int band = i / (8 * t.tiles_n), first = band * 8, rows = min(8, t.tiles_m - first);
    i -= band * 8 * t.tiles_n;
    q.m = first + i % rows;
    q.n = i / rows;
    return q;
}

// 32 bytes in one access: a whole sector of a row per lane.
__device__ __forceinline__ void store_sector(void *to, const uint32_t (&q)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]), "r"(q[4]),
                 "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
}
__device__ __forceinline__ void put(bf16 *to, float v) { *to = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float *to, float v) { *to = v; }
__device__ __forceinline__ void store_whole(bf16 *out, const float (&v)[32]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = pack_bf16(v[16 * k + 2 * e], v[16 * k + 2 * e + 1]);
        store_sector(out + 16 * k, q);
    }
}
__device__ __forceinline__ void store_whole(float *out, const float (&v)[32]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(v[8 * k + e]);
        store_sector(out + 8 * k, q);
    }
}
// 32 rows of a warp, 32 columns: v is this lane's row, `first` the warp's first row, of which `rows` belong to the output, as
// `inside` of the columns.  Rows of whole sectors go out by lanes; others turn in shared memory, so that a row's neighbours leave
// together.
template <class T> __device__ __forceinline__ void store_rows(T *first, long long ld, const float (&v)[32], int rows, int inside, bool wide, float (*turn)[33]) {
    const int lane = threadIdx.x & 31;
    if (wide && inside >= 32) {
        if (lane < rows) store_whole(first + lane * ld, v);
        return;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 32; ++k) turn[lane][k] = v[k];
    __syncwarp();
    if constexpr (sizeof(T) == 2)
        if ((inside >= 32 || inside % 2 == 0) && ((reinterpret_cast<uintptr_t>(first) | (uintptr_t)ld * 2) & 3) == 0) {   // pairs, two rows at a time
            const int c = lane % 16 * 2;
            first += lane / 16 * ld + c;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 8) {
                uint32_t q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float *from = turn[r0 + 2 * k + lane / 16] + c;
                    q[k] = pack_bf16(from[0], from[1]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k, first += 2 * ld)
                    if (r0 + 2 * k + lane / 16 < rows && c < inside) *reinterpret_cast<uint32_t *>(first) = q[k];
            }
            return;
        }
    first += lane;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {
        float q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = turn[r0 + k][lane];
#pragma unroll
        for (int k = 0; k < 8; ++k, first += ld)
            if (r0 + k < rows && lane < inside) put(first, q[k]);
    }
}
__device__ __forceinline__ bool wide_rows(const void *p, long long ld, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 31) == 0 && ld * es % 32 == 0;
}

// The outputs of a warp's 32 rows from row0 (of the call), `rows` of which belong to it, and a tile's columns.  get(c, v): this
// lane's row of 32 accumulator columns from c.
template <Mode MODE, class Get>
__device__ __forceinline__ void finish(const TcArgs &t, const Tile &q, long long row0, int rows, float (*turn)[33], Get get) {
    const GluParams &p = t.p;
    if constexpr (MODE == FWD || MODE == RECOMPUTE) {
        const int n0 = q.n * HALF;
        const bool wide = MODE == FWD ? wide_rows(p.h, p.ld_h, 2) : wide_rows(p.dg, p.ld_d, 2) && wide_rows(p.du, p.ld_d, 2);
        const bool keep = wide_rows(p.g, p.F, 4) && wide_rows(p.u, p.F, 4);
#pragma unroll 1
        for (int c = 0; c < HALF; c += 32) {
            float g[32], u[32];
            __syncwarp();                                // (the loads from TMEM are the whole warp's)
            get(c, g);
            get(HALF + c, u);
            const int n = n0 + c, inside = p.F - n;
            if (inside <= 0 || rows <= 0) continue;
            if constexpr (MODE == FWD) {
                if (p.g) {
                    store_rows(p.g + row0 * p.F + n, p.F, g, rows, inside, keep, turn);
                    store_rows(p.u + row0 * p.F + n, p.F, u, rows, inside, keep, turn);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) u[k] *= act(g[k], p.gelu);
                store_rows(static_cast<bf16 *>(p.h) + row0 * p.ld_h + n, p.ld_h, u, rows, inside, wide, turn);
            } else {
                const int lane = threadIdx.x & 31;
                const bf16 *dh = static_cast<const bf16 *>(p.dh) + (row0 + min(lane, rows - 1)) * p.ld_dh + n;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const Act f = act_and_slope(g[k], p.gelu);
                    const float d = k < inside ? __bfloat162float(dh[k]) : 0.f;
                    g[k] = d * u[k] * f.d;
                    u[k] = d * f.v;
                }
                store_rows(static_cast<bf16 *>(p.dg) + row0 * p.ld_d + n, p.ld_d, g, rows, inside, wide, turn);
                store_rows(static_cast<bf16 *>(p.du) + row0 * p.ld_d + n, p.ld_d, u, rows, inside, wide, turn);
            }
        }
    } else {
        const int n0 = q.n * COLS;
        const bool second = MODE == DW && q.z;
        bf16 *out = static_cast<bf16 *>(MODE == DX ? p.dx : second ? p.dwu : p.dwg);
        const long long ld = MODE == DX ? p.ld_dx : second ? p.ld_dwu : p.ld_dwg;
        const bool wide = wide_rows(out, ld, 2), whole = wide_rows(t.part, t.pitch, 4);
#pragma unroll 1
        for (int c = 0; c < COLS; c += 32) {
            float v[32];
            __syncwarp();
            get(c, v);
            const int inside = p.D - n0 - c;
            if (inside <= 0 || rows <= 0) continue;
            if (t.splits > 1) {
                const long long all = MODE == DW ? p.F : p.M, z = (long long)q.split * (MODE == DW ? 2 : 1) + q.z;
                store_rows(t.part + (z * all + row0) * t.pitch + n0 + c, t.pitch, v, rows, inside, whole, turn);
            } else store_rows(out + row0 * ld + n0 + c, ld, v, rows, inside, wide, turn);
        }
    }
}

// ------------------------------------------------------------------------------------- kernel
template <bool PAIR, Mode MODE> __global__ void __launch_bounds__(THREADS, 1) glu_tc_kernel(const __grid_constant__ TcArgs t) {
    using C = Cfg<PAIR>;
    constexpr bool A_MN = MODE == DW, B_MN = MODE == DX || MODE == DW;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = PAIR ? cluster_ctarank() : 0;
    const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&sh.full[s], PAIR ? 2 : 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], EPI_WARPS * (PAIR ? 2 : 1));
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        sh.issued[0] = sh.issued[1] = 0;
        fence_mbar_init();
    }
    if (warp == 0) alloc<PAIR>(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int budget = t.status ? t.status[kda::kStatusBoundWord] : 0;
    const Waits wait{&sh.abort, t.status, budget > 0 ? (uint32_t)budget : kWaitBound};
    unsigned used = 0;                                   // stages that the products have waited for

    if (warp == 0) {
        if (lane == 0) {
            unsigned it = 0;
            bool ok = true;
            for (int i = worker; ok && i < t.tiles; i += workers) {
                const Tile q = tile_of(t, i);
                const int m0 = q.m * C::ROWS + (int)rank * HALF, n0 = q.n * (B_MN ? COLS : HALF);
                for (int k = q.k0; k < q.k1; ++k, ++it) {
                    const int s = it % C::STAGES;
                    if (it >= C::STAGES && !(ok = wait(&sh.empty[s], it / C::STAGES - 1 & 1))) break;
                    const uint32_t bar = leader_bar(&sh.full[s]);
                    if (PAIR && rank) mbar_arrive_expect_tx_remote(bar, C::STAGE);
                    else mbar_arrive_expect_tx(&sh.full[s], C::STAGE);
                    unsigned char *a = tiles + s * C::STAGE, *b = a + UNIT;
                    const bool second = MODE == DX ? k >= t.kb : MODE == DW && q.z;
                    const int k0 = (MODE == DX && second ? k - t.kb : k) * BK;
                    const CUtensorMap *ma = second ? &t.a1 : &t.a0;
                    if constexpr (A_MN) {
                        tma_load<PAIR>(a, ma, bar, m0, k0);
                        tma_load<PAIR>(a + UNIT / 2, ma, bar, m0 + 64, k0);
                    } else {
                        tma_load<PAIR>(a, ma, bar, k0, m0);
                    }
                    if constexpr (B_MN) {
                        const CUtensorMap *mb = MODE == DX && second ? &t.b1 : &t.b0;
#pragma unroll
                        for (int u = 0; u < 2 * C::B_UNITS; ++u)
                            tma_load<PAIR>(b + u * (UNIT / 2), mb, bar, n0 + (int)rank * HALF + u * 64, k0);
                    } else if constexpr (PAIR) {
                        tma_load<PAIR>(b, rank ? &t.b1 : &t.b0, bar, k0, n0);
                    } else {
                        tma_load<PAIR>(b, &t.b0, bar, k0, n0);
                        tma_load<PAIR>(b + UNIT, &t.b1, bar, k0, n0);
                    }
                }
            }
            sh.issued[rank] = it;
            if (PAIR && rank) {                          // the leader lets this CTA's copies arrive too, where work was broken off
                const uint32_t at = map_to_rank(smem_u32(&sh.issued[1]), 0);
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(it) : "memory");
            }
            // every stage has been given back: no arrival is on its way any more
            for (unsigned j = it > C::STAGES ? it - C::STAGES : 0; ok && j < it; ++j) ok = wait(&sh.empty[j % C::STAGES], j / C::STAGES & 1);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_bf16(C::ROWS, COLS, A_MN, B_MN);
            const uint32_t base = smem_u32(tiles);
            unsigned it = 0, n = 0;
            bool ok = true;
            for (int i = worker; ok && i < t.tiles; i += workers, ++n) {
                const int buf = n & 1;
                if (n >= 2 && !(ok = wait(&sh.acc_empty[buf], (n / 2 - 1) & 1))) break;
                tc_fence_after();
                const Tile q = tile_of(t, i);
                for (int k = q.k0; k < q.k1; ++k, ++it) {
                    const int s = it % C::STAGES;
                    if (!(ok = wait(&sh.full[s], it / C::STAGES & 1))) break;
                    tc_fence_after();
                    const uint32_t a = base + s * C::STAGE, b = a + UNIT;
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ++ks)
                        mma<PAIR>(tmem + buf * COLS, A_MN ? desc_mnmajor(a, BK, ks) : desc_kmajor(a, HALF, ks),
                                  B_MN ? desc_mnmajor(b, BK, ks) : desc_kmajor(b, HALF, ks), idesc, k > q.k0 || ks > 0);
                    commit<PAIR>(&sh.empty[s]);
                }
                if (ok) commit<PAIR>(&sh.acc_full[buf]);
            }
            used = it;
        }
    } else {
        const int quarter = warp & 3;                    // the lanes of TMEM that this warp may read
        unsigned n = 0;
        int ok = 1;                                      // until a tile was not finished: none after it is, and its buffer's phase stands still
        for (int i = worker; i < t.tiles; i += workers, ++n) {
            const Tile q = tile_of(t, i);
            const int buf = n & 1;
            if (ok && lane == 0) ok = wait(&sh.acc_full[buf], n / 2 & 1);
            ok = __shfl_sync(~0u, ok, 0);
            tc_fence_after();
            const long long row0 = (long long)q.m * C::ROWS + rank * HALF + quarter * 32;
            const int rows = (int)max(0LL, min(32LL, (MODE == DW ? (long long)t.p.F : t.p.M) - row0));
            const uint32_t at = tmem + ((uint32_t)quarter << 21) + buf * COLS;
            if (ok) {
                finish<MODE>(t, q, row0, rows, sh.turn[quarter], [&](int c, float (&v)[32]) { tmem_ld32(at + c, v); });
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(leader_bar(&sh.acc_empty[buf]));
            } else {                                     // broken off: the tile's outputs say so
                const float bad = __int_as_float(0x7fc00000);
                finish<MODE>(t, q, row0, rows, sh.turn[quarter], [&](int, float (&v)[32]) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = bad;
                });
            }
        }
    }
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    // Broken off: copies and products that began still arrive, before TMEM and shared memory are given back.
    if (warp == 1 && lane == 0 && rank == 0) {
        const unsigned i0 = sh.issued[0], i1 = PAIR ? sh.issued[1] : i0;
        for (unsigned j = used; j < max(i0, i1); ++j) {
            uint64_t *bar = &sh.full[j % C::STAGES];
            if (j >= i0 || j >= i1) mbar_arrive(bar);    // for the CTA that did not begin this stage
            drain(bar, j / C::STAGES & 1);
        }
        if (used < max(i0, i1) || sh.abort) {
            if constexpr (PAIR)
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&sh.drain)) : "memory");
            else mma_commit(&sh.drain);
            drain(&sh.drain, 0);
        }
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    if (warp == 0) dealloc<PAIR>(tmem);
}

// ------------------------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// A matrix [rows][cols] with row stride ld (of a single row, which has no next one, any); boxes of 64 columns by `box` rows, 128-byte
// swizzle.
bool make_map(CUtensorMap *m, const void *p, long long rows, long long cols, long long ld, int box) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(rows > 1 ? ld : (cols + 7) / 8 * 8) * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, one[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, Mode MODE> cudaError_t launch(TcArgs &t, cudaStream_t s) {
    using C = Cfg<PAIR>;
    constexpr auto kernel = glu_tc_kernel<PAIR, MODE>;
    const cudaError_t e = allow_shared<glu_tc_kernel<PAIR, MODE>>(C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = PAIR ? 2 : 1;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int workers = sm_count();
    if (PAIR) {                             // pairs of SMs that can run at once: a pair past them would run alone, after the others
        static std::atomic<int> pairs[DEVICES];
        const int dev = current_device();
        int n = dev < DEVICES ? pairs[dev].load(std::memory_order_relaxed) : 0;
        if (n < 1) {
            cfg.gridDim = dim3(2 * (workers / 2));
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) n = workers / 2;
            if (dev < DEVICES) pairs[dev].store(n, std::memory_order_relaxed);
        }
        workers = n;
    }
    if (workers > t.tiles) workers = t.tiles;
    cfg.gridDim = dim3((PAIR ? 2 : 1) * workers);
    return cudaLaunchKernelEx(&cfg, kernel, t);
}

// The joined sums of the parts of K, in their order: four columns per thread.
__global__ void __launch_bounds__(256) glu_join_kernel(const float *part, int splits, long long rows, int cols, long long pitch, long long apart, bf16 *out,
                                                        long long ld) {
    const long long per = pitch / 4, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const long long r = i / per;
    const int c = (int)(i - r * per) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < splits; ++k) {
        const float4 g = *reinterpret_cast<const float4 *>(part + k * apart + r * pitch + c);
        v.x += g.x;
        v.y += g.y;
        v.z += g.z;
        v.w += g.w;
    }
    bf16 *to = out + r * ld + c;
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (c + k < cols) to[k] = __float2bfloat16_rn(f[k]);
}

// Where the tiles of one of the backward's products (or pairs of CTAs for them) leave half of the SMs idle, K is cut into parts that fill
// them, each of four blocks of 64 at least.  (The forward's is not cut: its epilogue needs whole sums.)
struct Shape {
    bool pair;
    long long tm, tn, kbs;
    int splits;
    long long pitch;
};
template <Mode MODE> Shape shape_of(const GluParams &p) {
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE;
    Shape q;
    const long long ms = MODE == DW ? p.F : p.M, ks = DUAL ? p.D : MODE == DX ? p.F : p.M;
    q.pair = ms > HALF;
    const int rows = q.pair ? 2 * HALF : HALF, cols = DUAL ? HALF : COLS;
    q.tm = (ms + rows - 1) / rows;
    q.tn = ((DUAL ? p.F : p.D) + (long long)cols - 1) / cols;
    q.kbs = (ks + BK - 1) / BK * (MODE == DX ? 2 : 1);
    q.splits = 1;
    q.pitch = (p.D + 7LL) / 8 * 8;
    if (!DUAL) {
        const long long places = sm_count() / (q.pair ? 2 : 1), tiles = q.tm * q.tn * (MODE == DW ? 2 : 1);
        const long long n = places / tiles, most = q.kbs / 4;
        if (n > 1 && most > 1) q.splits = (int)(n < most ? n : most);
    }
    return q;
}
template <Mode MODE> size_t part_bytes(const GluParams &p) {
    const Shape q = shape_of<MODE>(p);
    return q.splits > 1 ? (size_t)q.splits * (MODE == DW ? 2 * (size_t)p.F : (size_t)p.M) * q.pitch * 4 : 0;
}

template <Mode MODE> cudaError_t run(const GluParams &p, int *status, cudaStream_t s) {
    TcArgs t;
    t.p = p;
    t.status = status;
    constexpr bool DUAL = MODE == FWD || MODE == RECOMPUTE;
    const Shape q = shape_of<MODE>(p);
    const bool pair = q.pair;
    if (q.tm * q.tn * 2 * q.splits > 0x7fffffffLL) return cudaErrorNotSupported;
    t.tiles_m = (int)q.tm;
    t.tiles_n = (int)q.tn;
    t.splits = q.splits;
    t.part = static_cast<float *>(p.part);
    t.pitch = q.pitch;
    t.tiles = (int)(q.tm * q.tn * (MODE == DW ? 2 : 1) * q.splits);
    t.segments = MODE == DX ? 2 : 1;
    t.kb = (int)(q.kbs / t.segments);
    bool ok;
    if constexpr (DUAL) {
        ok = make_map(&t.a0, p.x, p.M, p.D, p.ld_x, HALF) && make_map(&t.b0, p.wg, p.F, p.D, p.ld_wg, HALF) &&
             make_map(&t.b1, p.wu, p.F, p.D, p.ld_wu, HALF);
        t.a1 = t.a0;
    } else if constexpr (MODE == DX) {
        ok = make_map(&t.a0, p.dg, p.M, p.F, p.ld_d, HALF) && make_map(&t.a1, p.du, p.M, p.F, p.ld_d, HALF) &&
             make_map(&t.b0, p.wg, p.F, p.D, p.ld_wg, BK) && make_map(&t.b1, p.wu, p.F, p.D, p.ld_wu, BK);
    } else {
        ok = make_map(&t.a0, p.dg, p.M, p.F, p.ld_d, BK) && make_map(&t.a1, p.du, p.M, p.F, p.ld_d, BK) &&
             make_map(&t.b0, p.x, p.M, p.D, p.ld_x, BK);
        t.b1 = t.b0;
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = pair ? launch<true, MODE>(t, s) : launch<false, MODE>(t, s);
    if (e != cudaSuccess || q.splits == 1) return e;
    const long long rows = MODE == DW ? p.F : p.M, apart = rows * q.pitch * (MODE == DW ? 2 : 1);
    const unsigned grid = (unsigned)((rows * (q.pitch / 4) + 255) / 256);
    for (int z = 0; z < (MODE == DW ? 2 : 1); ++z) {
        bf16 *out = static_cast<bf16 *>(MODE == DX ? p.dx : z ? p.dwu : p.dwg);
        glu_join_kernel<<<grid, 256, 0, s>>>(t.part + z * rows * q.pitch, q.splits, rows, p.D, q.pitch, apart, out,
                                             MODE == DX ? p.ld_dx : z ? p.ld_dwu : p.ld_dwg);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t glu_tc_part_bytes(const GluParams &p) {
    const size_t x = part_bytes<DX>(p), w = part_bytes<DW>(p);
    return x > w ? x : w;
}
cudaError_t launch_glu_tc_fwd(const GluParams &p, cudaStream_t s) { return run<FWD>(p, p.status, s); }
cudaError_t launch_glu_tc_grads(const GluParams &p, cudaStream_t s) { return run<RECOMPUTE>(p, p.status, s); }
cudaError_t launch_glu_tc_dx(const GluParams &p, cudaStream_t s) { return run<DX>(p, p.status, s); }
cudaError_t launch_glu_tc_dw(const GluParams &p, cudaStream_t s) { return run<DW>(p, p.status, s); }

}  // namespace mixer
