// Gated recurrence (one state per channel), forward, backward and single tokens.
//
// All rows of a chain of sequences form one axis.  Tiles of it go to the blocks of a cluster in turn; each
// block holds a tile of 64 rows (backward: 32) by 64 channels in registers, every warp 8 (4) neighbouring rows, a lane two
// channels.  A warp reduces its rows to h_out = h + A h_in, the block's warps and then the cluster's blocks
// exchange these pairs through shared memory, and each warp walks its rows again from the state that enters them.
// So every tensor is read once and written once, whatever the sequences' lengths, and the order of the sums is
// fixed.  Where a sequence begins inside a tile the link is cut by selection (never by a product with 0: a state
// of an earlier sequence may be an infinity).
//
// The backward runs the same walk from the end, with G_t = dy_t + a_{t+1} G_{t+1}; the states that enter its
// tiles are the forward's, saved every 32 rows in float32 (6 % of one bfloat16 tensor), so that it too reads each tensor once.
#include "gated_scan.cuh"
#include "tc_common.cuh"

namespace mixer {
namespace {

using namespace gs;

// 16 bytes into the same place of another block's shared memory.
__device__ __forceinline__ void store_remote(const float4 *at, unsigned rank, float4 v) {
    const uint32_t a = kda::tc::map_to_rank((uint32_t)__cvta_generic_to_shared(at), rank);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void store_remote(const int *at, unsigned rank, int v) {
    const uint32_t a = kda::tc::map_to_rank((uint32_t)__cvta_generic_to_shared(at), rank);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ float4 quad(f2 a, f2 b) {
    float4 r;
    unpack2(a, r.x, r.y);
    unpack2(b, r.z, r.w);
    return r;
}

constexpr int MAX_CLUSTER = 8;
static_assert(MAX_CLUSTER <= WARPS, "warp k writes to block k of the cluster");

// What the warps of a block and the blocks of a cluster tell each other of a tile, in two sets that take turns:
// h_out = h + A h_in of their rows (A, h), or h_out = h alone where a sequence begins (ends, in the backward).
struct Exchange {
    float4 warp[2][WARPS][32];
    float4 block[2][MAX_CLUSTER][32];
    int warp_cut[2][WARPS], block_cut[2][MAX_CLUSTER];
};

// h_out of the rows that (A, h) stand for, and the composition of two such.
__device__ __forceinline__ f2 through(float4 g, bool cut, f2 h) {
    return cut ? pack2(g.z, g.w) : fma2(pack2(g.x, g.y), h, pack2(g.z, g.w));
}

// The state (or its gradient) that enters this warp's rows, and the one that leaves the cluster's tiles (carry).
// REV: warps and blocks count from the last row.  prod, out: this warp's pair.
template <bool REV>
__device__ __forceinline__ f2 enter(Exchange &ex, int buf, int warp, int lane, unsigned rank, int blocks, f2 prod, f2 out, bool cut,
                                    f2 &carry) {
    ex.warp[buf][warp][lane] = quad(prod, out);
    if (lane == 0) ex.warp_cut[buf][warp] = cut;
    __syncthreads();
    if (blocks == 1) {
        f2 mine = carry;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            const int k = REV ? WARPS - 1 - i : i;
            if (k == warp) mine = carry;
            carry = through(ex.warp[buf][k][lane], ex.warp_cut[buf][k], carry);
        }
        return mine;
    }
    // the block's pair, and the pair of the warps before this one
    f2 pa = both(1.f), ph = both(0.f), ma = pa, mh = ph;
    bool pc = false, mc = false;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const int k = REV ? WARPS - 1 - i : i;
        if (k == warp) ma = pa, mh = ph, mc = pc;
        const float4 g = ex.warp[buf][k][lane];
        const bool c = ex.warp_cut[buf][k];
        ph = i == 0 ? pack2(g.z, g.w) : through(g, c, ph);
        pa = mul2(pa, pack2(g.x, g.y));
        pc |= c;
    }
    if (warp < blocks) {
        store_remote(&ex.block[buf][rank][lane], warp, quad(pa, ph));
        if (lane == 0) store_remote(&ex.block_cut[buf][rank], warp, (int)pc);
    }
    kda::tc::cluster_sync_all();
    f2 into = carry;
    for (int i = 0; i < blocks; ++i) {
        const int k = REV ? blocks - 1 - i : i;
        if (k == (int)rank) into = carry;
        carry = through(ex.block[buf][k][lane], ex.block_cut[buf][k], carry);
    }
    const bool first = REV ? warp == WARPS - 1 : warp == 0;
    return first ? into : mc ? mh : fma2(ma, into, mh);
}

// ------------------------------------------------------------------------------------------ forward
constexpr int FROWS = 8, FTILE = FROWS * WARPS;

template <class T, bool VEC>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 3 : 2) gated_scan_fwd_kernel(GatedScanParams p) {
    __shared__ Exchange ex;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = p.cluster;
    const unsigned rank = blockIdx.x % blocks;
    const int c = (int)(blockIdx.x / blocks) * COLS + lane * 2, D = p.D;
    const bool on = c < D;
    const int cl = on ? c : D - (VEC ? 2 : 1);       // idle lanes read the last channels and write nothing
    const Chain k = chain_of(p.cu_seqlens, p.B, p.T, p.chains, blockIdx.y);
    if (p.cu_seqlens && p.ht && rank == 0 && on)     // empty sequences: the state passes through
        for (int s = k.s0 + warp; s < k.s1; s += WARPS) {
            const int lo = clamped(p.cu_seqlens[s], 0, p.T), hi = clamped(p.cu_seqlens[s + 1], lo, p.T);
            if (lo == hi) store_state(p.ht + (long long)s * D, c, D, p.h0 ? load_state(p.h0 + (long long)s * D, c, D) : both(0.f));
        }
    if (k.c0 >= k.c1) return;                        // (the whole cluster)
    const T *px = static_cast<const T *>(p.x), *pd = static_cast<const T *>(p.decay), *pg = static_cast<const T *>(p.gate);
    if (blocks > 1) kda::tc::cluster_sync_all();     // every block has begun: its shared memory may be written
    const f2 coef = coefficients(p, cl);
    const long long tile0 = k.c0 / FTILE, tiles = ((long long)k.c1 + FTILE - 1) / FTILE - tile0;
    const int turns = (int)((tiles + blocks - 1) / blocks);

    Raw<T, VEC> x[FROWS], d[FROWS], g[FROWS];
    auto fetch = [&](long long r0) {                 // rows outside the chain: its first or last row instead
#pragma unroll
        for (int j = 0; j < FROWS; ++j) {
            const long long r = r0 + j < k.c0 ? k.c0 : r0 + j >= k.c1 ? k.c1 - 1 : r0 + j;
            x[j].load(px + r * p.ld_x, cl, D);
            d[j].load(pd + r * p.ld_decay, cl, D);
            g[j].load(pg + r * p.ld_gate, cl, D);
        }
    };
    long long r0 = (tile0 + rank) * FTILE + warp * FROWS;
    fetch(r0);
    Marks<FROWS> marks;
    f2 carry = both(0.f);
    for (int i = 0; i < turns; ++i, r0 += (long long)blocks * FTILE) {
        f2 a[FROWS], v[FROWS];
#pragma unroll
        for (int j = 0; j < FROWS; ++j) {
            f2 w;
            decay_of(mul2(coef, sigmoid2(d[j].pair())), a[j], w);
            v[j] = mul2(mul2(sqrt2(w), sigmoid2(g[j].pair())), x[j].pair());
        }
        if (i + 1 < turns) fetch(r0 + (long long)blocks * FTILE);
        marks.find(p, k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        f2 h = v[0], prod = a[0];
#pragma unroll
        for (int j = 0; j < FROWS; ++j) {
            if (starts >> j & 1) {
                h = p.h0 ? fma2(a[j], load_state(p.h0 + (long long)marks.sequence(j) * D, cl, D), v[j]) : v[j];
                v[j] = h;                            // the walk below begins here anew
            } else if (j) {
                h = fma2(a[j], h, v[j]);
            }
            if (j) prod = mul2(prod, a[j]);
        }
        h = enter<false>(ex, i & 1, warp, lane, rank, blocks, prod, h, starts != 0, carry);
        if (p.states && r0 % SAVE == 0 && r0 >= k.c0 && r0 < k.c1 && on) store_state(p.states + r0 / SAVE * D, c, D, h);
#pragma unroll
        for (int j = 0; j < FROWS; ++j) {
            h = starts >> j & 1 ? v[j] : fma2(a[j], h, v[j]);
            const long long r = r0 + j;
            if (on && r >= k.c0 && r < k.c1 && p.y) store_pair<T, VEC>(static_cast<T *>(p.y) + r * p.ld_y, c, D, h);
            if (ends >> j & 1) {
                const int s = marks.sequence(j);
                if (p.ht && on) store_state(p.ht + (long long)s * D, c, D, h);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------ backward
// With q the exponent, s and u the two sigmoids, v = u x and G_t the gradient of h_t:
//     dq = G (v a^2 / m - a h_{t-1}),  ddecay = dq c s (1 - s),  drate = scale sigmoid(rate) sum dq s,
//     dx = G m u,  dgate = G m x u (1 - u),  dh0 = a G of the first token.
constexpr int BROWS = 4, BTILE = BROWS * WARPS;
static_assert(BTILE == SAVE, "a saved state enters every tile");

template <class T, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) gated_scan_bwd_kernel(GatedScanParams p) {
    __shared__ Exchange ex;
    __shared__ float4 fwd[2][WARPS][32];             // (A, h) of the warps' rows, first to last
    __shared__ int fwd_cut[2][WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = p.cluster;
    const unsigned rank = blockIdx.x % blocks;
    const int c = (int)(blockIdx.x / blocks) * COLS + lane * 2, D = p.D;
    const bool on = c < D;
    const int cl = on ? c : D - (VEC ? 2 : 1);
    const Chain k = chain_of(p.cu_seqlens, p.B, p.T, p.chains, blockIdx.y);
    float *part = p.part + ((long long)blockIdx.y * blocks + rank) * D;
    if (p.cu_seqlens && p.dh0 && rank == 0 && on)    // empty sequences hand the gradient through
        for (int s = k.s0 + warp; s < k.s1; s += WARPS) {
            const int lo = clamped(p.cu_seqlens[s], 0, p.T), hi = clamped(p.cu_seqlens[s + 1], lo, p.T);
            if (lo == hi) store_state(p.dh0 + (long long)s * D, c, D, p.dht ? load_state(p.dht + (long long)s * D, c, D) : both(0.f));
        }
    if (k.c0 >= k.c1) {                              // (the whole cluster)
        if (warp == 0 && on) store_state(part, c, D, both(0.f));
        return;
    }
    const T *px = static_cast<const T *>(p.x), *pd = static_cast<const T *>(p.decay), *pg = static_cast<const T *>(p.gate);
    const T *py = static_cast<const T *>(p.dy);
    if (blocks > 1) kda::tc::cluster_sync_all();     // every block has begun: its shared memory may be written
    const f2 coef = coefficients(p, cl), minus = both(-1.f), one = both(1.f);
    const long long tile0 = k.c0 / BTILE, tiles = ((long long)k.c1 + BTILE - 1) / BTILE - tile0;
    const int turns = (int)((tiles + blocks - 1) / blocks);

    Raw<T, VEC> nx[BROWS], nd[BROWS], ng[BROWS], ny[BROWS];
    f2 saved;                                        // the state that enters the tile
    auto fetch = [&](long long r0) {
#pragma unroll
        for (int j = 0; j < BROWS; ++j) {
            const long long r = r0 + j < k.c0 ? k.c0 : r0 + j >= k.c1 ? k.c1 - 1 : r0 + j;
            nx[j].load(px + r * p.ld_x, cl, D);
            nd[j].load(pd + r * p.ld_decay, cl, D);
            ng[j].load(pg + r * p.ld_gate, cl, D);
            ny[j].load(py + r * p.ld_dy, cl, D);
        }
        const long long top = r0 - warp * BROWS;     // (a tile that begins outside the chain has no saved state and needs none)
        saved = top >= k.c0 && top < k.c1 ? load_state(p.states + top / SAVE * D, cl, D) : both(0.f);
    };
    // The cluster's tiles of a turn are neighbours, the last block's the last; turns go from the end.
    long long r0 = (tile0 + (long long)(turns - 1) * blocks + rank) * BTILE + warp * BROWS;
    fetch(r0);
    Marks<BROWS> marks;
    f2 carry = both(0.f), sum = both(0.f);
    for (int i = 0; i < turns; ++i, r0 -= (long long)blocks * BTILE) {
        f2 a[BROWS], m[BROWS], rm[BROWS], s[BROWS], u[BROWS], x[BROWS], gy[BROWS];
#pragma unroll
        for (int j = 0; j < BROWS; ++j) {
            f2 w;
            s[j] = sigmoid2(nd[j].pair());
            u[j] = sigmoid2(ng[j].pair());
            x[j] = nx[j].pair();
            gy[j] = ny[j].pair();
            decay_of(mul2(coef, s[j]), a[j], w);
            float w0, w1;
            unpack2(w, w0, w1);                      // 1 - a^2 of 0 (no decay at all): its root's reciprocal stays finite, so that times q = 0 it is 0
            rm[j] = pack2(rsqrt_fast(fmaxf(w0, 1e-36f)), rsqrt_fast(fmaxf(w1, 1e-36f)));
            m[j] = mul2(w, rm[j]);
        }
        f2 h = saved;
        if (i + 1 < turns) fetch(r0 - (long long)blocks * BTILE);
        marks.find(p, k, r0);
        const unsigned starts = marks.starts, ends = marks.ends;
        // both walks over this warp's rows alone: the states from 0, the gradients from 0
        f2 hw = both(0.f), prod = a[0], gw = both(0.f);
#pragma unroll
        for (int j = 0; j < BROWS; ++j) {
            const f2 v = mul2(mul2(m[j], u[j]), x[j]);
            if (starts >> j & 1) hw = p.h0 ? fma2(a[j], load_state(p.h0 + (long long)marks.sequence(j) * D, cl, D), v) : v;
            else hw = j ? fma2(a[j], hw, v) : v;
            if (j) prod = mul2(prod, a[j]);
        }
        fwd[i & 1][warp][lane] = quad(prod, hw);
        if (lane == 0) fwd_cut[i & 1][warp] = starts != 0;
#pragma unroll
        for (int j = BROWS - 1; j >= 0; --j) {
            if (ends >> j & 1) {
                gw = p.dht ? load_state(p.dht + (long long)marks.sequence(j) * D, cl, D) : both(0.f);
                gy[j] = add2(gy[j], gw);             // the walk below begins here anew
                gw = mul2(a[j], gy[j]);
            } else {
                gw = mul2(a[j], j == BROWS - 1 ? gy[j] : add2(gy[j], gw));
            }
        }
        f2 grad = enter<true>(ex, i & 1, warp, lane, rank, blocks, prod, gw, ends != 0, carry);
#pragma unroll
        for (int q = 0; q < WARPS - 1; ++q)
            if (q < warp) h = through(fwd[i & 1][q][lane], fwd_cut[i & 1][q], h);
        f2 before[BROWS];                            // the state before each row
#pragma unroll
        for (int j = 0; j < BROWS; ++j) {
            if (starts >> j & 1) h = p.h0 ? load_state(p.h0 + (long long)marks.sequence(j) * D, cl, D) : both(0.f);
            before[j] = h;
            h = fma2(a[j], h, mul2(mul2(m[j], u[j]), x[j]));
        }
#pragma unroll
        for (int j = BROWS - 1; j >= 0; --j) {
            const long long r = r0 + j;
            const f2 G = ends >> j & 1 ? gy[j] : add2(gy[j], grad);
            grad = mul2(a[j], G);
            if (starts >> j & 1) {
                const int q = marks.sequence(j);
                if (p.dh0 && on) store_state(p.dh0 + (long long)q * D, c, D, grad);
            }
            if (r < k.c0 || r >= k.c1) continue;     // (a warp's rows are the same for all its lanes)
            const f2 v = mul2(u[j], x[j]), gm = mul2(G, m[j]);
            // a G (v a / m - h)
            const f2 dq = mul2(grad, fma2(mul2(v, a[j]), rm[j], mul2(before[j], minus)));
            const f2 ds = mul2(dq, s[j]);
            sum = add2(sum, ds);
            if (!on) continue;
            store_pair<T, VEC>(static_cast<T *>(p.ddecay) + r * p.ld_ddecay, c, D, mul2(mul2(ds, coef), fma2(s[j], minus, one)));
            store_pair<T, VEC>(static_cast<T *>(p.dx) + r * p.ld_dx, c, D, mul2(gm, u[j]));
            store_pair<T, VEC>(static_cast<T *>(p.dgate) + r * p.ld_dgate, c, D, mul2(mul2(gm, v), fma2(u[j], minus, one)));
        }
    }
    __syncthreads();                                 // the exchange's last set has been read
    ex.warp[0][warp][lane] = quad(sum, sum);
    __syncthreads();
    if (warp == 0 && on) {
        f2 t = both(0.f);
#pragma unroll
        for (int q = 0; q < WARPS; ++q) t = add2(t, pack2(ex.warp[0][q][lane].x, ex.warp[0][q][lane].y));
        const float e0 = p.rate[c], e1 = p.rate[min(c + 1, D - 1)];
        store_state(part, c, D, mul2(t, pack2(p.scale * sigmoid(e0), p.scale * sigmoid(e1))));
    }
}

// ------------------------------------------------------------------------------------------ single tokens
template <class T, bool VEC> __global__ void __launch_bounds__(128) gated_scan_step_kernel(GatedScanParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int pairs = (p.D - 1) / 2 + 1, D = p.D;
    const long long b = i / pairs;
    if (b >= p.B) return;
    const int c = (int)(i - b * pairs) * 2;
    const int slot = p.slot ? p.slot[b] : (int)b;
    T *y = static_cast<T *>(p.y) + b * p.ld_y;
    if (slot < 0 || slot >= p.slots) {
        store_pair<T, VEC>(y, c, D, both(0.f));
        return;
    }
    Raw<T, VEC> x, d, g;
    x.load(static_cast<const T *>(p.x) + b * p.ld_x, c, D);
    d.load(static_cast<const T *>(p.decay) + b * p.ld_decay, c, D);
    g.load(static_cast<const T *>(p.gate) + b * p.ld_gate, c, D);
    float *state = p.state + (long long)slot * D;
    const f2 old = load_state(state, c, D);
    f2 a, w;
    decay_of(mul2(coefficients(p, c), sigmoid2(d.pair())), a, w);
    const f2 h = fma2(a, old, mul2(mul2(sqrt2(w), sigmoid2(g.pair())), x.pair()));
    store_state(state, c, D, h);
    store_pair<T, VEC>(y, c, D, h);
}

bool vectors(const GatedScanParams &p, bool bf16) {
    const size_t es = bf16 ? 2 : 4, n = 2 * es;
    return p.D % 2 == 0 && rows_aligned(p.x, p.ld_x, es, n) && rows_aligned(p.decay, p.ld_decay, es, n) &&
           rows_aligned(p.gate, p.ld_gate, es, n) && rows_aligned(p.y, p.ld_y, es, n) && rows_aligned(p.dy, p.ld_dy, es, n) &&
           rows_aligned(p.dx, p.ld_dx, es, n) && rows_aligned(p.ddecay, p.ld_ddecay, es, n) && rows_aligned(p.dgate, p.ld_dgate, es, n);
}

cudaError_t launch(void (*kernel)(GatedScanParams), const GatedScanParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.D - 1) / COLS + 1) * p.cluster, p.chains);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

long long rows_of(const GatedScanParams &p) { return (long long)(p.cu_seqlens ? 1 : p.B) * p.T; }

}  // namespace

size_t gated_scan_saved_rows(const GatedScanParams &p) { return (size_t)((rows_of(p) + SAVE - 1) / SAVE); }

// Chains side by side cost nothing, so there are as many as fill the GPU (three blocks to an SM), up to one per
// sequence; what they leave idle, clusters of up to eight blocks fill by sharing a chain's tiles.
void gated_scan_split(GatedScanParams &p, int tile) {
    const long long cols = (p.D - 1) / COLS + 1, want = 3LL * sm_count(), rows = rows_of(p);
    const long long chains = (want + cols - 1) / cols;
    p.chains = (int)(chains < p.B ? chains : p.B);
    p.cluster = 1;
    while (p.cluster < MAX_CLUSTER && cols * p.chains * p.cluster < want && rows > (long long)tile * p.chains * p.cluster) p.cluster *= 2;
}

size_t gated_scan_part_floats(const GatedScanParams &p) {
    GatedScanParams q = p;
    gated_scan_split(q, BTILE);
    return (size_t)q.chains * q.cluster * p.D;
}

cudaError_t launch_gated_scan_fwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    gated_scan_split(p, FTILE);
    const bool v = vectors(p, bf16_);
    if (bf16_) return launch(v ? gated_scan_fwd_kernel<bf16, true> : gated_scan_fwd_kernel<bf16, false>, p, s);
    return launch(v ? gated_scan_fwd_kernel<float, true> : gated_scan_fwd_kernel<float, false>, p, s);
}

cudaError_t launch_gated_scan_bwd(const GatedScanParams &q, bool bf16_, cudaStream_t s) {
    GatedScanParams p = q;
    gated_scan_split(p, BTILE);
    const bool v = vectors(p, bf16_);
    const cudaError_t e = bf16_ ? launch(v ? gated_scan_bwd_kernel<bf16, true> : gated_scan_bwd_kernel<bf16, false>, p, s)
                                : launch(v ? gated_scan_bwd_kernel<float, true> : gated_scan_bwd_kernel<float, false>, p, s);
    if (e != cudaSuccess) return e;
    return launch_sum_rows(p.part, p.chains * p.cluster, SumOut{p.drate, p.D, false}, SumOut{nullptr, 0, false}, s);
}

cudaError_t launch_gated_scan_step(const GatedScanParams &p, bool bf16_, cudaStream_t s) {
    const long long n = (long long)p.B * ((p.D - 1) / 2 + 1);
    const unsigned grid = (unsigned)((n + 127) / 128);
    const bool v = vectors(p, bf16_);
    if (bf16_) {
        if (v) gated_scan_step_kernel<bf16, true><<<grid, 128, 0, s>>>(p);
        else gated_scan_step_kernel<bf16, false><<<grid, 128, 0, s>>>(p);
    } else {
        if (v) gated_scan_step_kernel<float, true><<<grid, 128, 0, s>>>(p);
        else gated_scan_step_kernel<float, false><<<grid, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace mixer
