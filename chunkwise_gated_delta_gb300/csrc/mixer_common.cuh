// Loads, stores and sums shared by the kernels behind mixer.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mixer_seq.cuh"

namespace mixer {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }

// One element as it lies in memory, in a register of its own: pairs of 16-bit values would share
// one, and the load would be waited for where they are put together.  Loads of what a kernel only reads
// are told apart from those of what it writes (__ldg): they may then move ahead of its stores.
__device__ __forceinline__ uint32_t load_bits(const float *p) { return __float_as_uint(__ldg(p)); }
__device__ __forceinline__ uint32_t load_bits(const bf16 *p) { return __ldg(reinterpret_cast<const unsigned short *>(p)); }
template <class T> __device__ __forceinline__ float bits_f(uint32_t v) {
    return __uint_as_float(sizeof(T) == 4 ? v : v << 16);
}

// A parameter vector stored as bfloat16 or float32 (uniform over the launch).
__device__ __forceinline__ float load_w(const void *p, long long i, bool is_bf16) {
    return is_bf16 ? __uint_as_float(load_bits(static_cast<const bf16 *>(p) + i) << 16) : __ldg(static_cast<const float *>(p) + i);
}
__device__ __forceinline__ void store_w(void *p, long long i, bool is_bf16, float v) {
    if (is_bf16) static_cast<bf16 *>(p)[i] = from_f<bf16>(v);
    else static_cast<float *>(p)[i] = v;
}

// V neighbouring parameters from element i (a multiple of V; V elements of a 16-byte aligned vector).
template <int V> __device__ __forceinline__ void load_params(float (&o)[V], const void *p, long long i, bool is_bf16);

// V neighbouring elements in one access of V sizeof(T) bytes, kept packed.  At most 16 bytes: no pointer is
// known to be aligned to more, neither the caller's tensors nor the workspaces.
template <class T, int V> struct alignas(V * sizeof(T)) Vec {
    static_assert(V * sizeof(T) <= 16, "an access takes at most 16 bytes");
    T e[V];
};
template <class T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, V> *>(p);
}
// The same of data that the kernel does not write.
template <class T, int V> __device__ __forceinline__ Vec<T, V> load_const(const T *p) {
    constexpr int N = V * sizeof(T);
    static_assert(N == 2 || N == 4 || N == 8 || N == 16, "one access");
    Vec<T, V> v;
    if constexpr (N == 2) {
        const unsigned short q = __ldg(reinterpret_cast<const unsigned short *>(p));
        memcpy(&v, &q, N);
    } else if constexpr (N == 4) {
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(p));
        memcpy(&v, &q, N);
    } else if constexpr (N == 8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p));
        memcpy(&v, &q, N);
    } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
        memcpy(&v, &q, N);
    }
    return v;
}
template <class T, int V> __device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v) {
    *reinterpret_cast<Vec<T, V> *>(p) = v;
}

template <int V> __device__ __forceinline__ void load_params(float (&o)[V], const void *p, long long i, bool is_bf16) {
    if (is_bf16) {
        const Vec<bf16, V> v = load_const<bf16, V>(static_cast<const bf16 *>(p) + i);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = to_f(v.e[e]);
    } else {
        constexpr int F = V < 4 ? V : 4;
#pragma unroll
        for (int k = 0; k < V / F; ++k) {
            const Vec<float, F> v = load_const<float, F>(static_cast<const float *>(p) + i + k * F);
#pragma unroll
            for (int e = 0; e < F; ++e) o[k * F + e] = v.e[e];
        }
    }
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }

// Two float32 values in one 64-bit register: the packed forms of the FMA pipe do both in one issue
// slot (the same arithmetic rate, half the instructions, and issue slots are what runs short).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// v sigmoid(v) of two values at once.
__device__ __forceinline__ f2 silu2(f2 v) {
    float lo, hi;
    unpack2(mul2(v, both(-kLog2e)), lo, hi);
    unpack2(add2(pack2(ex2(lo), ex2(hi)), both(1.f)), lo, hi);
    return mul2(v, pack2(rcp(lo), rcp(hi)));
}

// sigmoid of two values at once.
__device__ __forceinline__ f2 sigmoid2(f2 v) {
    float lo, hi;
    unpack2(mul2(v, both(-kLog2e)), lo, hi);
    unpack2(add2(pack2(ex2(lo), ex2(hi)), both(1.f)), lo, hi);
    return pack2(rcp(lo), rcp(hi));
}

// Four neighbouring elements as they lie in memory.
template <class T> struct RawQuad;
template <> struct RawQuad<float> {
    using type = float4;
    static __device__ __forceinline__ float4 floats(float4 v) { return v; }
};
template <> struct RawQuad<bf16> {
    using type = uint2;
    static __device__ __forceinline__ float4 floats(uint2 v) {
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
};

// V neighbouring elements of a row: as they lie in memory in registers, then as pairs of float32 (of one
// element, V = 1, the upper half is 0 and means nothing).
template <class T, int V> struct Lanes {
    static constexpr int P = (V + 1) / 2, WORDS = (V * (int)sizeof(T) + 3) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V * sizeof(T) < 4) w[0] = load_bits(p);
        else {
            const Vec<uint32_t, WORDS> v = load_const<uint32_t, WORDS>(reinterpret_cast<const uint32_t *>(p));
#pragma unroll
            for (int k = 0; k < WORDS; ++k) w[k] = v.e[k];
        }
    }
    __device__ __forceinline__ void load_shared(const void *p) {      // (V sizeof(T) >= 4)
        const Vec<uint32_t, WORDS> v = load_vec<uint32_t, WORDS>(static_cast<const uint32_t *>(p));
#pragma unroll
        for (int k = 0; k < WORDS; ++k) w[k] = v.e[k];
    }
    // These elements, or zeros.
    __device__ __forceinline__ Lanes kept(bool on) const {
        Lanes r;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) r.w[k] = w[k] & (on ? ~0u : 0u);
        return r;
    }
    __device__ __forceinline__ f2 pair(int k) const {
        if constexpr (V == 1) return pack2(bits_f<T>(w[0]), 0.f);
        else if constexpr (sizeof(T) == 4) return pack2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        else return pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
};
template <class T, int V> __device__ __forceinline__ void store_lanes(T *p, const f2 (&v)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        float lo, hi;
        unpack2(v[0], lo, hi);
        *p = from_f<T>(lo);
    } else {
        constexpr int E = V * sizeof(T) <= 16 ? V : 16 / (int)sizeof(T);      // elements per access
#pragma unroll
        for (int a = 0; a < V; a += E) {
            Vec<T, E> o;
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                float lo, hi;
                unpack2(v[a / 2 + k], lo, hi);
                o.e[2 * k] = from_f<T>(lo);
                o.e[2 * k + 1] = from_f<T>(hi);
            }
            store_vec<T, E>(p + a, o);
        }
    }
}
// N bytes (4, 8 or 16) from global to shared memory, asynchronously.
template <int N> __device__ __forceinline__ void copy_async(void *to, const void *from) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this thread's copies have arrived.
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int V> __device__ __forceinline__ float pair_sum(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return V == 1 ? lo : lo + hi;
}
// V neighbouring parameters as pairs.
template <int V> __device__ __forceinline__ void load_param_pairs(f2 (&o)[(V + 1) / 2], const void *p, long long i, bool is_bf16) {
    float v[V];
    load_params<V>(v, p, i, is_bf16);
    if constexpr (V == 1) o[0] = pack2(v[0], 0.f);
    else
#pragma unroll
        for (int k = 0; k < V / 2; ++k) o[k] = pack2(v[2 * k], v[2 * k + 1]);
}


__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
}

// Sums `rows` rows of partial sums [rows][cols], in row order within each of 32 strided groups,
// into two vectors that lie side by side in a row.
struct SumOut {
    void *out;          // NULL: not written
    long long cols;
    bool bf16;
};
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *part, int rows, long long cols, SumOut o0, SumOut o1);
cudaError_t launch_sum_rows(const float *part, int rows, SumOut o0, SumOut o1, cudaStream_t s);

// Streaming multiprocessors of the current device (152 if the query fails: sizes only).
int sm_count();

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Rows of `es`-byte elements that may be read n bytes at a time (a NULL pointer may).
inline bool rows_aligned(const void *p, long long ld, size_t es, size_t n) {
    return !p || (aligned_to(p, n) && (size_t)ld * es % n == 0);
}

}  // namespace mixer
