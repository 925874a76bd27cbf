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
// one, and the load would be waited for where they are put together.
__device__ __forceinline__ uint32_t load_bits(const float *p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t load_bits(const bf16 *p) { return *reinterpret_cast<const unsigned short *>(p); }
template <class T> __device__ __forceinline__ float bits_f(uint32_t v) {
    return __uint_as_float(sizeof(T) == 4 ? v : v << 16);
}

// A parameter vector stored as bfloat16 or float32 (uniform over the launch).
__device__ __forceinline__ float load_w(const void *p, long long i, bool is_bf16) {
    return is_bf16 ? to_f(static_cast<const bf16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_w(void *p, long long i, bool is_bf16, float v) {
    if (is_bf16) static_cast<bf16 *>(p)[i] = from_f<bf16>(v);
    else static_cast<float *>(p)[i] = v;
}

// V neighbouring elements in one access of V sizeof(T) bytes, kept packed.
template <class T, int V> struct alignas(V * sizeof(T)) Vec {
    T e[V];
};
template <class T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, V> *>(p);
}
template <class T, int V> __device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v) {
    *reinterpret_cast<Vec<T, V> *>(p) = v;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
}

// Sums `rows` rows of partial sums [rows][cols], in row order within each of 8 strided groups,
// into up to three vectors that lie side by side in a row.
struct SumOut {
    void *out;          // NULL: not written
    long long cols;
    bool bf16;
};
__global__ void __launch_bounds__(256) sum_rows_kernel(const float *part, int rows, long long cols, SumOut o0, SumOut o1,
                                                       SumOut o2);
cudaError_t launch_sum_rows(const float *part, int rows, SumOut o0, SumOut o1, SumOut o2, cudaStream_t s);

// Streaming multiprocessors of the current device (152 if the query fails: sizes only).
int sm_count();

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Rows of `es`-byte elements that may be read n bytes at a time (a NULL pointer may).
inline bool rows_aligned(const void *p, long long ld, size_t es, size_t n) {
    return !p || (aligned_to(p, n) && (size_t)ld * es % n == 0);
}

}  // namespace mixer
