// Second step of the sums over tokens: partial sums of blocks, in a fixed order.
#include "mixer_common.cuh"

namespace mixer {

// 32 columns x 32 groups of rows per block.  A few MB at most, from L2: bound by latency, so the
// groups run side by side and each thread keeps four loads in flight.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *part, int rows, long long cols, SumOut o0, SumOut o1) {
    __shared__ float sm[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < cols) {
        const float *p = part + c;
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        int r = ty;
        for (; r + 96 < rows; r += 128) {
            a0 += p[(long long)r * cols];
            a1 += p[(long long)(r + 32) * cols];
            a2 += p[(long long)(r + 64) * cols];
            a3 += p[(long long)(r + 96) * cols];
        }
        for (; r < rows; r += 32) a0 += p[(long long)r * cols];
        s = (a0 + a1) + (a2 + a3);
    }
    sm[ty][tx] = s;
    __syncthreads();
    s = warp_sum(sm[tx][ty]);            // warp ty: column ty's 32 groups
    const long long k = (long long)blockIdx.x * 32 + ty;
    if (tx == 0 && k < cols) {
        if (k < o0.cols) {
            if (o0.out) store_w(o0.out, k, o0.bf16, s);
        } else if (o1.out) {
            store_w(o1.out, k - o0.cols, o1.bf16, s);
        }
    }
}

cudaError_t launch_sum_rows(const float *part, int rows, SumOut o0, SumOut o1, cudaStream_t s) {
    const long long cols = o0.cols + o1.cols;
    sum_rows_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(part, rows, cols, o0, o1);
    return cudaGetLastError();
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        n < 1)
        return 152;
    return n;
}

}  // namespace mixer
