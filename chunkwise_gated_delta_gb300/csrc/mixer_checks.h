// Argument checks shared by the C-ABI layers of mixer.h's operators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mixer.h"
#include "mixer_common.cuh"

namespace {

// A block of `rows` rows of `cols` elements with a row stride of `ld`, as bytes.
struct Block {
    const void *p;
    long long rows, cols, ld;
    size_t es;
};

size_t es_of(kda_dtype d) { return d == KDA_F32 ? 4 : 2; }
bool dtype_ok(kda_dtype d) { return d == KDA_BF16 || d == KDA_F32; }

long long stride_or(long long ld, long long cols) { return ld ? ld : cols; }

bool overlap(const Block &a, const Block &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.cols < 1 || b.cols < 1) return false;
    const unsigned long long x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const unsigned long long sa = (unsigned long long)a.ld * a.es, sb = (unsigned long long)b.ld * b.es;
    const unsigned long long wa = (unsigned long long)a.cols * a.es, wb = (unsigned long long)b.cols * b.es;
    const unsigned long long ea = x + (a.rows - 1) * sa + wa, eb = y + (b.rows - 1) * sb + wb;
    if (!(x < eb && y < ea)) return false;
    if (sa != sb) return true;
    // equal strides: parts of one buffer's rows, apart when their columns are
    const unsigned long long d = (y >= x ? y - x : x - y) % sa;
    const unsigned long long first = y >= x ? wa : wb, second = y >= x ? wb : wa;
    return d < first || sa - d < second;
}

// Every output apart from every input and from the other outputs; every pointer aligned to its
// element, every stride at least the row.
template <size_t NI, size_t NO> bool blocks_ok(const Block (&in)[NI], const Block (&out)[NO]) {
    for (const Block &b : in)
        if (!mixer::aligned_to(b.p, b.es) || b.ld < b.cols || b.ld > (1LL << 40)) return false;
    for (const Block &b : out)
        if (!mixer::aligned_to(b.p, b.es) || b.ld < b.cols || b.ld > (1LL << 40)) return false;
    for (size_t i = 0; i < NO; ++i) {
        for (const Block &b : in)
            if (overlap(out[i], b)) return false;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

// A packed batch has T rows whatever B is.
bool sizes_ok(int B, int T, int D, bool packed = false) {
    return B >= 1 && T >= 1 && D >= 1 && (packed || (long long)B * T <= 0x7fffffffLL) && (long long)B * D <= (1LL << 40);
}

Block dense(const void *p, long long rows, long long cols, size_t es) { return {p, rows, cols, cols, es}; }

kda_status from(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    cudaGetLastError();                  // a launch that was refused is this call's answer, not the next one's too
    return e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

kda_status check_space(const void *ws, size_t have, size_t need) {
    if (!ws || have < need) return KDA_ERR_WORKSPACE;
    return mixer::aligned_to(ws, 16) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

cudaStream_t stream_of(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace
