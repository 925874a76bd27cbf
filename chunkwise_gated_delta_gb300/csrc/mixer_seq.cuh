// Rows and segment slots of the sequences of a dense or packed batch, for segments of a length
// chosen at run time (host and device).
//
// Dense: sequence b holds rows b T .. b T + T - 1 and slots b n .. b n + n - 1, n = ceil(T / seg).
// Packed (cu_seqlens): sequence b holds rows lo .. hi - 1, offsets clamped into [0, T], and slots
// b + floor(lo / seg) + i.  The next sequence's first slot lies at least ceil((hi - lo) / seg) and
// at least 1 further on, so no two sequences share a slot, an empty sequence has one to itself
// (its states pass through it), and B + ceil(T / seg) slots hold them all.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mixer {

struct Segment {
    int b;           // sequence
    int i, n;        // segment of it, and how many it has (1 for an empty sequence)
    int t0, len;     // first token within the sequence, tokens
    int total;       // tokens of the whole sequence
    long long row0;  // row of the sequence's first token
};

__host__ __device__ inline long long segment_slots(int B, int T, int seg, bool packed) {
    const long long n = (T + (long long)seg - 1) / seg;
    return packed ? B + n : B * n;
}

__host__ __device__ inline int clamped(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__host__ __device__ inline long long first_slot(const int32_t *cu, int T, int seg, int b) {
    return (long long)b + clamped(cu[b], 0, T) / seg;
}

// The segment in slot s.  False for a slot that no sequence uses.
__host__ __device__ inline bool segment_of(const int32_t *cu, int B, int T, int seg, long long s, Segment &g) {
    if (!cu) {
        const int n = (int)((T + (long long)seg - 1) / seg);
        g.b = (int)(s / n);
        g.i = (int)(s - (long long)g.b * n);
        g.n = n;
        g.total = T;
        g.row0 = (long long)g.b * T;
    } else {
        int lo = 0, hi = B - 1;   // the last sequence whose first slot is at or before s
        while (lo < hi) {
            const int mid = (int)(((long long)lo + hi + 1) >> 1);
            if (first_slot(cu, T, seg, mid) <= s) lo = mid;
            else hi = mid - 1;
        }
        const int r0 = clamped(cu[lo], 0, T), r1 = clamped(cu[lo + 1], r0, T);
        g.b = lo;
        g.total = r1 - r0;
        g.row0 = r0;
        g.n = g.total > 0 ? (int)((g.total + (long long)seg - 1) / seg) : 1;
        const long long i = s - first_slot(cu, T, seg, lo);
        if (i < 0 || i >= g.n) return false;
        g.i = (int)i;
    }
    g.t0 = g.i * seg;
    g.len = g.total - g.t0 < seg ? g.total - g.t0 : seg;
    return true;
}

// Slot of the segment that begins at token t0 of sequence b, for segments of another length.
__host__ __device__ inline long long slot_at(const int32_t *cu, int T, int seg, int b, int t0) {
    return (cu ? first_slot(cu, T, seg, b) : b * ((T + (long long)seg - 1) / seg)) + t0 / seg;
}

// The rows that the sequences of a call cover, for kernels that cut them in segments whatever the sequences' lengths.
struct Extent {
    int lo, hi;
};
__host__ __device__ inline Extent extent_of(const int32_t *cu, int B, int T) {
    if (!cu) return {0, (int)((long long)B * T)};
    const int lo = clamped(cu[0], 0, T);
    return {lo, clamped(cu[B], lo, T)};
}
// Whether any of the rows r0 .. r0 + n - 1 is covered.  (No row is where all sequences are empty, wherever they lie.)
__host__ __device__ inline bool covers(const Extent &k, long long r0, int n) { return k.lo < k.hi && r0 < k.hi && r0 + n > k.lo; }
// The covered row nearest to r, of an extent that covers some.
__host__ __device__ inline long long nearest_row(const Extent &k, long long r) { return r < k.lo ? k.lo : r >= k.hi ? k.hi - 1 : r; }

// A kernel that walks `len` tokens in tiles counts tokens past the end too: the last tile's, and those of the
// tiles that it looks ahead.  Lengths reach 2^31 - 1, so these positions have no sign.
__host__ __device__ inline int tiles_of(int len, int tile) { return (int)(((unsigned)len + tile - 1) / tile); }
__host__ __device__ inline unsigned tile_token(int k, int tile, int t) { return (unsigned)k * tile + t; }
__host__ __device__ inline bool inside(unsigned pos, int len) { return pos < (unsigned)len; }
// Row at a position, the last one past the end (len > 0).
__host__ __device__ inline long long row_or_last(unsigned pos, int len) { return inside(pos, len) ? pos : (unsigned)len - 1; }

}  // namespace mixer
