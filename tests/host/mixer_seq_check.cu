// Host check of the segment-slot arithmetic of mixer_seq.cuh: for random packings and segment
// lengths, every token of every sequence lies in exactly one segment, segments stay inside their
// sequence and the slots inside the count that sizes the workspaces, an empty sequence owns one
// slot, and offsets out of range or decreasing stay in bounds.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mixer_seq.cuh"

static int check(const int *cu, int B, int T, int seg, bool monotone) {
    using namespace mixer;
    const long long slots = segment_slots(B, T, seg, cu != nullptr);
    std::vector<int> seen(cu ? T : (size_t)B * T, 0), owned(B, 0);
    for (long long s = 0; s < slots; ++s) {
        Segment g{};
        if (!segment_of(cu, B, T, seg, s, g)) continue;
        if (g.b < 0 || g.b >= B || g.i < 0 || g.i >= g.n) return 1;
        if (g.len < 0 || g.len > seg || g.t0 < 0 || g.t0 + g.len > g.total) return 2;
        if (g.row0 < 0 || g.row0 + g.total > (long long)seen.size()) return 3;
        if (g.len == 0 && g.total != 0) return 4;
        ++owned[g.b];
        for (int t = 0; t < g.len; ++t) ++seen[g.row0 + g.t0 + t];
    }
    if (!monotone) return 0;
    for (int b = 0; b < B; ++b) {
        const int lo = cu ? clamped(cu[b], 0, T) : b * T, hi = cu ? clamped(cu[b + 1], lo, T) : b * T + T;
        for (int r = lo; r < hi; ++r)
            if (seen[r] != 1) return 5;
        const int n = hi > lo ? (hi - lo + seg - 1) / seg : 1;
        if (owned[b] != n) return 6;
    }
    return 0;
}

int main() {
    srand(4321);
    for (int trial = 0; trial < 6000; ++trial) {
        const int B = 1 + rand() % 9, T = 1 + rand() % 300, seg = 1 + rand() % 130;
        const bool monotone = rand() % 4 != 0;
        int rc = check(nullptr, B, T, seg, true);
        std::vector<int> cu(B + 1);
        for (int i = 0; i <= B; ++i) cu[i] = monotone ? rand() % (T + 1) : rand() % (3 * T) - T;
        if (monotone) {
            for (int i = 0; i <= B; ++i)
                for (int j = i + 1; j <= B; ++j)
                    if (cu[j] < cu[i]) { int x = cu[i]; cu[i] = cu[j]; cu[j] = x; }
            cu[0] = 0;
            if (rand() % 3) cu[B] = T;
        }
        if (!rc) rc = check(cu.data(), B, T, seg, monotone);
        if (rc) {
            printf("trial %d: check %d failed (B %d T %d seg %d)\n", trial, rc, B, T, seg);
            return 1;
        }
    }
    puts("ok");
    return 0;
}
