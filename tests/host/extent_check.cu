// Host check of the rows that the gated recurrence reads: for dense calls and packings of every kind (gaps before and behind, empty
// sequences, none but empty ones wherever they lie, offsets out of range or decreasing), the segments that work are those that hold a
// covered row, and every row that one of them brings, eight at a time, is a row of the call.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mixer_seq.cuh"

static int check(const int *cu, int B, int T, int seg) {
    using namespace mixer;
    const long long rows = (long long)(cu ? 1 : B) * T, segs = (rows + seg - 1) / seg;
    const Extent k = extent_of(cu, B, T);
    if (k.lo < 0 || k.hi < k.lo || k.hi > rows) return 1;
    for (long long s = 0; s < segs; ++s) {
        const long long r0 = s * seg, end = k.hi < r0 + seg ? k.hi : r0 + seg;
        bool any = false;
        for (long long r = r0; r < r0 + seg; ++r) any |= r >= k.lo && r < k.hi;
        if (covers(k, r0, seg) != any) return 2;
        if (!any) continue;
        if (end <= r0) return 3;
        for (long long next = r0; next <= r0 + (end - 1 - r0) / 8 * 8; next += 8)
            for (int j = 0; j < 8; ++j) {
                const long long r = next >= k.lo && next + 8 <= k.hi ? next + j : nearest_row(k, next + j);
                if (r < k.lo || r >= k.hi || r >= rows) return 4;
            }
    }
    return 0;
}

int main() {
    srand(99);
    for (int trial = 0; trial < 20000; ++trial) {
        const int B = 1 + rand() % 6, T = 1 + rand() % 200, seg = 8 * (1 + rand() % 16);
        std::vector<int> cu(B + 1);
        const int kind = rand() % 3, at = rand() % 3 ? T : rand() % (T + 20);
        for (int i = 0; i <= B; ++i) cu[i] = kind == 0 ? at : kind == 1 ? rand() % (3 * T) - T : rand() % (T + 1);
        if (kind == 2)
            for (int i = 0; i <= B; ++i)
                for (int j = i + 1; j <= B; ++j)
                    if (cu[j] < cu[i]) { const int x = cu[i]; cu[i] = cu[j]; cu[j] = x; }
        int rc = check(nullptr, B, T, seg);
        if (!rc) rc = check(cu.data(), B, T, seg);
        if (rc) {
            printf("trial %d: check %d failed (B %d T %d seg %d, offsets %d to %d)\n", trial, rc, B, T, seg, cu[0], cu[B]);
            return 1;
        }
    }
    puts("ok");
    return 0;
}
