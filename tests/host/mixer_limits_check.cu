// Host check of the positions that the scan's forward counts (mixer_seq.cuh): for lengths up to
// 2^31 - 1 and every tile, the number of tiles covers the length, and the rows that are fetched up to
// five tiles past the end exist.
#include <cstdio>

#include "mixer_seq.cuh"

int main() {
    using namespace mixer;
    const int most = 0x7fffffff;
    const int lens[] = {1, 2, 15, 16, 17, 31, 32, 33, 1000, 1 << 30, most - 200, most - 64, most - 63, most - 33, most - 32, most - 31, most - 1, most};
    const int sizes[] = {16, 32, 64};
    for (int len : lens)
        for (int tile : sizes) {
            const long long want = ((long long)len + tile - 1) / tile;
            const int tiles = tiles_of(len, tile);
            if (tiles != want) {
                printf("len %d tile %d: %d tiles\n", len, tile, tiles);
                return 1;
            }
            for (int k = tiles > 3 ? tiles - 3 : 0; k <= tiles + 5; ++k)
                for (int t = 0; t < tile; ++t) {
                    const long long pos = (long long)k * tile + t;
                    const unsigned p = tile_token(k, tile, t);
                    const long long row = row_or_last(p, len);
                    if (inside(p, len) != (pos < len) || row != (pos < len ? pos : len - 1LL)) {
                        printf("len %d tile %d position %lld: row %lld\n", len, tile, pos, row);
                        return 1;
                    }
                }
        }
    puts("ok");
    return 0;
}
