// Test driver for the rule that picks a product's tile (csrc/product_tile.hpp), built by
// tests/test_product_tiles.py.  Reads lines "swiglu M G N offsets" and prints for each the
// tile's matrix rows, rows, waves and stages.
#include <cstdio>

#include "product_tile.hpp"

int main() {
    int swiglu, offsets;
    long long M, G, N;
    while (std::scanf("%d %lld %lld %lld %d", &swiglu, &M, &G, &N, &offsets) == 5) {
        auto print = [](auto t) { return std::printf("%d %d %d %d\n", t.TW, t.TT, t.WAVES, t.S); };
        if (swiglu) moe::product_tile<true>(M, G, N, offsets != 0, print);
        else moe::product_tile<false>(M, G, N, offsets != 0, print);
    }
    return 0;
}
