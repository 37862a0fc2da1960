// Test driver for the rules that pick an expert product's tile and that of a matrix' gradient
// (csrc/product_tile.hpp), built by tests/test_expert_tiles.py.  Reads lines "rule bf16 M G N K offsets"
// and prints for each the tile's columns, rows, bytes of a stage's row and stages, and the parts.
#include <cstdio>

#include "product_tile.hpp"

int main() {
    char rule;
    int bf16, offsets;
    long long M, G, N, K;
    while (std::scanf(" %c %d %lld %lld %lld %lld %d", &rule, &bf16, &M, &G, &N, &K, &offsets) == 7) {
        auto print = [](auto t, int parts) { return std::printf("%d %d %d %d %d\n", t.PA, t.PB, t.RB, t.S, parts); };
        if (rule == 'm') moe::matrix_tile(M, G, N, K, print);
        else if (rule == 's') moe::expert_tile<true>(bf16 != 0, M, G, N, offsets != 0, [&](auto t) { return print(t, 1); });
        else moe::expert_tile<false>(bf16 != 0, M, G, N, offsets != 0, [&](auto t) { return print(t, 1); });
    }
    return 0;
}
