// Test driver for how a launch's workgroups are laid out (csrc/product_tile.hpp), built by tests/test_grid.py.
// Reads lines "workgroups waves" and prints for each the columns and rows.
#include <cstdio>

#include "product_tile.hpp"

int main() {
    long long n;
    int waves;
    while (std::scanf("%lld %d", &n, &waves) == 2) {
        const moe::Grid g = moe::grid_of(n, waves);
        std::printf("%lld %lld\n", (long long)g.columns, (long long)g.rows);
    }
    return 0;
}
