// Test driver for what fp32 leaves open in the grouped router (csrc/route_doubt.hpp), built by
// tests/test_route_doubt.py.  Reads lines "one two pairs off" and prints what a group is compared by and
// what that may be off (pairs = 2: 1 if the choice two may lie above one, else 0).
#include <cstdio>

#include "route_doubt.hpp"

int main() {
    float one, two, off;
    int pairs;
    while (std::scanf("%f %f %d %f", &one, &two, &pairs, &off) == 4) {
        if (pairs == 2) {
            std::printf("%d\n", moe::near_choices(one, two, off));
            continue;
        }
        const moe::GroupSum s = moe::group_sum(one, two, pairs != 0, off);
        std::printf("%a %a\n", (double)s.value, (double)s.off);
    }
    return 0;
}
