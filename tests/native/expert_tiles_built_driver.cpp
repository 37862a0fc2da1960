// Test driver for which tiles expert_tile (csrc/product_tile.hpp) has a program build for a format that is
// known to the compiler, built by tests/test_expert_tiles_built.py.  First prints the tiles that are built, in
// lines "swiglu bf16 columns rows", then reads lines "swiglu bf16 M G N offsets" and prints the tile each takes.
#include <cstdio>
#include <set>
#include <tuple>
#include <type_traits>

#include "product_tile.hpp"

typedef std::tuple<int, int, int, int> Name;
static std::set<Name>& built() {
    static std::set<Name> all;
    return all;
}

// Its value is taken before main, for every tile that the rule's f is built with.
template <bool SWIGLU, class Bf16, class C>
struct Built {
    static const bool value;
};
template <bool SWIGLU, class Bf16, class C>
const bool Built<SWIGLU, Bf16, C>::value = built().insert(Name{SWIGLU, Bf16::value, C::PA, C::PB}).second;

template <bool SWIGLU, class Bf16>
static int tile(long long M, long long G, long long N, bool offsets) {
    return moe::expert_tile<SWIGLU>(Bf16{}, M, G, N, offsets, [](auto t) {
        return Built<SWIGLU, Bf16, decltype(t)>::value ? std::printf("%d %d\n", t.PA, t.PB) : 0;
    });
}

int main() {
    for (const auto& [s, b, columns, rows] : built()) std::printf("%d %d %d %d\n", s, b, columns, rows);
    std::printf("end\n");
    int swiglu, bf16, offsets;
    long long M, G, N;
    while (std::scanf("%d %d %lld %lld %lld %d", &swiglu, &bf16, &M, &G, &N, &offsets) == 6) {
        if (swiglu) bf16 ? tile<true, std::true_type>(M, G, N, offsets) : tile<true, std::false_type>(M, G, N, offsets);
        else bf16 ? tile<false, std::true_type>(M, G, N, offsets) : tile<false, std::false_type>(M, G, N, offsets);
    }
    return 0;
}
