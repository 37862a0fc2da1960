// Where fp32 leaves the grouped router's order open (host and device, no GPU needed).
#pragma once

namespace moe {

constexpr float magnitude(float v) { return v < 0.0f ? -v : v; }

// What a group is compared by, and what that may be off: its largest choice, or half the sum of its
// two largest (halves do not run over fp32; two = -inf: there is only one).  A choice is off by off / 2
// and by half a step of itself, and the sum and what is added to or taken from it are rounded: four half
// steps at most of |one| + |two|, and not of the sum, for choices of opposite signs cancel.
struct GroupSum {
    float value, off;
};
constexpr GroupSum group_sum(float one, float two, bool pairs, float off) {
    // of an infinite choice, which is one in fp64 too, nothing is off
    const bool finite = magnitude(one) < __builtin_inff();
    if (!pairs) return {one, finite ? 0.5f * off + magnitude(one) * 0x1p-23f : 0.0f};
    const bool both = two > -__builtin_inff();
    const float second = both ? 0.5f * two : 0.0f;
    return {0.5f * one + second, finite ? 0.5f * off + (0.5f * magnitude(one) + magnitude(second)) * 0x1p-22f : 0.0f};
}

// May the choice y, no larger than x, lie above it in fp64?  Each is off by off / 2 and by half a step.
// Next to an infinite choice the order is in no doubt: masked experts (-inf) are behind all others, and
// among themselves in id order.
constexpr bool near_choices(float x, float y, float off) {
    const float gap = x - y;                           // of equal infinities NaN
    return gap < __builtin_inff() && gap <= off + (magnitude(x) + magnitude(y)) * 0x1p-23f;
}

}  // namespace moe
