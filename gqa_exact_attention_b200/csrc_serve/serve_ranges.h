// The arithmetic of the ranges schedule: all units' steps in one row, cut into one range per CTA.
// A unit whose steps lie in several ranges has parts, each CTA's first piece in slot 2 cta and its
// last in slot 2 cta + 1 of the partials; the blocks of each boundary inside a unit join a share
// of its items.  Plain C++ on the host, so that a test can walk the schedules that the kernels walk.
#pragma once

#include <cstdint>

namespace gqa {

// floor(a * b / c): 64-bit division is slow, and rarely needed
__host__ __device__ inline long long mul_div(long long a, int b, long long c) {
    const long long ab = a * b;
    if ((unsigned long long)ab < (1ull << 32) && c < (1ll << 32)) return (uint32_t)ab / (uint32_t)c;
    return ab / c;
}

// CTAs that take part: each has at least min_blocks steps, if there are
__host__ __device__ inline int range_ctas(long long all, int min_blocks, int grid) {
    const long long n = mul_div(all, 1, min_blocks);
    return n < 1 ? 1 : (n < grid ? (int)n : grid);
}
// CTA c takes steps [range_start(c), range_start(c + 1)); no range is empty while ctas <= all
__host__ __device__ inline long long range_start(long long all, int ctas, int cta) { return mul_div(all, cta, ctas); }
// the CTA of step x: the last whose range starts at or before it, c < (x + 1) ctas / all
__host__ __device__ inline int range_cta(long long all, int ctas, long long x) {
    return (int)mul_div((x + 1) * ctas - 1, 1, all);
}

// How the unit of steps [begin, begin + steps) is shared.
struct UnitShares {
    int cta0;        // the CTA that begins it
    int parts;       // CTAs that share it
    int first_slot;  // where the first one's partials are
};
__host__ __device__ inline UnitShares unit_shares(long long all, int ctas, long long begin, int steps) {
    UnitShares u;
    u.cta0 = range_cta(all, ctas, begin);
    u.parts = range_cta(all, ctas, begin + steps - 1) - u.cta0 + 1;
    u.first_slot = 2 * u.cta0 + (range_start(all, ctas, u.cta0) == begin ? 0 : 1);
    return u;
}
// the slot of a CTA's piece, and that of a unit's part i
__host__ __device__ inline int piece_slot(int cta, bool first_of_range) { return 2 * cta + (first_of_range ? 0 : 1); }
__host__ __device__ inline int part_slot(int cta0, int first_slot, int i) { return i == 0 ? first_slot : 2 * (cta0 + i); }

// Of a unit's `items`, block `block` of `blocks` at the begin of CTA cta's range joins [lo, hi).
struct JoinShare {
    int lo, hi;
};
__host__ __device__ inline JoinShare join_share(int items, int cta, int cta0, int parts, int block, int blocks) {
    const int shares = (parts - 1) * blocks, share = (cta - cta0 - 1) * blocks + block;
    return {items * share / shares, items * (share + 1) / shares};
}

}  // namespace gqa
