// evict_select.cuh -- how an eviction finds the rows that stay, as plain arithmetic: what the kernel computes per
// thread, and what a host program can walk through (no CUDA needed beyond the qualifiers).
#pragma once

#include <cstdint>

namespace e2d2 {

// Ranks are looked at by 11, 11 and 10 bits in turn; a histogram has a bin for each value of the first two.
constexpr int kEvictBins = 2048;
__host__ __device__ constexpr int evict_pass_bits(int pass) { return pass < 2 ? 11 : 10; }
__host__ __device__ constexpr int evict_pass_shift(int pass) { return pass == 0 ? 21 : (pass == 1 ? 10 : 0); }

// Whether rows of a head must be chosen.  Not for keep = 0: nothing stays, and no bin holds the 0-th largest rank.
__host__ __device__ constexpr bool evict_selects(int P, int keep) { return keep > 0 && P > keep; }

// What the passes know so far: the leading bits of the threshold (the rank of the last row that stays), how many rows
// with those bits stay, and how many there are.
struct EvictPick {
    uint32_t prefix, need, equal;
};

// One of the threads that share a pass's bins, from the largest down: thread tid has mine[i], the count of bin
// 2047 - BINS tid - i, `sum` rows in all, `above` rows in the bins before it.  True for the one thread that has the
// bin where the count from above reaches `need` (1 at least); `pick` then goes on to that bin.
template <int BINS>
__host__ __device__ inline bool evict_pick(const uint32_t (&mine)[BINS], uint32_t above, uint32_t sum, uint32_t need,
                                           int tid, int bits, uint32_t prefix, EvictPick& pick) {
    if (above >= need || need > above + sum) return false;
    int i = 0;
    while (i < BINS - 1 && above + mine[i] < need) above += mine[i++];
    pick.prefix = (prefix << bits) | ((2047u - BINS * tid - i) & ((1u << bits) - 1u));
    pick.need = need - above;
    pick.equal = mine[i];
    return true;
}

}  // namespace e2d2
