// Split tiles of the grouped and of the scaled products: who joins the partials,
// and the device words of their plans.
#pragma once
#include "ptx.cuh"

namespace psm {

enum : int { G_STATUS_PIPE_TIMEOUT = 2 };
// a plan's device words: the status; how often a timeout has been reported; and,
// for tests, the unit that gives up, counted from 1
enum : int { G_WORD_STATUS, G_WORD_TIMEOUTS, G_WORD_GIVE_UP, G_WORDS };

// The counter of a split tile holds (tag << 16) | count.  A word with another
// tag (of another run, or whatever the workspace held) counts as none, so the
// workspace needs no clearing, and the last arrival leaves 0, so that a replay
// of the same launch starts afresh.  The tile's first contributor opens the
// counter long before anyone arrives; an arrival is then one atomic add.  (With
// a compare-and-swap an arrival, five contributors took up to 6 us to count.)
// An arrival that finds it unopened opens it itself.
//
// A run whose waits ran out leaves counts behind, and a replay of it has the
// same run number.  So the tag also counts the plan's reported timeouts: what
// such a run left then reads as another run's.
__device__ __forceinline__ uint64_t grouped_tag(uint64_t epoch, const int* words) {
    return (epoch + (uint64_t)(uint32_t)words[G_WORD_TIMEOUTS] * 0x9e3779b97f4a7c15ull) & 0xffffffffffffull;
}

__device__ __forceinline__ void grouped_open_counter(unsigned long long* f, uint64_t tag) {
    uint64_t cur = *reinterpret_cast<volatile unsigned long long*>(f);
#pragma unroll 1
    for (int tries = 0; tries < (1 << 20) && (cur >> 16) != tag; ++tries) {
        const uint64_t prev = atom_cas_acq_rel_u64(f, cur, tag << 16);
        if (prev == cur) return;
        cur = prev;
    }
}

// Count one contribution in; true when it was the last of n.
__device__ __forceinline__ bool grouped_count_in(unsigned long long* f, uint64_t tag, uint32_t n) {
    uint64_t have = atom_add_acq_rel_u64(f, 1);
    if ((have >> 16) != tag) {
        uint64_t cur = have + 1;  // what the add left; it has not counted
#pragma unroll 1
        for (int tries = 0; tries < (1 << 20); ++tries) {
            const uint64_t base = (cur >> 16) == tag ? cur : tag << 16;
            const uint64_t prev = atom_cas_acq_rel_u64(f, cur, base + 1);
            if (prev == cur) {
                have = base;
                break;
            }
            cur = prev;
        }
    }
    const bool last = (have & 0xffffu) + 1 == n;
    if (last) *reinterpret_cast<volatile unsigned long long*>(f) = 0;
    return last;
}

}  // namespace psm
