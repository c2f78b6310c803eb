// qm_attend_parts.h -- of cache_attend's cut into runs what needs no warp: shares of the
// units, and how the CTAs that share an item tell of its parts. Plain C++, so that a test
// on the host compiles it as it stands.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QM_BOTH __host__ __device__ __forceinline__
#else
#define QM_BOTH inline
#endif

namespace qm {
namespace attend {

// total * c / runs, in 32 bits where they hold it.
QM_BOTH int64_t share(int64_t total, int c, int runs) {
    if (total < (1 << 22) && c < 1024) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(runs);
    return total * c / runs;
}

// Whether every item has a CTA to itself: there are enough of them, and no item is so long that splitting it
// would be quicker (cost: what a split costs, in units). items: how many, the longest of `most` units; `total`
// units on `used` of `runs` CTAs (none where no sequence has rows).
QM_BOTH bool item_each(int items, int most, int64_t total, int used, int runs, int cost) {
    return used > 0 && items <= runs && most <= share(total, 1, used) + cost;
}

// attend_tiles_kernel, for attend_join_kernel: eight ints of each CTA. [0] its first part; [1] 1 if
// its last part begins an item that it does not finish, whose [2] first token, [3] key
// head, [4] first row, [5] rows and [6] position of its sequence's first new token follow.
constexpr int kDesc = 8;
enum : int {
    kNoPart = 0,  // its run begins with an item, or is empty, or was abandoned
    kInner = 1,   // neither end of its item
    kLast = 2,    // its item's last
};

// The CTA that has the last part of the item that CTA c's last part begins; -1 where c
// begins none, or where a part of it is missing: a CTA whose wait gave up leaves its
// descriptor as a run without parts.
QM_BOTH int last_part(const int* desc, int c, int runs) {
    if (desc[c * kDesc + 1] == 0) return -1;
    for (int i = c + 1; i < runs; ++i) {
        if (desc[i * kDesc] == kLast) return i;
        if (desc[i * kDesc] != kInner) return -1;
    }
    return -1;
}

// attend_rows_kernel: a CTA's flag is at the call's mark (odd) from when its part of an item that goes on
// is there until the item's joiner has seen it. A captured call keeps its mark in every replay, so
// no flag may stay at it when the kernel ends, whatever ended it: a joiner whose wait gave
// up leaves the mark's complement, and the later of the two takes the flag back.
// F: swap(v) exchanges the flag for v (acquire and release), set(v) stores it.
template <class F>
QM_BOTH void take_back(F f, unsigned long long before, unsigned long long mark) {  // by the part's CTA: `before` the mark
    if (before == ~mark) f.set(0);
}
template <class F>
QM_BOTH bool give_up(F f, unsigned long long mark) {  // by the joiner; true: the part came after all
    if (f.swap(~mark) != mark) return false;
    f.set(0);
    return true;
}

}  // namespace attend
}  // namespace qm
