// qm_attend_parts.h -- how the CTAs that share an item of cache_attend tell of its
// parts. Plain C++, so that a test on the host compiles it as it stands.
#pragma once

#ifdef __CUDACC__
#define QM_BOTH __host__ __device__ __forceinline__
#else
#define QM_BOTH inline
#endif

namespace qm {
namespace attend {

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

}  // namespace attend
}  // namespace qm
