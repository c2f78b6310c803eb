// qm_router.cu -- the choice of each token's experts from its router logits
// (select_kernel) and the weighted sum of what those experts gave
// (combine_kernel).
//
// Choice. Keys are s + bias, s = softmax(l) or sigmoid(l); without a bias the order
// of the logits is the order of the keys, and they are compared as they are. A
// warp takes a token and holds its logits in registers: 32 / G' lanes to a group (G'
// the groups rounded up to a power of two), a group's experts dealt to its lanes in
// turn. Keys are order-preserving integers from then on. Group scores meet by shuffles
// within a group's lanes, and each group counts those before it. The topk-th largest
// of the lanes' own largest keys is a bound that at least topk keys reach and seldom
// many more: those move to a list, a lane each, and each counts the entries before
// its own, which is its place. (One maximum after another over all keys: 57 us for the
// case below; a list: 36.)
//
// Keys that are sums or exponentials carry float32 roundings, and two of them may
// lie closer than those. Neighbours in the order (and group scores about the border)
// nearer than a bound on their errors, unless their logit and bias are the same, are
// compared by float64 keys of the candidates concerned, one to a lane; what does not fit
// a list goes to select_ties (many equal keys, one after another) or select_exact (all of
// a token in float64).
//
// It reads each logit once; what bounds it is instructions, some 500 a token without a
// bias or groups and 1080 with both, at 70 % of the issue slots: 16384 tokens of 256
// experts take 9.6 us (top 8 of all) and 22 us (sigmoid, bias, 4 of 8 groups by their
// two best), against 2.6 us of memory time. Some 60 of the latter's tokens need float64,
// whose chain of operations at 1/64 of float32's rate the last of them shows: 3 us. Asking
// for the next token's logits ahead changed nothing (32 warps to an SM hide them).
//
// Sum. Eight columns of one token to a thread, up to eight of its experts' rows asked for
// before the first is used: 4096 tokens x 8 rows of 2880 take 34 us, 6.9 TB/s.
#include <cuda_runtime.h>

#include <algorithm>

#include "qm_device.cuh"
#include "qm_epilogue.cuh"
#include "qm_internal.h"

namespace qm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSelectWarps = 4;

struct Select {
    const void* logits;
    int64_t stride;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t T;
    int dtype;
    int gsize;        // experts of a group
    int groups, topk_groups, top2;
    int lanes_log2;   // log2 of a group's lanes
    int topk;
    int sigmoid, renormalize;
    float scale;
};

QM_DEV float load_logit(const Select& a, int64_t t, int e) {
    const int64_t i = t * a.stride + e;
    if (a.dtype == QM_F32) return __ldca(static_cast<const float*>(a.logits) + i);
    const uint32_t h = __ldca(static_cast<const uint16_t*>(a.logits) + i);
    return a.dtype == QM_F16 ? f16_bits_to_f32(h) : bf16_bits_to_f32(h);
}

// Float order as unsigned order, zeros of both signs as one, shifted so that -infinity is 0:
// what stands for an expert that cannot be chosen. +infinity is kTop, a NaN of either sign above it.
constexpr uint32_t kNone = 0u, kLow = 0x007FFFFFu, kTop = 0xFF800000u - kLow;
QM_DEV uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u)) - kLow;
}
QM_DEV float unordered(uint32_t k) {
    k += kLow;
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 1 / (1 + exp(-x)) for a weight: expf is within 2 units and the sum and quotient
// within half a unit each, so it is off by at most 2^-22 of itself.
QM_DEV float sigmoid_weight(float x) {
    const float t = expf(-fabsf(x));
    return __fdiv_rn(x < 0.0f ? t : 1.0f, 1.0f + t);
}

// Where this lane's experts lie: expert i is base + (i << lanes_log2), for i < count.
struct Place {
    int group, base, count;
    QM_DEV Place(const Select& a, int lane) {
        const int lanes = 1 << a.lanes_log2, sub = lane & (lanes - 1);
        group = lane >> a.lanes_log2;
        base = group * a.gsize + sub;
        count = group < a.groups && sub < a.gsize ? ((a.gsize - 1 - sub) >> a.lanes_log2) + 1 : 0;
    }
};

// The choice by float64 keys: lane r receives the r-th chosen expert (-1: none).
template <int V>
static __device__ __noinline__ int select_exact(const Select& a, int64_t t, int lane) {
    const Place at(a, lane);
    double key[V], score[V];
    double top = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const float l = i < at.count ? load_logit(a, t, at.base + (i << a.lanes_log2)) : -INFINITY;
        score[i] = l > -INFINITY ? l : -INFINITY;  // NaN
        top = fmax(top, score[i]);
    }
    if (a.sigmoid) {
#pragma unroll 1
        for (int i = 0; i < V; ++i) score[i] = score[i] > -INFINITY ? 1.0 / (1.0 + exp(-score[i])) : -INFINITY;
    } else {  // softmax rows that come here are finite or -infinity
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
        double sum = 0.0;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            const bool live = score[i] > -INFINITY;
            score[i] = live ? exp(score[i] - top) : -INFINITY;
            sum += live ? score[i] : 0.0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
#pragma unroll 1
        for (int i = 0; i < V; ++i) score[i] /= sum;
    }
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        key[i] = score[i];
        if (a.bias && i < at.count) {
            const float b = __ldg(a.bias + at.base + (i << a.lanes_log2));
            key[i] = score[i] > -INFINITY && b > -INFINITY ? score[i] + b : -INFINITY;
        }
    }
    if (a.groups > 1) {
        double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            m2 = fmax(m2, fmin(m1, key[i]));
            m1 = fmax(m1, key[i]);
        }
        for (int o = 1; o < (1 << a.lanes_log2); o <<= 1) {
            const double p1 = __shfl_xor_sync(kFull, m1, o), p2 = __shfl_xor_sync(kFull, m2, o);
            m2 = fmax(fmin(m1, p1), fmax(m2, p2));
            m1 = fmax(m1, p1);
        }
        const double mine = a.top2 ? (m2 > -INFINITY ? m1 + m2 : -INFINITY) : m1;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl_sync(kFull, mine, g << a.lanes_log2);
            rank += other > mine || (other == mine && g < at.group);
        }
        if (rank >= a.topk_groups) {
#pragma unroll 1
            for (int i = 0; i < V; ++i) key[i] = -INFINITY;
        }
    }
    // without a bias the logits order the experts, as in the float32 path
    int got = -1;
    uint64_t taken = 0u;  // of this lane's experts
    for (int r = 0; r < a.topk; ++r) {
        double best = -INFINITY;
        int idx = 0x7FFFFFFF, slot = 0;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            if (!(key[i] > -INFINITY) || ((taken >> i) & 1u)) continue;
            const int e = at.base + (i << a.lanes_log2);
            const double k = a.bias ? key[i] : static_cast<double>(load_logit(a, t, e));
            if (idx == 0x7FFFFFFF || k > best) {
                best = k;
                idx = e;
                slot = i;
            }
        }
        const int own = idx;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(kFull, best, o);
            const int oi = __shfl_xor_sync(kFull, idx, o);
            if (oi != 0x7FFFFFFF && (idx == 0x7FFFFFFF || ob > best || (ob == best && oi < idx))) {
                best = ob;
                idx = oi;
            }
        }
        if (idx == 0x7FFFFFFF) break;  // none left, for every lane
        if (idx == own) taken |= uint64_t(1) << slot;
        if (lane == r) got = idx;
    }
    return got;
}

// Scores for the order alone. exp2 of the scaled argument is off by 2^-22 and 2^-23 for each
// unit of the argument (softmax: and 2^-24, the difference's rounding), the reciprocal and the
// sum below it by 2^-22.4. z exp(-z) stays below 0.37, so of a score, at most 1, the error is
// below 2^-20; softmax adds up to 37 roundings of its sum, below 2^-18 in all. Results below 2^-126 are 0.
QM_DEV float exp_fast(float v) {
    float t;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(v * 1.44269504f));
    return t;
}
QM_DEV float sigmoid_score(float l) {
    const float t = exp_fast(-fabsf(l));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    return l < 0.0f ? t * r : r;
}
QM_DEV float score_of(const Select& a, float l, float top, float inv_sum) {
    return a.sigmoid ? sigmoid_score(l) : exp_fast(l - top) * inv_sum;
}
QM_DEV float most_error(const Select& a) { return a.sigmoid ? 0x1p-20f : 0x1p-17f; }

// The key of expert e with logit l, as an ordered integer.
QM_DEV uint32_t key_of(const Select& a, float l, int e, float top, float inv_sum) {
    float k = l;
    if (a.bias) k = l > -INFINITY ? score_of(a, l, top, inv_sum) + __ldg(a.bias + e) : -INFINITY;
    const uint32_t key = ordered(k);
    return key <= kTop ? key : kNone;  // NaN
}

// Keys nearer than this may change places: both errors, the sums' roundings, and as much again.
QM_DEV float key_margin(const Select& a, float k) { return 4.0f * most_error(a) + 0x1p-21f * fabsf(k); }

// The choice among many equal or nearly equal keys, one after another (`stays`: this lane's group
// does): lane r receives the r-th chosen expert (-1: none). Sets *near where float32 cannot tell the order.
template <int V>
static __device__ __noinline__ int select_ties(const Select& a, int64_t t, int lane, bool stays, float top, float inv_sum, bool* near) {
    const Place at(a, lane);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = at.base + (i << a.lanes_log2);
        key[i] = stays && i < at.count ? key_of(a, load_logit(a, t, e), e, top, inv_sum) : kNone;
    }
    int idx = -1;
    uint32_t picked = kNone;
    const int picks = a.topk + (a.bias ? 1 : 0);
    for (int r = 0; r < picks; ++r) {
        uint32_t mk = kNone;
        int mi = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > mk) {
                mk = key[i];
                mi = i;
            }
        const uint32_t best = __reduce_max_sync(kFull, mk);
        if (best == kNone) break;
        const int mine = mk == best ? at.base + (mi << a.lanes_log2) : 0x7FFFFFFF;
        const int low = __reduce_min_sync(kFull, mine);
        if (mine == low) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == mi) key[i] = kNone;
        }
        if (lane == r) {
            idx = low;
            picked = best;
        }
    }
    *near = false;
    if (a.bias) {
        const uint32_t next = __shfl_down_sync(kFull, picked, 1);
        const int next_idx = __shfl_down_sync(kFull, idx, 1);
        bool close = false;
        if (lane < a.topk && idx >= 0 && next_idx >= 0) {
            const float x = unordered(picked), y = unordered(next);
            if (!(x - y > key_margin(a, x)))
                close = load_logit(a, t, idx) != load_logit(a, t, next_idx) || __ldg(a.bias + idx) != __ldg(a.bias + next_idx);
        }
        *near = __any_sync(kFull, close);
    }
    return lane < a.topk ? idx : -1;
}

// Float64 order as signed order, zeros of both signs as one: float64 arithmetic has 1/64 of float32's
// rate here, its comparisons too.
QM_DEV int64_t ordered64(double v) {
    const int64_t u = __double_as_longlong(v);
    return u < 0 ? static_cast<int64_t>(0x8000000000000000ull) - u : u;
}
QM_DEV double unordered64(int64_t k) {
    return __longlong_as_double(k < 0 ? static_cast<int64_t>(0x8000000000000000ull) - k : k);
}
constexpr int64_t kNone64 = static_cast<int64_t>(0x8000000000000001ull);  // below -infinity

// A key whose order counts, from a logit and its bias: of softmax without a bias up to a factor.
static __device__ __noinline__ double key_exact(const Select& a, float l, float b, float top) {
    return (a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : exp(static_cast<double>(l) - static_cast<double>(top))) + b;
}

// A warp's list of candidates: key above, complement of the expert's index below, so that
// the greater entry goes first. 0: none.
QM_DEV uint64_t entry_of(uint32_t key, int e) { return (static_cast<uint64_t>(key) << 32) | ~static_cast<uint32_t>(e); }
QM_DEV int expert_of(uint64_t entry) { return static_cast<int>(~static_cast<uint32_t>(entry)); }

// Every lane's keys from `from` on, side by side in the list; returns how many (more than 32:
// the list is not whole). Its first 32 entries are otherwise 0.
template <int V>
QM_DEV int gather(const Select& a, const uint32_t (&key)[V], uint32_t from, int base, uint64_t* list) {
    const int lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u;
    list[lane] = 0u;
    __syncwarp();
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = key[i] >= from;
        const uint32_t who = __ballot_sync(kFull, in);
        const int at = n + __popc(who & before);
        if (in && at < 32) list[at] = entry_of(key[i], base + (i << a.lanes_log2));
        n += __popc(who);
    }
    __syncwarp();
    return n;
}

// Two largest keys over a group's lanes.
QM_DEV void join_top2(const Select& a, uint32_t& m1, uint32_t& m2) {
#pragma unroll 1
    for (int o = 1; o < (1 << a.lanes_log2); o <<= 1) {
        const uint32_t p1 = __shfl_xor_sync(kFull, m1, o), p2 = __shfl_xor_sync(kFull, m2, o);
        m2 = max(min(m1, p1), max(m2, p2));
        m1 = max(m1, p1);
    }
}

// Two largest keys of a lane's group: its own experts', then over the group's lanes.
template <int V>
QM_DEV void group_top2(const Select& a, const uint32_t (&key)[V], uint32_t& m1, uint32_t& m2) {
    m1 = m2 = kNone;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
    }
    join_top2(a, m1, m2);
}

// A group's score from its two largest keys (-infinity: kNone), and a bound on its error:
// of a sum of scores that no bias joins relative to them and up to a factor that all share.
QM_DEV uint32_t group_score(const Select& a, uint32_t m1, uint32_t m2, float top, float inv_sum, float* err) {
    *err = a.bias ? most_error(a) : 0.0f;
    if (!a.top2) return m1;
    if (m2 == kNone) return kNone;
    const float k1 = unordered(m1), k2 = unordered(m2);
    if (a.bias) {
        *err = 2.0f * most_error(a);
        return ordered(k1 + k2);
    }
    const float s1 = score_of(a, k1, top, inv_sum), s2 = score_of(a, k2, top, inv_sum);
    const float z1 = fabsf(a.sigmoid ? k1 : k1 - top), z2 = fabsf(a.sigmoid ? k2 : k2 - top);
    *err = s1 * fmaf(z1, 0x1p-22f, 0x1p-20f) + s2 * fmaf(z2, 0x1p-22f, 0x1p-20f) + 0x1p-124f;
    return ordered(s1 + s2);
}

// Whether this lane's group stays, where scores about the border lie nearer than float32 can tell:
// the groups within `tol` of the last that stayed, x, and the first that did not, y, are ranked
// anew by float64 keys. One above x + tol is passed only by groups that stay as well, one below
// y - tol by any that stays. Sets *all where more than that is to be done in float64.
// What a rare call waits for is its instructions: it takes the keys as they are (a copy of this
// lane's), and its loops are not unrolled.
template <int V>
static __device__ __noinline__ bool regroup(const Select& a, int64_t t, int lane, const uint32_t* key, uint32_t mine, uint32_t m1, uint32_t m2,
                                            float top, float x, float y, float tol, uint64_t* list, int64_t* exact, bool* all) {
    const Place at(a, lane);
    const float m = unordered(mine);
    const bool real = at.group < a.groups && mine != kNone;
    const bool above = real && m > x + tol, band = real && !above && !(m < y - tol);
    // the elements that may be a group's largest: within both errors of the last of them
    const uint32_t cut = a.top2 ? m2 : m1;
    const float cv = unordered(cut);
    const uint32_t from = !band || cut == kNone ? 0xFFFFFFFFu : (a.bias ? max(ordered(cv - key_margin(a, cv)), 1u) : cut);
    list[lane] = 0u;
    __syncwarp();
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const bool in = i < at.count && key[i] >= from;
        const uint32_t who = __ballot_sync(kFull, in);
        const int place = n + __popc(who & ((1u << lane) - 1u));
        if (in && place < 32) list[place] = entry_of(key[i], at.base + (i << a.lanes_log2));
        n += __popc(who);
    }
    __syncwarp();
    *all = n > 32 || (a.bias && !a.sigmoid) || !(fabsf(x) < INFINITY);
    if (*all) return false;
    if (lane < n) {
        const int e = expert_of(list[lane]);
        exact[lane] = ordered64(key_exact(a, load_logit(a, t, e), a.bias ? __ldg(a.bias + e) : 0.0f, top));
    }
    __syncwarp();
    int64_t e1 = kNone64, e2 = kNone64;
    const int first = at.group * a.gsize;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int e = expert_of(list[j]) - first;
        if (e < 0 || e >= a.gsize) continue;
        e2 = max(e2, min(e1, exact[j]));
        e1 = max(e1, exact[j]);
    }
    const int64_t score = a.top2 && band ? ordered64(unordered64(e1) + unordered64(e2)) : e1;
    const uint32_t in_band = __ballot_sync(kFull, band), over = __ballot_sync(kFull, above);
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
        const int leader = g << a.lanes_log2;
        const int64_t other = __shfl_sync(kFull, score, leader);
        if ((over >> leader) & 1u) ++rank;
        else if ((in_band >> leader) & 1u) rank += other > score || (other == score && g < at.group);
    }
    __syncwarp();  // the list is written again
    return above || (band && rank < a.topk_groups);
}

// HALF: 16-bit logits.
template <int V, bool GROUPS, bool HALF>
__global__ void __launch_bounds__(kSelectWarps * 32, V <= 8 ? 8 : 1) select_kernel(const __grid_constant__ Select a) {
    __shared__ uint64_t s_list[kSelectWarps][32];
    __shared__ int64_t s_exact[kSelectWarps][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    uint64_t* list = s_list[threadIdx.x >> 5];
    const int64_t nw = static_cast<int64_t>(gridDim.x) * kSelectWarps;
    const Place at(a, lane);
    const int step = GROUPS ? a.lanes_log2 : 5;
    const bool keyed = a.bias != nullptr;          // keys are sums, else the logits themselves
    const bool softmax_sum = !a.sigmoid && (keyed || !a.renormalize);
    const int picks = a.topk + (keyed ? 1 : 0);    // with inexact keys one more: the first not chosen
    float bias[V];
    if (keyed) {
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = i < at.count ? __ldg(a.bias + at.base + (i << step)) : 0.0f;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kSelectWarps + (threadIdx.x >> 5); t < a.T; t += nw) {
        uint32_t key[V];
        uint32_t mk = kNone;  // the largest of this lane's keys
        float top = 0.0f, inv_sum = 1.0f;
        {
            float l[V];
            if constexpr (HALF) {
                const uint16_t* row = static_cast<const uint16_t*>(a.logits) + t * a.stride + at.base;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t h = i < at.count ? __ldca(row + (i << step)) : 0u;
                    l[i] = a.dtype == QM_F16 ? f16_bits_to_f32(h) : bf16_bits_to_f32(h);
                    if (i >= at.count) l[i] = -INFINITY;
                }
            } else {
                const float* row = static_cast<const float*>(a.logits) + t * a.stride + at.base;
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = i < at.count ? __ldca(row + (i << step)) : -INFINITY;
            }
            if (!(keyed && a.sigmoid)) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    key[i] = ordered(l[i]);
                    mk = max(mk, key[i]);
                }
            }
            if (!a.sigmoid) {
                const uint32_t best = __reduce_max_sync(kFull, mk);
                if (best >= kTop) {  // NaN or +infinity: no softmax
                    if (lane < a.topk) {
                        a.ids[t * a.topk + lane] = -1;
                        a.weights[t * a.topk + lane] = __uint_as_float(0x7FC00000u);
                    }
                    continue;
                }
                top = unordered(best);
                if (softmax_sum) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += key[i] != kNone ? expf(l[i] - top) : 0.0f;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                    inv_sum = 1.0f / sum;
                }
            }
            if (keyed) {
                mk = kNone;
                if (a.sigmoid) {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = ordered(l[i] > -INFINITY ? sigmoid_score(l[i]) + bias[i] : -INFINITY);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = ordered(l[i] > -INFINITY ? exp_fast(l[i] - top) * inv_sum + bias[i] : -INFINITY);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) mk = max(mk, key[i]);
            }
            if (mk > kTop) {  // a NaN is never chosen
                mk = kNone;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (key[i] > kTop) key[i] = kNone;
                    mk = max(mk, key[i]);
                }
            }
        }
        bool exact_all = false;  // for select_exact
        bool stays = true;       // this lane's group
        if (GROUPS) {
            uint32_t m1, m2;
            group_top2<V>(a, key, m1, m2);
            float err;
            const uint32_t mine = group_score(a, m1, m2, top, inv_sum, &err);
            // how many groups go before this one: its lanes look at a share of them each
            const int lanes = 1 << a.lanes_log2;
            int rank = 0;
            for (int g0 = 0; g0 < a.groups; g0 += lanes) {
                const int g = g0 + (lane & (lanes - 1));
                const uint32_t other = __shfl_sync(kFull, mine, (g << a.lanes_log2) & 31);
                rank += g < a.groups && (other > mine || (other == mine && g < at.group));
            }
            for (int o = 1; o < lanes; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
            const bool real = at.group < a.groups;
            stays = real && rank < a.topk_groups;
            if (keyed || a.top2) {
                const uint32_t low = __reduce_min_sync(kFull, stays ? mine : 0xFFFFFFFFu);
                const uint32_t high = __reduce_max_sync(kFull, real && !stays ? mine : kNone);
                if (low != kNone && high != kNone) {  // the last group that stays, the first that does not
                    const float x = unordered(low), y = unordered(high);
                    if (!keyed) err = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(real ? err : 0.0f)));
                    else err = a.top2 ? 2.0f * most_error(a) : most_error(a);
                    // both errors, the sums' roundings, and as much again
                    const float tol = 4.0f * err + 0x1p-21f * (fabsf(x) + fabsf(y));
                    if (!(x - y > tol)) {
                        uint32_t copy[V];
                        bool all;
#pragma unroll
                        for (int i = 0; i < V; ++i) copy[i] = key[i];
                        stays = regroup<V>(a, t, lane, copy, mine, m1, m2, top, x, y, tol, list, s_exact[threadIdx.x >> 5], &all);
                        exact_all = all;
                    }
                }
            }
            if (!stays) mk = kNone;
        }
        // Candidates: every key from the topk-th largest of the lanes' own largest on (with inexact keys the
        // next, and a margin), no fewer than are chosen and seldom many more. A lane each.
        int n = 0, expert = -1, rank = 32;  // this lane's candidate and its place
        if (!exact_all) {
            uint32_t from = kNone;
            for (int r = 0; r < picks; ++r) {
                from = __reduce_max_sync(kFull, mk);
                if (mk == from) mk = kNone;
            }
            if (from == kNone) {
                from = 1u;  // all there are
            } else if (keyed) {
                const float f = unordered(from);
                from = fabsf(f) < INFINITY ? max(ordered(f - key_margin(a, f)), 1u) : 1u;
            }
            n = gather<V>(a, key, stays ? from : 0xFFFFFFFFu, at.base, list);
            if (n > 32) {  // as many equal or nearly equal keys
                bool near;
                expert = select_ties<V>(a, t, lane, stays, top, inv_sum, &near);
                exact_all = near;
                rank = expert >= 0 ? lane : 32;
                n = __popc(__ballot_sync(kFull, expert >= 0));
            } else {
                const uint64_t own = list[lane];
                rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) rank += list[j] > own;
                if (lane < n) expert = expert_of(own);
                else rank = 32;
                if (keyed) {
                    const float kf = unordered(static_cast<uint32_t>(own >> 32)), tol = key_margin(a, kf);
                    __syncwarp();
                    if (lane < n) list[rank] = own;  // in order now; beyond n still 0
                    __syncwarp();
                    const uint32_t k0 = static_cast<uint32_t>(list[lane] >> 32), k1 = lane + 1 < n ? static_cast<uint32_t>(list[lane + 1] >> 32) : kNone;
                    // neighbours nearer than their errors
                    bool close = lane < a.topk && k1 != kNone && !(unordered(k0) - unordered(k1) > key_margin(a, unordered(k0)));
                    if (__any_sync(kFull, close)) {
                        const float l = lane < n ? load_logit(a, t, expert) : 0.0f, b = lane < n ? __ldg(a.bias + expert) : 0.0f;
                        close = false;  // but not the same sum of the same two
#pragma unroll 1
                        for (int j = 0; j < n; ++j) {
                            const float lj = __shfl_sync(kFull, l, j), bj = __shfl_sync(kFull, b, j);
                            const float kj = __shfl_sync(kFull, kf, j);
                            close = close || (!(fabsf(kf - kj) > tol) && (lj != l || bj != b));
                        }
                        if (__any_sync(kFull, close && rank < a.topk)) {
                            if (!a.sigmoid) {
                                exact_all = true;
                            } else {
                                int64_t* exact = s_exact[threadIdx.x >> 5];
                                const int64_t mine = ordered64(key_exact(a, l, b, top));
                                exact[lane] = mine;
                                __syncwarp();
                                rank = 0;
#pragma unroll 1
                                for (int j = 0; j < n; ++j) {
                                    const int ej = __shfl_sync(kFull, expert, j);
                                    rank += exact[j] > mine || (exact[j] == mine && ej < expert);
                                }
                                if (lane >= n) rank = 32;
                            }
                        }
                    }
                }
            }
            __syncwarp();  // the list is written again
        }
        if (exact_all) {  // lane r holds the r-th
            expert = select_exact<V>(a, t, lane);
            rank = expert >= 0 ? lane : 32;
            n = __popc(__ballot_sync(kFull, expert >= 0));
        }
        const bool on = rank < a.topk;
        const float l = on ? load_logit(a, t, expert) : -INFINITY;
        float w = 0.0f;
        if (a.renormalize) {
            // scores over their sum, all of them times exp(-high) where that is below zero: no score of
            // very negative logits is lost
            const float high = unordered(__reduce_max_sync(kFull, ordered(l)));
            const float shift = a.sigmoid ? fminf(high, 0.0f) : high;
            if (on) {
                if (!a.sigmoid) w = expf(l - shift);
                else w = l <= 0.0f ? __fdividef(expf(l - shift), 1.0f + expf(l)) : sigmoid_weight(l);
            }
            float all = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
            if (on) w = __fdividef(w, all);  // all is in [1/2, 31]
        } else if (on) {
            w = a.sigmoid ? sigmoid_weight(l) : expf(l - top) * inv_sum;
        }
        if (on) {
            a.ids[t * a.topk + rank] = expert;
            a.weights[t * a.topk + rank] = w * a.scale;
        }
        if (lane >= n && lane < a.topk) {  // fewer than topk to choose from
            a.ids[t * a.topk + lane] = -1;
            a.weights[t * a.topk + lane] = 0.0f;
        }
    }
}

template <int V, bool GROUPS>
cudaError_t launch_select(const Select& a, cudaStream_t st) {
    // twice as many blocks as stay resident: a warp reads the bias once for a token or two, and what
    // one of them waits for (float64) the rest is not dealt out to wait behind (8 an SM 24.1, 16 23.8, 32 25.5 us)
    const int64_t blocks = std::min<int64_t>((a.T + kSelectWarps - 1) / kSelectWarps, int64_t(num_sms()) * 16);
    return launch_pdl(a.dtype == QM_F32 ? select_kernel<V, GROUPS, false> : select_kernel<V, GROUPS, true>, static_cast<unsigned>(blocks),
                      kSelectWarps * 32, 0, st, a);
}

cudaError_t by_width(const Select& a, int width, cudaStream_t st) {
    if (a.groups > 1) {
        if (width <= 4) return launch_select<4, true>(a, st);
        if (width <= 8) return launch_select<8, true>(a, st);
        if (width <= 16) return launch_select<16, true>(a, st);
        if (width <= 32) return launch_select<32, true>(a, st);
        return launch_select<64, true>(a, st);  // 1024 experts in 2^i + 1 .. groups: fewer than twice 32 to a lane
    }
    if (width <= 4) return launch_select<4, false>(a, st);
    if (width <= 8) return launch_select<8, false>(a, st);
    if (width <= 16) return launch_select<16, false>(a, st);
    return launch_select<32, false>(a, st);
}

}  // namespace

cudaError_t launch_experts_select(const qm_router& r, const void* logits, int dtype, int64_t stride, int64_t T, int32_t* ids,
                                  float* weights, cudaStream_t st) {
    Select a{};
    a.logits = logits;
    a.stride = stride;
    a.bias = r.bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.dtype = dtype;
    // all groups stay: the same choice as from one
    a.groups = r.topk_groups < r.groups ? r.groups : 1;
    a.topk_groups = a.groups > 1 ? r.topk_groups : 1;
    a.gsize = r.experts / a.groups;
    a.top2 = r.group_score == QM_GROUP_TOP2;
    a.topk = r.topk;
    a.sigmoid = r.score == QM_SCORE_SIGMOID;
    a.renormalize = r.renormalize;
    a.scale = r.scale;
    int g2 = 0;
    while ((1 << g2) < a.groups) ++g2;
    a.lanes_log2 = 5 - g2;
    const int width = ((a.gsize - 1) >> a.lanes_log2) + 1;  // logits that a lane holds
    return by_width(a, width, st);
}

// ---------------------------------------------------------------- the sum over a token's experts
namespace {

struct Combine {
    const uint16_t* y;
    const float* weights;
    const uint16_t* residual;
    uint16_t* out;
    int64_t residual_stride, n, T;
    int topk;
};

QM_DEV void add8(float (&s)[8], uint4 v, float w) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), s[2 * i]);
        s[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xFFFF0000u), s[2 * i + 1]);
    }
}

QM_DEV uint32_t pair_bf16(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// Up to eight elements at an even address, as loaded: a first one where the address is odd in
// words, then words (a half where only their first element is live). Packed later, so that
// several rows' loads are under way at once.
struct Loose {
    uint32_t first, word[4];
};
QM_DEV Loose load_loose(const uint16_t* p, int live) {
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
    Loose r;
    r.first = odd && live > 0 ? __ldca(p) : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 2 * k + odd;
        r.word[k] = 0u;
        if (e + 1 < live) r.word[k] = __ldca(reinterpret_cast<const uint32_t*>(p + e));
        else if (e < live) r.word[k] = __ldca(p + e);
    }
    return r;
}
QM_DEV uint4 packed(const Loose& r, const uint16_t* p) {
    if (!(reinterpret_cast<uintptr_t>(p) & 2)) return make_uint4(r.word[0], r.word[1], r.word[2], r.word[3]);
    return make_uint4(r.first | r.word[0] << 16, __funnelshift_r(r.word[0], r.word[1], 16), __funnelshift_r(r.word[1], r.word[2], 16),
                      __funnelshift_r(r.word[2], r.word[3], 16));
}
QM_DEV void store_loose(uint16_t* p, const uint32_t (&v)[4], int live) {
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
    if (odd) p[0] = static_cast<uint16_t>(v[0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 2 * k + odd;
        const uint32_t w = odd ? __funnelshift_r(v[k], k < 3 ? v[k + 1] : 0u, 16) : v[k];
        if (e + 1 < live) *reinterpret_cast<uint32_t*>(p + e) = w;
        else if (e < live) p[e] = static_cast<uint16_t>(w);
    }
}

// VEC: n a multiple of 8, so that every row of y and out is in 16-byte pieces, and the residual's too; else rows begin at
// any even address, and a row's last piece may be short (n = 1001: 43 us an element at a time, 4096
// tokens x 8 rows; now 25). ROWS of them are asked for before the first is used; the blocks to an SM leave
// the registers for that (8 rows of 2880: 34 us with 6 blocks, 36 with 8, 44 and more without a bound).
template <bool VEC, int ROWS>
__global__ void __launch_bounds__(128, VEC && ROWS == 2 ? 12 : VEC && ROWS == 8 ? 6 : 8) combine_kernel(const __grid_constant__ Combine a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t per = (a.n + 7) / 8, total = a.T * per, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = total <= 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per)) : i / per;
        const int64_t c = (i - t * per) * 8;
        const int live = VEC ? 8 : static_cast<int>(min(static_cast<int64_t>(8), a.n - c));
        const uint16_t* yr = a.y + t * a.topk * a.n + c;
        const float* wr = a.weights + t * a.topk;
        const uint16_t* rr = a.residual + t * a.residual_stride + c;
        float s[8] = {};
        uint4 res = make_uint4(0u, 0u, 0u, 0u);
        Loose loose_res{};
        if (a.residual) {
            if constexpr (VEC) res = __ldca(reinterpret_cast<const uint4*>(rr));
            else loose_res = load_loose(rr, live);
        }
        for (int j = 0; j < a.topk; j += ROWS) {
            uint4 v[ROWS];
            Loose r[ROWS];
            float w[ROWS];
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                const bool on = j + q < a.topk;
                if constexpr (VEC) v[q] = on ? __ldcs(reinterpret_cast<const uint4*>(yr + (j + q) * a.n)) : make_uint4(0u, 0u, 0u, 0u);
                else r[q] = load_loose(yr + (j + q) * a.n, on ? live : 0);
                w[q] = on ? __ldg(wr + j + q) : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                if constexpr (!VEC) v[q] = packed(r[q], yr + (j + q) * a.n);
                add8(s, v[q], w[q]);
            }
        }
        if (a.residual) {
            if constexpr (!VEC) res = packed(loose_res, rr);
            add8(s, res, 1.0f);
        }
        const uint32_t o[4] = {pair_bf16(s[0], s[1]), pair_bf16(s[2], s[3]), pair_bf16(s[4], s[5]), pair_bf16(s[6], s[7])};
        uint16_t* out = a.out + t * a.n + c;
        if constexpr (VEC) *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
        else store_loose(out, o, live);
    }
}

}  // namespace

cudaError_t launch_experts_combine(const void* y, const float* weights, int64_t T, int64_t topk, int64_t n, const void* residual,
                                   int64_t residual_stride, void* out, cudaStream_t st) {
    Combine a{static_cast<const uint16_t*>(y), weights, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
              residual_stride, n, T, static_cast<int>(topk)};
    const bool vec = n % 8 == 0 && (!residual || (aligned16(residual) && residual_stride % 8 == 0));
    const int64_t items = T * ((n + 7) / 8);
    const int64_t blocks = std::min<int64_t>((items + 127) / 128, int64_t(1) << 22);
    return launch_pdl(!vec ? combine_kernel<false, 4>
                           : topk > 4 ? combine_kernel<true, 8>
                           : topk > 2 ? combine_kernel<true, 4>
                                      : combine_kernel<true, 2>,
                      static_cast<unsigned>(blocks), 128, 0, st, a);
}

}  // namespace qm
