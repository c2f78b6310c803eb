// qm_router.cu -- the choice of each token's experts from its router logits
// (select_kernel) and the weighted sum of what those experts gave
// (combine_kernel).
//
// Choice. Keys are s + bias, s = softmax(l) or sigmoid(l); without a bias the order
// of the logits is the order of the keys, and they are compared as they are. A
// warp takes a token and holds its logits in registers: 32 / G' lanes to a group (G'
// the groups rounded up to a power of two), a group's experts dealt to its lanes in
// turn. Group scores then meet by shuffles within a group's lanes, each
// group's rank is counted over all of them, and the topk largest keys are taken one after
// another: a warp maximum over order-preserving integers, the lowest index where
// several lanes hold it.
//
// Keys that are sums or exponentials carry float32 roundings, and two of them may
// lie closer than those. Neighbours in the order (and group scores about the border)
// nearer than a bound on their errors, unless their logit and bias are the same, send the
// token to select_exact, which orders it anew by float64 keys.
//
// Sum. Eight columns of one token to a thread, the rows of its experts loaded
// together before the first is used.
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

// Float order as unsigned order; 0 is below every number. Zeros of both signs meet.
QM_DEV uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
QM_DEV float unordered(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

constexpr uint32_t kNone = 0u;

// 1 / (1 + exp(-x)): expf is within 2 units and the sum and quotient within half a
// unit each, so it is off by at most 2^-22 of itself.
QM_DEV float sigmoid_key(float x) {
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

template <int V, bool GROUPS>
__global__ void __launch_bounds__(kSelectWarps * 32) select_kernel(const __grid_constant__ Select a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t nw = static_cast<int64_t>(gridDim.x) * kSelectWarps;
    const Place at(a, lane);
    const bool keyed = a.bias != nullptr;          // keys are sums, else the logits themselves
    const bool softmax_sum = !a.sigmoid && (keyed || !a.renormalize || (GROUPS && a.top2));
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kSelectWarps + (threadIdx.x >> 5); t < a.T; t += nw) {
        float l[V];
        uint32_t key[V];
        bool bad = false;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = i < at.count ? load_logit(a, t, at.base + (i << a.lanes_log2)) : -INFINITY;
            bad = bad || l[i] != l[i] || l[i] == INFINITY;
            top = fmaxf(top, l[i]);
        }
        if (!a.sigmoid && __any_sync(kFull, bad)) {  // no softmax
            if (lane < a.topk) {
                a.ids[t * a.topk + lane] = -1;
                a.weights[t * a.topk + lane] = __uint_as_float(0x7FC00000u);
            }
            continue;
        }
        float sum = 1.0f;
        if (softmax_sum) {
            top = unordered(__reduce_max_sync(kFull, ordered(top)));
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        }
        // A score's error, relative to it: sigmoid 2^-22; softmax 2^-17 (2^-22 for the exponential, up to
        // 104 * 2^-24 for its argument, 37 * 2^-24 for the sum). Of a score, at most 1, it is no more
        // than 2^-18, since s log(1 / s) < 1/2. A key adds half a unit of its sum with the bias.
        const float rel = a.sigmoid ? 0x1p-22f : 0x1p-17f, most_err = a.sigmoid ? 0x1p-22f : 0x1p-18f;
        auto score = [&](float v) { return a.sigmoid ? sigmoid_key(v) : expf(v - top) / sum; };
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float k = l[i];
            if (keyed && i < at.count) {
                const float b = __ldg(a.bias + at.base + (i << a.lanes_log2));
                k = l[i] > -INFINITY && b > -INFINITY ? score(l[i]) + b : -INFINITY;
            }
            key[i] = k > -INFINITY ? ordered(k) : kNone;
        }
        bool near = false;  // an order that float32 cannot tell
        if (GROUPS) {
            uint32_t m1 = kNone, m2 = kNone;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                m2 = max(m2, min(m1, key[i]));
                m1 = max(m1, key[i]);
            }
            for (int o = 1; o < (1 << a.lanes_log2); o <<= 1) {
                const uint32_t p1 = __shfl_xor_sync(kFull, m1, o), p2 = __shfl_xor_sync(kFull, m2, o);
                m2 = max(min(m1, p1), max(m2, p2));
                m1 = max(m1, p1);
            }
            uint32_t mine = m1;
            if (a.top2) {
                if (m2 == kNone) mine = kNone;
                else if (keyed) mine = ordered(unordered(m1) + unordered(m2));
                else mine = ordered(score(unordered(m1)) + score(unordered(m2)));
            }
            int rank = 0;
            for (int g = 0; g < a.groups; ++g) {
                const uint32_t other = __shfl_sync(kFull, mine, g << a.lanes_log2);
                rank += other > mine || (other == mine && g < at.group);
            }
            const bool real = at.group < a.groups, stays = rank < a.topk_groups;
            if (keyed || a.top2) {
                const uint32_t least = __reduce_min_sync(kFull, real && stays ? mine : 0xffffffffu);
                const uint32_t most = __reduce_max_sync(kFull, real && !stays ? mine : kNone);
                if (least != kNone && most != kNone) {
                    const float x = unordered(least), y = unordered(most);
                    // two keys' errors and their sum's rounding on either side, and as much again
                    near = !(x - y > (keyed ? 8.0f * most_err : 4.0f * rel * (x + y)) + 0x1p-21f * (fabsf(x) + fabsf(y)));
                }
            }
            if (!stays) {
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = kNone;
            }
        }
        // the largest keys one after another; with inexact keys one more, the first that is not chosen
        int idx = -1;
        uint32_t picked = kNone;
        if (!near) {
            uint32_t mk = kNone;
            int mi = 0;
            auto local_best = [&]() {
                mk = kNone;
                mi = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] > mk) {
                        mk = key[i];
                        mi = i;
                    }
            };
            local_best();
            const int picks = a.topk + (keyed ? 1 : 0);
            for (int r = 0; r < picks; ++r) {
                const uint32_t best = __reduce_max_sync(kFull, mk);
                if (best == kNone) break;
                const int mine = at.base + (mi << a.lanes_log2);
                uint32_t who = __ballot_sync(kFull, mk == best);
                if (who & (who - 1)) {  // several lanes: the lowest index
                    const int low = __reduce_min_sync(kFull, mk == best ? mine : 0x7FFFFFFF);
                    who = __ballot_sync(kFull, mk == best && mine == low);
                }
                const int src = __ffs(who) - 1;
                const int e = __shfl_sync(kFull, mine, src);
                if (lane == r) {
                    idx = e;
                    picked = best;
                }
                if (lane == src) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i == mi) key[i] = kNone;
                    local_best();
                }
            }
            if (keyed) {
                // neighbours of the order nearer than their errors, but not the same sum of the same two
                const uint32_t next = __shfl_down_sync(kFull, picked, 1);
                const int next_idx = __shfl_down_sync(kFull, idx, 1);
                bool close = false;
                if (lane < a.topk && idx >= 0 && next_idx >= 0) {
                    const float x = unordered(picked), y = unordered(next);
                    const float bx = __ldg(a.bias + idx), by = __ldg(a.bias + next_idx);
                    // both errors, and as much again
                    if (!(x - y > 2.0f * rel * (fabsf(x - bx) + fabsf(y - by)) + 0x1p-22f * (fabsf(x) + fabsf(y))))
                        close = load_logit(a, t, idx) != load_logit(a, t, next_idx) || bx != by;
                }
                near = __any_sync(kFull, close);
            }
        }
        if (near) idx = select_exact<V>(a, t, lane);
        // weights, from the chosen logits anew
        const bool on = lane < a.topk && idx >= 0;
        const float x = on ? load_logit(a, t, idx) : -INFINITY;
        float w = 0.0f;
        if (a.renormalize) {
            // scores over their sum, all of them times exp(-high) where that is below zero: no score of
            // very negative logits is lost
            const float high = unordered(__reduce_max_sync(kFull, ordered(x)));
            const float shift = a.sigmoid ? fminf(high, 0.0f) : high;
            if (on) {
                if (!a.sigmoid) w = expf(x - shift);
                else w = x <= 0.0f ? expf(x - shift) / (1.0f + expf(x)) : sigmoid_key(x);
            }
            float all = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
            if (on) w = w / all;
        } else if (on) {
            w = a.sigmoid ? sigmoid_key(x) : expf(x - top) / sum;
        }
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = on ? idx : -1;
            a.weights[t * a.topk + lane] = w * a.scale;
        }
    }
}

template <int V, bool GROUPS>
cudaError_t launch_select(const Select& a, cudaStream_t st) {
    const int64_t blocks = std::min<int64_t>((a.T + kSelectWarps - 1) / kSelectWarps, int64_t(num_sms()) * 16);
    return launch_pdl(select_kernel<V, GROUPS>, static_cast<unsigned>(blocks), kSelectWarps * 32, 0, st, a);
}

template <bool GROUPS>
cudaError_t by_width(const Select& a, int width, cudaStream_t st) {
    if (width <= 1) return launch_select<1, GROUPS>(a, st);
    if (width <= 2) return launch_select<2, GROUPS>(a, st);
    if (width <= 4) return launch_select<4, GROUPS>(a, st);
    if (width <= 8) return launch_select<8, GROUPS>(a, st);
    if (width <= 16) return launch_select<16, GROUPS>(a, st);
    if (width <= 32) return launch_select<32, GROUPS>(a, st);
    return launch_select<64, GROUPS>(a, st);  // 1024 experts in 2^i + 1 .. groups: fewer than twice 32 to a lane
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
    return a.groups > 1 ? by_width<true>(a, width, st) : by_width<false>(a, width, st);
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
    int vec_residual;  // residual rows in 16-byte pieces
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

// VEC: n a multiple of 8, so that every row of y and out is in 16-byte pieces.
template <bool VEC>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Combine a) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int W = VEC ? 8 : 1;
    const int64_t per = a.n / W, total = a.T * per, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = total <= 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per)) : i / per;
        const int64_t c = (i - t * per) * W;
        const uint16_t* yr = a.y + t * a.topk * a.n + c;
        const float* wr = a.weights + t * a.topk;
        if constexpr (VEC) {
            float s[8] = {};
            uint4 res = make_uint4(0u, 0u, 0u, 0u);
            if (a.residual && a.vec_residual) {
                res = __ldca(reinterpret_cast<const uint4*>(a.residual + t * a.residual_stride + c));
            } else if (a.residual) {
                const uint16_t* r = a.residual + t * a.residual_stride + c;
                uint32_t u[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) u[q] = static_cast<uint32_t>(__ldca(r + 2 * q)) | (static_cast<uint32_t>(__ldca(r + 2 * q + 1)) << 16);
                res = make_uint4(u[0], u[1], u[2], u[3]);
            }
            for (int j = 0; j < a.topk; j += 4) {
                uint4 v[4];
                float w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool live = j + q < a.topk;
                    v[q] = live ? __ldg(reinterpret_cast<const uint4*>(yr + (j + q) * a.n)) : make_uint4(0u, 0u, 0u, 0u);
                    w[q] = live ? __ldg(wr + j + q) : 0.0f;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) add8(s, v[q], w[q]);
            }
            add8(s, res, 1.0f);
            *reinterpret_cast<uint4*>(a.out + t * a.n + c) =
                make_uint4(pair_bf16(s[0], s[1]), pair_bf16(s[2], s[3]), pair_bf16(s[4], s[5]), pair_bf16(s[6], s[7]));
        } else {
            float s = 0.0f;
            for (int j = 0; j < a.topk; ++j) s = fmaf(__ldg(wr + j), bf16_bits_to_f32(__ldg(yr + j * a.n)), s);
            if (a.residual) s += bf16_bits_to_f32(__ldca(a.residual + t * a.residual_stride + c));
            a.out[t * a.n + c] = bf16_bits(s);
        }
    }
}

}  // namespace

cudaError_t launch_experts_combine(const void* y, const float* weights, int64_t T, int64_t topk, int64_t n, const void* residual,
                                   int64_t residual_stride, void* out, cudaStream_t st) {
    Combine a{static_cast<const uint16_t*>(y), weights, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
              residual_stride, n, T, static_cast<int>(topk), 0};
    a.vec_residual = aligned16(residual) && residual_stride % 8 == 0;
    const bool vec = n % 8 == 0;
    const int64_t items = T * (vec ? n / 8 : n);
    const int64_t blocks = std::min<int64_t>((items + 127) / 128, int64_t(num_sms()) * 16);
    return launch_pdl(vec ? combine_kernel<true> : combine_kernel<false>, static_cast<unsigned>(blocks), 128, 0, st, a);
}

}  // namespace qm
