// qm_attend_tc.cu -- attention of new tokens over a paged cache for many rows to
// a key head (attend_tiles_kernel: chunks of prompts), on the 5th-generation
// tensor cores.
//
// The mathematics is qm_attend.cu's: one pass over the keys with the running
// maximum and total of every row in float32. An item is 256 rows, two tiles of 128,
// over the same keys; a unit of 128 keys costs each tile two products, S = Q K^T and
// O += P V, of 128 x 128 x dim. What bounds it is those products as long as the
// exponentials (one for every element of S) fit beside them, so the two tiles take
// turns: while one tile's weights are formed, the tensor cores work on the other's.
// One CTA per SM, three warpgroups:
//  * warpgroups 0 and 1, one tile each, one row a thread: S from tensor memory to
//    registers, weights P = 2^(t - ref) rounded to 16 bits back over it. ref follows
//    the running maximum lazily: only when it has grown by kSlack (a factor of 2^8
//    or 2^4) is O rescaled, which is exact in float32 whenever it happens; weights stay
//    below 2^8 (bfloat16) or 2^12 (float16, lifted by 2^8: all bits down to 2^-22 of the
//    row's largest, none past 2^-33).
//  * warp 8: issues the products: Q and K from shared memory (128-byte swizzle, K
//    major), P from tensor memory, V from shared memory as it lies in the cache
//    (rows of keys: MN major); S and O of both tiles fill the 512 tensor-memory columns.
//  * warps 9..11: fill a ring of 32 KB slots (a unit's keys, then its values), each
//    row's place looked up in the page table, a unit ahead. Where pages are multiples of 32
//    tokens that is one TMA box for each page and 64 elements, by lanes of warp 9; the
//    units with a length's ragged end, and other page sizes, are 16-byte asynchronous
//    copies of all three warps, zeros where there is nothing. Copies arrive on the
//    slot's barrier as they land, so the loaders only issue; the issuer of the products
//    orders them before its reads with a proxy fence. 8-bit codes pass through the
//    loaders' registers on the way and enter the products exactly.
// Every wait is bounded; a wait that gives up raises the device flag and the CTA
// winds down with its copies and products drained.
// Measured (16 / 8 heads of 128): chunk of 4096 over 32768 706 us, 1460 TFLOP/s, 0.77 of the
// products' rate in a burst (757 to 767 us after a second of nothing else, when power holds the clock at
// some 1700 MHz: 0.79 of the sustained rate); of 4096 over 16384 364 us in pages of 64, 373 in pages of 16 or 20. A unit takes
// 3300 clocks, 2048 of them products: a tile's scores wait 1700 for their weights, then
// those 1500 for the products and the next scores, and the tiles' turns hide most but not all of it.
// Over 8-bit codes 1168 us (4096 over 16384): the scales, broadcast from shared memory to every row,
// and the products share its bandwidth.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qm_attend.cuh"

namespace qm {
namespace attend {
namespace {

__device__ uint32_t g_err_attend = 0;

constexpr int kRows = kTileRows;
constexpr int kThreads = 384;
constexpr int kLoaders = 3;  // warps

// Shared memory: Q (two tiles of 128 rows x DP), the ring, scales of 8-bit codes,
// barriers.
template <int DP, bool I8>
struct Lay {
    static constexpr int kPanel = 128 * 128;           // 128 rows of 64 16-bit elements
    static constexpr int kTile = kPanel * (DP / 64);   // 128 rows of a head
    static constexpr int kQ = 2 * kTile;
    static constexpr int kSlots = I8 ? 4 : DP == 128 ? 5 : 8;
    static constexpr int kScale = kQ + kSlots * kTile;  // [2][3][128] floats: key scales, value scales, their logarithms
    static constexpr int kFar = kScale + 2 * 3 * 512;   // [2] ints: a value scale is out of float16's reach
    static constexpr int kBars = kScale + (I8 ? 2 * 3 * 512 + 16 : 0);
    static constexpr int kCursors = kBars + 256;       // of the warps that form weights: they are out of registers
    static constexpr int kSmem = kCursors + 8 * 96;
};

QM_DEV bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

// Descriptors of operands in shared memory, 128-byte swizzled, 8-row groups 1024
// bytes apart: their constant high words, and the low words at an address. The
// issuer adds steps to low words alone: it has some 60 clocks for each product.
// Keys and queries (rows of 64 elements of the product's K) ...
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
QM_DEV uint32_t desc_k_major(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | 1u << 16; }
// ... and values as they lie: rows of keys (the product's K), 64 elements (its N) to a
// row, panels of 64 elements `panel` bytes apart.
QM_DEV uint32_t desc_rows_of_k(uint32_t addr, uint32_t panel) { return ((addr >> 4) & 0x3FFFu) | (panel >> 4) << 16; }

QM_DEV void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 da, db;\n"
        "mov.b64 da, {%1, %5};\n"
        "mov.b64 db, {%2, %5};\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
        "}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "n"(kDescHigh)
        : "memory");
}
QM_DEV void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 db;\n"
        "mov.b64 db, {%2, %5};\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n"
        "}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "n"(kDescHigh)
        : "memory");
}

// Instruction descriptor, kind::f16, f32 sums, 128 x N; B K-major or (mn) MN-major.
QM_DEV uint32_t idesc16(bool bf16, int N, bool mn) {
    const uint32_t f = bf16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

QM_DEV void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

QM_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

QM_DEV void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr) : "memory");
}

// Where 16-byte piece c of row r lies in a tile.
template <int DP>
QM_DEV uint32_t at16(int r, int c) {
    return (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Four lanes with pieces 0..3 of a row each: afterwards lane l of the quad has piece
// l of the rows of lanes 0..3.
QM_DEV void quad_transpose(uint32_t (&w)[4][8]) {
    const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b0 ? w[p][e] : w[p + 1][e], 1);
            (b0 ? w[p][e] : w[p + 1][e]) = got;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? w[p][e] : w[p + 2][e], 2);
            (b1 ? w[p][e] : w[p + 2][e]) = got;
        }
    }
}

// O[row] += P[row] V over the unit's keys that the row sees, product by product:
// for a unit in which rows see different keys and a value is infinite or NaN (0
// times it would be NaN in rows that do not see it). p: the row's weights in tensor memory
// (16-bit pairs; WIDE: float32), o: its sums, zeros instead if `fresh`; keys [a, b] are seen.
template <int DP, bool BF16, bool WIDE>
__device__ __noinline__ void exact_values(uint32_t p, uint32_t o, bool fresh, uint32_t v, int a, int b) {
#pragma unroll 1
    for (int c = 0; c < DP / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(o + 32 * c, r);
        tmem_wait_ld();
        float acc[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = fresh ? 0.f : __uint_as_float(r[i]);
#pragma unroll 1
        for (int kb = 0; kb < 8; ++kb) {
            uint32_t w[WIDE ? 16 : 8];
            if constexpr (WIDE) tmem_ld16(p + 16 * kb, w);
            else tmem_ld8(p + 8 * kb, w);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int key = 16 * kb + k;
                float pk;
                if constexpr (WIDE) {
                    pk = __uint_as_float(w[k]);
                } else {
                    const uint32_t h = (k & 1) ? w[k / 2] >> 16 : w[k / 2] & 0xFFFFu;
                    pk = BF16 ? __uint_as_float(h << 16) : f16_bits_to_f32(h);
                }
                const bool see = key >= a && key <= b;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 x = lds_v4(v + at16<DP>(key, 4 * c + q));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v0 = BF16 ? __uint_as_float(xs[e] << 16) : f16_bits_to_f32(xs[e] & 0xFFFFu);
                        const float v1 = BF16 ? __uint_as_float(xs[e] & 0xFFFF0000u) : f16_bits_to_f32(xs[e] >> 16);
                        if (see) {
                            acc[8 * q + 2 * e] = fmaf(pk, v0, acc[8 * q + 2 * e]);
                            acc[8 * q + 2 * e + 1] = fmaf(pk, v1, acc[8 * q + 2 * e + 1]);
                        }
                    }
                }
            }
        }
        uint32_t lo[16], hi[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = __float_as_uint(acc[i]);
            hi[i] = __float_as_uint(acc[16 + i]);
        }
        tmem_st16(o + 32 * c, lo);
        tmem_st16(o + 32 * c + 16, hi);
        tmem_wait_st();
    }
}

// A unit of codes with a far value scale: the row's scores in tensor memory become its weights in float32,
// which meet the values the same way. sc: the unit's key scales, value scales and their logarithms; keys [a, b]
// are seen. From and to the row's reference and total.
template <int DP>
__device__ __noinline__ float2 far_unit(uint32_t p, uint32_t o, bool fresh, uint32_t v, const float* sc, int a, int b, float ref, float total) {
    const auto score = [&](int key, uint32_t raw) { return key >= a && key <= b ? __uint_as_float(raw) * sc[key] : -INFINITY; };
    float top = -INFINITY;
#pragma unroll 1
    for (int kb = 0; kb < 8; ++kb) {
        uint32_t w[16];
        tmem_ld16(p + 16 * kb, w);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, score(16 * kb + k, w[k]) + sc[256 + 16 * kb + k]);
    }
    const float old = ref;
    ref = fminf(fmaxf(ref, top - 8.f), FLT_MAX);  // the lift of float16 weights
    const float base = reference(ref), f = ex2(old - base);
    total *= f;
#pragma unroll 1
    for (int c = 0; c < DP / 16 && !fresh; ++c) {
        uint32_t r[16];
        tmem_ld16(o + 16 * c, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
        tmem_st16(o + 16 * c, r);
    }
#pragma unroll 1
    for (int kb = 0; kb < 8; ++kb) {
        uint32_t w[16];
        tmem_ld16(p + 16 * kb, w);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int key = 16 * kb + k;
            const float x = ex2(score(key, w[k]) - base);
            total += x;
            w[k] = key >= a && key <= b ? __float_as_uint(x * sc[128 + key]) : 0u;
        }
        tmem_st16(p + 16 * kb, w);
    }
    tmem_wait_st();
    exact_values<DP, false, true>(p, o, fresh, v, a, b);
    return make_float2(ref, total);
}

struct TileArgs {
    CUtensorMap tk, tv;  // keys and values [pages][heads][page_size][dim], boxes of 64 elements x box_rows tokens
    CUtensorMap tq;      // queries [1][tokens][heads][dim], boxes of 64 elements x group heads x 128 / group tokens
    Args a;
    int box_rows;  // 0: no tensor maps of the cache
    int q_boxes;   // the queries' map is there
};

template <int DP, bool BF16, bool I8>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const __grid_constant__ TileArgs ta) {
    const Args& a = ta.a;
    using L = Lay<DP, I8>;
    constexpr int NS = L::kSlots;
    constexpr bool PBF = BF16 && !I8;  // type of the weights and values in their product
    constexpr float kLift = PBF ? 0.f : 8.f, kSlack = PBF ? 8.f : 4.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sq = smem_u32(smem), ring = sq + L::kQ, b0 = sq + L::kBars;
    auto kv_full = [&](int i) { return b0 + 8 * i; };
    auto kv_free = [&](int i) { return b0 + 8 * (NS + i); };
    const uint32_t q_free = b0 + 8 * (2 * NS), done = q_free + 8;
    auto s_full = [&](int t) { return q_free + 16 + 8 * t; };
    auto p_full = [&](int t) { return q_free + 32 + 8 * t; };
    auto o_full = [&](int t) { return q_free + 48 + 8 * t; };
    auto agreed = [&](int t) { return q_free + 64 + 8 * t; };
    const uint32_t q_full = q_free + 80;
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kBars + 8 * (2 * NS) + 88);
    uint32_t* tmem_slot = words;
    volatile uint32_t* skip = words + 1;  // [2]: the tile's values were added without the tensor cores
    uint32_t* odd_word = words + 3;       // [3][2]: a warp of the tile saw a value that is infinite or NaN

    grid_launch_dependents();
    grid_dependency_wait();
    // What the workspace held is no descriptor: one that is never published, by an empty run or one
    // that a wait made give up, reads as a run without parts.
    if (threadIdx.x < 2) a.desc[blockIdx.x * kDesc + threadIdx.x] = 0;
    // the run's start, its end, the barriers and the tensor memory, a warp each
    struct Run {
        Cursor<kRows> start;
        int64_t from, to;
    };
    static_assert(sizeof(Run) <= 8 * 96, "run");
    Run* run = reinterpret_cast<Run*>(smem + L::kCursors);
    if (warp < 2) {
        // a split costs some 9 units of an item of one tile and 14 of one of two: 16 chunks of 512 88 -> 54 us against
        // splitting everywhere, 10 batches of 6 to 15 ragged chunks in a window of 2000 (16 / 4 heads of 96) 0.2 to 35 %
        // less, the largest 222 -> 192 (220 with 5 and 8 units). An item to each CTA, where
        // there are enough, keeps runs from holding the ends of two: those chunks, 140 items of up to 17 units, 78 -> 49 us,
        // 144 items of 9 to 11 units 60 -> 34.
        const Load work = measure<kRows>(a, gridDim.x);
        int64_t at;
        const bool each = item_each(work.items, work.most, work.total, work.runs, gridDim.x, 8);
        const Cursor<kRows> k = run_start<kRows>(a, work, blockIdx.x + (each ? 0 : warp), each, Split{9, 9}, Split{14, 14}, at);
        if (each) at = warp == 0 ? 0 : k.u1 - k.u;
        if (lane == 0) {
            if (warp == 0) {
                run->start = k;
                run->from = at;
            } else {
                run->to = at;
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(kv_full(i), 32 * kLoaders);
                mbar_init(kv_free(i), 1);
            }
            mbar_init(q_free, 1);
            mbar_init(q_full, 32 * kLoaders);
            mbar_init(done, 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(s_full(t), 1);
                mbar_init(p_full(t), 4);
                mbar_init(o_full(t), 1);
                mbar_init(agreed(t), 4);
                skip[t] = odd_word[t] = odd_word[2 + t] = odd_word[4 + t] = 0;
            }
            fence_mbar_init();
        }
    } else if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    Cursor<kRows> start = run->start;
    start.left = run->to - run->from;
    __syncthreads();  // the cursors of the warps that form weights lie there from here on
    const uint32_t tmem = *tmem_slot;
    if (start.left <= 0) {
        if (warp == 8) tmem_dealloc(tmem, 512);
        return;
    }
    auto give_up = [&]() { atomicOr(&g_err_attend, DEV_ERR_TIMEOUT); };
    // every wait is a whole warp's, and so is its verdict
    auto wait = [](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
    const int ksteps = (a.dim + 15) / 16;
    // units of the run's part that `now` is in
    auto part_units = [](const Cursor<kRows>& c) { return static_cast<int>(min(static_cast<int64_t>(c.u1 - c.u), c.left)); };
    auto skip_part = [&](Cursor<kRows>& c, int n) {
        c.left -= n;
        c.u += n;
        if (c.u == c.u1 && c.left > 0) c.next_item(a);
    };

    if (warp < 8) {
        // ------------------------------------------------------------ weights of one tile
        const int t = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
        int nth = 0, parts = 0, checks = 0;  // units, parts and value checks of this tile so far
        uint32_t index = 0;      // units of the CTA so far
        int first_part = kNoPart;
        bool ok = true;
        static_assert(sizeof(Cursor<kRows>) <= 96, "cursor");
        Cursor<kRows>* now = reinterpret_cast<Cursor<kRows>*>(smem + L::kCursors + 96 * warp);
        if (lane == 0) *now = start;
        __syncwarp();
        while (now->left > 0 && ok) {
            const int n = part_units(*now);
            // (what only the part's end needs is read again there: the units' loop has no register to spare)
            int kmin = 0, kmax = -1;
            if (128 * t + row < now->span.rows) {
                const int at = now->seq.len - now->seq.fresh + static_cast<int>(token_of(a, now->tile * kRows + 128 * t + row));
                kmin = first_seen(a, at);
                kmax = min(at, a.cap - 1);
            }
            float ref = -INFINITY, total = 0.f;
            if (128 * t < now->span.rows) {
                // keys that every row of the item sees lie within [all_lo, all_hi]
                const int all_hi = min(now->span.p0, a.cap - 1), all_lo = first_seen(a, now->span.p1);
                const bool differ = now->span.p0 != now->span.p1;
                int j = 0;
                while (true) {
                    for (; j < n; ++j, ++nth) {
                        const int key0 = (now->u + j) * kUnit;
                        const bool cut = key0 + kUnit - 1 > all_hi || key0 < all_lo;
                        const int sa = max(kmin - key0, 0), sb = min(kmax - key0, kUnit - 1);  // the unit's keys that the row sees
                        const uint32_t vi = 2 * (index + j) + 1;  // the values' slot
                        const int slot = vi % NS;
                        const float* sc = reinterpret_cast<const float*>(smem + L::kScale) + (I8 ? ((index + j) & 1) * 384 : 0);
                        // (only then is the unit's slot in turn: a tile that sat out an item runs ahead of the copies)
                        if (!wait(s_full(t), nth & 1)) { ok = false; break; }
                        bool odd = false;
                        if constexpr (!I8) {
                            // 0 times an infinity or NaN is NaN: where rows see different keys, a look at the
                            // unit's values (each thread at one key's) tells whether the tensor cores may add them
                            if (cut && differ) {
                                if (!wait(kv_full(slot), (vi / NS) & 1)) { ok = false; break; }
                                const uint32_t v = ring + slot * L::kTile;
                                uint32_t high = 0;
#pragma unroll
                                for (int c = 0; c < DP / 8; ++c)
                                    if (c < 2 * ksteps) high = top_exponents<BF16>(high, lds_v4(v + at16<DP>(row, c)));
                                uint32_t* word = odd_word + 2 * (checks % 3) + t;
                                // the next check's word, which every warp read two checks ago
                                if (row == 0) odd_word[2 * ((checks + 1) % 3) + t] = 0;
                                if (nonfinite<BF16>(high)) atomicOr(word, 1u);
                                __syncwarp();
                                if (lane == 0) mbar_arrive(agreed(t));
                                if (!wait(agreed(t), checks & 1)) { ok = false; break; }
                                odd = *reinterpret_cast<volatile uint32_t*>(word) != 0;
                                ++checks;
                            }
                        }
                        if (I8 && !wait(kv_full(slot), (vi / NS) & 1)) { ok = false; break; }
                        tc_fence_after();
                        if (I8 && *reinterpret_cast<const volatile int*>(smem + L::kFar + 4 * ((index + j) & 1))) break;  // see below
                        uint32_t raw[4][32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, raw[c]);
                        tmem_wait_ld();
                        float s[128];
#pragma unroll
                        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(raw[i / 32][i % 32]);
                        if constexpr (I8) {
#pragma unroll
                            for (int i = 0; i < 128; i += 4) {
                                const float4 k = *reinterpret_cast<const float4*>(sc + i);
                                s[i] *= k.x; s[i + 1] *= k.y; s[i + 2] *= k.z; s[i + 3] *= k.w;
                            }
                        }
                        if (cut) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {  // where the warp's rows all see 32 keys, nothing is compared
                                if (__any_sync(0xffffffffu, sb < 32 * c + 31)) {
#pragma unroll
                                    for (int i = 32 * c; i < 32 * c + 32; ++i) s[i] = i <= sb ? s[i] : -INFINITY;
                                }
                                if (__any_sync(0xffffffffu, sa > 32 * c)) {
#pragma unroll
                                    for (int i = 32 * c; i < 32 * c + 32; ++i) s[i] = i >= sa ? s[i] : -INFINITY;
                                }
                            }
                        }
                        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        if constexpr (I8) {
#pragma unroll
                            for (int i = 0; i < 128; i += 4) {
                                const float4 lv = *reinterpret_cast<const float4*>(sc + 256 + i);
                                m[0] = fmaxf(m[0], s[i] + lv.x);
                                m[1] = fmaxf(m[1], s[i + 1] + lv.y);
                                m[2] = fmaxf(m[2], s[i + 2] + lv.z);
                                m[3] = fmaxf(m[3], s[i + 3] + lv.w);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 128; i += 8) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) m[e] = max3(m[e], s[i + e], s[i + 4 + e]);
                            }
                        }
                        // scores of 8-bit codes are in powers of two already (their key scales hold the factor)
                        const float top = max3(max3(m[0], m[1], m[2]), m[3], m[3]) * (I8 ? 1.f : a.scale2) - kLift;
                        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
                            const float old = ref;
                            ref = fminf(fmaxf(ref, top), FLT_MAX);
                            const float f = ex2(old - (ref == -INFINITY ? 0.f : ref));
                            total *= f;
                            if (j > 0) {
#pragma unroll 1
                                for (int c = 0; c < DP / 16; ++c) {
                                    uint32_t r[16];
                                    tmem_ld16(to + 16 * c, r);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                                    tmem_st16(to + 16 * c, r);
                                }
                            }
                        }
                        const float base = ref == -INFINITY ? 0.f : ref;
                        const float2 sc2 = I8 ? make_float2(1.f, 1.f) : make_float2(a.scale2, a.scale2), nb = make_float2(-base, -base);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int k = 32 * c + 2 * i;
                                const float2 x = fma2(make_float2(s[k], s[k + 1]), sc2, nb);
                                float2 p = make_float2(ex2(x.x), ex2(x.y));
                                sum[i & 1] = add2(sum[i & 1], p);
                                if constexpr (I8) {
                                    p = mul2(p, *reinterpret_cast<const float2*>(sc + 128 + k));
                                    if (cut) {  // a scale that the row does not see may be infinite or NaN
                                        if (k < sa || k > sb) p.x = 0.f;
                                        if (k + 1 < sa || k + 1 > sb) p.y = 0.f;
                                    }
                                }
                                w[i] = pack16<PBF>(p.x, p.y);
                            }
                            tmem_st16(ts + 16 * c, w);
                        }
                        total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                        tmem_wait_st();
                        if constexpr (!I8) {
                            if (odd) exact_values<DP, BF16, false>(ts, to, j == 0, ring + slot * L::kTile, sa, sb);
                        }
                        if (row == 0) skip[t] = odd ? 1u : 0u;
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_full(t));
                    }
                    if (!I8 || !ok || j == n) break;
                    // a unit with a far value scale, out of the loop's way (within it, 1146 us of a chunk of 4096 over 16384
                    // became 1220; so 1168)
                    const int key0 = (now->u + j) * kUnit;
                    const float* sc = reinterpret_cast<const float*>(smem + L::kScale) + ((index + j) & 1) * 384;
                    const float2 at = far_unit<DP>(ts, to, j == 0, ring + (2 * (index + j) + 1) % NS * L::kTile, sc, max(kmin - key0, 0),
                                                   min(kmax - key0, kUnit - 1), ref, total);
                    ref = at.x;
                    total = at.y;
                    if (row == 0) skip[t] = 1u;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(t));
                    ++j;
                    ++nth;
                }
                // ---- the part's end
                const bool starts = now->first(), done_here = starts && now->u + n == now->u1;
                const int rows = now->span.rows;
                const unsigned R = now->tile * kRows + 128 * t + row;
                const bool mine = 128 * t + row < rows;
                const int pos = now->seq.len - now->seq.fresh + static_cast<int>(token_of(a, R));
                if (ok && !wait(o_full(t), parts & 1)) ok = false;
                ++parts;
                tc_fence_after();
                const int part = 2 * blockIdx.x + (starts ? 1 : 0);
                uint16_t* y = nullptr;
                int64_t lse_at = 0;
                float inv = 1.f;
                if (mine && done_here) {
                    y = out_row(a, now->seq.first, now->h, R, lse_at);
                    inv = inverse_total(a, pos, total);
                }
                // A warp's rows lie apart in memory: quads of lanes exchange pieces of 32 bytes so
                // that each store of a quad is 128 bytes of one row (row by row from its own
                // lane, an item's 64 KB took some 8000 clocks of the SM's memory path).
                const int l4 = lane & 3;
                uint16_t* yrow[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    yrow[k] = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(y), (lane & ~3) + k));
                if (done_here) {
#pragma unroll 1
                    for (int c = 0; c < DP / 64; ++c) {
                        uint32_t w[4][8];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[32];
                            tmem_ld32(to + 64 * c + 32 * h, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[2 * h + (e >> 3)][e & 7] = pack16<BF16>(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
                        }
                        quad_transpose(w);
                        const int col = 64 * c + 16 * l4;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (!yrow[k] || !ok) continue;
                            uint16_t* to16 = yrow[k] + col;
                            if (col + 16 <= a.dim && (reinterpret_cast<uintptr_t>(to16) & 31) == 0) {
                                st_global_32(to16, w[k]);
                            } else {
                                if (col < a.dim) *reinterpret_cast<uint4*>(to16) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                                if (col + 8 < a.dim) *reinterpret_cast<uint4*>(to16 + 8) = make_uint4(w[k][4], w[k][5], w[k][6], w[k][7]);
                            }
                        }
                    }
                } else {
                    float* po = a.part + (static_cast<int64_t>(part) * kRows + 128 * t + 32 * (warp & 3) + (lane & ~3)) * DP + 8 * l4;
                    const int left = rows - (128 * t + 32 * (warp & 3) + (lane & ~3));  // of the quad's rows, those that are
#pragma unroll 1
                    for (int c = 0; c < DP / 32; ++c) {
                        uint32_t r[32], w[4][8];
                        tmem_ld32(to + 32 * c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e >> 3][e & 7] = r[e];
                        quad_transpose(w);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < left && ok) st_global_32(po + k * DP + 32 * c, w[k]);
                    }
                }
                tc_fence_before();  // the next part's products come after these reads
                if (mine && ok) {
                    if (done_here) {
                        if (a.lse) a.lse[lse_at] = log_total(ref, total);
                    } else {
                        a.ml[part * kRows + 128 * t + row] = make_float2(ref, total);
                    }
                }
            }
            const bool starts = now->first(), ends = now->u + n == now->u1;
            if (!starts) first_part = ends ? kLast : kInner;
            if (threadIdx.x == 0 && now->left == n && ok) {  // the run's last part
                int* desc = a.desc + blockIdx.x * kDesc;
                desc[0] = first_part;
                if (starts && !ends) {
                    desc[1] = 1;
                    desc[2] = now->seq.first;
                    desc[3] = now->h;
                    desc[4] = static_cast<int>(now->tile * kRows);
                    desc[5] = now->span.rows;
                    desc[6] = now->seq.len - now->seq.fresh;
                }
            }
            index += n;
            Cursor<kRows> then = *now;
            skip_part(then, n);
            __syncwarp();
            if (lane == 0) *now = then;
            __syncwarp();
        }
        if (!ok) give_up();
    } else if (warp == 8) {
        // ------------------------------------------------------------ products
        const uint32_t id_s = idesc16(BF16, 128, false), id_o = idesc16(PBF, 16 * ksteps, true);
        uint32_t i = 0;  // slots so far
        int nth[2] = {0, 0}, parts = 0;
        bool ok = true;
        auto wait_slot = [&](uint32_t k) { return wait(kv_full(k % NS), (k / NS) & 1); };
        auto scores = [&](int t, uint32_t k) {  // S of tile t over the keys in slot k
            if (elect_one()) {
                const uint32_t qd = desc_k_major(sq + t * L::kTile), kd = desc_k_major(ring + (k % NS) * L::kTile);
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
                    if (kk < ksteps) {
                        const uint32_t off = ((kk >> 2) * L::kPanel + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + 128 * t, qd + off, kd + off, id_s, kk > 0);
                    }
                umma_commit(s_full(t));
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t bar) {
            if (elect_one()) umma_commit(bar);
            __syncwarp();
        };
        Cursor<kRows> now = start;
        while (now.left > 0 && ok) {
            const int n = part_units(now);
            const int tiles = now.span.rows > 128 ? 2 : 1;
            if (!(ok = wait(q_full, parts & 1) && wait_slot(i))) break;
            ++parts;
            fence_proxy_async_smem();
            tc_fence_after();
            for (int t = 0; t < tiles; ++t) scores(t, i);
            commit(kv_free(i % NS));
            if (n == 1) commit(q_free);
            for (int j = 0; j < n && ok; ++j) {
                for (int t = 0; t < tiles; ++t) {
                    if (!(ok = wait(p_full(t), nth[t] & 1))) break;
                    ++nth[t];
                    if (t == 0 && !(ok = wait_slot(i + 1))) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    if (!skip[t] && elect_one()) {
                        const uint32_t vd = desc_rows_of_k(ring + ((i + 1) % NS) * L::kTile, L::kPanel);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * kk, vd + ((kk * 2048) >> 4), id_o, j > 0 || kk > 0);
                    }
                    __syncwarp();
                    if (t == tiles - 1) commit(kv_free((i + 1) % NS));
                    if (j == n - 1) {
                        commit(o_full(t));
                    } else {
                        if (t == 0 && !(ok = wait_slot(i + 2))) break;
                        fence_proxy_async_smem();
                        tc_fence_after();
                        scores(t, i + 2);
                    }
                }
                if (!ok) break;
                if (j < n - 1) {
                    commit(kv_free((i + 2) % NS));
                    if (j == n - 2) commit(q_free);
                }
                i += 2;
            }
            skip_part(now, n);
        }
        if (!ok) give_up();
        commit(done);  // drains whatever was issued
        (void)mbar_wait(done, 0);
    } else {
        // ------------------------------------------------------------ copies
        const int lw = warp - 9;
        constexpr int C = DP / 8;           // 16-byte pieces of a 16-bit row
        const int pieces = 2 * ksteps;      // of which the products read these
        uint32_t i = 0;                     // slots so far
        int parts = 0;
        bool ok = true;
        auto landed = [&](uint32_t bar) {  // arrives when this thread's copies so far have landed
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        };
        auto take_slot = [&]() {  // waits until slot i is free
            return i < NS || wait(kv_free(i % NS), ((i / NS) & 1) ^ 1u);
        };
        Cursor<kRows> now = start;
        // A warp copies `per` rows at once, the same rows of each quarter of 32 of a
        // slot; their places, each found by one lane, are passed round once for a
        // unit's keys and values, and the shared-memory addresses stay the same.
        constexpr int CB = I8 ? DP / 16 : C;  // 16-byte pieces of a row as it lies in the cache
        constexpr int per = 32 / CB, turns = (32 / per + kLoaders - 1) / kLoaders;
        const int pc = lane % CB;
        uint32_t place[4], off[4][turns];  // of row 32 x + lane; of the rows that the lane copies
        int64_t splace[4];
        Lookup found[4];  // rows 32 x + lane of the next unit
        int head = 0;
        bool all_there = false;
        // With tensor maps a unit is some boxes of box_rows tokens of one page each, one a
        // lane: pages that are not there, and boxes outside the keys to be read, lie at
        // page `pages`, which reads as zeros. A unit with a box partly outside is copied
        // row by row.
        const int box_rows = ta.box_rows, boxes = box_rows ? kUnit / box_rows * (DP / 64) : 0;
        const int box_i = DP == 128 ? lane >> 1 : lane, box_x = DP == 128 ? (lane & 1) * 64 : 0;
        const uint32_t box_dst = static_cast<uint32_t>((DP == 128 ? (lane & 1) * L::kPanel : 0) + box_i * box_rows * 128);
        bool next_boxed = false, boxed = false;
        Lookup box_at = {0, 0};
        int box_head = 0;
        auto look = [&](const Cursor<kRows>& c) {
            head = c.h;
            const int k0 = c.u * kUnit, k1 = k0 + (kUnit - 1);
            next_boxed = box_rows && c.span.hi > c.span.lo && (k1 < c.span.hi || c.span.hi % box_rows == 0) &&
                         (k0 >= c.span.lo || c.span.lo % box_rows == 0);
            if (next_boxed) {
                found[0] = begin_lookup(a, c.s, k0 + box_i * box_rows, c.span.lo, c.span.hi);
                return;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) found[x] = begin_lookup(a, c.s, c.u * kUnit + 32 * x + lane, c.span.lo, c.span.hi);
        };
        auto pass_round = [&]() {
            boxed = next_boxed;
            if (boxed) {
                box_at = found[0];
                if (box_at.row < 0 || static_cast<unsigned>(box_at.id) >= static_cast<unsigned>(a.pages)) box_at = Lookup{a.pages, 0};
                box_head = head;
                return;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) place[x] = finish_lookup<I8>(a, found[x], head, splace[x]);
            all_there = __all_sync(0xffffffffu, place[0] != kNoRow && place[1] != kNoRow && place[2] != kNoRow && place[3] != kNoRow);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < turns; ++y) {
                    off[x][y] = __shfl_sync(0xffffffffu, place[x], ((lw + kLoaders * y) * per + lane / CB) & 31);
                    if ((I8 ? 16 : 8) * pc >= a.dim) off[x][y] = kNoRow;
                }
        };
        uint32_t dst16[turns];  // where the lane's piece of its row in turn y of a quarter lies in a tile
#pragma unroll
        for (int y = 0; y < turns; ++y) dst16[y] = at16<DP>(((lw + kLoaders * y) * per + lane / CB) & 31, I8 ? 2 * pc : pc);
        const bool full_rows = C * 8 == a.dim;  // every piece of a row holds elements
        auto load_q = [&]() {
            if (ta.q_boxes) {  // a tile's rows are a box's: tokens, and within each the group's heads
                const int tiles = now.span.rows > 128 ? 2 : 1, per_tile = 128 / a.group;
                if (lw == 0) {
                    if (lane < tiles * (DP / 64)) {
                        const int t = DP == 128 ? lane >> 1 : lane, panel = DP == 128 ? lane & 1 : 0;
                        tma_load_4d(sq + t * L::kTile + panel * L::kPanel, &ta.tq, 64 * panel, now.h * a.group,
                                    now.seq.first + (2 * static_cast<int>(now.tile) + t) * per_tile, 0, q_full);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(q_full, tiles * L::kTile);
                }
                if (lane == 0) mbar_arrive_n(q_full, 32);
                return;
            }
            constexpr int qper = 32 / C;
            const int c = lane % C;
            const int tiles = now.span.rows > 128 ? 2 : 1;
            const int rows = now.span.rows;
            const uint16_t* base = a.q + now.seq.first * a.q_ts + now.h * a.group * a.q_hs + 8 * c;
#pragma unroll 8
            for (int r = lw * qper + lane / C; r < 128 * tiles; r += kLoaders * qper) {
                const unsigned R = now.tile * kRows + r, tok = token_of(a, R), g = R - tok * a.group;
                const bool on = r < rows && 8 * c < a.dim;
                if (c < pieces)
                    cp_async16(sq + (r >> 7) * L::kTile + at16<DP>(r & 127, c), base + static_cast<int64_t>(tok) * a.q_ts + static_cast<int64_t>(g) * a.q_hs, on, a.q);
            }
            landed(q_full);
        };
        Cursor<kRows> next = now;  // the unit that places are looked up for: one ahead of the copies
        auto look_on = [&]() {
            next.step(a);
            if (next.left > 0) look(next);
        };
        look(now);
        while (now.left > 0 && ok) {
            const int n = part_units(now);
            if (parts > 0) {
                if (!(ok = wait(q_free, (parts - 1) & 1))) break;
            }
            ++parts;
            load_q();
            for (int j = 0; j < n && ok; ++j) {
                pass_round();
                if constexpr (!I8) {
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        const int slot = i % NS;
                        if (!(ok = take_slot())) break;
                        const uint32_t dst = ring + slot * L::kTile;
                        const uint8_t* src = (v ? a.v : a.k) + 16 * pc;
                        if (boxed) {
                            if (lw == 0) {
                                if (lane < boxes)
                                    tma_load_4d(dst + box_dst, v ? &ta.tv : &ta.tk, box_x, box_at.row, box_head, box_at.id, kv_full(slot));
                                __syncwarp();
                                if (lane == 0) mbar_expect_tx(kv_full(slot), L::kTile);
                            }
                            // every loader arrives, so that none falls a whole turn of the ring behind
                            if (lane == 0) mbar_arrive_n(kv_full(slot), 32);
                            ++i;
                            if (v == 0) look_on();
                            continue;
                        }
                        if (all_there && full_rows) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
#pragma unroll
                                for (int y = 0; y < turns; ++y)
                                    if (lw + kLoaders * y < 32 / per)
                                        cp_async16(dst + dst16[y] + 32 * 128 * x, src + static_cast<uint64_t>(off[x][y]) * 16);
                        } else if (pc < pieces) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
#pragma unroll
                                for (int y = 0; y < turns; ++y)
                                    if (lw + kLoaders * y < 32 / per) {
                                        cp_async16(dst + dst16[y] + 32 * 128 * x, src + static_cast<uint64_t>(off[x][y]) * 16,
                                                   off[x][y] != kNoRow, a.q);
                                    }
                        }
                        landed(kv_full(slot));
                        ++i;
                        if (v == 0) look_on();
                    }
                } else {
                    // codes: through registers, as exact 16-bit values
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        const uint8_t* src = (v ? a.v : a.k) + 16 * pc;
                        uint4 w[4][turns];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int y = 0; y < turns; ++y) {
                                w[x][y] = make_uint4(0u, 0u, 0u, 0u);
                                if (lw + kLoaders * y < 32 / per && off[x][y] != kNoRow)
                                    w[x][y] = *reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(off[x][y]) * 16);
                            }
                        const int slot = i % NS;
                        if (!(ok = take_slot())) break;
                        uint8_t* dst = smem + L::kQ + slot * L::kTile;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int y = 0; y < turns; ++y) {
                                if (lw + kLoaders * y < 32 / per && 2 * pc < pieces) {
                                    const uint32_t ws[4] = {w[x][y].x, w[x][y].y, w[x][y].z, w[x][y].w};
                                    uint32_t o[8];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const uint32_t lo = prmt(ws[e], 0u, 0x4140), hi = prmt(ws[e], 0u, 0x4342);
                                        o[2 * e] = v ? codes16<false>(lo) : codes16<BF16>(lo);
                                        o[2 * e + 1] = v ? codes16<false>(hi) : codes16<BF16>(hi);
                                    }
                                    // pieces 2 pc and 2 pc + 1 of a swizzled row: the other of a pair of addresses
                                    *reinterpret_cast<uint4*>(dst + dst16[y] + 32 * 128 * x) = make_uint4(o[0], o[1], o[2], o[3]);
                                    *reinterpret_cast<uint4*>(dst + (dst16[y] ^ 16u) + 32 * 128 * x) = make_uint4(o[4], o[5], o[6], o[7]);
                                }
                            }
                        if (v == 1 && lw < 2) {  // a warp for the key scales, one for the values'
                            // the values two units back have been used, so their scales have been read
                            float* sc = reinterpret_cast<float*>(smem + L::kScale) + ((i >> 1) & 1) * 384;
                            const float* from = lw ? a.vs : a.ks;
                            float got[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) got[x] = place[x] != kNoRow ? __ldg(from + splace[x]) : 0.f;
                            if (lw == 0) {
#pragma unroll
                                for (int x = 0; x < 4; ++x) sc[32 * x + lane] = got[x] * a.scale2;
                            } else {
                                bool far = false;
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    sc[128 + 32 * x + lane] = got[x];
                                    sc[256 + 32 * x + lane] = scale_log2(got[x]);
                                    far |= far_scale(got[x]);
                                }
                                far = __any_sync(0xffffffffu, far);
                                if (lane == 0) reinterpret_cast<int*>(smem + L::kFar)[(i >> 1) & 1] = far;
                            }
                        }
                        mbar_arrive(kv_full(slot));
                        ++i;
                        if (v == 1) look_on();
                    }
                }
                if (!ok) break;
                now.step(a);
            }
        }
        cp_async_wait_all();
        if (lw == 0 && parts > 0) (void)mbar_wait(q_full, (parts - 1) & 1);
        if (lw == 0)  // boxes too have landed before the CTA ends, whoever gave up
            for (uint32_t k = i < NS ? 0 : i - NS; k < i; ++k) (void)mbar_wait(kv_full(k % NS), (k / NS) & 1);
        if (!ok) give_up();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP, bool BF16, bool I8>
cudaError_t run_tiles(const TileArgs& a, int runs, cudaStream_t st) {
    auto kern = attend_tiles_kernel<DP, BF16, I8>;
    constexpr int smem = Lay<DP, I8>::kSmem;
    static_assert(smem <= 227 * 1024 && 16 * Lay<DP, I8>::kSlots + 124 <= 256, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(runs), kThreads, smem, st, a);
}

// Tensor maps of the queries where a tile of 128 rows is whole tokens, and
// of a 16-bit cache whose pages are multiples of 32 tokens and whose heads have at least a
// box's 64 elements. Against the loaders' own copies, chunk of 4096 over 16384 (16 / 8 heads of 128):
// boxes of 16 rows, 2 KB, 475 us to 372; of 32 rows 379 to 371, but 125 to 147 for 2048 over 8192 with heads of 96,
// 48 to 51 for 16 x 512 and 287 to 292 for 8192 over itself; of 64 rows 362 to 372.
void make_maps(TileArgs& t, const qm_cache& c) {
    const Args& a = t.a;
    // the stride of an axis of one never counts, but has to be one that a map can have
    const auto stride = [](int64_t n, int64_t s) { return static_cast<uint64_t>(n > 1 ? 2 * s : 256); };
    if (a.dim >= 64 && 128 % a.group == 0 && (a.tokens == 1 || a.q_ts > 0) && (a.heads == 1 || a.q_hs > 0)) {
        const uint64_t qd[4] = {static_cast<uint64_t>(a.dim), static_cast<uint64_t>(a.heads), static_cast<uint64_t>(a.tokens), 1};
        const uint64_t qs[3] = {stride(a.heads, a.q_hs), stride(a.tokens, a.q_ts), 256};
        t.q_boxes = make_tmap_4d_16(&t.tq, a.q, qd, qs, 64, a.group, 128 / a.group);
    }
    if (c.dtype == QM_I8 || c.page_size % 32 != 0 || c.dim < 64 || c.pages < 1) return;
    int rows = kUnit;
    while (c.page_size % rows != 0) rows /= 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(c.dim), static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(c.heads),
                              static_cast<uint64_t>(c.pages)};
    const uint64_t strides[3] = {stride(c.page_size, c.token_stride), stride(c.heads, c.head_stride), stride(c.pages, c.page_stride)};
    if (make_tmap_4d_16(&t.tk, c.k, dims, strides, 64, rows) && make_tmap_4d_16(&t.tv, c.v, dims, strides, 64, rows)) t.box_rows = rows;
}

}  // namespace

cudaError_t launch_tiles(const Args& args, const qm_cache& c, int runs, bool bf16, cudaStream_t st) {
    TileArgs a = {};
    a.a = args;
    make_maps(a, c);
    const bool i8 = c.dtype == QM_I8;
    if (c.dim <= 64) {
        if (i8) return bf16 ? run_tiles<64, true, true>(a, runs, st) : run_tiles<64, false, true>(a, runs, st);
        return bf16 ? run_tiles<64, true, false>(a, runs, st) : run_tiles<64, false, false>(a, runs, st);
    }
    if (i8) return bf16 ? run_tiles<128, true, true>(a, runs, st) : run_tiles<128, false, true>(a, runs, st);
    return bf16 ? run_tiles<128, true, false>(a, runs, st) : run_tiles<128, false, false>(a, runs, st);
}

}  // namespace attend

uint32_t attend_read_clear_error() {
    uint32_t v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, attend::g_err_attend, sizeof(v));
    cudaMemcpyToSymbol(attend::g_err_attend, &z, sizeof(z));
    return v;
}

}  // namespace qm
