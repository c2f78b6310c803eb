// qm_attend.cuh -- what the kernels of cache_attend share: the arguments, how
// the work is cut, and the join of items that several CTAs worked on.
//
// The work. Query heads that share a key head are rows over the same keys: a
// sequence's new tokens and its group of G query heads make new*G rows (row r:
// token r / G, head r % G of the group), cut into tiles of R rows. An item is one
// row tile of one key head of one sequence; its work is its span of keys in units
// of 128 or 256 keys, from the first key that any of its rows sees to the last (one
// unit where they see none, whose rows are then written as empty). The units of
// all items, in order of sequence, key head, tile and key, are cut into as many
// equal runs as there are CTAs: lengths of any mix keep every SM busy to the end,
// and the host needs to know none of them. Each CTA finds its run from the
// lengths itself. A CTA that has all of an item writes its rows; one that has a
// part leaves its unnormalised sums, with their maximum and total, in the
// workspace. An item's parts are then added in order of key: in attend_rows_kernel
// by the CTA with its last part, once its own run is done (it waits for flags of the
// CTAs before it, whose runs are as long; a second launch costs more), after
// attend_tiles_kernel, whose parts are up to 128 KB each, by attend_join_kernel. The
// cut depends on the lengths alone, and so does the order of every sum: the same
// call gives the same bits.
#pragma once

#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "qm_attend_parts.h"
#include "qm_device.cuh"
#include "qm_internal.h"

namespace qm {
namespace attend {

constexpr int kUnit = 128;      // keys of a unit of work (attend_rows_kernel may take 256)
constexpr int kTileRows = 256;  // rows of an item of attend_tiles_kernel

struct Args {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    int64_t q_ts, q_hs, o_ts, o_hs;
    const uint8_t *k, *v;
    const float *ks, *vs;
    uint32_t page_stride, head_stride, token_stride;  // in 16-byte pieces
    int64_t sps, shs, sts;
    const int32_t *lens, *table, *q_off;
    int64_t table_stride;
    int cap;  // keys that the page table has room for
    int seqs, tokens, each;
    int heads, group, kv_heads, dim;
    int page_size, pages;
    // quotients of numbers below 2^31: n / page_size = (n * page_mul) >> (32 + page_shift),
    // and by `group` likewise; a factor of 0 for a divisor of 1
    uint32_t page_mul, group_mul;
    int page_shift, group_shift;
    int window;  // 0: none
    float scale2;  // scale * log2(e): scores are kept in powers of two
    // workspace
    int* desc;     // [grid][kDesc] (attend_tiles_kernel)
    unsigned long long* done;  // [grid] (attend_rows_kernel): `call` once the CTA's part of an item that goes on is there
    unsigned long long call;   // marks this call
    float2* ml;    // [grid][2][R]: maximum and total of each row
    float* part;   // [grid][2][R][DP]
};

QM_DEV uint32_t quotient(uint32_t n, uint32_t mul, int shift) { return mul ? __umulhi(n, mul) >> shift : n; }
// The token (of its sequence's new ones) that a row belongs to.
QM_DEV uint32_t token_of(const Args& a, uint32_t row) { return quotient(row, a.group_mul, a.group_shift); }

QM_DEV int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// One sequence of the batch: first row, new tokens, length.
struct Seq {
    int first, fresh, len;
};

QM_DEV Seq load_seq(const Args& a, int s) {
    Seq q;
    if (a.q_off) {
        q.first = clampi(__ldg(a.q_off + s), 0, a.tokens);
        q.fresh = clampi(__ldg(a.q_off + s + 1), q.first, a.tokens) - q.first;
    } else {
        q.first = s * a.each;
        q.fresh = a.each;
    }
    q.len = max(__ldg(a.lens + s), 0);
    return q;
}

// The first key that position p sees.
QM_DEV int first_seen(const Args& a, int p) { return a.window && p >= a.window ? p - a.window + 1 : 0; }

// The keys [lo, hi) that rows r0 .. r0 + R - 1 of a sequence see between them (hi
// <= lo: none); p0 and p1: the first and last row's positions.
template <int U>
struct Span {
    int lo, hi, p0, p1, rows;
    QM_DEV int u0() const { return hi > lo ? lo / U : 0; }
    QM_DEV int u1() const { return hi > lo ? (hi - 1) / U + 1 : 1; }
};

template <int R, int U>
QM_DEV Span<U> tile_span(const Args& a, const Seq& s, unsigned tile) {
    const unsigned r0 = tile * R, all = static_cast<unsigned>(s.fresh) * a.group;
    Span<U> t;
    t.rows = static_cast<int>(min(static_cast<unsigned>(R), all - r0));
    const int base = s.len - s.fresh;
    t.p0 = base + static_cast<int>(token_of(a, r0));
    t.p1 = base + static_cast<int>(token_of(a, r0 + t.rows - 1));
    t.hi = min(a.cap, t.p1 + 1);
    t.lo = first_seen(a, t.p0);
    return t;
}

template <int R>
QM_DEV unsigned tiles_of(const Args& a, const Seq& s) {
    return (static_cast<unsigned>(s.fresh) * a.group + R - 1) / R;
}

// Units of tile `t` of a sequence; 0 past its last.
template <int R, int U>
QM_DEV int tile_units(const Args& a, const Seq& s, unsigned t, unsigned tiles) {
    if (t >= tiles) return 0;
    const Span<U> p = tile_span<R, U>(a, s, t);
    return p.u1() - p.u0();
}

QM_DEV Seq shfl_seq(const Seq& s, int src) {
    Seq o;
    o.first = __shfl_sync(0xffffffffu, s.first, src);
    o.fresh = __shfl_sync(0xffffffffu, s.fresh, src);
    o.len = __shfl_sync(0xffffffffu, s.len, src);
    return o;
}

// Units of one key head of each lane's sequence (0 for a lane without one); `most` grows
// to those of the longest item seen. The warp goes through the tiles of a sequence of many together.
template <int R, int U>
QM_DEV int64_t head_units(const Args& a, const Seq& s, bool mine, int& most) {
    const int lane = threadIdx.x & 31;
    const unsigned tiles = mine ? tiles_of<R>(a, s) : 0;
    int64_t n = 0;
    constexpr unsigned kAlone = 12;
    if (tiles <= kAlone)
        for (unsigned t = 0; t < tiles; ++t) {
            const int units = tile_units<R, U>(a, s, t, tiles);
            n += units;
            if constexpr (R == kTileRows) most = max(most, units);
        }
    for (unsigned many = __ballot_sync(0xffffffffu, tiles > kAlone); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const Seq q = shfl_seq(s, src);
        const unsigned all = __shfl_sync(0xffffffffu, tiles, src);
        int64_t sum = 0;
        for (unsigned t = lane; t < all; t += 32) {
            const int units = tile_units<R, U>(a, q, t, all);
            sum += units;
            if constexpr (R == kTileRows) most = max(most, units);
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == src) n = sum;
    }
    return n;
}

// A place in a CTA's run of units.
template <int R, int U = kUnit>
struct Cursor {
    int64_t left;  // units of the run still to come, this one among them
    int s, h;
    unsigned tile, tiles;
    Seq seq;
    Span<U> span;
    int u, u1;

    QM_DEV void enter(const Args& a) {  // the item's first unit
        span = tile_span<R, U>(a, seq, tile);
        u = span.u0();
        u1 = span.u1();
    }
    QM_DEV bool first() const { return u == span.u0(); }
    QM_DEV void next_item(const Args& a) {
        if (++tile == tiles) {
            tile = 0;
            if (++h == a.kv_heads) {
                h = 0;
                do {
                    if (++s >= a.seqs) return;  // only past the last unit
                    seq = load_seq(a, s);
                    tiles = tiles_of<R>(a, seq);
                } while (tiles == 0);
            }
        }
        enter(a);
    }
    QM_DEV void step(const Args& a) {
        --left;
        if (++u == u1 && left > 0) next_item(a);
    }
};

// The calling warp's cursor at unit g (every lane returns the same; left is not
// set). seq and units: the lane's sequence and its units of one key head, of
// sequences 0..31. each: g counts items, and units their row tiles.
template <int R, int U>
QM_DEV Cursor<R, U> locate(const Args& a, int64_t g, Seq seq, int64_t units, bool each) {
    const int lane = threadIdx.x & 31;
    Cursor<R, U> k = {};
    int64_t at = 0;  // units before sequence s0
    for (int s0 = 0; s0 < a.seqs; s0 += 32) {
        if (s0 > 0) {
            const bool mine = s0 + lane < a.seqs;
            if (mine) seq = load_seq(a, s0 + lane);
            int most = 0;
            units = each ? (mine ? tiles_of<R>(a, seq) : 0) : head_units<R, U>(a, seq, mine, most);
        }
        const int64_t n = units * a.kv_heads;
        int64_t upto = n;  // units up to and with this lane's sequence
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + upto > g);
        if (past) {
            const int src = __ffs(past) - 1;
            const int64_t before = at + __shfl_sync(0xffffffffu, upto - n, src);
            const int64_t per_head = __shfl_sync(0xffffffffu, units, src);
            k.s = s0 + src;
            k.seq = shfl_seq(seq, src);
            k.tiles = tiles_of<R>(a, k.seq);
            int64_t rem = g - before;
            k.h = (rem >> 31) == 0 && (per_head >> 31) == 0
                      ? static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(per_head))
                      : static_cast<int>(rem / per_head);
            rem -= k.h * per_head;
            for (unsigned t0 = 0; t0 < k.tiles; t0 += 32) {  // the tile that unit `rem` of the head is in
                int sum = each ? t0 + lane < k.tiles : tile_units<R, U>(a, k.seq, t0 + lane, k.tiles);
                const int own = sum;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, sum, m);
                    if (lane >= m) sum += o;
                }
                const unsigned beyond = __ballot_sync(0xffffffffu, sum > rem);
                if (beyond) {
                    const int hit = __ffs(beyond) - 1;
                    k.tile = t0 + hit;
                    k.enter(a);
                    k.u += static_cast<int>(rem) - __shfl_sync(0xffffffffu, sum - own, hit);
                    return k;
                }
                rem -= __shfl_sync(0xffffffffu, sum, 31);
            }
            return k;  // not reached: the head's tiles have per_head units
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
    }
    return k;
}

// The units in all, and those of one key head of the lane's sequence among the first 32.
struct Load {
    int64_t total, units0;
    Seq seq0;
    int runs;   // that have units
    // of attend_tiles_kernel:
    int items;  // (2^16 stands for any more)
    int most;   // units of the longest
};
template <int R, int U = kUnit>
QM_DEV Load measure(const Args& a, int runs) {
    const int lane = threadIdx.x & 31;
    Load w = {};
    for (int s0 = 0; s0 < a.seqs; s0 += 32) {
        Seq seq = {};
        const bool mine = s0 + lane < a.seqs;
        if (mine) seq = load_seq(a, s0 + lane);
        int64_t n = head_units<R, U>(a, seq, mine, w.most);
        if constexpr (R == kTileRows) {
            const unsigned items = __reduce_add_sync(0xffffffffu, mine ? min(tiles_of<R>(a, seq), 1u << 16) : 0u);
            w.items = min(w.items + static_cast<int>(min(items, 1u << 16)), 1 << 16);
        }
        if (s0 == 0) {
            w.seq0 = seq;
            w.units0 = n;
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) n += __shfl_xor_sync(0xffffffffu, n, m);
        w.total += n;
    }
    if constexpr (R == kTileRows) {
        w.most = __reduce_max_sync(0xffffffffu, w.most);
        w.items = static_cast<int>(min(static_cast<int64_t>(w.items) * a.kv_heads, static_cast<int64_t>(1 << 16)));
    }
    w.total *= a.kv_heads;
    w.runs = w.total < runs ? static_cast<int>(w.total) : runs;  // the CTAs past the last unit have nothing
    return w;
}

// The items that are not split: of up to `inside` units where runs are at least as long, else
// of up to `beyond` more than a run.
struct Split {
    int inside, beyond;
};

// Where run `c` begins: unit `at`, and the cursor there (the calling warp's; every
// lane returns the same, left is not set); the last one's end for c = runs. Moved to an
// end of the item it falls in where splitting that would cost more (its parts are written
// and joined) than uneven runs: whole items of s units leave the longest of the runs that
// should have L units each with s where s > L, and with up to s more than L else. An item's
// span alone decides, so it is cut at all the runs' ends in it or at none. small and
// large: for items of at most R / 2 rows and of more. each: run c is item c.
template <int R, int U = kUnit>
QM_DEV Cursor<R, U> run_start(const Args& a, const Load& w, int c, bool each, Split small, Split large, int64_t& at) {
    Cursor<R, U> k = {};
    at = each ? 0 : w.total;
    if (c >= (each ? w.items : w.runs)) return k;
    if (!each) at = share(w.total, c, w.runs);
    k = locate<R, U>(a, each ? c : at, w.seq0, each ? tiles_of<R>(a, w.seq0) : w.units0, each);
    if (each) return k;
    const int64_t even = share(w.total, 1, w.runs);
    const int span = k.span.u1() - k.span.u0(), in = k.u - k.span.u0();
    const Split cost = k.span.rows > R / 2 ? large : small;
    if (in > 0 && (span <= even ? span <= cost.inside : span <= even + cost.beyond)) {
        if (2 * in < span) {
            at -= in;
            k.u = k.span.u0();
        } else {
            at += span - in;
            k.left = 1;  // only so that next_item looks at what follows
            if (at < w.total) k.next_item(a);
        }
    }
    return k;
}

// Where key `key`'s row of head h lies: its offset in 16-byte pieces (a part of the
// cache spans less than 2^32 - 1 of them, 64 GB), or kNoRow where it is not to be
// read; and its scale's offset.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
// A lookup is begun and finished apart, so that what lies between hides the page
// table's latency (and no branch keeps several of them from overlapping).
struct Lookup {
    int id, row;  // page id as the table has it, row in the page; row -1: not to be read
};
QM_DEV Lookup begin_lookup(const Args& a, int s, int key, int lo, int hi) {
    Lookup l = {0, -1};
    if (lo >= hi) return l;  // the same for the whole warp
    const int k = clampi(key, lo, hi - 1);
    const int p = static_cast<int>(quotient(k, a.page_mul, a.page_shift));
    l.id = __ldg(a.table + s * a.table_stride + p);
    l.row = k == key ? k - p * a.page_size : -1;
    return l;
}
template <bool I8>
QM_DEV uint32_t finish_lookup(const Args& a, const Lookup& l, int h, int64_t& scale_off) {
    const bool there = l.row >= 0 && static_cast<unsigned>(l.id) < static_cast<unsigned>(a.pages);
    if constexpr (I8) scale_off = l.id * a.sps + h * a.shs + l.row * a.sts;
    const uint32_t at = l.id * a.page_stride + h * a.head_stride + l.row * a.token_stride;
    return there ? at : kNoRow;
}

QM_DEV void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 zeros instead where not `on` (`any`: an address that is then not read).
QM_DEV void cp_async16(uint32_t dst, const void* src, bool on, const void* any) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(on ? src : any), "r"(on ? 16u : 0u) : "memory");
}
QM_DEV void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
QM_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
QM_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QM_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

QM_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What exponents are taken against, given a running maximum: 0 where there is none yet, and for +infinity
// the largest float32, so that the total becomes infinity, as its definition has it, and not infinity less infinity.
QM_DEV float reference(float top) { return top == -INFINITY ? 0.f : fminf(top, FLT_MAX); }

template <bool BF16>
QM_DEV uint32_t pack16(float lo, float hi) {
    if constexpr (BF16) {
        uint32_t d;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    } else {
        return pack_f16x2(lo, hi);
    }
}

template <bool BF16>
QM_DEV void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
    }
}

// Signed bytes 0 and 2 of x as a pair of 16-bit values, exactly. bfloat16 has eight
// significant bits: 128 + the low seven bits, less 128 or 256 by the sign bit;
// float16: 1024 + the code with its sign bit turned (code + 128), less 1152.
template <bool BF16>
QM_DEV uint32_t codes16(uint32_t x) {
    if constexpr (BF16) {
        const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&d);
    } else {
        const uint32_t a = (x & 0x00FF00FFu) ^ 0x64806480u, b = 0x64806480u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
}

// The four codes of a word as two pairs of float16.
QM_DEV void codes4(uint32_t word, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = word ^ 0x80808080u, b = 0x64806480u;
    const uint32_t x = prmt(u, 0x64646464u, 0x4140), y = prmt(u, 0x64646464u, 0x4342);
    const __half2 c = *reinterpret_cast<const __half2*>(&b);
    const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), c), q = __hsub2(*reinterpret_cast<const __half2*>(&y), c);
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
}

// A row of bfloat16 as float16: the power of two that brings its largest magnitude
// to 2^14 .. 2^15, and its inverse; beside an infinity or NaN the finite elements stay
// finite. The eight bits of every element above 2^-31 of the largest stay whole.
struct RowScale {
    float by, back;
};
QM_DEV RowScale row_scale(float largest) {
    const uint32_t e0 = (__float_as_uint(largest) >> 23) & 255u;
    const uint32_t e = min(max(e0, 15u), 254u);
    return RowScale{__uint_as_float((268u - e) << 23), __uint_as_float((e - 14u) << 23)};
}
QM_DEV float largest2(uint32_t pair) {  // of two bfloat16 magnitudes (a NaN as an integer above infinity)
    return __uint_as_float(max((pair << 16) & 0x7FFF0000u, pair & 0x7FFF0000u));
}
QM_DEV float larger(float a, float b) { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); }
QM_DEV uint32_t to_f16x2(uint32_t pair, float by) {
    return pack_f16x2(__uint_as_float(pair << 16) * by, __uint_as_float(pair & 0xFFFF0000u) * by);
}

// Value scales. A weight is 2^(s - m) times its value's scale, rounded to float16, and m the running maximum
// of s + log2 |scale|: within [0, 2^12] with the kernels' lift and slack, and whole down to 2^-22 of the row's largest. The
// logarithm is held within 2^+-80 (zero and NaN: the low end), so that the totals, sums of
// 2^(s - m), stay in float32: at most 2^92 for a key, at least 2^-72 for the largest. A finite scale
// beyond that is a far one: its products are formed one by one in float32, as a user will
// hardly ever have them (2^80 is 10^24), and their range is float32's.
constexpr int kFarLog2 = 80;
QM_DEV float scale_log2(float s) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(fabsf(s)));
    return fminf(fmaxf(y, static_cast<float>(-kFarLog2)), static_cast<float>(kFarLog2));
}
QM_DEV bool far_scale(float s) {  // finite, not zero, and past 2^+-80
    const uint32_t u = __float_as_uint(s) & 0x7FFFFFFFu, e = u >> 23;
    return u != 0u && e != 255u && (e < 127u - kFarLog2 || e >= 127u + kFarLog2);
}

// Whether an infinity or NaN is among pairs of 16-bit values: the largest exponents
// of the low and high halves so far, and the verdict on them.
template <bool BF16>
QM_DEV uint32_t top_exponents(uint32_t top, const uint4& v) {
    constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u;
    return __vmaxu2(__vmaxu2(__vmaxu2(top, v.x & kExp), __vmaxu2(v.y & kExp, v.z & kExp)), v.w & kExp);
}
template <bool BF16>
QM_DEV bool nonfinite(uint32_t top) {
    constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
    return (top & 0xFFFFu) == kExp || (top >> 16) == kExp;
}

// 32 bytes to a 32-byte aligned address in one access.
QM_DEV void st_global_32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Where row r of an item goes: its token and query head.
QM_DEV uint16_t* out_row(const Args& a, int first, int h, unsigned r, int64_t& lse_at) {
    const unsigned i = token_of(a, r), g = r - i * a.group;
    const int head = h * a.group + static_cast<int>(g);
    const int64_t t = first + static_cast<int64_t>(i);
    lse_at = t * a.heads + head;
    return a.out + t * a.o_ts + head * a.o_hs;
}

// 1 / total; where the row sees keys but their weights add up to nothing (every score
// -infinity) the quotient is the definition's 0/0, and 0 where it sees none.
QM_DEV float inverse_total(const Args& a, int pos, float total) {
    if (first_seen(a, pos) >= min(a.cap, pos + 1)) return 0.f;
    return 1.0f / total;
}

// The sum of an item's parts, four elements to a thread, against a reference m.
struct Sum4 {
    float m, total;
    float4 o;
    QM_DEV void add(float em, float et, const float4& v) {
        const float mn = fmaxf(m, em), ref = reference(mn);
        const float f = ex2(m - ref), fe = ex2(em - ref);
        total = total * f + et * fe;
        o.x = o.x * f + v.x * fe; o.y = o.y * f + v.y * fe;
        o.z = o.z * f + v.z * fe; o.w = o.w * f + v.w * fe;
        m = mn;
    }
};
// Parts i0, i0 + di, ... of a row: the item's first part lies at slot 2 c + 1, part i
// after it at slot 2 (c + i).
template <int R, int DP>
QM_DEV Sum4 sum_parts(const Args& a, int c, int parts, int row, int c4, int i0, int di) {
    Sum4 s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int i = i0; i < parts; i += di) {
        const int64_t at = static_cast<int64_t>(2 * (c + i) + (i == 0 ? 1 : 0)) * R + row;
        const float2 e = __ldcg(a.ml + at);
        s.add(e.x, e.y, __ldcg(reinterpret_cast<const float4*>(a.part + at * DP + 4 * c4)));
    }
    return s;
}

QM_DEV float log_total(float top, float total) {
    return total == 0.f ? __int_as_float(0xff800000) : (top + log2f(total)) * 0.69314718055994531f;
}

// Writes four elements of row r of an item from its whole sum.
template <bool BF16>
QM_DEV void write_row4(const Args& a, int first, int h, unsigned r, int p0, int c4, const Sum4& s) {
    int64_t lse_at;
    uint16_t* y = out_row(a, first, h, r, lse_at);
    const float inv = inverse_total(a, p0 + static_cast<int>(token_of(a, r)), s.total);
    if (4 * c4 < a.dim)
        *reinterpret_cast<uint2*>(y + 4 * c4) = make_uint2(pack16<BF16>(s.o.x * inv, s.o.y * inv), pack16<BF16>(s.o.z * inv, s.o.w * inv));
    if (a.lse && c4 == 0) a.lse[lse_at] = log_total(s.m, s.total);
}

// attend_tiles_kernel (qm_attend_tc.cu).
cudaError_t launch_tiles(const Args& a, const qm_cache& c, int runs, bool bf16, cudaStream_t st);

}  // namespace attend
}  // namespace qm
