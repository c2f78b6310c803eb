// qm_attend.cu -- attention of new tokens over a paged cache for few rows to a
// key head (attend_rows_kernel: decode steps, drafted tokens), and the join of
// items cut between CTAs (attend_join_kernel).
//
// o = sum_j w_j v_j, w = softmax over the keys j that a row sees of scale (q . k_j),
// in one pass over the keys: with m the running maximum of the scores (in powers
// of two: t = scale log2(e) (q . k)), l = sum 2^(t_j - m) and o = sum 2^(t_j - m) v_j are
// rescaled by 2^(m - m') when m grows to m'. Scores, weights' sums and o are float32;
// a weight is rounded to the values' 16-bit type to enter its product (a relative 2^-8 or
// 2^-11 at most that does not add up over keys, as the output's own rounding).
//
// Every key and value is read once for up to 16 rows, 2 flops a byte and row: what
// bounds it is HBM. One CTA per SM, eight warps; a warp takes an eighth of a unit's keys and
// streams them through its own ring of shared-memory stages with 16-byte
// asynchronous copies (whole 2 * DP-byte rows; the pages' places are looked up one
// step ahead), so that warps wait for nothing but their own copies and an SM keeps
// 64 to 139 KB in flight. A step is 16 keys of 256-byte rows and 32 of shorter ones: with 16 the
// step's own latency and its fixed instructions (place, maxima, rescaling) are what bounds those (8-bit
// codes, below; 32 x 2 tokens of 7 query heads of 64 over 8192 38.9 -> 32.5 us). The products are m16n8k16 tensor-core instructions on 16
// rows (rows that the item lacks are zeros: the tensor pipe has time to spare). At the
// end of an item the warps' sums are added through shared memory in warp order while
// the next item's copies are already under way. Up to 32 rows (48 of heads of 64
// elements: the sums fit in registers) take two or three such tiles of rows at once, their queries
// in shared memory; against attend_tiles_kernel 113 to 117 us for 32 x 8 tokens of 4 query
// heads to a key head over 4096, 124 to 339 over 8-bit codes, and 28 to 36 for 32 x 5 drafted tokens (7 heads of 64).
// Measured: one token of 64 ragged sequences of up to 8192 (16 / 8 heads of 128,
// 1.08 GB) 176 to 179 us, 6.0 to 6.1 TB/s, 0.9 of the copy rate (184 with 64 / 8 heads); of one sequence of 1500
// 8.5 us, of one of 32768 30 us (4.4 TB/s).
//
// 8-bit codes are exact in both 16-bit types, so they enter the products as they
// are: a key's scale multiplies its score, a value's scale its weight. All operands
// are float16 whatever q's type: a code takes fewer instructions to become one than to become
// bfloat16, bfloat16 queries fit after an exact power of two for each row, and scaled weights
// have three bits more (the running maximum includes the values' scales, which
// keeps them within 2^+-8; beside a scale past 2^+-80 the values' products are formed one by one in
// float32). Instructions, not bytes, are what bounds it: 4 sequences
// of 65 to 131 thousand tokens (32 / 8 heads) 174 us, 4.7 TB/s (205 in steps of 16 keys, 238 with keys also turned into
// bfloat16); 16 x 2 tokens of 8 query heads to a key head over 8192 73 us (84, 93).
//
// Float16 weights, here and over a float16 cache: lifted by 2^8, a weight (times its value's scale)
// keeps all its bits down to 2^-22 of the row's largest, fewer below, and none past 2^-33.
// It shows where the values of a row's large weights are zero in an element.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "qm_attend.cuh"

namespace qm {
namespace attend {
namespace {

constexpr int kWarps = 8;
constexpr float kNegInf = -INFINITY;

// Stage and shared-memory layout of a kernel variant.
template <int DP, bool I8, int MT>
struct Lay {
    static constexpr int kRows = 16 * MT;
    static constexpr int kRowBytes = I8 ? DP : 2 * DP;
    static constexpr int kKeys = kRowBytes == 256 ? 16 : 32;       // of a warp's step
    static constexpr int kPart = kKeys * kRowBytes;                // keys, or values, of a step
    static constexpr int kStage = 2 * kPart + (I8 ? 8 * kKeys : 0);  // and their scales
    static constexpr int kStages = I8 ? (DP == 128 ? 2 : 5) : 3;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kRed = kWarps * 8 * DP * 4;               // sums of eight rows; between, the queries of several tiles
    static constexpr int kMl = kWarps * kRows * 8;
    static constexpr int kRun = kWarps * kStages * kStage + kRed + kMl;  // the CTA's run
    static constexpr int kSmem = kRun + 384;
    // where 16-byte piece c of row r lies: rows that one access reads together
    // must differ in bank group
    static QM_DEV uint32_t k_at(int r, int c) {
        if constexpr (!I8) return r * kRowBytes + ((c ^ (r & 7)) << 4);
        else if constexpr (DP == 128) return r * kRowBytes + ((c ^ ((r & 1) << 2)) << 4);
        else return r * kRowBytes + (c << 4);
    }
    static QM_DEV uint32_t v_at(int r, int c) {
        if constexpr (!I8) return r * kRowBytes + ((c ^ (r & 7)) << 4);
        else if constexpr (DP == 128) return r * kRowBytes + ((c ^ (((r >> 1) & 3) << 1)) << 4);
        else return r * kRowBytes + ((c ^ (((r >> 1) & 1) << 1)) << 4);
    }
    static QM_DEV uint32_t q_at(int r, int c) { return r * 2 * DP + ((c ^ (r & 7)) << 4); }
};

QM_DEV void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
QM_DEV void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ uint32_t g_err_rows = 0;

struct Flag {
    unsigned long long* p;
    QM_DEV unsigned long long swap(unsigned long long v) const {
        unsigned long long old;
        asm volatile("atom.acq_rel.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
        return old;
    }
    QM_DEV void set(unsigned long long v) const { *reinterpret_cast<volatile unsigned long long*>(p) = v; }
};
QM_DEV unsigned long long load_acquire(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

// An item whose last part this CTA has.
struct Join {
    int owner;  // the CTA with its first part; -1: there is no such item
    int first, h;
    unsigned row0;
    int rows, base;
};

template <int DP, bool BF16, bool I8, int MT>
__global__ void __launch_bounds__(kWarps * 32, 1) attend_rows_kernel(const __grid_constant__ Args a) {
    using L = Lay<DP, I8, MT>;
    constexpr int kRows = L::kRows;
    constexpr int ST = L::kStages;
    constexpr int KK = DP / 16;
    constexpr int KEYS = L::kKeys, NT = KEYS / 8, KP = KEYS / 16;
    constexpr int U = kWarps * KEYS;            // keys of a unit
    constexpr bool PBF = BF16 && !I8;           // type of the operands
    constexpr float kLift = PBF ? 0.f : 8.f;    // float16 weights in [0, 2^8]: the small ones keep their bits
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * ST * L::kStage;
    float* red = reinterpret_cast<float*>(smem + kWarps * ST * L::kStage);
    float2* ml = reinterpret_cast<float2*>(smem + kWarps * ST * L::kStage + L::kRed);

    grid_launch_dependents();
    grid_dependency_wait();
    struct Run {
        Cursor<kRows, U> start;
        int64_t from, to, total;  // the run's first unit, the unit after it, units in all
        int runs;
        float back[kRows];  // see below
    };
    static_assert(sizeof(Run) <= 384, "run");
    Run* run = reinterpret_cast<Run*>(smem + L::kRun);
    if (warp < 2) {  // the run's start and its end
        const Load work = measure<kRows, U>(a, gridDim.x);
        // Runs of one unit have one part each, and a join costs little more than a second unit;
        // longer ones may have two, and write or join both. Against splitting everywhere: 32 x 5 tokens (7 query
        // heads of 64 to a key head) over 100 to 4000 32.3 -> 27.9 us, over 1024 19.4 -> 15.1; 32 x 4
        // (4 heads of 128) over 512 26.0 -> 21.9, over 1024 37.3 -> 33.3; one token over 256 7.4 -> 6.5.
        // One token over 512 to 1024 loses 2 % to looking; left whole it would lose 20 to 60.
        const Split split = {1024 / U, work.total <= gridDim.x ? 1 : U == 256 ? 3 : 2};
        int64_t at;
        const Cursor<kRows, U> k = run_start<kRows, U>(a, work, blockIdx.x + warp, false, split, split, at);
        if (lane == 0 && warp == 0) {
            run->from = at;
            run->total = work.total;
            run->runs = work.runs;
            run->start = k;
        }
        if (lane == 0 && warp == 1) run->to = at;
    }
    __syncthreads();
    Cursor<kRows, U> now = run->start;
    now.left = run->to - run->from;
    if (now.left <= 0) return;
    Cursor<kRows, U> ahead = now;
    Join join = {-1, 0, 0, 0, 0, 0};

    // ---- copies: the place of key row lane % KEYS of the step `ahead` is at
    Lookup found = {0, -1};
    int head = 0;
    auto look = [&]() {
        if (ahead.left > 0) {
            head = ahead.h;
            found = begin_lookup(a, ahead.s, ahead.u * U + warp * KEYS + lane % KEYS, ahead.span.lo, ahead.span.hi);
        }
    };
    auto issue = [&](int slot) {
        const uint32_t base = ring + slot * L::kStage;
        int64_t splace;
        const uint32_t place = finish_lookup<I8>(a, found, head, splace);
        constexpr int per = 32 / L::kChunks;  // rows that the warp copies at once
        const int c = lane % L::kChunks;
        const int step = I8 ? 16 : 8;  // elements of a piece
#pragma unroll
        for (int i = 0; i < KEYS / per; ++i) {
            const int r = i * per + lane / L::kChunks;
            const uint32_t off = __shfl_sync(0xffffffffu, place, r);
            const bool on = off != kNoRow && c * step < a.dim;
            const uint64_t at = (static_cast<uint64_t>(off) + c) * 16;
            cp_async16(base + L::k_at(r, c), a.k + at, on, a.q);
            cp_async16(base + L::kPart + L::v_at(r, c), a.v + at, on, a.q);
        }
        if constexpr (I8) {
            static_assert(KEYS == 32, "a lane for every key");
            const bool on = place != kNoRow;
            cp_async4(base + 2 * L::kPart + 4 * lane, on ? a.ks + splace : reinterpret_cast<const float*>(a.q), on ? 4u : 0u);
            cp_async4(base + 2 * L::kPart + 4 * KEYS + 4 * lane, on ? a.vs + splace : reinterpret_cast<const float*>(a.q), on ? 4u : 0u);
        }
    };
    look();
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) {
        if (ahead.left > 0) {
            issue(i);
            ahead.step(a);
            look();
        }
        cp_async_commit();
    }

    uint32_t qa[MT == 1 ? KK : 1][4];
    const uint32_t sq = smem_u32(red);
    float acc[MT][DP / 8][4];
    float top[MT][2], sum[MT][2];
    float back[MT][2];             // bfloat16 queries over codes: what their scores are still to be multiplied by
    int kmin[MT][2], kmax[MT][2];  // of rows 16 mt + g and + 8: the keys they see, [kmin, kmax]
    bool begin = true;             // the next step begins a part of an item
    bool whole_start = false;
    int slot = 0;
    while (now.left > 0) {
        if (begin) {
            begin = false;
            whole_start = now.first();
            const auto query = [&](int r) -> const uint16_t* {  // row r of the item; null past its last
                if (r >= now.span.rows) return nullptr;
                const unsigned R = now.tile * kRows + r, i = token_of(a, R), gg = R - i * a.group;
                return a.q + (now.seq.first + static_cast<int64_t>(i)) * a.q_ts + (now.h * a.group + static_cast<int>(gg)) * a.q_hs;
            };
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 16 * mt + g + 8 * x;
                    const int at = now.seq.len - now.seq.fresh + static_cast<int>(token_of(a, now.tile * kRows + r));
                    top[mt][x] = kNegInf;
                    sum[mt][x] = 0.f;
                    kmin[mt][x] = r < now.span.rows ? first_seen(a, at) : 0;
                    kmax[mt][x] = r < now.span.rows ? min(at, a.cap - 1) : -1;
                    if constexpr (MT == 1) {
                        const uint16_t* qrow = query(r);
#pragma unroll
                        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                // codes come four to a lane: their products take the head's elements in that order
                                const int d = I8 ? 64 * (kk / 4) + 16 * t + 4 * (kk % 4) + 2 * y : 16 * kk + 8 * y + 2 * t;
                                qa[kk][2 * y + x] = qrow && d < a.dim ? *reinterpret_cast<const uint32_t*>(qrow + d) : 0u;
                            }
                        if constexpr (I8 && BF16) {
                            float big = 0.f;
#pragma unroll
                            for (int kk = 0; kk < KK; ++kk) big = larger(big, larger(largest2(qa[kk][x]), largest2(qa[kk][2 + x])));
                            big = larger(big, __shfl_xor_sync(0xffffffffu, big, 1));
                            big = larger(big, __shfl_xor_sync(0xffffffffu, big, 2));
                            const RowScale rs = row_scale(big);
                            back[mt][x] = rs.back;
#pragma unroll
                            for (int kk = 0; kk < KK; ++kk) {
                                qa[kk][x] = to_f16x2(qa[kk][x], rs.by);
                                qa[kk][2 + x] = to_f16x2(qa[kk][2 + x], rs.by);
                            }
                        }
                    }
                }
            if constexpr (MT > 1) {  // kept where the warps' sums meet at a part's end
                for (int i = threadIdx.x; i < kRows * (DP / 8); i += kWarps * 32) {
                    const int r = i / (DP / 8), c = i % (DP / 8);
                    const uint16_t* qrow = query(r);
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (qrow && 8 * c < a.dim) v = *reinterpret_cast<const uint4*>(qrow + 8 * c);
                    if constexpr (I8 && BF16) {  // the lanes of a row agree on its scale
                        float big = larger(larger(largest2(v.x), largest2(v.y)), larger(largest2(v.z), largest2(v.w)));
#pragma unroll
                        for (int m = 1; m < DP / 8; m <<= 1) big = larger(big, __shfl_xor_sync(0xffffffffu, big, m));
                        const RowScale rs = row_scale(big);
                        v = make_uint4(to_f16x2(v.x, rs.by), to_f16x2(v.y, rs.by), to_f16x2(v.z, rs.by), to_f16x2(v.w, rs.by));
                        if (c == 0) run->back[r] = rs.back;
                    }
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(red) + L::q_at(r, c)) = v;
                }
                __syncthreads();
                if constexpr (I8 && BF16) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) back[mt][x] = run->back[16 * mt + g + 8 * x];
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) acc[mt][j][0] = acc[mt][j][1] = acc[mt][j][2] = acc[mt][j][3] = 0.f;
        }
        cp_async_wait<ST - 2>();
        __syncwarp();  // the stage is whole, and its predecessor is free in every lane
        if (ahead.left > 0) {
            issue(slot == 0 ? ST - 1 : slot - 1);
            ahead.step(a);
            look();
        }
        cp_async_commit();

        const int key0 = now.u * U + warp * KEYS;
        const Span<U>& sp = now.span;
        if (key0 < sp.hi && key0 + KEYS - 1 >= sp.lo) {
            const uint32_t kb = ring + slot * L::kStage, vb = kb + L::kPart;
            float s[MT][NT][4] = {};
            // queries of tile mt, step kk
            const auto queries = [&](int mt, int kk, uint32_t (&q)[4]) {
                if constexpr (MT == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = qa[kk][i];
                } else if constexpr (!I8) {
                    ldsm4(sq + L::q_at(16 * mt + (lane & 15), 2 * kk + (lane >> 4)), q);
                } else {
                    const int d = 64 * (kk / 4) + 16 * t + 4 * (kk % 4);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 v = lds_v2(sq + L::q_at(16 * mt + g + 8 * x, d / 8) + 2 * (d % 8));
                        q[x] = v.x;
                        q[2 + x] = v.y;
                    }
                }
            };
            if constexpr (!I8) {
                const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b[KP][4];
#pragma unroll
                    for (int h = 0; h < KP; ++h) ldsm4(kb + L::k_at(16 * h + r, 2 * kk + c), b[h]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t q[4];
                        queries(mt, kk, q);
#pragma unroll
                        for (int h = 0; h < KP; ++h) {
                            mma16<BF16>(s[mt][2 * h], q, b[h][0], b[h][1]);
                            mma16<BF16>(s[mt][2 * h + 1], q, b[h][2], b[h][3]);
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][n][e] *= a.scale2;
            } else {
#pragma unroll
                for (int h = 0; h < KK / 4; ++h) {
                    uint4 w[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) w[n] = lds_v4(kb + L::k_at(8 * n + g, 4 * h + t));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t word = i == 0 ? w[n].x : i == 1 ? w[n].y : i == 2 ? w[n].z : w[n].w;
                            codes4(word, b[n][0], b[n][1]);
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t q[4];
                            queries(mt, 4 * h + i, q);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma16<false>(s[mt][n], q, b[n][0], b[n][1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 sc = lds_v2(kb + 2 * L::kPart + 4 * (8 * n + 2 * t));
                    const float s0 = __uint_as_float(sc.x) * a.scale2, s1 = __uint_as_float(sc.y) * a.scale2;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (BF16) {
                            s[mt][n][0] *= back[mt][0]; s[mt][n][1] *= back[mt][0]; s[mt][n][2] *= back[mt][1]; s[mt][n][3] *= back[mt][1];
                        }
                        s[mt][n][0] *= s0; s[mt][n][1] *= s1; s[mt][n][2] *= s0; s[mt][n][3] *= s1;
                    }
                }
            }
            // rows differ in what they see, or the step's keys end or begin in between
            const bool cut = key0 + KEYS - 1 > min(sp.p0, a.cap - 1) || (a.window && key0 < first_seen(a, sp.p1));
            uint32_t hidden[MT] = {};  // bit 4n + e
            if (cut) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 8 * n + 2 * t + (e & 1), x = e >> 1;
                            if (key < kmin[mt][x] || key > kmax[mt][x]) {
                                s[mt][n][e] = kNegInf;
                                hidden[mt] |= 1u << (4 * n + e);
                            }
                        }
            }
            float vs[NT][2], lv[NT][2];  // value scales of keys 8n + 2t + e, and their logarithms
            bool far = false;            // a value scale is out of float16's reach
            if constexpr (I8) {
                far = __any_sync(0xffffffffu, far_scale(__uint_as_float(lds_u32(kb + 2 * L::kPart + 4 * KEYS + 4 * lane))));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 sc = lds_v2(kb + 2 * L::kPart + 4 * KEYS + 4 * (8 * n + 2 * t));
                    vs[n][0] = __uint_as_float(sc.x);
                    vs[n][1] = __uint_as_float(sc.y);
                    lv[n][0] = scale_log2(vs[n][0]);
                    lv[n][1] = scale_log2(vs[n][1]);
                }
            }
            uint32_t pa[MT][KP][4];
            float p[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float from[2];
                bool grown = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float m = top[mt][x];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) m = fmaxf(m, I8 ? s[mt][n][2 * x + e] + lv[n][e] : s[mt][n][2 * x + e]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    grown = grown || m > top[mt][x];
                    from[x] = top[mt][x];
                    top[mt][x] = m;
                }
                if (__any_sync(0xffffffffu, grown)) {
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        f[x] = ex2(from[x] - reference(top[mt][x]));
                        sum[mt][x] *= f[x];
                    }
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j) {
                        acc[mt][j][0] *= f[0]; acc[mt][j][1] *= f[0];
                        acc[mt][j][2] *= f[1]; acc[mt][j][3] *= f[1];
                    }
                }
                const float ref[2] = {reference(top[mt][0]) - kLift, reference(top[mt][1]) - kLift};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[mt][n][e] = ex2(s[mt][n][e] - ref[e >> 1]);
                        sum[mt][e >> 1] += p[mt][n][e];
                        if constexpr (I8) p[mt][n][e] = (hidden[mt] >> (4 * n + e)) & 1 ? 0.f : p[mt][n][e] * vs[n][e & 1];
                    }
#pragma unroll
                for (int h = 0; h < KP; ++h) {
                    pa[mt][h][0] = pack16<PBF>(p[mt][2 * h][0], p[mt][2 * h][1]);
                    pa[mt][h][1] = pack16<PBF>(p[mt][2 * h][2], p[mt][2 * h][3]);
                    pa[mt][h][2] = pack16<PBF>(p[mt][2 * h + 1][0], p[mt][2 * h + 1][1]);
                    pa[mt][h][3] = pack16<PBF>(p[mt][2 * h + 1][2], p[mt][2 * h + 1][3]);
                }
            }
            if constexpr (!I8) {
                // A value that only some of the rows see must not reach the others: 0 times an
                // infinity or NaN is NaN. Where the rows differ and such a value is there, the
                // products are formed one by one.
                bool odd = false;
                if (cut && sp.p0 != sp.p1) {
                    uint32_t high = 0;
#pragma unroll
                    for (int i = 0; i < L::kPart / 512; ++i) high = top_exponents<BF16>(high, lds_v4(vb + 16 * (32 * i + lane)));
                    odd = __any_sync(0xffffffffu, nonfinite<BF16>(high));
                }
                if (!odd) {
                    const int r = (lane & 7) + (((lane >> 3) & 1) << 3), c = lane >> 4;
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j) {
#pragma unroll
                        for (int h = 0; h < KP; ++h) {
                            uint32_t b[4];
                            ldsm4_t(vb + L::v_at(16 * h + r, 2 * j + c), b);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma16<BF16>(acc[mt][2 * j], pa[mt][h], b[0], b[1]);
                                mma16<BF16>(acc[mt][2 * j + 1], pa[mt][h], b[2], b[3]);
                            }
                        }
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < KEYS; ++k) {
                        // p[row g + 8x][key k] is in lane 4g + (k % 8) / 2, entry [k / 8][2x + k % 2]
                        const int src = 4 * g + ((k & 7) >> 1);
                        float pk[MT][2];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                uint32_t mine = 0;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mine |= __float_as_uint((k & 1) ? p[mt][n][2 * x + 1] : p[mt][n][2 * x]) & (k >> 3 == n ? ~0u : 0u);
                                pk[mt][x] = __uint_as_float(__shfl_sync(0xffffffffu, mine, src));
                            }
#pragma unroll
                        for (int j = 0; j < DP / 8; ++j) {
                            const uint32_t w = lds_u32(vb + L::v_at(k, j) + 4 * t);
                            const float v0 = BF16 ? __uint_as_float(w << 16) : f16_bits_to_f32(w & 0xFFFFu);
                            const float v1 = BF16 ? __uint_as_float(w & 0xFFFF0000u) : f16_bits_to_f32(w >> 16);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    if (key0 + k >= kmin[mt][x] && key0 + k <= kmax[mt][x]) {
                                        acc[mt][j][2 * x] = fmaf(pk[mt][x], v0, acc[mt][j][2 * x]);
                                        acc[mt][j][2 * x + 1] = fmaf(pk[mt][x], v1, acc[mt][j][2 * x + 1]);
                                    }
                        }
                    }
                }
            } else if (far) {
#pragma unroll 1
                for (int k = 0; k < KEYS; ++k) {
                    const int src = 4 * g + ((k & 7) >> 1);  // (as above for 16-bit values)
                    float pk[MT][2];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t mine = 0;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mine |= __float_as_uint((k & 1) ? p[mt][n][2 * x + 1] : p[mt][n][2 * x]) & (k >> 3 == n ? ~0u : 0u);
                            pk[mt][x] = __uint_as_float(__shfl_sync(0xffffffffu, mine, src));
                        }
#pragma unroll
                    for (int jb = 0; jb < DP / 32; ++jb) {  // elements 32 jb + 8 t + 4 z + i
                        const uint2 w = lds_v2(vb + L::v_at(k, 2 * jb + (t >> 1)) + 8 * (t & 1));
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float v = static_cast<float>(static_cast<int8_t>((z ? w.y : w.x) >> (8 * i)));
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                    for (int x = 0; x < 2; ++x) acc[mt][4 * jb + i][2 * x + z] = fmaf(pk[mt][x], v, acc[mt][4 * jb + i][2 * x + z]);
                            }
                    }
                }
            } else {
                // column n of tile i of 32 elements jb: element 32 jb + 4 n + i
#pragma unroll
                for (int jb = 0; jb < DP / 32; ++jb) {
                    uint32_t w[KP][4];
#pragma unroll
                    for (int h = 0; h < KP; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 16 * h + 2 * t + (i & 1) + 8 * (i >> 1);
                            w[h][i] = lds_u32(vb + L::v_at(r, 2 * jb + (g >> 2)) + 4 * (g & 3));
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t pick = 0x0400u + 0x0101u * i;  // byte i of the two keys, to bytes 0 and 2
#pragma unroll
                        for (int h = 0; h < KP; ++h) {
                            const uint32_t b0 = codes16<PBF>(prmt(w[h][0], w[h][1], pick)), b1 = codes16<PBF>(prmt(w[h][2], w[h][3], pick));
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) mma16<PBF>(acc[mt][4 * jb + i], pa[mt][h], b0, b1);
                        }
                    }
                }
            }
        }
        slot = slot + 1 == ST ? 0 : slot + 1;

        const bool ends = now.u + 1 == now.u1;
        if (ends || now.left == 1) {
            // ---- the part's end: add the warps' sums
#pragma unroll
            for (int x = 0; x < 2 * MT; ++x) {
                float total = sum[x >> 1][x & 1];
                total += __shfl_xor_sync(0xffffffffu, total, 1);
                total += __shfl_xor_sync(0xffffffffu, total, 2);
                if (t == 0) ml[warp * kRows + g + 8 * x] = make_float2(top[x >> 1][x & 1], total);
            }
            __syncthreads();
            const int rows = now.span.rows;
            const bool done = whole_start && ends;
            const int part = 2 * blockIdx.x + (whole_start ? 1 : 0);
            // swaps 16-byte pieces of row g of `red` so that the rows' writes differ in bank
            auto piece = [](int row, int c4) { return c4 ^ (2 * (row & 3) | (row >> 2)); };
#pragma unroll
            for (int x = 0; x < 2 * MT; ++x) {
                if (8 * x >= rows) break;
                const int mt = x >> 1, y = x & 1;
                float m = kNegInf;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * kRows + g + 8 * x].x);
                const float f = ex2(top[mt][y] - reference(m));
                float* mine = red + (warp * 8 + g) * DP;
                if constexpr (!I8) {
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j)
                        *reinterpret_cast<float2*>(mine + 4 * piece(g, 2 * j + (t >> 1)) + 2 * (t & 1)) =
                            make_float2(acc[mt][j][2 * y] * f, acc[mt][j][2 * y + 1] * f);
                } else {
#pragma unroll
                    for (int jb = 0; jb < DP / 32; ++jb)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            *reinterpret_cast<float4*>(mine + 4 * piece(g, 8 * jb + 2 * t + z)) =
                                make_float4(acc[mt][4 * jb][2 * y + z] * f, acc[mt][4 * jb + 1][2 * y + z] * f,
                                            acc[mt][4 * jb + 2][2 * y + z] * f, acc[mt][4 * jb + 3][2 * y + z] * f);
                }
                __syncthreads();
                const int rr = threadIdx.x / (DP / 4), c4 = threadIdx.x % (DP / 4);
                const int row = rr + 8 * x;
                if (rr < 8 && row < rows) {
                    float mm = kNegInf;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * kRows + row].x);
                    const float mr = reference(mm);
                    float total = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 e = ml[w * kRows + row];
                        total += e.y * ex2(e.x - mr);
                        const float4 v = *reinterpret_cast<const float4*>(red + (w * 8 + rr) * DP + 4 * piece(rr, c4));
                        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
                    }
                    if (done) {
                        const unsigned R = now.tile * kRows + row;
                        int64_t lse_at;
                        uint16_t* y = out_row(a, now.seq.first, now.h, R, lse_at);
                        const int at = now.seq.len - now.seq.fresh + static_cast<int>(token_of(a, R));
                        const float inv = inverse_total(a, at, total);
                        if (4 * c4 < a.dim)
                            *reinterpret_cast<uint2*>(y + 4 * c4) = make_uint2(pack16<BF16>(o.x * inv, o.y * inv), pack16<BF16>(o.z * inv, o.w * inv));
                        if (a.lse && c4 == 0) a.lse[lse_at] = log_total(mm - kLift, total);
                    } else {
                        *reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(part) * kRows + row) * DP + 4 * c4) = o;
                        if (c4 == 0) a.ml[part * kRows + row] = make_float2(mm - kLift, total);
                    }
                }
                __syncthreads();
            }
            if (!done && ends) {  // the item's last part: the CTA joins the item when its run is done
                const int64_t at = run->to - now.left;  // this unit
                const int64_t first_unit = at - (now.u - now.span.u0());
                const int owner = static_cast<int>(((first_unit + 1) * run->runs - 1) / run->total);  // the run that holds it
                join = Join{owner, now.seq.first, now.h, now.tile * kRows, rows, now.seq.len - now.seq.fresh};
            }
            begin = true;
        }
        now.step(a);
    }
    cp_async_wait<0>();
    const Flag own = {a.done + blockIdx.x};
    unsigned long long before = 0;
    if (now.u != now.u1) {  // the run's last part is for a later CTA to join
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) before = own.swap(a.call);
    }
    bool there = join.owner >= 0;
    // ---- the parts of the item that this CTA's first part ended: all but its own are
    // the last of the runs before, which end when this one does
    const int parts = static_cast<int>(blockIdx.x) - join.owner + 1;
    if (there && threadIdx.x < parts - 1) {
        const Flag flag = {a.done + join.owner + threadIdx.x};
        const uint64_t t0 = globaltimer();
        uint64_t round = 0;
        while (there && load_acquire(flag.p) != a.call)
            there = globaltimer() - t0 <= kWaitLimitNs && ++round <= kWaitLimitNs;
        if (there) flag.set(0);
        else if (!(there = give_up(flag, a.call))) atomicOr(&g_err_rows, DEV_ERR_TIMEOUT);
    }
    if (threadIdx.x == 0) take_back(own, before, a.call);
    if (!__syncthreads_and(there)) return;
    // groups of DP / 4 threads: as many rows at once as there are, the rest of the groups over the parts
    constexpr int C4 = DP / 4, G = kWarps * 32 / C4;
    int side = 1;  // rows at once
    while (side < join.rows && side < G) side *= 2;
    const int grp = threadIdx.x / C4, c4 = threadIdx.x % C4, per = G / side;
    for (int r0 = 0; r0 < join.rows; r0 += side) {
        const int row = r0 + grp / per;
        Sum4 s = {kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (row < join.rows) s = sum_parts<kRows, DP>(a, join.owner, parts, row, c4, grp % per, per);
        float* mine = red + (grp * C4 + c4) * 8;
        *reinterpret_cast<float4*>(mine) = s.o;
        *reinterpret_cast<float2*>(mine + 4) = make_float2(s.m, s.total);
        __syncthreads();
        if (grp % per == 0 && row < join.rows) {
            for (int k = 1; k < per; ++k) {
                const float* other = red + ((grp + k) * C4 + c4) * 8;
                const float2 e = *reinterpret_cast<const float2*>(other + 4);
                s.add(e.x, e.y, *reinterpret_cast<const float4*>(other));
            }
            write_row4<BF16>(a, join.first, join.h, join.row0 + row, join.base, c4, s);
        }
        __syncthreads();
    }
}

// Joins the parts of one item of attend_tiles_kernel: block x of a CTA whose last part begins an item
// adds that part and the first parts of the CTAs after it, up to the item's last.
template <int R, int DP, bool BF16>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ Args a, int runs) {
    constexpr int C4 = DP / 4, G = 256 / C4;  // groups of threads that take every G-th part
    __shared__ float4 so[G][C4];
    __shared__ float2 sm[G];
    grid_dependency_wait();
    const int c = blockIdx.x;
    const int last = last_part(a.desc, c, runs);
    if (last < 0) return;
    const int* d = a.desc + c * kDesc;
    const int first = d[2], h = d[3], r0 = d[4], rows = d[5], base = d[6];
    if (static_cast<int>(blockIdx.y) >= rows) return;
    const int parts = last - c + 1;
    const int grp = threadIdx.x / C4, c4 = threadIdx.x % C4;
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        Sum4 s = sum_parts<R, DP>(a, c, parts, row, c4, grp, G);
        so[grp][c4] = s.o;
        if (c4 == 0) sm[grp] = make_float2(s.m, s.total);
        __syncthreads();
        if (grp == 0) {
            for (int w = 1; w < G; ++w) s.add(sm[w].x, sm[w].y, so[w][c4]);
            write_row4<BF16>(a, first, h, static_cast<unsigned>(r0) + row, base, c4, s);
        }
        __syncthreads();
    }
}

template <int DP, bool BF16, bool I8, int MT>
cudaError_t run_rows(const Args& a, int runs, cudaStream_t st) {
    auto kern = attend_rows_kernel<DP, BF16, I8, MT>;
    constexpr int smem = Lay<DP, I8, MT>::kSmem;
    static_assert(smem <= 227 * 1024, "shared memory");
    static_assert(Lay<DP, I8, MT>::kRows * DP * 2 <= Lay<DP, I8, MT>::kRed, "queries");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(runs), kWarps * 32, smem, st, a);
}

template <int DP, int MT>
cudaError_t rows_of_type(const Args& a, int runs, bool bf16, bool i8, cudaStream_t st) {
    if (i8) return bf16 ? run_rows<DP, true, true, MT>(a, runs, st) : run_rows<DP, false, true, MT>(a, runs, st);
    return bf16 ? run_rows<DP, true, false, MT>(a, runs, st) : run_rows<DP, false, false, MT>(a, runs, st);
}

cudaError_t launch_rows(const Args& a, int runs, int dp, int rows, bool bf16, bool i8, cudaStream_t st) {
    if (dp == 64) return rows == 16 ? rows_of_type<64, 1>(a, runs, bf16, i8, st) : rows_of_type<64, 3>(a, runs, bf16, i8, st);
    return rows == 16 ? rows_of_type<128, 1>(a, runs, bf16, i8, st) : rows_of_type<128, 2>(a, runs, bf16, i8, st);
}

cudaError_t launch_join(const Args& a, int runs, int dp, bool bf16, cudaStream_t st) {
    const dim3 grid(runs, 16);
    if (dp == 64)
        return bf16 ? launch_pdl(attend_join_kernel<kTileRows, 64, true>, grid, 256, 0, st, a, runs)
                    : launch_pdl(attend_join_kernel<kTileRows, 64, false>, grid, 256, 0, st, a, runs);
    return bf16 ? launch_pdl(attend_join_kernel<kTileRows, 128, true>, grid, 256, 0, st, a, runs)
                : launch_pdl(attend_join_kernel<kTileRows, 128, false>, grid, 256, 0, st, a, runs);
}

// Marks calls apart in the parts' flags: 64 scattered bits, never 0, so that what a
// workspace happens to hold is not taken for one.
unsigned long long next_call() {
    static std::atomic<unsigned long long> next{static_cast<unsigned long long>(
        std::chrono::system_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ull};
    return next.fetch_add(0x9E3779B97F4A7C15ull, std::memory_order_relaxed) | 1ull;
}

// Workspace: [runs][kDesc] int or [runs] flags, [runs][2][R] float2, [runs][2][R][DP] float.
struct Ws {
    size_t ml, part, all;
};
Ws workspace_layout(int runs, int rows, int dp) {
    Ws w;
    w.ml = (static_cast<size_t>(runs) * kDesc * 4 + 255) / 256 * 256;
    w.part = w.ml + (static_cast<size_t>(runs) * 2 * rows * 8 + 255) / 256 * 256;
    w.all = w.part + static_cast<size_t>(runs) * 2 * rows * dp * 4;
    return w;
}

// With 2^(l-1) < d <= 2^l and mul = ceil(2^(31+l) / d), n * mul exceeds n 2^(31+l) / d
// by less than 2^(31+l) / d for every n < 2^31: the quotient is exact.
void set_quotient(int d, uint32_t* mul, int* shift) {
    *mul = 0;
    *shift = 0;
    if (d <= 1) return;
    int l = 1;
    while ((int64_t(1) << l) < d) ++l;
    *mul = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d);
    *shift = l - 1;
}

// Rows of an item: by the rows that share a key head (the most of any sequence, if
// the caller said; else the average). Up to 16, and up to 32 of heads over 64
// elements or 48 of others, go to attend_rows_kernel, more to attend_tiles_kernel. So one chunk takes the
// sequences that decode beside it to items of 256 rows: against a call for each kind, 60 decoding sequences and a
// chunk of 64 or 512, all of 1024 to 8192 tokens, take 0.61 to 0.77 of the time (14 / 2 heads of 64; 0.9 to 1.03 of 8192)
// and 0.77 to 1.09 (16 / 8 and 32 / 8 of 128: ahead at 1024, up to 9 % behind at 8192).
int item_rows(const qm_batch& b, int group, int dp) {
    const int64_t most = b.max_new > 0 ? std::min<int64_t>(b.max_new, b.tokens) : (b.tokens + b.seqs - 1) / b.seqs;
    const int64_t rows = most * group;
    const int several = dp == 64 ? 48 : 32;
    return rows <= 16 ? 16 : rows <= several ? several : kTileRows;
}

}  // namespace
}  // namespace attend

using namespace attend;

uint32_t attend_rows_read_clear_error() {
    uint32_t v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_err_rows, sizeof(v));
    cudaMemcpyToSymbol(g_err_rows, &z, sizeof(z));
    return v;
}

size_t attend_workspace_bytes(const qm_cache& c, const qm_batch& b, int q_heads) {
    const int dp = c.dim <= 64 ? 64 : 128;
    return workspace_layout(num_sms(), item_rows(b, q_heads / c.heads, dp), dp).all;
}

cudaError_t launch_cache_attend(const qm_cache& c, const qm_batch& b, const qm_heads& q, const qm_heads& out,
                                float* lse, float scale, int64_t window, void* workspace, cudaStream_t st) {
    const int dp = c.dim <= 64 ? 64 : 128;
    const int runs = num_sms();
    const int rows = item_rows(b, q.heads / c.heads, dp);
    const bool few = rows != kTileRows;
    const Ws ws = workspace_layout(runs, rows, dp);
    uint8_t* wb = static_cast<uint8_t*>(workspace);
    Args a = {};
    a.q = static_cast<const uint16_t*>(q.data);
    a.out = static_cast<uint16_t*>(out.data);
    a.lse = lse;
    a.q_ts = q.token_stride;
    a.q_hs = q.head_stride;
    a.o_ts = out.token_stride;
    a.o_hs = out.head_stride;
    a.k = static_cast<const uint8_t*>(c.k);
    a.v = static_cast<const uint8_t*>(c.v);
    a.ks = c.k_scales;
    a.vs = c.v_scales;
    const int step = c.dtype == QM_I8 ? 16 : 8;
    a.page_stride = static_cast<uint32_t>(c.page_stride / step);
    a.head_stride = static_cast<uint32_t>(c.head_stride / step);
    a.token_stride = static_cast<uint32_t>(c.token_stride / step);
    a.sps = c.scale_page_stride;
    a.shs = c.scale_head_stride;
    a.sts = c.scale_token_stride;
    a.lens = b.lens;
    a.table = b.page_table;
    a.q_off = b.q_offsets;
    a.table_stride = b.table_stride;
    int64_t cap = 0;
    a.cap = mul_ok(b.table_width, c.page_size, &cap) && cap <= INT_MAX ? static_cast<int>(cap) : INT_MAX;
    a.seqs = b.seqs;
    a.tokens = static_cast<int>(b.tokens);
    a.each = b.q_offsets ? 0 : static_cast<int>(b.tokens / b.seqs);
    a.heads = q.heads;
    a.kv_heads = c.heads;
    a.group = q.heads / c.heads;
    a.dim = c.dim;
    a.page_size = c.page_size;
    a.pages = static_cast<int>(c.pages);
    set_quotient(c.page_size, &a.page_mul, &a.page_shift);
    set_quotient(a.group, &a.group_mul, &a.group_shift);
    a.window = static_cast<int>(std::min<int64_t>(window, INT_MAX));
    a.scale2 = scale * 1.4426950408889634f;
    a.desc = reinterpret_cast<int*>(wb);
    a.done = reinterpret_cast<unsigned long long*>(wb);
    a.call = few ? next_call() : 0;
    a.ml = reinterpret_cast<float2*>(wb + ws.ml);
    a.part = reinterpret_cast<float*>(wb + ws.part);
    const bool bf16 = q.dtype == QM_BF16, i8 = c.dtype == QM_I8;
    const cudaError_t e = few ? launch_rows(a, runs, dp, rows, bf16, i8, st) : launch_tiles(a, c, runs, bf16, st);
    if (e != cudaSuccess) return e;
    return few ? cudaSuccess : launch_join(a, runs, dp, bf16, st);
}

}  // namespace qm
