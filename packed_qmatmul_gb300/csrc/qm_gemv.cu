// qm_gemv.cu -- the tensor-map GEMV's plans and entry points, and its kernels without an
// epilogue. The kernel and its pipeline are in qm_gemv_kernel.cuh.
#include "qm_gemv_kernel.cuh"

namespace qm {

uint32_t gemv_read_clear_error() { return gemv::read_clear_flag() | gemv::fused_read_clear_flag(); }

namespace gemv {

// ---------------------------------------------------------------- host planning
static uint32_t round_up(uint64_t v, uint64_t a) { return static_cast<uint32_t>((v + a - 1) / a * a); }

// Bytes of codes for `kk` values of one row.
static int64_t code_bytes(const WDesc& w, int64_t kk) {
    if (w.fmt == QM_Q8_0) return kk / 32 * 34;
    if (w.fmt == QM_MXFP4_BLOCKS) return kk / 32 * 17;
    return kk * w.bits / 8;
}

__global__ void cluster_probe_kernel() {}

// Clusters of S CTAs (`threads` threads and `smem` bytes each) that can be
// resident at once; cached per (device, S, CTAs per SM), which fixes the other two.
static int max_clusters(int S, int per_sm, int threads, size_t smem) {
    static int cache[64][9][2];
    int dev = 0;
    cudaGetDevice(&dev);
    if (S <= 1) return num_sms();
    int* slot = (dev >= 0 && dev < 64) ? &cache[dev][S][per_sm - 1] : nullptr;
    if (slot && *slot > 0) return *slot;
    int n = 0;
    cudaFuncSetAttribute(cluster_probe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         static_cast<int>(smem));
    cudaFuncSetAttribute(cluster_probe_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S * 64);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = S;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, cluster_probe_kernel, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = num_sms() / S;
    }
    if (slot) *slot = n;
    return n;
}

// A plan for S CTAs per cluster (splitting k) and `per_sm` CTAs per SM, the
// matrix getting `share` of the GPU's CTA slots (other chunks of a grouped
// product take the rest).
static bool plan_for(const WDesc& w, int64_t M, int S, int per_sm, Plan* out, double share = 1.0) {
    if (w.k % S) return false;
    const int64_t kr = w.k / S;
    if (kr % w.gs) return false;
    const int NT = M > 8 ? 2 : 1;
    const int64_t cseg = code_bytes(w, kr);
    if (cseg % 16 || w.code_row_bytes % 16) return false;
    int64_t sseg = 0;
    if (w.fmt == QM_AFFINE) sseg = kr / w.gs * 2;
    if (w.fmt == QM_MXFP4) sseg = kr / 32;
    // scales by 2-d boxes of this CTA's part, where a box can take it; else
    // whole rows as a span (k whole, or a part that is no 16-byte multiple)
    const bool boxes = S > 1 && sseg % 16 == 0 && sseg <= 256 && w.scale_row_bytes % 16 == 0;
    if (S > 1 && !boxes && M > 1) return false;  // whole scale rows per rank: measured slower with several tokens
    Params& p = out->p;
    p = Params{};
    p.code_seg = static_cast<uint32_t>(cseg);
    p.nbox = static_cast<uint32_t>((cseg + 127) / 128);
    p.scale_seg = static_cast<uint32_t>(sseg);
    p.scale_span = boxes ? 0 : 1;
    p.scale_pitch = static_cast<uint32_t>(boxes ? sseg : w.scale_row_bytes);
    const uint32_t codes_bytes = p.nbox * kRows * 128;
    const uint32_t sc_bytes = round_up(kRows * (sseg ? p.scale_pitch : 0), 128);
    p.off_scales = codes_bytes;
    p.off_biases = codes_bytes + sc_bytes;
    p.stage_bytes = round_up(codes_bytes + sc_bytes * (w.fmt == QM_AFFINE ? 2 : 1), 1024);  // swizzled boxes
    const int64_t groups = kr / w.gs;
    const int64_t budget = (per_sm == 2 ? (max_smem_optin() + 1024) / 2 : max_smem_optin()) - 1024;
    // work split: clusters of S CTAs, per_sm CTAs to an SM
    p.n_stages = (w.n + kRows - 1) / kRows;
    const int cw = per_sm == 1 ? 16 : 8;
    int64_t G = std::max<int64_t>(1, static_cast<int64_t>(num_sms() * per_sm * share) / S);
    if (S > 1) G = std::max<int64_t>(1, std::min<int64_t>(G, max_clusters(S, per_sm, kThreadsOf(cw), budget)));
    G = std::min<int64_t>(G, p.n_stages);
    const int64_t spc = (p.n_stages + G - 1) / G;
    G = (p.n_stages + spc - 1) / spc;
    // shared memory: fixed part, then as many stage slots as fit
    auto layout = [&]() -> int64_t {
        p.off_tokscale = 512;  // [16] 2^-E, [16] unused, [16] max |x| bits
        p.off_tok = p.off_tokscale + 256;
        p.off_xfrag = round_up(p.off_tok + groups * 16 * 8, 128);
        // B fragments: 16 bytes per k value and token tile, or 2 for exactly one token
        const uint64_t xfrag_bytes = M == 1 ? static_cast<uint64_t>(kr) * 2 : static_cast<uint64_t>(kr) * 16 * NT;
        const uint64_t red_bytes = M == 1 ? static_cast<uint64_t>(cw) * 2 * 32 * 4
                                          : static_cast<uint64_t>(cw) * 2 * 2 * NT * 32 * 4 * 4;
        const uint64_t partial_bytes = S > 1 ? static_cast<uint64_t>(spc) * kRows * 16 * 4 : 0;
        const uint64_t xraw_bytes = static_cast<uint64_t>(M) * kr * 2;
        // The raw activations are dead once the fragments are built (a barrier of
        // all consumers), so the team sums, which start after it, reuse their
        // room; with a k split the stages' partial sums take that room instead.
        p.off_xraw = round_up(p.off_xfrag + xfrag_bytes, 128);
        uint64_t end;
        if (S == 1) {
            p.off_red = p.off_xraw;
            end = p.off_xraw + std::max(xraw_bytes, red_bytes);
        } else {
            p.off_red = round_up(p.off_xraw + std::max(partial_bytes, xraw_bytes), 128);
            end = p.off_red + red_bytes;
        }
        // split k: rank 0 receives the other ranks' sums apart from everything it may still be reading
        const uint64_t recv_bytes = S > 1 ? static_cast<uint64_t>(S - 1) * spc * kRows * M * 4 : 0;
        p.off_recv = round_up(end, 128);
        p.off_stages = round_up(p.off_recv + recv_bytes, 1024);
        const int64_t room = budget - p.off_stages;
        return std::min<int64_t>(std::min<int64_t>(kMaxStages, room / p.stage_bytes), std::max<int64_t>(2, spc));
    };
    const int64_t nst = layout();
    if (nst < 2) return false;
    // teams: one per stage a CTA can hold in flight, each warp at least one group
    int teams = 1;
    while (teams * 2 <= kMaxTeams && teams * 2 <= spc && teams * 2 <= nst) teams *= 2;
    int T = cw / teams;
    while (T > 1 && T > groups && cw / (T / 2) <= kMaxTeams) T /= 2;
    p.team = T;
    p.nstage = static_cast<uint32_t>(nst);
    p.S = S;
    p.krange = kr;
    p.stages_per_cluster = static_cast<int>(spc);
    out->S = S;
    out->cw = cw;
    out->grid = G * S;
    out->smem = p.off_stages + nst * p.stage_bytes;
    out->ok = true;
    return true;
}

// Pick the k split and CTAs per SM: least per-CTA work (stages x k range,
// halved where two CTAs share an SM) plus a fixed cost per extra rank of a k
// split, then fewest splits; a plan that keeps three stages in flight beats
// one that cannot.
static Plan make_plan(const WDesc& w, int64_t M, double share = 1.0) {
    Plan best;
    double best_cost = 1e300;
    for (int per_sm = 2; per_sm >= 1; --per_sm)
        for (int S = 1; S <= 8; ++S) {
            Plan pl;
            if (!plan_for(w, M, S, per_sm, &pl, share)) continue;
            const bool shallow = pl.p.nstage < 3 && pl.p.stages_per_cluster >= 3;
            // one token: each extra rank of a k split costs a fixed hand-off
            // (its partial sums reach rank 0 through distributed shared memory),
            // measured on GB300 to be worth about 1024 k values of one stage; with
            // more tokens the activation work per CTA favors the wider splits
            const double cost = static_cast<double>(pl.p.stages_per_cluster) * pl.p.krange / per_sm *
                                    (1.0 + 0.03 * (S - 1)) * (shallow ? 2.0 : 1.0) +
                                (M == 1 ? 1024.0 * (S - 1) : 0.0);
            if (cost < best_cost * 0.999) {
                best_cost = cost;
                best = pl;
            }
        }
    return best;
}

}  // namespace gemv

namespace gemv {

// A plan with the weight's fields and tensor maps filled in: everything of a
// launch that depends only on the weight descriptor, M and the device.
struct Prepared {
    Plan pl;
    bool maps = false;  // the driver encoded the tensor maps (else the plain kernel runs)
};

static void prepare(const WDesc& w, int64_t M, Prepared* out) {
    out->pl = make_plan(w, M);
    out->maps = false;
    if (!out->pl.ok) return;
    Params& p = out->pl.p;
    p.codes = w.codes;
    p.scales = w.scales;
    p.biases = w.biases;
    p.n = w.n;
    p.k = w.k;
    p.M = static_cast<int>(M);
    p.sdt = w.sdt;
    p.code_row_bytes = w.code_row_bytes;
    p.scale_row_bytes = w.scale_row_bytes;
    p.static_w = w.is_static ? 1 : 0;
    bool maps = make_tmap_2d(&p.tm_codes, w.codes, w.code_row_bytes, w.n, w.code_row_bytes, 128, kRows, true);
    if (maps && !p.scale_span && p.scale_seg) {
        maps = make_tmap_2d(&p.tm_scales, w.scales, w.scale_row_bytes, w.n, w.scale_row_bytes, p.scale_seg,
                            kRows, false);
        if (maps && w.biases)
            maps = make_tmap_2d(&p.tm_biases, w.biases, w.scale_row_bytes, w.n, w.scale_row_bytes, p.scale_seg,
                                kRows, false);
    }
    out->maps = maps;
}

// What a prepared plan depends on, with no padding bytes (compared bytewise).
struct PlanKey {
    const void* codes;
    const void* scales;
    const void* biases;
    int64_t n, k, code_row_bytes, scale_row_bytes;
    int32_t fmt, bits, gs, sdt, M, is_static, dev, unused;
};
static_assert(sizeof(PlanKey) == 3 * 8 + 4 * 8 + 8 * 4, "PlanKey has padding");

struct PlanKeyHash {
    size_t operator()(const PlanKey& k) const {
        uint64_t h = 1469598103934665603ull;  // FNV-1a over the key's bytes
        const unsigned char* b = reinterpret_cast<const unsigned char*>(&k);
        for (size_t i = 0; i < sizeof k; ++i) h = (h ^ b[i]) * 1099511628211ull;
        return static_cast<size_t>(h);
    }
};
struct PlanKeyEq {
    bool operator()(const PlanKey& a, const PlanKey& b) const { return std::memcmp(&a, &b, sizeof a) == 0; }
};

// Prepared plans, memoized per calling thread: a decode step calls the same
// few hundred (weight, M) pairs over and over, and planning plus tensor-map
// encoding costs microseconds of host time per call. Only host-side launch
// metadata is kept (at most kMaxPlans entries, then the table starts over);
// no device memory is held.
static const Prepared* prepared(const WDesc& w, int64_t M, cudaError_t* err = nullptr) {
    PlanKey key;
    std::memset(&key, 0, sizeof key);
    key.codes = w.codes;
    key.scales = w.scales;
    key.biases = w.biases;
    key.n = w.n;
    key.k = w.k;
    key.code_row_bytes = w.code_row_bytes;
    key.scale_row_bytes = w.scale_row_bytes;
    key.fmt = w.fmt;
    key.bits = w.bits;
    key.gs = w.gs;
    key.sdt = w.sdt;
    key.M = static_cast<int32_t>(M);
    key.is_static = w.is_static ? 1 : 0;
    const cudaError_t e = cudaGetDevice(&key.dev);
    if (e != cudaSuccess) {
        if (err) *err = e;
        return nullptr;
    }
    constexpr size_t kMaxPlans = 4096;
    thread_local std::unordered_map<PlanKey, Prepared, PlanKeyHash, PlanKeyEq> table;
    auto it = table.find(key);
    if (it != table.end()) return &it->second;
    if (table.size() >= kMaxPlans) table.clear();
    Prepared& pr = table[key];
    prepare(w, M, &pr);
    return &pr;
}

}  // namespace gemv

bool gemv_supported(const WDesc& w, int64_t M) {
    if (M < 1 || M > 16 || w.ndim != 2 || !pipelined_format(w)) return false;
    const gemv::Prepared* pr = gemv::prepared(w, M);
    return pr && pr->pl.ok;
}

qm_status launch_gemv(const WDesc& w, const Epi& ep, const void* x, int64_t M, void* y, cudaStream_t st) {
    using namespace gemv;
    cudaError_t err = cudaSuccess;
    const Prepared* pr = prepared(w, M, &err);
    if (!pr) return cuda_fail(err, "cudaGetDevice");
    if (!pr->pl.ok) return fail(QM_ENOTSUP, "w: no decode plan for this shape");
    if (!pr->maps) {  // the driver refused a descriptor for this shape: the plain kernel
        cudaError_t e = launch_apply_simple(w, ep, x, M, y, st);
        return e == cudaSuccess ? QM_OK : cuda_fail(e, "apply launch");
    }
    Plan pl = pr->pl;
    Params& p = pl.p;
    p.x = static_cast<const uint16_t*>(x);
    p.y = static_cast<uint16_t*>(y);
    p.ep = ep;
    const int ntk = M > 8 ? 2 : (M > 1 ? 1 : 0);
    const cudaError_t e = ep.on ? dispatch_fused(w, pl, ntk, st) : dispatch<false>(w, pl, ntk, st);
    if (e != cudaSuccess) return cuda_fail(e, "gemv launch");
    return QM_OK;
}

// ---------------------------------------------------------------- grouped (apply_experts)
// Chunks of Q routed positions of one expert, each a decode product over that
// expert's [n, k] matrix. The chunk list lives on the device (the routing
// offsets), so the grid covers the most chunks P positions can make; slots
// past the last chunk exit at once.
namespace gemv {

static int grouped_q(int64_t P, int64_t E) { return P <= 8 * E ? 8 : 16; }

static bool grouped_plan(const WDesc& w, int64_t P, Plan* out, int64_t* slots) {
    const int64_t E = w.shape[0];
    if (w.ndim != 3 || E < 1 || P < 1 || E * w.n >= (int64_t(1) << 31) || !pipelined_format(w)) return false;
    if ((w.n * w.scale_row_bytes) % 16) return false;  // each expert's scales start 16-byte aligned
    const int Q = grouped_q(P, E);
    *slots = std::min<int64_t>(P, P / Q + E);  // sum over experts of ceil(count / Q) is below P/Q + E
    // chunks expected when ids spread evenly: every expert used, about half a chunk extra each
    const int64_t est = std::max<int64_t>(1, std::min<int64_t>(*slots, (P + Q - 1) / Q + std::min(E, P) / 2));
    *out = make_plan(w, Q, 1.0 / static_cast<double>(est));
    return out->ok;
}

}  // namespace gemv

bool gemv_grouped_supported(const WDesc& w, int64_t P) {
    gemv::Plan pl;
    int64_t slots = 0;
    return gemv::grouped_plan(w, P, &pl, &slots);
}

qm_status launch_gemv_grouped(const WDesc& w, const Epi& ep, const int32_t* offsets, const int32_t* perm, int64_t P,
                              int xdiv, const void* x, void* y, cudaStream_t st) {
    using namespace gemv;
    Plan pl;
    int64_t slots = 0;
    if (!grouped_plan(w, P, &pl, &slots)) return fail(QM_ENOTSUP, "w: no grouped decode plan for this shape");
    const int64_t E = w.shape[0];
    const int Q = grouped_q(P, E);
    Params& p = pl.p;
    p.codes = w.codes;
    p.scales = w.scales;
    p.biases = w.biases;
    p.x = static_cast<const uint16_t*>(x);
    p.y = static_cast<uint16_t*>(y);
    p.ep = ep;
    p.n = w.n;
    p.k = w.k;
    p.M = Q;
    p.sdt = w.sdt;
    p.code_row_bytes = w.code_row_bytes;
    p.scale_row_bytes = w.scale_row_bytes;
    p.static_w = 0;
    p.g_off = offsets;
    p.g_perm = perm;
    p.g_E = static_cast<int>(E);
    p.g_Q = Q;
    p.g_xdiv = xdiv;
    p.g_wclusters = static_cast<int>(pl.grid / pl.S);
    const int64_t rows = E * w.n;
    bool maps = make_tmap_2d(&p.tm_codes, w.codes, w.code_row_bytes, rows, w.code_row_bytes, 128, kRows, true);
    if (maps && !p.scale_span && p.scale_seg) {
        maps = make_tmap_2d(&p.tm_scales, w.scales, w.scale_row_bytes, rows, w.scale_row_bytes, p.scale_seg,
                            kRows, false);
        if (maps && w.biases)
            maps = make_tmap_2d(&p.tm_biases, w.biases, w.scale_row_bytes, rows, w.scale_row_bytes, p.scale_seg,
                                kRows, false);
    }
    if (!maps) return fail(QM_ENOTSUP, "w: no tensor map for the grouped decode product");
    if (pl.grid * slots >= (int64_t(1) << 31)) return fail(QM_ENOTSUP, "ids: too many positions for one launch");
    if (pl.S > 1) {
        pl.grid *= slots;
    } else {
        // a CTA for every place and every chunk there may be; where the chunks may take more than
        // half the places, three waves, so that they can be cut finer (CTAs past the last share exit)
        p.g_resident = num_sms() * (pl.cw == 16 ? 1 : 2);
        pl.grid = std::max<int64_t>(slots, p.g_resident * (2 * slots > p.g_resident ? 3 : 1));
    }
    const bool two = Q > 8;
    const cudaError_t e = ep.on ? dispatch_fused(w, pl, two ? 2 : 1, st) : dispatch<false>(w, pl, two ? 2 : 1, st);
    if (e != cudaSuccess) return cuda_fail(e, "grouped gemv launch");
    return QM_OK;
}

}  // namespace qm
