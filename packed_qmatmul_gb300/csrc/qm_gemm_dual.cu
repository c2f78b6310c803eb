// qm_gemm_dual.cu -- plain products of at most 128 tokens (dual layout),
// instantiated here so that they compile beside qm_gemm.cu.
#include "qm_gemm_kernel.cuh"

namespace qm {
namespace gemm {

uint32_t dual_read_clear_flag() { return read_clear_flag(); }

namespace {
struct Dual {
    Params& p;
    const WDesc& w;
    const void* x;
    cudaStream_t st;
    template <int FMT, int BITS, int GS>
    cudaError_t run() const {
        return launch_t<FMT, BITS, GS, 128, true>(p, w, x, st);
    }
};
}  // namespace

cudaError_t dispatch_dual(Params& p, const WDesc& w, const void* x, cudaStream_t st) {
    return by_format(p, w, Dual{p, w, x, st});
}

}  // namespace gemm
}  // namespace qm
