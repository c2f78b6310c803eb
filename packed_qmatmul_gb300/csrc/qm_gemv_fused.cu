// qm_gemv_fused.cu -- the tensor-map GEMV's kernels with an epilogue, instantiated
// here so that they compile beside qm_gemv.cu.
#include "qm_gemv_kernel.cuh"

namespace qm {
namespace gemv {

uint32_t fused_read_clear_flag() { return read_clear_flag(); }

cudaError_t dispatch_fused(const WDesc& w, const Plan& pl, int ntk, cudaStream_t st) { return dispatch<true>(w, pl, ntk, st); }

}  // namespace gemv
}  // namespace qm
