// qm_gemm_fused.cu -- 256-token tiles with an epilogue,
// instantiated here so that they compile beside qm_gemm.cu.
#include "qm_gemm_kernel.cuh"

namespace qm {
namespace gemm {

uint32_t wide_fused_read_clear_flag() { return read_clear_flag(); }

cudaError_t dispatch_wide_fused(Params& p, const WDesc& w, const void* x, cudaStream_t st) { return dispatch_tiles<256, false, true>(p, w, x, st); }

}  // namespace gemm
}  // namespace qm
