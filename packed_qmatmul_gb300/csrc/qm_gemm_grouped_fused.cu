// qm_gemm_grouped_fused.cu -- the grouped products' 128-token tiles (classic
// layout) with an epilogue,
// instantiated here so that they compile beside qm_gemm.cu.
#include "qm_gemm_kernel.cuh"

namespace qm {
namespace gemm {

uint32_t grouped_fused_read_clear_flag() { return read_clear_flag(); }

cudaError_t dispatch_grouped_fused(Params& p, const WDesc& w, const void* x, cudaStream_t st) { return dispatch_tiles<128, false, true>(p, w, x, st); }

}  // namespace gemm
}  // namespace qm
