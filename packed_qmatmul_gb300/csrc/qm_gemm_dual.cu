// qm_gemm_dual.cu -- plain products of at most 128 tokens (dual
// layout),
// instantiated here so that they compile beside qm_gemm.cu.
#include "qm_gemm_kernel.cuh"

namespace qm {
namespace gemm {

uint32_t dual_read_clear_flag() { return read_clear_flag(); }

cudaError_t dispatch_dual(Params& p, const WDesc& w, const void* x, cudaStream_t st) { return dispatch_tiles<128, true, false>(p, w, x, st); }

}  // namespace gemm
}  // namespace qm
