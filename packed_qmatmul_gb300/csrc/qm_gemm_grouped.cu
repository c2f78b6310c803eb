// qm_gemm_grouped.cu -- the grouped products' 128-token tiles (classic
// layout),
// instantiated here so that they compile beside qm_gemm.cu.
#include "qm_gemm_kernel.cuh"

namespace qm {
namespace gemm {

uint32_t grouped_read_clear_flag() { return read_clear_flag(); }

cudaError_t dispatch_grouped(Params& p, const WDesc& w, const void* x, cudaStream_t st) { return dispatch_tiles<128, false, false>(p, w, x, st); }

}  // namespace gemm
}  // namespace qm
