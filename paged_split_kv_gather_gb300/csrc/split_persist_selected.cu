// split_persist_selected.cu -- instantiations of the persistent tensor-core split kernel
// for fdec_run_selected (16-bit caches, every head_dim, both stage layouts).
#include "split_persist_kernel.cuh"

namespace fdec {

cudaError_t launch_split_mma_persist_selected(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                              int head_dim, bool bf16, dim3 grid, cudaStream_t s, bool launch) {
    return launch_persist(p, tk, tv, head_dim, bf16, grid, s, launch);
}

}  // namespace fdec
