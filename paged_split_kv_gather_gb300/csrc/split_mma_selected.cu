// split_mma_selected.cu -- instantiations of the tensor-core split kernel for
// fdec_run_selected (the head_dims and caches of split_mma.cu).
#include "split_mma_kernel.cuh"

namespace fdec {

cudaError_t launch_split_mma_selected(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                      bool bf16, bool kv8, dim3 grid, cudaStream_t s, bool launch) {
    return launch_mma(p, tk, tv, head_dim, bf16, kv8, grid, s, launch);
}

}  // namespace fdec
