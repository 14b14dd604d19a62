// split_persist.cu -- instantiations of the persistent tensor-core split kernel
// (16-bit caches, every head_dim), each in two stage layouts: box-major for pages of
// 8 or 16 tokens (one TMA box per page), region-major for every other page size.
#include "split_persist_kernel.cuh"

namespace fdec {

cudaError_t launch_split_mma_persist(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                     bool bf16, dim3 grid, cudaStream_t s, bool launch) {
    if (!launch || p.per_head) {  // set-up (plan upload): both forms' kernel attributes
        const cudaError_t e = launch_split_mma_persist_selected(p, tk, tv, head_dim, bf16, grid, s, launch);
        if (e != cudaSuccess || launch) return e;
    }
    return launch_persist(static_cast<const SplitParams&>(p), tk, tv, head_dim, bf16, grid, s, launch);
}

}  // namespace fdec
