// split_d128.cu -- split-kernel instantiations for head_dim 128.
#include "split_kernel.cuh"

namespace fdec {

cudaError_t launch_split_d128(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch) {
    return launch_split_d<128>(p, tk, tv, rc, bf16, grid, s, launch);
}

}  // namespace fdec
