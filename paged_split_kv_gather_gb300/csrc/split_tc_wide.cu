// split_tc_wide.cu -- instantiations of the tcgen05 dense-query split kernel for
// head_dim 192 and 256: one 128-row query tile per CTA (the S/P buffers and an O
// of 192 or 256 columns fill the 512 tensor-memory columns of one CTA).
#include "split_tc_kernel.cuh"

namespace fdec {

template <typename P>
static cudaError_t launch_wide(const P& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim, bool bf16, dim3 grid,
                               cudaStream_t s, bool launch) {
    if (head_dim == 192)
        return bf16 ? launch_split_tc_one<1, 192, true>(p, tk, tv, grid, s, launch)
                    : launch_split_tc_one<1, 192, false>(p, tk, tv, grid, s, launch);
    if (head_dim == 256)
        return bf16 ? launch_split_tc_one<1, 256, true>(p, tk, tv, grid, s, launch)
                    : launch_split_tc_one<1, 256, false>(p, tk, tv, grid, s, launch);
    return cudaErrorInvalidValue;
}

cudaError_t launch_split_tc_wide(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                 bool bf16, dim3 grid, cudaStream_t s, bool launch) {
    if (!launch || p.per_head) {  // set-up (plan upload): both forms' kernel attributes
        const cudaError_t e = launch_wide(p, tk, tv, head_dim, bf16, grid, s, launch);
        if (e != cudaSuccess || launch) return e;
    }
    return launch_wide(static_cast<const SplitParams&>(p), tk, tv, head_dim, bf16, grid, s, launch);
}

size_t split_tc_wide_smem_bytes(int head_dim) {
    return head_dim == 192 ? TcLayout<1, 192>::SMEM : TcLayout<1, 256>::SMEM;
}

}  // namespace fdec
