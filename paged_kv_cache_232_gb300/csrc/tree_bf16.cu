// tree_bf16.cu -- the bf16 instantiations of the tree-attention kernels, and their dispatch by type.
#include "tree_launch.cuh"

namespace pa {

extern template cudaError_t launch_tree_dtype<false>(int, int, const TreeParams&, const CUtensorMap&, const CUtensorMap&,
                                                     const CUtensorMap&, int, cudaStream_t);

cudaError_t launch_tree(int bf16, int head_dim, int unit_rows, const TreeParams& p, const CUtensorMap& k, const CUtensorMap& v,
                        const CUtensorMap& q, int ctas, cudaStream_t st) {
    return bf16 ? launch_tree_dtype<true>(head_dim, unit_rows, p, k, v, q, ctas, st)
                : launch_tree_dtype<false>(head_dim, unit_rows, p, k, v, q, ctas, st);
}

}  // namespace pa
