// tree_f16.cu -- the fp16 instantiations of the tree-attention kernels.
#include "tree_launch.cuh"

namespace pa {

template cudaError_t launch_tree_dtype<false>(int, int, const TreeParams&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, int, cudaStream_t);

}  // namespace pa
