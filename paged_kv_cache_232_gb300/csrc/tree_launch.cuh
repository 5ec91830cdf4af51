// tree_launch.cuh -- the tree-attention launcher, shared by its instantiation units (tree_bf16.cu, tree_f16.cu).
#pragma once
#include "tree_kernel.cuh"

namespace pa {

template <bool BF16, int D, int NR>
static cudaError_t launch_tree_t(const TreeParams& p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, int ctas,
                                 cudaStream_t st) {
    static std::atomic<unsigned long long> s_done{0};
    using C = tree::Cfg<D, NR>;
    auto kern = tree_kernel<BF16, D, NR>;
    cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, s_done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p, k, v, q);
    if (e != cudaSuccess) return e;
    // the merge: a block for 16 query rows of each CTA's cut units
    cfg.gridDim = dim3((unsigned)ctas, NR / 16);
    cfg.blockDim = dim3(tree::MERGE_THREADS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<BF16, D, NR>, p);
}

template <bool BF16, int D>
static cudaError_t tree_by_rows(int unit_rows, const TreeParams& p, const CUtensorMap& k, const CUtensorMap& v,
                                const CUtensorMap& q, int ctas, cudaStream_t st) {
    switch (unit_rows) {
        case 32: return launch_tree_t<BF16, D, 32>(p, k, v, q, ctas, st);
        case 64: return launch_tree_t<BF16, D, 64>(p, k, v, q, ctas, st);
        default: return launch_tree_t<BF16, D, 128>(p, k, v, q, ctas, st);
    }
}

template <bool BF16>
cudaError_t launch_tree_dtype(int head_dim, int unit_rows, const TreeParams& p, const CUtensorMap& k, const CUtensorMap& v,
                              const CUtensorMap& q, int ctas, cudaStream_t st) {
    if (head_dim == 64) return tree_by_rows<BF16, 64>(unit_rows, p, k, v, q, ctas, st);
    if (head_dim == 128) return tree_by_rows<BF16, 128>(unit_rows, p, k, v, q, ctas, st);
    return tree_by_rows<BF16, 256>(unit_rows, p, k, v, q, ctas, st);
}

}  // namespace pa
