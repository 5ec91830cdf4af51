// latent.cu -- instantiations of the latent-cache attention kernels.
#include "latent_pair_kernel.cuh"

namespace pa {

template <bool BF16, int DL, int NR>
static cudaError_t launch_latent_t(const LatentParams& p, const CUtensorMap& tmC, const CUtensorMap& tmQ, int ctas,
                                   cudaStream_t st) {
    static std::atomic<unsigned long long> s_done{0};
    cudaError_t e;
    if constexpr (NR == 128) {
        using C = latp::Cfg<DL>;
        auto kern = latent_pair_kernel<BF16, DL>;
        if ((e = smem_limit_once(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, s_done)) != cudaSuccess) return e;
        e = launch_dependent(kern, (unsigned)ctas, C::THREADS, C::SMEM_BYTES, st, p, tmC, tmQ);
    } else {
        using C = lat::Cfg<DL, NR>;
        auto kern = latent_kernel<BF16, DL, NR>;
        if ((e = smem_limit_once(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, s_done)) != cudaSuccess) return e;
        e = launch_dependent(kern, (unsigned)ctas, C::THREADS, C::SMEM_BYTES, st, p, tmC, tmQ);
    }
    if (e != cudaSuccess) return e;
    // the merge: a block for 16 query rows of each range
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(NR == 128 ? ctas / 2 : ctas), NR / 16);
    cfg.blockDim = dim3(lat::merge_threads(NR));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_merge_kernel<BF16, DL, NR>, p);
}

template <bool BF16, int DL>
static cudaError_t by_rows(int unit_rows, const LatentParams& p, const CUtensorMap& c, const CUtensorMap& q, int ctas,
                           cudaStream_t st) {
    switch (unit_rows) {
        case 16: return launch_latent_t<BF16, DL, 16>(p, c, q, ctas, st);
        case 32: return launch_latent_t<BF16, DL, 32>(p, c, q, ctas, st);
        case 64: return launch_latent_t<BF16, DL, 64>(p, c, q, ctas, st);
        default: return launch_latent_t<BF16, DL, 128>(p, c, q, ctas, st);
    }
}

cudaError_t launch_latent(int bf16, int latent_dim, int unit_rows, const LatentParams& p, const CUtensorMap& tmC,
                          const CUtensorMap& tmQ, int ctas, cudaStream_t st) {
    if (latent_dim == 512)
        return bf16 ? by_rows<true, 512>(unit_rows, p, tmC, tmQ, ctas, st) : by_rows<false, 512>(unit_rows, p, tmC, tmQ, ctas, st);
    return bf16 ? by_rows<true, 256>(unit_rows, p, tmC, tmQ, ctas, st) : by_rows<false, 256>(unit_rows, p, tmC, tmQ, ctas, st);
}

}  // namespace pa
