// fa_paged_launch.h -- launch of the paged attention, shared by the translation
// units that instantiate it: fa_paged.cu (16 bits) and fa_paged_e4m3.cu (8 bits).
#pragma once

#include <type_traits>

#include "fa_host.h"
#include "fa_paged_kernel.cuh"

namespace fa_launch {

// CTAs that an SM takes of the kernel for `tile_rows` query rows to a tile (8, 16, 32 or 64).
inline int paged_ctas(int D, int bits, int tile_rows)
{
    using namespace fa::paged;
    if (tile_rows == 8)
        return bits == 8 ? (D == 64 ? kCtas<64, 8, 1> : kCtas<128, 8, 1>) : (D == 64 ? kCtas<64, 16, 1> : kCtas<128, 16, 1>);
    return bits == 8 ? (D == 64 ? kCtas<64, 8, 2> : kCtas<128, 8, 2>) : (D == 64 ? kCtas<64, 16, 2> : kCtas<128, 16, 2>);
}

fa_status launch_paged(const fa::paged::Params &p, int D, bool bf16, int tile_rows, int grid, cudaStream_t s, int dev);
fa_status launch_paged_e4m3(const fa::paged::Params &p, int D, bool bf16, int tile_rows, int grid, cudaStream_t s, int dev);

// (internal linkage: see fa_launch.cuh)
namespace {

template <int D, bool BF16, int BITS, int NT, int NRB>
fa_status launch_paged_t(const fa::paged::Params &p, int grid, cudaStream_t s, int dev)
{
    namespace paged = fa::paged;
    constexpr int smem = paged::Smem<D, BITS, NT>::kBytes;
    static bool set[fa_host::kMaxDevices] = {};
    auto kern = paged::attend_kernel<D, BF16, BITS, NT, NRB>;
    const fa_status st = fa_host::allow_smem(reinterpret_cast<const void *>(kern), smem, dev, set);
    if (st != FA_OK)
        return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(paged::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    if (p.cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    if (p.cluster)
        return FA_OK;
    // right behind it (programmatic dependent launch): the join of split tiles
    cfg.gridDim = dim3((unsigned)(grid - 1));
    cfg.blockDim = dim3(paged::kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, paged::merge_kernel<D, BF16, 8 * NT * NRB>, p, grid) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

template <int BITS>
fa_status launch_paged_bits(const fa::paged::Params &p, int D, bool bf16, int tile_rows, int grid, cudaStream_t s, int dev)
{
    auto run = [&](auto d, auto b) -> fa_status {
        constexpr int DD = decltype(d)::value;
        constexpr bool BB = decltype(b)::value;
        switch (tile_rows) {
        case 8: return launch_paged_t<DD, BB, BITS, 1, 1>(p, grid, s, dev);
        case 16: return launch_paged_t<DD, BB, BITS, 2, 1>(p, grid, s, dev);
        case 32: return launch_paged_t<DD, BB, BITS, 2, 2>(p, grid, s, dev);
        default: return launch_paged_t<DD, BB, BITS, 2, 4>(p, grid, s, dev);
        }
    };
    using T = std::true_type;
    using F = std::false_type;
    if (D == 64)
        return bf16 ? run(std::integral_constant<int, 64>{}, T{}) : run(std::integral_constant<int, 64>{}, F{});
    return bf16 ? run(std::integral_constant<int, 128>{}, T{}) : run(std::integral_constant<int, 128>{}, F{});
}

}  // namespace

}  // namespace fa_launch
