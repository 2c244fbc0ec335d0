// fa_bwd_pass.cuh -- launch of one backward pass, shared by the translation
// units that instantiate them: fa_bwd.cu and fa_bwd_sink.cu.
#pragma once

#include <mutex>
#include <utility>

#include "fa_bwd_kernel.cuh"
#include "fa_bwd_launch.h"

namespace fa_launch {

// (internal linkage: see fa_launch.cuh)
namespace {

constexpr int kMaxDev = 64;

// Launch `kern` on `stream` allowing programmatic dependent launch: it may
// start while the previous kernel on the stream finishes, and waits for that
// kernel's completion with griddepcontrol.wait before reading its results.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args &&...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <int D, bool BF16, bool CAUSAL, bool KV, bool FQ = false, class P = fa::bwd::Params>
fa_status launch_pass(const CUtensorMap &r0, const CUtensorMap &r1, const CUtensorMap &s0, const CUtensorMap &s1,
                      const CUtensorMap &dq, const P &p, int grid, cudaStream_t stream, int dev)
{
    static std::mutex mu;
    static bool attr_set[kMaxDev] = {};
    auto kern = fa::bwd::fa_bwd_sm103<D, BF16, CAUSAL, KV, FQ, P>;
    constexpr int smem = fa::bwd::BCfg<D, KV, FQ>::kSmem;
    if (dev < 0 || dev >= kMaxDev)
        return FA_ERR_UNSUPPORTED_DEVICE;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
                cudaGetLastError();
                return FA_ERR_CUDA;
            }
            attr_set[dev] = true;
        }
    }
    // right behind the previous kernel (programmatic dependent launch): see fa_bwd_sm103
    if (launch_dependent(kern, dim3(grid), dim3(FQ ? fa::bwd::kThreadsFused : fa::bwd::kThreads), smem, stream, r0, r1,
                         s0, s1, dq, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

}  // namespace

}  // namespace fa_launch
