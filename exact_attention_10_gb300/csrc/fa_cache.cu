// fa_cache.cu -- the 4-bit key/value cache's entry points (include/fa.h):
// argument checks, kernel choice and launch; the kernels are in
// fa_cache_kernel.cuh.
#include "fa.h"

#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "fa_cache_kernel.cuh"
#include "fa_cache_rows.h"
#include "fa_host.h"

namespace {

using fa_host::Arg;
namespace cache = fa::cache;

fa_status launched()
{
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// What every cache call checks of its sizes.
bool sizes_ok(int B, int Hkv, long long N, int C, int D, fa_dtype dtype)
{
    if (dtype != FA_BF16 && dtype != FA_FP16)
        return false;
    if (D != 64 && D != 128)
        return false;
    if (B < 1 || Hkv < 1 || N < 1 || C < 1)
        return false;
    const long long BH = (long long)B * Hkv;
    return BH <= fa_host::kMaxRows && BH * N <= fa_host::kMaxRows && BH * C <= fa_host::kMaxRows;
}

bool queries_ok(int B, int H, int Hkv, int Nq)
{
    if (H < 1 || Hkv < 1 || H % Hkv != 0 || Nq < 1)
        return false;
    return (long long)B * H <= fa_host::kMaxRows && (long long)B * H * Nq <= fa_host::kMaxRows;
}

// Query rows per tile: 8 where a key head has no more, else 16 (a tile's rows
// share the unpacked codes, but their accumulators fill the registers of one CTA
// per SM instead of two: 108 us for 16 rows against 79 for 8, see
// fa_cache_kernel.cuh, which also says what more rows cost).
int row_tiles(int rows)
{
    return rows <= 8 ? 1 : 2;
}

int row_blocks(int rows, int nt)
{
    return (rows + 8 * nt - 1) / (8 * nt);
}

int attend_grid(int sms, int nt)
{
    return sms * (nt == 1 ? 2 : 1);
}

// Whether tiles (sequence, key head, row block) are left whole: cutting them up
// to share the tokens out evenly costs a second launch, which joins the parts.
// Measured, whole against cut, D = 128, H / Hkv = 4, us: capacity 1024: 7.9
// against 7.7 for 8 tiles, 7.9 / 10.2 for 64, 21.0 / 26.7 for 512; 2048: 11.0 /
// 9.1, 11.4 / 15.5, 35.7 / 40.3; 4096: 17.7 / 12.3, 18.2 / 19.0, 60.5 / 61.1 --
// and beyond, a batch of different lengths is better cut.
bool whole_tiles(long long tiles, int C)
{
    return C <= 1024 || (C <= 2048 && tiles >= 64);
}

size_t attend_workspace(int sms, int nt, long long tiles, int C, int D)
{
    if (whole_tiles(tiles, C))
        return 0;
    return (size_t)2 * attend_grid(sms, nt) * 8 * nt * (D * sizeof(float) + sizeof(float2));
}

template <int D, bool BF16, int NT>
fa_status launch_attend_t(const cache::Params &p, int sms, cudaStream_t s, int dev)
{
    constexpr int smem = cache::AttendSmem<D, NT>::kBytes;
    static bool set[fa_host::kMaxDevices] = {};
    const fa_status st = fa_host::allow_smem(reinterpret_cast<const void *>(&cache::attend_kernel<D, BF16, NT>), smem, dev, set);
    if (st != FA_OK)
        return st;
    const long long tiles = (long long)p.B * p.Hkv * p.RB;
    const int grid = p.whole && tiles < attend_grid(sms, NT) ? (int)tiles : attend_grid(sms, NT);
    cache::attend_kernel<D, BF16, NT><<<grid, cache::kThreads, smem, s>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return FA_ERR_CUDA;
    if (p.whole)
        return FA_OK;
    // right behind it (programmatic dependent launch): the join of split tiles
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(grid - 1));
    cfg.blockDim = dim3(cache::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache::merge_kernel<D, BF16, NT>, p, grid) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

template <int D, bool BF16, int NT>
fa_status launch_weights_t(const cache::Params &p, int sms, cudaStream_t s, int dev)
{
    constexpr int smem = cache::kWarps * cache::kStages * cache::Layout<D>::kKeyStage;
    static bool set[fa_host::kMaxDevices] = {};
    const fa_status st = fa_host::allow_smem(reinterpret_cast<const void *>(&cache::weights_kernel<D, BF16, NT>), smem, dev, set);
    if (st != FA_OK)
        return st;
    cache::weights_kernel<D, BF16, NT><<<sms * 2, cache::kThreads, smem, s>>>(p);
    return launched();
}

}  // namespace

extern "C" fa_status fa_cache_append(void *Kc, void *Kp, void *Vc, void *Vp, const void *K, const void *V,
                                     const int *start, const int *count, int B, int Hkv, int N, int C, int D,
                                     fa_dtype dtype, fa_stream_t stream)
{
    if (!sizes_ok(B, Hkv, N, C, D, dtype))
        return FA_ERR_INVALID_VALUE;
    const size_t rows = (size_t)B * Hkv * N, held = (size_t)B * Hkv * C;
    const Arg args[8] = {{Kc, held * D / 2, true, 16}, {Kp, held * 4, true, 4}, {Vc, held * D / 2, true, 16},
                         {Vp, held * 4, true, 4}, {K, rows * D * 2, false, 16}, {V, rows * D * 2, false, 16},
                         {start, (size_t)B * 4, false, 4}, {count, (size_t)B * 4, false, 4}};
    int dev;
    const fa_host::DeviceInfo *di;
    const fa_status st = fa_host::check_args(args, count ? 8 : 7, &dev, &di);
    if (st != FA_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto run = [&](auto kern, int tpr) {
        const size_t blocks = (rows * tpr + cache::kThreads - 1) / cache::kThreads;
        kern<<<(unsigned)blocks, cache::kThreads, 0, s>>>(
            static_cast<const uint16_t *>(K), static_cast<const uint16_t *>(V), static_cast<uint8_t *>(Kc),
            static_cast<uint32_t *>(Kp), static_cast<uint8_t *>(Vc), static_cast<uint32_t *>(Vp), start, count, Hkv, N, C,
            (uint32_t)rows);
        return launched();
    };
    if (D == 64)
        return dtype == FA_BF16 ? run(cache::append_kernel<64, true>, 4) : run(cache::append_kernel<64, false>, 4);
    return dtype == FA_BF16 ? run(cache::append_kernel<128, true>, 8) : run(cache::append_kernel<128, false>, 8);
}

extern "C" fa_status fa_cache_read(const void *Kc, const void *Kp, const void *Vc, const void *Vp, void *K, void *V,
                                   const int *start, const int *count, int B, int Hkv, int N, int C, int D,
                                   fa_dtype dtype, fa_stream_t stream)
{
    if (!sizes_ok(B, Hkv, N, C, D, dtype))
        return FA_ERR_INVALID_VALUE;
    const size_t rows = (size_t)B * Hkv * N, held = (size_t)B * Hkv * C;
    const Arg args[8] = {{Kc, held * D / 2, false, 16}, {Kp, held * 4, false, 4}, {Vc, held * D / 2, false, 16},
                         {Vp, held * 4, false, 4}, {K, rows * D * 2, true, 16}, {V, rows * D * 2, true, 16},
                         {start, (size_t)B * 4, false, 4}, {count, (size_t)B * 4, false, 4}};
    int dev;
    const fa_host::DeviceInfo *di;
    const fa_status st = fa_host::check_args(args, count ? 8 : 7, &dev, &di);
    if (st != FA_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto run = [&](auto kern, int tpr) {
        const size_t blocks = (rows * tpr + cache::kThreads - 1) / cache::kThreads;
        kern<<<(unsigned)blocks, cache::kThreads, 0, s>>>(
            static_cast<const uint8_t *>(Kc), static_cast<const uint32_t *>(Kp), static_cast<const uint8_t *>(Vc),
            static_cast<const uint32_t *>(Vp), static_cast<uint16_t *>(K), static_cast<uint16_t *>(V), start, count, Hkv, N,
            C, (uint32_t)rows);
        return launched();
    };
    if (D == 64)
        return dtype == FA_BF16 ? run(cache::read_kernel<64, true>, 8) : run(cache::read_kernel<64, false>, 8);
    return dtype == FA_BF16 ? run(cache::read_kernel<128, true>, 16) : run(cache::read_kernel<128, false>, 16);
}

extern "C" fa_status fa_cache_workspace(int B, int H, int Hkv, int Nq, int C, int D, size_t *bytes)
{
    if (!bytes || !sizes_ok(B, Hkv, 1, C, D, FA_BF16) || !queries_ok(B, H, Hkv, Nq))
        return FA_ERR_INVALID_VALUE;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_UNSUPPORTED_DEVICE;
    }
    const fa_host::DeviceInfo *di = fa_host::device_info(dev);
    if (!di || !di->supported)
        return FA_ERR_UNSUPPORTED_DEVICE;
    const int rows = (H / Hkv) * Nq, nt = row_tiles(rows);
    *bytes = attend_workspace(di->sms, nt, (long long)B * Hkv * row_blocks(rows, nt), C, D);
    return FA_OK;
}

extern "C" fa_status fa_cache_fwd(const void *Q, const void *Kc, const void *Kp, const void *Vc, const void *Vp,
                                  const int *lens, void *O, float *LSE, int B, int H, int Hkv, int Nq, int C, int D,
                                  int window_left, int sinks, float scale, fa_dtype dtype, void *workspace,
                                  size_t workspace_bytes, fa_stream_t stream)
{
    if (!sizes_ok(B, Hkv, 1, C, D, dtype) || !queries_ok(B, H, Hkv, Nq) || sinks < 0)
        return FA_ERR_INVALID_VALUE;
    if (!std::isfinite(scale) || !(scale > 0.f))
        return FA_ERR_INVALID_VALUE;
    const size_t qrows = (size_t)B * H * Nq, held = (size_t)B * Hkv * C;
    const Arg args[9] = {{Q, qrows * D * 2, false, 16}, {Kc, held * D / 2, false, 16}, {Kp, held * 4, false, 4},
                         {Vc, held * D / 2, false, 16}, {Vp, held * 4, false, 4}, {lens, (size_t)B * 4, false, 4},
                         {O, qrows * D * 2, true, 16}, {LSE, qrows * 4, true, 4}, {workspace, workspace_bytes, true, 16}};
    int dev;
    const fa_host::DeviceInfo *di;
    const fa_status st = fa_host::check_args(args, workspace ? 9 : 8, &dev, &di);
    if (st != FA_OK)
        return st;
    const int rows = (H / Hkv) * Nq, nt = row_tiles(rows);
    const int blocks = row_blocks(rows, nt);
    const size_t need = attend_workspace(di->sms, nt, (long long)B * Hkv * blocks, C, D);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return FA_ERR_INVALID_VALUE;
    cache::Params p{};
    p.kc = static_cast<const uint8_t *>(Kc);
    p.kp = static_cast<const uint32_t *>(Kp);
    p.vc = static_cast<const uint8_t *>(Vc);
    p.vp = static_cast<const uint32_t *>(Vp);
    p.q = Q;
    p.o = O;
    p.lse = LSE;
    p.lens = lens;
    p.B = B;
    p.Hkv = Hkv;
    p.C = C;
    p.rows = rows;
    p.Nq = Nq;
    p.RB = blocks;
    p.left = window_left < 0 ? -1 : window_left;
    p.sinks = sinks;
    p.qk2 = scale * cache::kLog2e;
    p.whole = need == 0;
    if (!p.whole) {
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)2 * attend_grid(di->sms, nt) * 8 * nt * D);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == FA_BF16;
    if (D == 64) {
        if (nt == 1)
            return bf16 ? launch_attend_t<64, true, 1>(p, di->sms, s, dev) : launch_attend_t<64, false, 1>(p, di->sms, s, dev);
        return bf16 ? launch_attend_t<64, true, 2>(p, di->sms, s, dev) : launch_attend_t<64, false, 2>(p, di->sms, s, dev);
    }
    if (nt == 1)
        return bf16 ? launch_attend_t<128, true, 1>(p, di->sms, s, dev) : launch_attend_t<128, false, 1>(p, di->sms, s, dev);
    return bf16 ? launch_attend_t<128, true, 2>(p, di->sms, s, dev) : launch_attend_t<128, false, 2>(p, di->sms, s, dev);
}

extern "C" fa_status fa_cache_weights(const void *Q, const void *Kc, const void *Kp, const float *LSE, const int *lens,
                                      float *acc, int accumulate, int B, int H, int Hkv, int Nq, int C, int D,
                                      int window_left, int sinks, float scale, fa_dtype dtype, fa_stream_t stream)
{
    if (!sizes_ok(B, Hkv, 1, C, D, dtype) || !queries_ok(B, H, Hkv, Nq) || sinks < 0)
        return FA_ERR_INVALID_VALUE;
    if (!std::isfinite(scale) || !(scale > 0.f) || (accumulate != 0 && accumulate != 1))
        return FA_ERR_INVALID_VALUE;
    const size_t qrows = (size_t)B * H * Nq, held = (size_t)B * Hkv * C;
    const Arg args[6] = {{Q, qrows * D * 2, false, 16}, {Kc, held * D / 2, false, 16}, {Kp, held * 4, false, 4},
                         {LSE, qrows * 4, false, 4}, {lens, (size_t)B * 4, false, 4}, {acc, held * 4, true, 4}};
    int dev;
    const fa_host::DeviceInfo *di;
    const fa_status st = fa_host::check_args(args, 6, &dev, &di);
    if (st != FA_OK)
        return st;
    const int rows = (H / Hkv) * Nq;
    cache::Params p{};
    p.kc = static_cast<const uint8_t *>(Kc);
    p.kp = static_cast<const uint32_t *>(Kp);
    p.q = Q;
    p.lse = const_cast<float *>(LSE);
    p.acc = acc;
    p.lens = lens;
    p.B = B;
    p.Hkv = Hkv;
    p.C = C;
    p.rows = rows;
    p.Nq = Nq;
    p.RB = 1;
    p.left = window_left < 0 ? -1 : window_left;
    p.sinks = sinks;
    p.accumulate = accumulate;
    p.qk2 = scale * cache::kLog2e;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == FA_BF16;
    auto run = [&](auto d, auto b) -> fa_status {
        constexpr int DD = decltype(d)::value;
        constexpr bool BB = decltype(b)::value;
        if (rows <= 8)
            return launch_weights_t<DD, BB, 1>(p, di->sms, s, dev);
        return rows <= 16 ? launch_weights_t<DD, BB, 2>(p, di->sms, s, dev) : fa_launch::launch_weights_rows(p, DD, BB, di->sms, s, dev);
    };
    using T = std::true_type;
    using F = std::false_type;
    if (D == 64)
        return bf16 ? run(std::integral_constant<int, 64>{}, T{}) : run(std::integral_constant<int, 64>{}, F{});
    return bf16 ? run(std::integral_constant<int, 128>{}, T{}) : run(std::integral_constant<int, 128>{}, F{});
}
