// fa_evict.cu -- eviction from the 4-bit cache by accumulated attention
// weight: which tokens stay (a selection per sequence and key head), and the
// copy of their rows into another cache.
//
// Of the n = lens[b] tokens of a sequence, the first `sinks` and the last
// `recent` stay, and of those between them the k = keep - sinks - recent with
// the largest accumulated weight (equal weights: the lowest position first),
// all in order of position; n <= keep keeps everything.
//
// Selection without sorting: weights become 32-bit keys that order as the
// weights do, and the k-th largest key is found digit by digit (four of 8
// bits, a histogram of the candidates per digit); one more pass ranks what is
// above it, and the first of those equal to it, by position.  A cluster of
// CTAs shares a row, each holding its slice of the keys in shared memory and
// adding the others' histograms through distributed shared memory, so the
// weights are read from memory once and a few long rows still occupy many
// SMs.  What it takes is a chain of short steps (8 rows of 130001 weights, 8
// CTAs each: 2 us of reading, then per digit a pass over 16 keys a thread, a
// cluster barrier, a histogram of 8 x 1 KB read from the neighbours, a scan),
// hence small histograms: 2048 bins took three digits instead of four, but
// 4100 cycles of reading each.
#include "fa.h"

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_host.h"

namespace {

namespace cg = cooperative_groups;
using fa_host::Arg;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxCluster = 8;         // the portable cluster size
constexpr int kMaxHeld = 40960;        // keys held in shared memory per CTA (160 KB); longer slices are read again
constexpr int kMinSlice = 2048;        // keys per CTA below which a row is not split further

struct EvictParams {
    const float *acc;
    const int *lens;
    const uint8_t *kc, *vc;
    const uint32_t *kp, *vp;
    float *acc2;
    int *lens2, *index;
    uint8_t *kc2, *vc2;
    uint32_t *kp2, *vp2;
    int Hkv, C, C2, keep, sinks, recent, held;
    long long BH;
};

// A key that orders as the weight does: larger weight, larger key; -0 equals
// 0, NaN is below every number.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x)
        return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 -> 0
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int clamped(int n, int C)
{
    return n < 0 ? 0 : (n > C ? C : n);
}

__device__ __forceinline__ int warp_scan(int v, int lane)   // inclusive
{
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m)
            v += u;
    }
    return v;
}

// One cluster per sequence and key head.  Two CTAs fit an SM (32 registers);
// one histogram per digit, so that a digit needs one cluster barrier.
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const EvictParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint32_t keys[];   // [held, rounded up to 4]
    __shared__ int hist[4][kBins];
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_count[2], s_found[2];
    static_assert(kSelWarps == 32, "one lane per warp's sum");
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const uint32_t bh = blockIdx.x / CS;
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    const int n = clamped(p.lens[bh / p.Hkv], p.C);
    const float *acc = p.acc + (size_t)bh * p.C;
    int *index = p.index + (size_t)bh * p.keep;
    if (rank == 0 && t == 0 && bh % p.Hkv == 0)
        p.lens2[bh / p.Hkv] = n < p.keep ? n : p.keep;
    if (n <= p.keep) {   // (the whole cluster leaves)
        for (int j = rank * kSelThreads + t; j < p.keep; j += CS * kSelThreads)
            index[j] = j < n ? j : -1;
        return;
    }
    // What always stays.
    for (int j = rank * kSelThreads + t; j < p.sinks; j += CS * kSelThreads)
        index[j] = j;
    for (int j = rank * kSelThreads + t; j < p.recent; j += CS * kSelThreads)
        index[p.keep - p.recent + j] = n - p.recent + j;
    const int k = p.keep - p.sinks - p.recent;
    if (k == 0)
        return;
    const int M = n - p.recent - p.sinks;             // candidates, more than k
    const int slice = (M + CS - 1) / CS;
    const int lo = p.sinks + (int)min((long long)rank * slice, (long long)M), cnt = min(slice, p.sinks + M - lo);
    const bool held = slice <= p.held;
    (&hist[0][0])[t] = 0;
    static_assert(4 * kBins == kSelThreads, "one bin per thread");
    __syncthreads();
    // The keys, and the histogram of their first digit as they come.
    constexpr int kBatch = 8;   // loads in flight per thread
    for (int i0 = 0; i0 < cnt; i0 += kBatch * kSelThreads) {
        float x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kSelThreads + t;
            x[u] = i < cnt ? __ldg(acc + lo + i) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kSelThreads + t;
            if (i < cnt) {
                const uint32_t key = key_of(x[u]);
                if (held)
                    keys[i] = key;
                atomicAdd(&hist[0][key >> 24], 1);
            }
        }
    }
    // Keys 4 v .. 4 v + 3 of the slice (what lies behind its end is not looked at).
    auto keys_at = [&](int v) -> uint4 {
        if (held)
            return reinterpret_cast<const uint4 *>(keys)[v];
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        x.x = key_of(__ldg(acc + lo + 4 * v));
        if (4 * v + 1 < cnt)
            x.y = key_of(__ldg(acc + lo + 4 * v + 1));
        if (4 * v + 2 < cnt)
            x.z = key_of(__ldg(acc + lo + 4 * v + 2));
        if (4 * v + 3 < cnt)
            x.w = key_of(__ldg(acc + lo + 4 * v + 3));
        return x;
    };
    const int vecs = (cnt + 3) / 4;

    uint32_t prefix = 0;   // the digits found so far
    int left = k;          // candidates still to take among the keys that share them
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        if (pass > 0) {
            __syncthreads();   // (pass 1: the keys are written)
            for (int v = t; v < vecs; v += kSelThreads) {
                const uint4 x = keys_at(v);
                const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if ((key[u] >> (shift + 8)) == prefix && 4 * v + u < cnt)
                        atomicAdd(&hist[pass][(key[u] >> shift) & 255u], 1);
            }
        }
        cluster.sync();
        // Counts of the bins from the top, one to each of 256 threads, over all slices.
        int c = 0, inc = 0;
        if (t < kBins) {
            const int bin = kBins - 1 - t;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                if (r < CS)
                    c += *cluster.map_shared_rank(&hist[pass][bin], r);
            inc = warp_scan(c, lane);
            if (lane == 31)
                s_gt[warp] = inc;
        }
        __syncthreads();
        if (t < kBins) {
            int before = inc - c;
#pragma unroll
            for (int w = 0; w < kBins / 32; ++w)
                before += w < warp ? s_gt[w] : 0;
            if (before < left && before + c >= left) {   // exactly one thread: the counts add up to at least `left`
                s_found[0] = kBins - 1 - t;
                s_found[1] = left - before;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)s_found[0];
        left = s_found[1];
    }
    // prefix is the k-th largest key; `left` of the keys equal to it are taken.

    // Rank by position: each thread counts its own consecutive part of the
    // slice; the slices, warps and lanes before it give its first rank.
    const int per = (vecs + kSelThreads - 1) / kSelThreads;
    const int v0 = min(t * per, vecs), v1 = min(v0 + per, vecs);
    int gt = 0, eq = 0;
    for (int v = v0; v < v1; ++v) {
        const uint4 x = keys_at(v);
        const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = 4 * v + u < cnt;
            gt += in && key[u] > prefix;
            eq += in && key[u] == prefix;
        }
    }
    const int gt_inc = warp_scan(gt, lane), eq_inc = warp_scan(eq, lane);
    if (lane == 31) {
        s_gt[warp] = gt_inc;
        s_eq[warp] = eq_inc;
    }
    __syncthreads();
    const int all_gt = warp_scan(s_gt[lane], lane), all_eq = warp_scan(s_eq[lane], lane);
    // (of the warps before this one: the sums up to and with it, less its own)
    int n_gt = __shfl_sync(0xffffffffu, all_gt, warp) - s_gt[warp] + gt_inc - gt;
    int n_eq = __shfl_sync(0xffffffffu, all_eq, warp) - s_eq[warp] + eq_inc - eq;
    if (t == 31) {
        s_count[0] = all_gt;
        s_count[1] = all_eq;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {   // taken for certain, and equal, in the slices before
        const int *o = cluster.map_shared_rank(s_count, r);
        n_gt += o[0];
        n_eq += o[1];
    }
    if (gt + eq > 0) {
        for (int v = v0; v < v1; ++v) {
            const uint4 x = keys_at(v);
            const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (4 * v + u >= cnt || key[u] < prefix)
                    continue;
                const bool g = key[u] > prefix;
                if (g || n_eq < left)
                    index[p.sinks + n_gt + min(n_eq, left)] = lo + 4 * v + u;
                n_gt += g;
                n_eq += !g;
            }
        }
    }
    cluster.sync();   // no CTA leaves while another may still read its counts
}

// Rows of the kept tokens into the other cache, 16 bytes a thread and row, and
// their weights (0 behind the last one).  Rows behind the last one are left as
// they are.  Each thread takes kGatherRows rows, so that as many reads at
// places of the index's choosing are in flight.
constexpr int kGatherRows = 4;

template <int D>
__global__ void __launch_bounds__(256) gather_kernel(const EvictParams p)
{
    constexpr int kHalf = D / 32;        // 16-byte chunks of codes per row, K or V
    constexpr int kTpr = 2 * kHalf;
    constexpr uint32_t kStep = 256 / kTpr;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection's index
    const uint32_t rows = (uint32_t)(p.BH * p.C2);       // (below 2^31)
    const uint32_t row0 = blockIdx.x * (kStep * kGatherRows) + threadIdx.x / kTpr;
    const int part = threadIdx.x % kTpr;
    const bool v = part >= kHalf;
    const int j = v ? part - kHalf : part;
    const uint8_t *codes = v ? p.vc : p.kc;
    const uint32_t *params = v ? p.vp : p.kp;
    long long from[kGatherRows];
    uint4 x[kGatherRows];
    uint32_t y[kGatherRows];
    float w[kGatherRows];
#pragma unroll
    for (int k = 0; k < kGatherRows; ++k) {
        const uint32_t row = row0 + k * kStep;
        from[k] = -1;
        if (row < rows) {
            const uint32_t bh = row / (uint32_t)p.C2;
            const int d = (int)(row - bh * p.C2);
            // (not through the read-only path: the index was written while this grid was already there)
            const int src = d < p.keep ? __ldcg(p.index + (size_t)bh * p.keep + d) : -1;
            if (src >= 0)
                from[k] = (long long)bh * p.C + src;
        }
    }
#pragma unroll
    for (int k = 0; k < kGatherRows; ++k) {
        if (from[k] >= 0) {
            x[k] = __ldg(reinterpret_cast<const uint4 *>(codes + from[k] * (D / 2)) + j);
            if (j == 0)
                y[k] = __ldg(params + from[k]);
            if (part == 1)
                w[k] = __ldg(p.acc + from[k]);
        } else {
            w[k] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < kGatherRows; ++k) {
        const uint32_t row = row0 + k * kStep;
        if (row >= rows)
            break;
        if (part == 1)
            p.acc2[row] = w[k];
        if (from[k] < 0)
            continue;
        reinterpret_cast<uint4 *>((v ? p.vc2 : p.kc2) + (size_t)row * (D / 2))[j] = x[k];
        if (j == 0)
            (v ? p.vp2 : p.kp2)[row] = y[k];
    }
}

// CTAs per row: more while every one of them still gets kMinSlice keys and
// the rows do not fill the SMs twice over by themselves.
int cluster_size(long long BH, int C, int sms)
{
    int cs = 1;
    while (cs < kMaxCluster && BH * cs * 2 <= 2ll * sms && C / (cs * 2) >= kMinSlice)
        cs *= 2;
    return cs;
}

fa_status launch_evict(const EvictParams &q, int D, int sms, cudaStream_t s, int dev)
{
    static bool set[fa_host::kMaxDevices] = {};
    const fa_status st = fa_host::allow_smem(reinterpret_cast<const void *>(&select_kernel), kMaxHeld * 4, dev, set);
    if (st != FA_OK)
        return st;
    EvictParams p = q;
    const int cs = cluster_size(p.BH, p.C, sms);
    const long long slice = ((long long)p.C + cs - 1) / cs;
    p.held = slice <= kMaxHeld ? (int)slice : 0;   // keys that fit are held; otherwise none are
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.BH * cs));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = ((size_t)p.held + 3) / 4 * 16;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, select_kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    const long long per = 256 / (D / 16) * kGatherRows;   // rows per block
    cudaLaunchConfig_t cg2{};
    cg2.gridDim = dim3((unsigned)((p.BH * p.C2 + per - 1) / per));
    cg2.blockDim = dim3(256);
    cg2.stream = s;
    cudaLaunchAttribute dep[1];
    dep[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dep[0].val.programmaticStreamSerializationAllowed = 1;
    cg2.attrs = dep;
    cg2.numAttrs = 1;
    const cudaError_t e = D == 64 ? cudaLaunchKernelEx(&cg2, gather_kernel<64>, p) : cudaLaunchKernelEx(&cg2, gather_kernel<128>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_cache_evict(const void *Kc, const void *Kp, const void *Vc, const void *Vp, const float *acc,
                                    const int *lens, void *Kc2, void *Kp2, void *Vc2, void *Vp2, float *acc2,
                                    int *lens2, int *index, int B, int Hkv, int C, int C2, int D, int keep, int sinks,
                                    int recent, fa_stream_t stream)
{
    if (D != 64 && D != 128)
        return FA_ERR_INVALID_VALUE;
    if (B < 1 || Hkv < 1 || C < 1 || C2 < 1 || keep < 1 || keep > C2 || sinks < 0 || recent < 0)
        return FA_ERR_INVALID_VALUE;
    if ((long long)sinks + recent > keep)
        return FA_ERR_INVALID_VALUE;
    const long long BH = (long long)B * Hkv;
    // (kMaxCluster CTAs per row at most, in one grid dimension)
    if (BH >= (1ll << 31) / kMaxCluster || BH * C > fa_host::kMaxRows || BH * C2 > fa_host::kMaxRows)
        return FA_ERR_INVALID_VALUE;
    const size_t from = (size_t)BH * C, to = (size_t)BH * C2;
    const Arg args[13] = {{Kc, from * D / 2, false, 16}, {Kp, from * 4, false, 4}, {Vc, from * D / 2, false, 16},
                          {Vp, from * 4, false, 4}, {acc, from * 4, false, 4}, {lens, (size_t)B * 4, false, 4},
                          {Kc2, to * D / 2, true, 16}, {Kp2, to * 4, true, 4}, {Vc2, to * D / 2, true, 16},
                          {Vp2, to * 4, true, 4}, {acc2, to * 4, true, 4}, {lens2, (size_t)B * 4, true, 4},
                          {index, (size_t)BH * keep * 4, true, 4}};
    int dev;
    const fa_host::DeviceInfo *di;
    const fa_status st = fa_host::check_args(args, 13, &dev, &di);
    if (st != FA_OK)
        return st;
    EvictParams p{};
    p.acc = acc;
    p.lens = lens;
    p.kc = static_cast<const uint8_t *>(Kc);
    p.kp = static_cast<const uint32_t *>(Kp);
    p.vc = static_cast<const uint8_t *>(Vc);
    p.vp = static_cast<const uint32_t *>(Vp);
    p.acc2 = acc2;
    p.lens2 = lens2;
    p.index = index;
    p.kc2 = static_cast<uint8_t *>(Kc2);
    p.kp2 = static_cast<uint32_t *>(Kp2);
    p.vc2 = static_cast<uint8_t *>(Vc2);
    p.vp2 = static_cast<uint32_t *>(Vp2);
    p.Hkv = Hkv;
    p.C = C;
    p.C2 = C2;
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.BH = BH;
    return launch_evict(p, D, di->sms, reinterpret_cast<cudaStream_t>(stream), dev);
}
