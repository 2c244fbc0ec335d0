// fa_bwd_sink.cu -- the backward for causal windows with sinks and shared key
// heads: the passes of fa_bwd_kernel.cuh with SinkParams, then the sum of the
// sink tiles' parts.
#include "fa_bwd_pass.cuh"

namespace fa_launch {

namespace {

template <int D, bool BF16>
fa_status launch_all(const BwdLaunch &a, cudaStream_t s, int dev)
{
    const long long rows = (long long)a.BH * a.Npad;
    const long long threads = rows * (D / 8);
    const bool fused = (D == 64) && a.fused;
    fa::bwd::fa_bwd_prep<D, BF16><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(
        static_cast<const uint16_t *>(a.O), static_cast<const uint16_t *>(a.dO), a.LSE, a.lg, a.dl,
        fused ? a.dqa : nullptr, a.N, a.Npad, rows);
    if (cudaGetLastError() != cudaSuccess)
        return FA_ERR_CUDA;
    fa::bwd::SinkParams p{};
    p.lg = a.lg;
    p.dl = a.dl;
    p.N = a.N;
    p.Nkv = a.Nkv;
    p.Npad = a.Npad;
    p.BH = a.BH;
    p.nqt = a.Npad / fa::bwd::kTile;
    p.nkt = (a.Nkv + fa::bwd::kTile - 1) / fa::bwd::kTile;
    p.off = a.Nkv - a.N;
    p.wl = a.wl;
    p.wr = 0;
    p.qk2 = a.scale * 1.4426950408889634f;
    p.scale = a.scale;
    p.sinks = a.sinks;
    p.ss = (a.sinks + fa::bwd::kTile - 1) / fa::bwd::kTile;
    p.group = a.group;
    p.BHkv = a.BHkv;
    p.nc = a.nc;
    p.part = a.part;
    if (!fused) {   // dQ in a pass of its own
        p.T = a.BH * p.nqt;
        p.dA = a.dQ;
        const int grid = p.T < a.sms ? p.T : a.sms;
        const fa_status st =
            launch_pass<D, BF16, true, false, false, fa::bwd::SinkParams>(a.tq, a.tdo, a.tk, a.tv, a.tq, p, grid, s, dev);
        if (st != FA_OK)
            return st;
    }
    p.T = a.BHkv * (p.ss * p.nc + p.nkt - p.ss);
    p.dA = a.dK;
    p.dB = a.dV;
    const int grid = p.T < a.sms ? p.T : a.sms;
    fa_status st;
    if constexpr (D == 64)
        st = fused ? launch_pass<D, BF16, true, true, true, fa::bwd::SinkParams>(a.tk, a.tv, a.tq, a.tdo, a.tdqa, p, grid, s, dev)
                   : launch_pass<D, BF16, true, true, false, fa::bwd::SinkParams>(a.tk, a.tv, a.tq, a.tdo, a.tq, p, grid, s, dev);
    else
        st = launch_pass<D, BF16, true, true, false, fa::bwd::SinkParams>(a.tk, a.tv, a.tq, a.tdo, a.tq, p, grid, s, dev);
    if (st != FA_OK)
        return st;
    if (p.ss > 0 && p.nc > 1) {
        const long long elems = (long long)p.BHkv * p.ss * 2 * fa::bwd::kTile * D;
        if (launch_dependent(fa::bwd::sink_reduce_kernel<D, BF16>, dim3((unsigned)((elems / 8 + 255) / 256)), dim3(256), 0,
                             s, p) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_CUDA;
        }
    }
    if (fused) {
        const long long elems = (long long)a.BH * a.N * D;
        if (launch_dependent(fa::bwd::fa_bwd_dq_convert<BF16>, dim3((unsigned)((elems / 8 + 255) / 256)), dim3(256), 0, s,
                             (const float *)a.dqa, static_cast<uint16_t *>(a.dQ), a.N, a.Npad, D, elems,
                             a.scale) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_CUDA;
        }
    }
    return FA_OK;
}

}  // namespace

int sink_parts_for(int BH, int BHkv, int N, int Nkv, int wl, int sinks, int sms)
{
    if (sinks < 1)
        return 1;
    const long long nqt = (N + fa::bwd::kTile - 1) / fa::bwd::kTile, nkt = (Nkv + fa::bwd::kTile - 1) / fa::bwd::kTile;
    const long long group = BH / BHkv, ss = (sinks + fa::bwd::kTile - 1) / fa::bwd::kTile;
    long long win = (long long)(wl / fa::bwd::kTile) + 2;   // query tiles that see an ordinary key tile, at most
    win = win < nqt ? win : nqt;
    const long long tall = group * nqt;                      // steps of the first sink tile
    const long long share = BHkv * (ss * group * nqt + (nkt - ss) * group * win) / sms;   // steps per CTA, about
    if (tall <= share)   // the sink tiles come first, the others fill up behind them
        return 1;
    long long per = share / 2;                               // a part: half a share, and at least an ordinary tile
    per = per < group * win ? group * win : per;
    const long long nc = (tall + per - 1) / per;
    return (int)(nc < 1 ? 1 : (nc > 64 ? 64 : nc));
}

fa_status launch_bwd_sink(const BwdLaunch &a, cudaStream_t s, int dev)
{
    if (a.D == 64)
        return a.bf16 ? launch_all<64, true>(a, s, dev) : launch_all<64, false>(a, s, dev);
    return a.bf16 ? launch_all<128, true>(a, s, dev) : launch_all<128, false>(a, s, dev);
}

unsigned int *status_word_bwd_sink()
{
    return fa::status_word_address();
}

}  // namespace fa_launch
