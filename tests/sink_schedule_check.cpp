// Exhaustive check, on the CPU, of the forward's work decomposition for causal
// windows with sinks (SinkSchedule in fa_schedule.h): the steps of a tile name
// distinct K/V tiles, a Q tile's steps are a prefix of its CTA tile's and hold
// every key tile that one of its rows sees; every (tile, step) belongs to one
// part; and the merge expects exactly the parts that hold work.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <utility>
#include <vector>

#include "fa_schedule.h"

using namespace fa;

static int fail(const char *what, int a, int b)
{
    std::printf("%s (%d, %d)\n", what, a, b);
    return 1;
}

static int check(int N, int Nkv, int BH, int sms, int mode, int left, int sinks)
{
    int wl = left, wr = 0;
    sched_band_normalize(N, Nkv, wl, wr);
    const SinkSchedule s = sched_plan_sink(N, Nkv, BH, 1, sms, mode, wl, sinks);
    if (s.G < 1 || s.G > kSchedMaxGrid)
        return fail("grid", s.G, 0);
    for (int ct = 0; ct < s.C; ++ct) {
        const TileKeys keys = sched_tile_keys(s, ct);
        const int n = sched_steps_ct(s, ct);
        std::set<int> seen;
        int last = -1;
        for (int j = 0; j < n; ++j) {
            const int k = keys.first_key(j);
            if (k % kSchedBN || k < 0 || k >= s.nkv * kSchedBN || k <= last)
                return fail("step key", ct, j);
            last = k;
            seen.insert(k / kSchedBN);
        }
        int longest = 0;
        for (int w = 0; w < 2; ++w) {
            const int nw = sched_kv_tiles(s, ct, w);
            if (nw > n)
                return fail("Q tile longer than its CTA tile", ct, w);
            longest = nw > longest ? nw : longest;
            std::set<int> mine;
            for (int j = 0; j < nw; ++j)
                mine.insert(keys.first_key(j) / kSchedBN);
            const int r0 = ct * kSchedCtaRows + w * kSchedBM;
            if (r0 < N && nw < 1)
                return fail("Q tile without a step", ct, w);
            for (int r = r0; r < r0 + kSchedBM && r < N; ++r) {
                const long long pos = (long long)r + Nkv - N;
                for (int t = 0; t < s.nkv; ++t) {   // does some key of tile t show?
                    const long long k0 = (long long)t * kSchedBN, k1 = k0 + kSchedBN - 1 < Nkv - 1 ? k0 + kSchedBN - 1 : Nkv - 1;
                    const long long lo = left < 0 ? 0 : (pos - left > 0 ? pos - left : 0);
                    const bool band = k0 <= pos && k1 >= lo, sink = left >= 0 && k0 <= pos && k0 < sinks;
                    if ((band || sink) && !mine.count(t))
                        return fail("key tile not visited", r, t);
                }
                // the row's own bounds, as the kernel masks with them
                const int lo = sched_row_lo(s, r), hi = sched_row_hi(s, r);
                if (hi != (pos + 1 < 0 ? 0 : (int)(pos + 1)) || lo != (left < 0 || pos - left < 0 ? 0 : (int)(pos - left)))
                    return fail("row bounds", lo, hi);
            }
        }
        if (longest != n)
            return fail("CTA tile longer than its Q tiles", ct, n);
    }
    // every (tile, step) once; partial slots distinct; the merge's count
    std::vector<std::vector<int>> got(s.T);
    for (int t = 0; t < s.T; ++t)
        got[t].assign(sched_steps(s, t), 0);
    std::set<int> slots;
    std::vector<int> parts0(s.T, 0), parts1(s.T, 0);
    for (int c = 0; c < s.G; ++c) {
        PartIter it;
        it.init(s, c);
        Part p;
        while (it.next(s, p)) {
            int bh, ct;
            sched_decode(s, p.tile, bh, ct);
            if (p.tile < 0 || p.tile >= s.T || bh < 0 || bh >= BH || ct < 0 || ct >= s.C || p.kb < 0 ||
                p.ke > (int)got[p.tile].size() || p.ke <= p.kb)
                return fail("part", c, p.tile);
            for (int j = p.kb; j < p.ke; ++j)
                ++got[p.tile][j];
            for (int w = 0; w < 2; ++w) {
                const int nw = sched_kv_tiles(s, ct, w);
                if (nw > p.kb)
                    ++(w ? parts1 : parts0)[p.tile];
            }
            const bool partial = p.kb > 0 || p.ke < (int)got[p.tile].size();   // (whole tiles use no slot)
            if (partial && (p.slot < 0 || p.slot >= 2 * s.G || !slots.insert(p.slot).second))
                return fail("slot", c, p.slot);
        }
    }
    for (int t = 0; t < s.T; ++t) {
        int bh, ct;
        sched_decode(s, t, bh, ct);
        for (int x : got[t])
            if (x != 1)
                return fail("step not run once", t, x);
        if (!s.split)
            continue;
        for (int w = 0; w < 2; ++w) {
            const int nw = sched_kv_tiles(s, ct, w);
            const int np = sched_part_slots(s, t, nw, nullptr, 0);
            if (np != (w ? parts1 : parts0)[t])
                return fail("merge parts", t, np);
            if (np > sched_max_parts(s))
                return fail("too many parts", t, np);
        }
    }
    return 0;
}

int main(int argc, char **argv)
{
    int n = 0;
    int N, Nkv, BH, sms, mode, left, sinks;
    while (std::scanf("%d %d %d %d %d %d %d", &N, &Nkv, &BH, &sms, &mode, &left, &sinks) == 7) {
        if (check(N, Nkv, BH, sms, mode, left, sinks)) {
            std::printf("FAIL N=%d Nkv=%d BH=%d sms=%d mode=%d left=%d sinks=%d\n", N, Nkv, BH, sms, mode, left, sinks);
            return 1;
        }
        ++n;
    }
    std::printf("ok %d\n", n);
    return 0;
}
