// CPU check of the tile sequence that the whole-tile kernel runs for causal
// windows with sinks (sched_next_whole in fa_schedule.h: its own serpentine
// rounds and a division by multiplication) against PartIter and sched_decode,
// and of its steps of a few sinks (SinkTile::few) against each row's keys.
#include <cstdio>

#include "fa_schedule.h"

using namespace fa;

static int fail(const char *what, int a, int b)
{
    std::printf("%s (%d, %d)\n", what, a, b);
    return 1;
}

static int check(int N, int Nkv, int BH, int sms, int left, int sinks)
{
    int wl = left, wr = 0;
    sched_band_normalize(N, Nkv, wl, wr);
    const SinkSchedule s = sched_plan_sink(N, Nkv, BH, 1, sms, 1, wl, sinks);   // whole tiles
    if (s.split)
        return fail("whole tiles were asked for", s.split, 0);
    if ((s.inv == 0) != ((double)s.T * BH >= 1099511627776.0))
        return fail("inverse", s.T, BH);
    for (int c = 0; c < s.G; ++c) {
        PartIter a, b;
        a.init(s, c);
        b.init_t<false>(s, c);
        for (;;) {
            Part pa, pb;
            SinkTile tile;
            int bh, ct, bh2, ct2;
            const bool more = a.next(s, pa);
            if (sched_next_whole(s, b, pb, bh, ct, tile) != more)
                return fail("number of tiles", c, pa.tile);
            if (!more)
                break;
            sched_decode(s, pa.tile, bh2, ct2);
            if (pa.tile != pb.tile || pa.kb != pb.kb || pa.ke != pb.ke || pa.slot != pb.slot || pa.ts != pb.ts)
                return fail("part", pa.tile, pb.tile);
            if (bh != bh2 || ct != ct2)
                return fail("head and row", pa.tile, bh);
            const TileKeys keys = sched_tile_keys(s, ct);
            if (tile.ssz != keys.ssz || tile.ks != keys.ks || tile.few != keys.few || tile.n != sched_steps_ct(s, ct) ||
                tile.nw[0] != sched_kv_tiles(s, ct, 0) || tile.nw[1] != sched_kv_tiles(s, ct, 1))
                return fail("steps", ct, tile.n);
        }
    }
    for (int ct = 0; ct < s.C; ++ct) {
        const SinkTile tile = sched_sink_tile(s, ct);
        // few exactly where the tile has one sink step, of at most kSchedFewSinks sinks, and no row's window reaches
        // into that step
        bool reaches = false;
        for (int r = ct * kSchedCtaRows; r < (ct + 1) * kSchedCtaRows && r < N; ++r) {
            const long long pos = (long long)r + Nkv - N;
            const long long lo = left < 0 || pos < left ? 0 : pos - left;
            reaches |= lo < kSchedBN;
        }
        const bool want = s.sinks > 0 && s.sinks <= kSchedFewSinks && tile.ssz == 1 && !reaches;
        if (tile.few != want)
            return fail("few", ct, tile.few);
    }
    return 0;
}

int main()
{
    int n = 0;
    int N, Nkv, BH, sms, left, sinks;
    while (std::scanf("%d %d %d %d %d %d", &N, &Nkv, &BH, &sms, &left, &sinks) == 6) {
        if (check(N, Nkv, BH, sms, left, sinks)) {
            std::printf("FAIL N=%d Nkv=%d BH=%d sms=%d left=%d sinks=%d\n", N, Nkv, BH, sms, left, sinks);
            return 1;
        }
        ++n;
    }
    std::printf("ok %d\n", n);
    return 0;
}
