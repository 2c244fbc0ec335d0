// The tiles of packed sequences (fa_packed.h) against their definition: reads lines
// "Lq Lk causal", checks which key tiles a query tile visits, which query tiles see a
// key tile, and the parts that steps are cut into; then lines of a batch, "batch H Hkv
// n Lq Lk Lq Lk ...", the room of its lists and the order of the plan's regions.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "fa_packed.h"

namespace pk = fa::packed;

static bool sees(long long i, long long j, long long Lq, long long Lk, bool causal)
{
    return j < Lk && i < Lq && (!causal || j <= i + Lk - Lq);
}

static int fail(const char *what, int Lq, int Lk, int causal)
{
    std::printf("%s: Lq %d Lk %d causal %d\n", what, Lq, Lk, causal);
    return 1;
}

static int sequence(int Lq, int Lk, int causal)
{
    for (int i = 0; i < Lq; ++i) {
        int n = 0;
        while (sees(i, n, Lq, Lk, causal))
            ++n;
        if (pk::row_end(i + Lk - Lq, Lk, causal) != n)
            return fail("keys of a row", Lq, Lk, causal);
    }
    for (int first = 0; first < Lq + 256; first += 128) {
        int want = first < Lq ? 1 : 0;
        for (int i = first; i < first + 128 && i < Lq; ++i)
            while (sees(i, want * 128, Lq, Lk, causal))
                ++want;
        if (pk::key_steps(first, Lq, Lk, causal) != want)
            return fail("steps of a query tile", Lq, Lk, causal);
        // the same from a tile of its own rows (the forward's slots)
        const int rows = Lq - first < 256 ? Lq - first : 256;
        if (first < Lq && (pk::tile_steps(0, rows, first + Lk - Lq, Lk, causal) != want ||
                           pk::tile_steps(128, rows, first + Lk - Lq, Lk, causal) != pk::key_steps(first + 128, Lq, Lk, causal)))
            return fail("steps of a tile", Lq, Lk, causal);
    }
    for (int kt = 0; kt * 128 < Lk; ++kt) {
        int want = -1;
        for (int i = 0; i < Lq && want < 0; ++i)
            for (int j = kt * 128; j < kt * 128 + 128 && want < 0; ++j)
                if (sees(i, j, Lq, Lk, causal))
                    want = i / 128;
        const int got = pk::first_query_tile(kt, Lq, Lk, causal);
        if (got != want || got * 128 >= (Lq > 0 ? Lq : 1))
            return fail("first query tile", Lq, Lk, causal);
    }
    for (int of = 1; of <= 16; ++of) {
        const int n = Lq + of;   // at least a step to a part
        int at = 0;
        for (int i = 0; i < of; ++i) {
            const int b = pk::part_step(n, i, of), e = pk::part_step(n, i + 1, of);
            if (b != at || e <= b)
                return fail("parts", n, of, i);
            at = e;
            const int x = pk::pack_part(Lk * 77 % (1 << 24), i, of);
            if (pk::part_tile(x) != Lk * 77 % (1 << 24) || pk::part_of(x) != i || pk::parts_of(x) != of)
                return fail("a packed part", Lk, i, of);
        }
        if (at != n)
            return fail("the last part", n, of, at);
    }
    for (int n = -20; n < 300; ++n) {
        const int ks = pk::tail_ksteps(n);
        if (ks < 1 || ks > 8 || (n < 128 ? 16 * ks < n : ks != 8) || (n > 0 && 16 * (ks - 1) >= n))
            return fail("k-steps", n, ks, 0);
    }
    return 0;
}

static int batch(int H, int Hkv, const std::vector<int> &q, const std::vector<int> &k)
{
    pk::Sizes z{(int)q.size(), 0, 0, H, Hkv};
    long long tiles[3] = {0, 0, 0}, longest = 0;
    for (size_t s = 0; s < q.size(); ++s) {
        z.Tq += q[s];
        z.Tk += k[s];
    }
    for (size_t s = 0; s < q.size(); ++s) {
        tiles[0] += (q[s] + pk::cta_rows(z) - 1) / pk::cta_rows(z);
        tiles[1] += (q[s] + 127) / 128;
        tiles[2] += (k[s] + 127) / 128;
        const long long n = (q[s] + 127) / 128 * (long long)(H / Hkv);
        longest = n > longest ? n : longest;
    }
    const int parts = pk::max_parts(z);
    if (parts < 1 || parts > 16 || (longest + pk::kPartSteps - 1) / pk::kPartSteps < 0 || tiles[2] > pk::key_tiles(z))
        return fail("key tiles", H, Hkv, parts);
    if (parts < 16 && (longest + pk::kPartSteps - 1) / pk::kPartSteps > parts &&
        pk::key_tiles(z) * Hkv * parts < 4 * pk::kOrderGrid)
        return fail("parts that there could be", H, Hkv, parts);
    if (parts > 1 && pk::key_tiles(z) > 32767)
        return fail("a key tile's number beside its head", H, Hkv, parts);
    for (int l = 0; l < 3; ++l) {
        const long long most = l == 2 ? tiles[2] * parts : tiles[l];
        const int G = pk::grid(z, l, 152), R = pk::rounds(z, l, G);
        if (most > pk::capacity(z, l) || (long long)G * R > pk::slots(z, l) || most * pk::heads_of(z, l) > (long long)G * R)
            return fail("room of a list", H, Hkv, l);
        if (pk::list_word(z, l) + 2 * pk::slots(z, l) != pk::entry_word(z, l) ||
            pk::entry_word(z, l) + 2 * pk::capacity(z, l) != pk::scratch_word(z, l) ||
            pk::scratch_word(z, l) + 2 * (z.S + 1) > pk::list_word(z, l + 1))
            return fail("regions of the plan", H, Hkv, l);
    }
    if (pk::list_word(z, 0) < 1 || pk::table_word(z) < pk::list_word(z, 3) ||
        pk::key_table_word(z) < pk::table_word(z) + tiles[1] + 1 ||
        pk::plan_words(z, true) < pk::key_table_word(z) + pk::key_tiles(z) || pk::plan_words(z, false) < pk::list_word(z, 1) ||
        pk::padded_rows(z) < (tiles[1] + 1) * 128)
        return fail("tables of the plan", H, Hkv, z.S);
    return 0;
}

int main()
{
    char word[64];
    int n = 0;
    while (std::scanf("%63s", word) == 1) {
        int bad;
        if (std::strcmp(word, "batch") == 0) {
            int H, Hkv, S;
            if (std::scanf("%d %d %d", &H, &Hkv, &S) != 3)
                return 2;
            std::vector<int> q(S), k(S);
            for (int s = 0; s < S; ++s)
                if (std::scanf("%d %d", &q[s], &k[s]) != 2)
                    return 2;
            bad = batch(H, Hkv, q, k);
        } else {
            int Lk, causal;
            if (std::scanf("%d %d", &Lk, &causal) != 2)
                return 2;
            bad = sequence(std::atoi(word), Lk, causal);
        }
        if (bad)
            return 1;
        ++n;
    }
    std::printf("ok %d\n", n);
    return 0;
}
