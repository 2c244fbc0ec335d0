// fa_packed.h -- packed sequences: the plan of a batch and the tiles it holds
// (host and device code).
//
// The tokens of S sequences stand behind one another; sequence s has the query
// rows cu_q[s] .. cu_q[s + 1] - 1 and the key rows cu_k[s] .. cu_k[s + 1] - 1.
// Lengths are device data, so a kernel on the device (fa_packed_plan.cu) lays
// out the work once per batch and every layer's calls read it: up to three
// lists of tiles, each longest first --
//   list 0  forward: CTA tiles of 256 query rows
//   list 1  dQ pass and the rows' statistics: query tiles of 128 rows
//   list 2  dK/dV pass: key tiles of 128 rows
// -- an entry of which is a tile of one sequence, and a tile of work one of its
// heads.  The persistent CTAs take a tile each in rounds: of a round's tiles the
// longest goes to the CTA whose tiles so far are the fewest steps, for kOrderRounds
// rounds, and then in serpentine order.  (Serpentine rounds alone leave the busiest
// of 152 CTAs 16 % above the mean in the dK/dV pass of 6 documents of 500 to 8001
// tokens, 572 tiles; so laid out, 5 %.)
//
// What a role of the kernels needs of a tile is one slot of two words, {q0, Lq, k0,
// Lk} and {tile, first query tile of the sequence, head, query tiles in all + 1},
// the last 0 where there is none; a CTA's slots follow one another, so after the
// first of four they are in L1.  (Looked up by way of order, entry and head, a tile
// began 0.7 us later.)
//
// Plan layout, in 16-byte words: a header {n0, n1, n2, 0} of entries per list; per
// list its slots, then scratch (its entries, longest first, and two words per
// sequence and two more); then list 1's table by query tile, {first row, rows, 0,
// 0}, in the sequences' order with one empty tile behind the last (the dK/dV pass's
// step of a key tile that no query sees).
#pragma once

#include <cstddef>
#include <cstdint>

#include "fa_schedule.h"

#ifdef __CUDACC__
#include <cuda_runtime.h>
#endif

namespace fa {
namespace packed {

constexpr int kTile = 128;
constexpr int kOrderRounds = 16;
constexpr int kOrderGrid = kSchedMaxGrid;   // CTAs, at most

struct Sizes {
    int S, Tq, Tk, H, Hkv;
};

// Entries that list l has room for, and all of it in 16-byte words.
FA_HD long long capacity(const Sizes &z, int l)
{
    return (l == 0 ? z.Tq / 256 : l == 1 ? z.Tq / kTile : z.Tk / kTile) + (long long)z.S;
}
FA_HD int heads_of(const Sizes &z, int l) { return l == 2 ? z.Hkv : z.H; }
// Slots that list l has room for (CTAs' rounds are as many for all of them).
FA_HD long long slots(const Sizes &z, int l) { return capacity(z, l) * heads_of(z, l) + kOrderGrid; }
FA_HD long long list_word(const Sizes &z, int l)   // first word of list l: its slots
{
    long long w = 1;
    for (int i = 0; i < l; ++i)
        w += 2 * (slots(z, i) + capacity(z, i) + z.S + 1);
    return w;
}
FA_HD long long entry_word(const Sizes &z, int l) { return list_word(z, l) + 2 * slots(z, l); }
FA_HD long long scratch_word(const Sizes &z, int l) { return entry_word(z, l) + 2 * capacity(z, l); }
FA_HD long long table_word(const Sizes &z) { return list_word(z, 3); }
// Words of a plan for the forward alone, or for both directions.
FA_HD long long plan_words(const Sizes &z, bool grad) { return grad ? table_word(z) + capacity(z, 1) + 1 : list_word(z, 1); }
// CTAs that walk list l, and the rounds that their slots have room for.
FA_HD int grid(const Sizes &z, int l, int sms)
{
    const long long t = capacity(z, l) * heads_of(z, l);
    const int top = sms < kOrderGrid ? sms : kOrderGrid;
    return (int)(t < top ? t : top);
}
FA_HD int rounds(const Sizes &z, int l, int G) { return (int)((capacity(z, l) * heads_of(z, l) + G - 1) / G); }
// Rows of the backward's row statistics per head: a whole number of query tiles.
FA_HD long long padded_rows(const Sizes &z) { return (capacity(z, 1) + 1) * kTile; }

// Keys that query row r of a sequence sees: [0, row_end).
FA_HD int row_end(int r, int Lq, int Lk, bool causal)
{
    if (!causal)
        return Lk;
    const int e = r + (Lk - Lq) + 1;
    return e < 0 ? 0 : (e > Lk ? Lk : e);
}
// Key tiles that query rows first .. first + 127 visit: at least one (rows that
// see nothing get their zeros from a masked step), none where there is no row.
FA_HD int key_steps(int first, int Lq, int Lk, bool causal)
{
    if (first >= Lq)
        return 0;
    const int last = first + kTile - 1 < Lq - 1 ? first + kTile - 1 : Lq - 1;
    const int n = (int)(((unsigned)row_end(last, Lq, Lk, causal) + kTile - 1) / kTile);
    return n < 1 ? 1 : n;
}
// First query tile that sees a key of key tile kt; -1 if none does.
FA_HD int first_query_tile(int kt, int Lq, int Lk, bool causal)
{
    if (Lq == 0)
        return -1;
    if (!causal)
        return 0;
    const long long i = (long long)kt * kTile - (Lk - (long long)Lq);
    return i <= 0 ? 0 : (int)(i / kTile);
}

// A tile's last rows.  The 128 rows of a tile that reaches behind its sequence
// hold the next sequence's rows there, whose products must not enter a sum over
// the tile's rows, not even with weight 0 (they may be infinite): such a product
// stops at the first multiple of 16 rows behind the sequence's, and the rows
// between are zeroed in shared memory before it.  k-steps (16 rows) of a product
// over a tile that holds n of the sequence's rows: at least one.
FA_HD int tail_ksteps(int n)
{
    return n <= 0 ? 1 : (n >= kTile ? kTile / 16 : (n + 15) / 16);
}

}  // namespace packed

#ifdef __CUDACC__

// The forward's schedule: list 0 of a plan.
struct PackedSchedule : Schedule {
    const int4 *slots;
    int rounds;         // slots of a CTA
    int group;          // query heads per key head
};

struct PackedTile {
    int q0, Lq, k0, Lk;   // the sequence
    int nw[2];            // key steps of its two Q tiles
    static constexpr bool few = false;
};

__device__ __forceinline__ int4 ld_plan(const int4 *p)
{
    return __ldg(p);
}

// CTA c's slot of round r; false: there is none.
__device__ __forceinline__ bool packed_slot(const int4 *slots, int rounds, int c, int r, int4 &seq, int4 &at)
{
    if (r >= rounds)
        return false;
    const int4 *p = slots + 2 * ((long long)c * rounds + r);
    seq = ld_plan(p);
    at = ld_plan(p + 1);
    return at.w != 0;
}

#endif

}  // namespace fa
