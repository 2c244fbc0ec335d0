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
// -- which the persistent CTAs walk in serpentine rounds, all heads of an entry
// next to one another.  The list is as long as the sequences make it; its
// length is in the plan's header, and its room is bounded by the token counts.
//
// Plan layout, in 16-byte words: a header {n0, n1, n2, 0}, then per list its
// entries (two words: {q0, Lq, k0, Lk}, {tile, first query tile of the
// sequence, 0, 0}) and two scratch words per sequence and two more; then list
// 1's table by query tile, {first row, rows, 0, 0}, in the sequences' order with one
// empty tile behind the last (the dK/dV pass's step of a key tile that no query
// sees).
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

struct Sizes {
    int S, Tq, Tk, H, Hkv;
};

// Entries that list l has room for, and all of it in 16-byte words.
FA_HD long long capacity(const Sizes &z, int l)
{
    return (l == 0 ? z.Tq / 256 : l == 1 ? z.Tq / kTile : z.Tk / kTile) + (long long)z.S;
}
FA_HD long long list_word(const Sizes &z, int l)   // first word of list l
{
    long long w = 1;
    for (int i = 0; i < l; ++i)
        w += 2 * (capacity(z, i) + z.S + 1);
    return w;
}
FA_HD long long scratch_word(const Sizes &z, int l) { return list_word(z, l) + 2 * capacity(z, l); }
FA_HD long long table_word(const Sizes &z) { return list_word(z, 3); }
// Words of a plan for the forward alone, or for both directions.
FA_HD long long plan_words(const Sizes &z, bool grad) { return grad ? table_word(z) + capacity(z, 1) + 1 : list_word(z, 1); }
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
    const int4 *list;
    const int *count;   // entries
    int H, group;       // query heads, and those per key head
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

#endif

}  // namespace fa
