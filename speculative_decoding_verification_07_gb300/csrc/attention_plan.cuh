// The list of items of attention calls with forms of the scores or shared prefixes:
// made by a kernel before the attention's, which reads it.
#pragma once

#include "attention.cuh"

namespace sv {

constexpr int kTile = 128;     // keys of a tile, and rows of a product
constexpr int kStageBox = 16;  // staged entries per TMA box
constexpr int kMembers = 32;   // requests whose rows share an item at most: a lane each
constexpr int kForms = 1, kShare = 2;

// A CTA's share of the work: [w, w1) of the list of all requests' items (head,
// row block), an item being kLead units for what it costs besides its tiles
// (queries in, outputs out) and then one unit a key tile.  64 requests of 128 to
// 8192 positions, bf16, single tokens / trees of 15 nodes: 193 / 215 us with a
// lead of 3, 191 / 208 with 4, 189 / 202 with 5, 192 / 200 with 6, 193 / 204 with 8.
constexpr int kLead = 6;
// Consecutive items: one a head and row block, T units each (with ranges: a head's row
// blocks together T units), `units` in all and `cum` before them.  A request alone has
// its rows in them, b = its number, S and n its extent, begin the first position that any
// row sees, tp the tiles of cached positions.  m > 0: m requests from b on that share their
// first S positions, n + 1 = m R entries, nb boxes of their own.
struct TcLot {
  int b, m, nb, S, n, begin, T, tp, blocks, cum, units, reserved;
};

struct TcList {
  const TcLot* lots;
  const int* head;    // units of all lots, and their number
  const int* ranges;  // the tiles that row blocks see, or null: see ranges_kernel
  int words;          // of a request in it
};

// A request's own boxes past the positions that it shares, the cached ones and all.
__device__ __forceinline__ int cached_boxes(const sv_attention_args& a, int box, int shift, int shared, Extent E) {
  const int keys = max(0, E.S - shared) + (a.stage.data ? 0 : E.n + 1);
  return E.n < 0 ? 0 : (keys + box - 1) >> shift;
}
__device__ __forceinline__ int own_boxes(const sv_attention_args& a, int box, int shift, int shared, Extent E) {
  return cached_boxes(a, box, shift, shared, E) + (a.stage.data ? (E.n + box) >> shift : 0);
}

// What the host decides of a call's lists.  Lists: of items of 128 rows and of 256
// (the attention's kernels have row tiles for one or the other); which: 1, 2 or 3 (both: a
// lot of more than 128 rows goes to the second).
struct TcPlanning {
  sv_attention_args a;
  int which, box, shift, group;
  bool sharing;
  int* ranges;  // of row blocks of the list's rows, or null
  int words;
  TcLot* lots[2];
  int* head;  // [2][2]
  int* err;
};

sv_status plan_launch(const TcPlanning& p, cudaStream_t stream);

}  // namespace sv
