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
// Items of 256 rows: a tile takes them 7000 cycles (8400 then), their start and end 15000.  Prompts of up to 2041
// entries under a window, listed with a lead of 6: 258 us; with 2: 245.
constexpr int kLeadWide = 2;
// Items of up to this many key tiles are not shared between CTAs: a tile is
// 0.9 us for a CTA alone, joining parts 3 us and more.  A single request leaves
// most of the GPU idle, so its items are shared earlier: one token over 777
// positions (7 tiles, 8 heads) 13.1 us shared, 14.8 whole; six trees over 100 to
// 1000 positions 20.7 shared, 18.6 whole; 64 over 16 to 520 51.2 and 42.8.
constexpr int kWholeOne = 6, kWhole = 12;
// Units of a share: more rows take longer to join.  One token (4 rows a head)
// over 2000 positions 16.7 us with 1, 14.6 with 2, 15.7 with 4, 22.1 with 10; a
// tree of 15 nodes (60 rows) 27.7, 22.4, 20.6 and 26.3.
constexpr int kLeastFew = 2, kLeastMany = 4, kFewRows = 32;

__device__ __forceinline__ int sharing_ctas(const sv_attention_args& a, int group, int grid, int total) {
  const int least = a.R * group <= kFewRows ? kLeastFew : kLeastMany;
  return min(grid, (total + least - 1) / least);
}

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
  const int* head;    // units of all lots, their number, and those of an item that stays whole
  const int* first;   // the lot in which each CTA's share starts
  const int* ranges;  // the tiles that row blocks see, or null: see ranges_kernel
  int words;          // of a request in it
  int lead;           // units of an item besides its tiles
};

// A request's own boxes past the positions that it shares, the cached ones and all.
__device__ __forceinline__ int cached_boxes(const sv_attention_args& a, int box, int shift, int shared, Extent E) {
  const int keys = max(0, E.S - shared) + (a.stage.data ? 0 : E.n + 1);
  return E.n < 0 ? 0 : (keys + box - 1) >> shift;
}
__device__ __forceinline__ int own_boxes(const sv_attention_args& a, int box, int shift, int shared, Extent E) {
  return cached_boxes(a, box, shift, shared, E) + (a.stage.data ? (E.n + box) >> shift : 0);
}

// What the host decides of a call's list.  rows: of an item, 128 or 256.
struct TcPlanning {
  sv_attention_args a;
  int rows, lead, box, shift, group, ctas;
  bool sharing;
  int* ranges;  // of row blocks of that many rows, or null
  int words;
  TcLot* lots;
  int *head, *first;
  int* err;
};

sv_status plan_launch(const TcPlanning& p, cudaStream_t stream);

}  // namespace sv
