// The (token, rank) pairs of a routed batch sorted by expert: the launcher that
// the sort call and the MXFP4 expert FFN share.
#pragma once

#include "common.cuh"

namespace si {

constexpr int kSortMaxExperts = 1024;
constexpr int kSortFewPairs = 4096;    // pairs that one launch sorts (5.5 us; two launches 5.6)
constexpr int kSortChunks = 64;        // chunks of a longer batch

// For pairs = n_tokens * top_k ids: position[i] = place of pair i (by expert,
// then by i) or -1 for ids outside [0, E); offsets[e] = first place of expert
// e, offsets[E] = number of kept pairs; order = the inverse of position, -1
// behind the kept pairs (either may be NULL).
// tile_rows > 0: every expert's places start at a multiple of tile_rows
// instead, and the tiles of tile_rows places that hold pairs are listed:
// tile_expert[i], tile_count[i] (pairs in the tile), *n_tiles.
struct SortArgs {
  const int32_t *ids;
  int64_t pairs;
  int n_experts;
  int32_t *order, *position, *offsets;
  int tile_rows;
  int32_t *tile_expert, *tile_count, *n_tiles;
  int32_t *counts;   // sort_workspace_bytes, for more than kSortFewPairs pairs
  int64_t chunk;     // set by sort_launch
};
size_t sort_workspace_bytes(int64_t pairs, int n_experts);
cudaError_t sort_launch(SortArgs a, cudaStream_t s);

// y[t] = sum_r w[t][r] rows[position[t][r]] over fp32 rows of `hidden` values
// (a multiple of 4, 16-byte aligned), fp32 sums in rank order, rounded to bf16.
cudaError_t combine_launch(const float *rows, int64_t n_rows, int n_tokens, int top_k, int64_t hidden,
                           const int32_t *position, const float *w, void *y, cudaStream_t s);

// Expert of a pair, E for a dropped one (negative ids are large unsigned ones).
SI_DEV int sort_expert(const SortArgs &a, int64_t i) {
  return static_cast<int>(min(static_cast<uint32_t>(__ldcg(a.ids + i)), static_cast<uint32_t>(a.n_experts)));
}
SI_DEV int sort_tiles(const SortArgs &a, int n) { return a.tile_rows > 0 ? (n + a.tile_rows - 1) / a.tile_rows : 0; }
// The list entries of expert e: its pairs, first tile `t`.
SI_DEV void sort_list(const SortArgs &a, int e, int count, int t, int from, int step) {
  for (int i = from; i * a.tile_rows < count; i += step) {
    a.tile_expert[t + i] = e;
    a.tile_count[t + i] = min(a.tile_rows, count - i * a.tile_rows);
  }
}

}  // namespace si
