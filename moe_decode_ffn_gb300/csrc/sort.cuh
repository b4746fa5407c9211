// The (token, rank) pairs of a routed batch sorted by expert: the launcher that
// the sort call and the MXFP4 expert FFN share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace si {

constexpr int kSortMaxExperts = 1024;
constexpr int kSortFewPairs = 2048;    // pairs that one launch sorts
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

// y[t] = sum_r w[t][r] rows[position[t][r]] over bf16 rows of `hidden` values
// (a multiple of 8, 16-byte aligned), fp32 sums in rank order.
cudaError_t combine_launch(const void *rows, int64_t n_rows, int n_tokens, int top_k, int64_t hidden,
                           const int32_t *position, const float *w, void *y, cudaStream_t s);

}  // namespace si
