// What the two kernels of chunk and cross attention (paged_chunk.cu,
// paged_chunk_tile.cu) have in common.
#pragma once

#include "tv_device.cuh"
#include "tv_kernels.h"

namespace tv {

// The running offset of a row that has seen no finite score: the lowest finite
// number.  Any finite score exceeds it, and a score of minus infinity (an infinity
// in K) against it is weight 0; against an offset of minus infinity it would be
// NaN.
constexpr float kNoOffset = -3.402823466e38f;

// The key tiles of a block, from the rows it covers.
struct TileBlock {
  int q_row;            // first query row in q / out
  int tb;               // query rows
  int first_limit;      // last key that the first row sees
  int key_end;          // keys that some row sees: [0, key_end)
};

template <bool kCausal>
__device__ __forceinline__ bool tile_block(const ChunkArgs& a, int seq,
                                           int blk, TileBlock* b) {
  const int qs = a.query_start_loc[seq];
  const int T = a.query_start_loc[seq + 1] - qs;
  const int cap = a.max_blocks_per_seq * (16 << a.page_shift);
  const int ctx = min(max(a.context_lens[seq], 0), cap);
  // what is out of range is flagged by the streaming kernel of this call
  if (T <= a.stream_rows || T > a.max_query_len || qs < 0 ||
      (int64_t)qs + T > a.num_query_rows || (kCausal && T > ctx))
    return false;
  const int rows = 256 >> a.group_shift;
  const int t0 = blk * rows;
  if (t0 >= T) return false;
  b->q_row = qs + t0;
  b->tb = min(rows, T - t0);
  b->first_limit = kCausal ? ctx - T + t0 : ctx - 1;
  b->key_end = kCausal ? b->first_limit + b->tb : ctx;
  return true;
}

}  // namespace tv
