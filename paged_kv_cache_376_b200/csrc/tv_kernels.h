// Internal launch interface between the C ABI (tv_api.cu) and the kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace tv {

// SMs of the current device (asked for once per device).
inline int device_sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed))
    return known[dev].load(std::memory_order_relaxed);
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
      cudaSuccess)
    return 0;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Launch with `bytes` of dynamic shared memory (the kernel's limit is raised
// once per device).  With `overlap` the grid may start before the stream's last
// kernel has ended (programmatic dependent launch); it waits for it with
// wait_for_last_kernel() (tv_device.cuh).
template <auto kKernel, typename... Args>
cudaError_t launch_kernel(dim3 grid, int threads, int bytes, bool overlap,
                          cudaStream_t stream, Args... args) {
  static std::atomic<uint64_t> raised;
  uint64_t bit = 0;
  bool known = true;
  if (bytes > 48 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    bit = dev < 64 ? 1ull << dev : 0;
    known = raised.load(std::memory_order_relaxed) & bit;
  }
  auto raise = [&]() {
    cudaError_t e = cudaFuncSetAttribute(
        kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_relaxed);
    return e;
  };
  if (!known) {
    cudaError_t e = raise();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kKernel, args...);
  if (e == cudaErrorInvalidValue && bit) {
    // a device that was reset has forgotten the limit
    (void)cudaGetLastError();
    e = raise();
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kKernel, args...);
  }
  return e;
}

struct DecodeArgs {
  __nv_bfloat16* out;            // [B][Hq][D]            (unsplit)
  float* partial_out;            // [B][Hq][maxP][D]      (split)
  float* partial_lse;            // [B][Hq][maxP]         (split)
  const __nv_bfloat16* q;        // [B][Hq][D]
  const __nv_bfloat16* k_new;    // [B][Hkv][D] (fused append; else null)
  const __nv_bfloat16* v_new;
  __nv_bfloat16* k_pool_w;       // pools, written by the fused append
  __nv_bfloat16* v_pool_w;
  const int32_t* block_tables;   // [B][max_blocks_per_seq]
  const int32_t* context_lens;   // [B]
  // nullable; grown[s] == 0 makes sequence s idle (no append, zero output):
  // the pool's marks of the sequences whose context the step's slot
  // reservation grew (tv_decode_step only)
  const int32_t* grown;
  uint32_t* err;                 // nullable
  // fused append only: RoPE of the new K row at position ctx-1 (nullable)
  const float* rope_cos_sin;     // [rope_max_position][2][32] fp32
  int rope_max_position;
  int max_blocks_per_seq;
  int num_q_heads;
  int num_pages;
  int partition_tokens;
  int max_partitions;
  float scale_log2;              // scale * log2(e)
  int page_shift;                // page_size = 16 << page_shift
  // work-balanced decode only
  int num_seqs;
  int num_kv_heads;
  int32_t* ws_counters;          // [warps of the grid], zero between launches
  float* ws_partials;            // [warps][2][kSlotFloats]
};

// Work-balanced decode (paged_decode_balanced.cu).
constexpr int kMaxBalancedSeqs = 512;    // prefix sums live in shared memory
constexpr int kMinPagesPerWarp = 4;      // smallest range a warp is given
constexpr int kMaxDecodeCtasPerSm = 4;   // of four warps each
constexpr int kSlotFloats = 16 + 8 * 64; // m[8], l[8], acc[8][64] per segment

int balanced_decode_ctas_per_sm(int group, bool append);
cudaError_t launch_balanced_decode(const DecodeArgs& a, const CUtensorMap& tk,
                                   const CUtensorMap& tv, int group, int ctas,
                                   cudaStream_t stream);

cudaError_t launch_paged_decode(const DecodeArgs& a, const CUtensorMap& tk,
                                const CUtensorMap& tv, int num_kv_heads,
                                int num_seqs, int group, bool split,
                                int parts, cudaStream_t stream);

// Device page pool (page_pool.cu).  Error bits beyond those of tv_device.cuh.
constexpr uint32_t DEVERR_POOL_EMPTY = 1u << 5;  // too few free pages
constexpr uint32_t DEVERR_BAD_SEQ = 1u << 6;     // bad fork / release index
constexpr uint32_t DEVERR_BAD_POSITION = 1u << 7;  // RoPE position off the table
constexpr int kPoolMaxSeqs = 1024;               // one thread per sequence

cudaError_t launch_pool_init(int32_t* state, int num_pages, int page_size,
                             const int32_t* bt, int mb, const int32_t* ctx,
                             int num_seqs, uint32_t* err, cudaStream_t stream);
cudaError_t launch_pool_append(int32_t* state, int num_pages, int page_size,
                               int32_t* bt, int mb, int32_t* ctx,
                               const int32_t* n_new, int num_seqs,
                               int32_t* slot_mapping, void* k_pool,
                               void* v_pool, int row_bytes, uint32_t* err,
                               cudaStream_t stream);
cudaError_t launch_pool_fork(int32_t* state, int num_pages, int32_t* bt,
                             int mb, int32_t* ctx, int num_seqs,
                             const int32_t* src, const int32_t* dst,
                             int num_pairs, uint32_t* err,
                             cudaStream_t stream);
cudaError_t launch_pool_release(int32_t* state, int num_pages, int32_t* bt,
                                int mb, int32_t* ctx, int num_seqs,
                                const int32_t* seqs, int num_release,
                                uint32_t* err, cudaStream_t stream);

cudaError_t launch_pool_truncate(int32_t* state, int num_pages, int32_t* bt,
                                 int mb, int32_t* ctx, const int32_t* new_lens,
                                 int num_seqs, uint32_t* err,
                                 cudaStream_t stream);
// Pools may be null (tables and moves only).
cudaError_t launch_pool_compact(int32_t* state, int num_pages, int page_size,
                                int32_t* bt, int mb, const int32_t* ctx,
                                int num_seqs, int32_t* move_src,
                                int32_t* move_dst, int32_t* num_moves,
                                void* k_pool, void* v_pool, int row_bytes,
                                uint32_t* err, cudaStream_t stream);
cudaError_t launch_page_copy(void* k_pool, void* v_pool, int num_pages,
                             int page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t max_pairs,
                             const int32_t* num_pairs, uint32_t* err,
                             cudaStream_t stream);

// Bounded-wait self-test (selftest.cu).
cudaError_t launch_wait_selftest(uint32_t* err, unsigned long long limit_ns,
                                 unsigned long long* waited_ns,
                                 cudaStream_t stream);

cudaError_t launch_kv_append_rope(const void* k_new, const void* v_new,
                                  const int32_t* slot_mapping,
                                  const int32_t* positions, int64_t num_tokens,
                                  void* k_pool, void* v_pool,
                                  int64_t num_slots, int num_kv_heads,
                                  const float* rope_cos_sin,
                                  int rope_max_position, uint32_t* err,
                                  cudaStream_t stream);

struct MropeArgs {
  __nv_bfloat16* q_out;          // [T][Hq][D], null: K and V only
  const __nv_bfloat16* q;        // token t at q + t * q_stride
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  const int32_t* slot_mapping;   // [T]
  const int32_t* positions;      // [num_axes][T]
  const int32_t* pair_axis;      // [D / 2]
  int64_t num_tokens;
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  int64_t num_slots;
  const float* cos_sin;          // [max_position][2][D / 2]
  uint32_t* err;
  int num_axes;
  int max_position;
  int num_q_heads;               // 0 when q_out is null
  int num_kv_heads;
};
cudaError_t launch_kv_append_mrope(const MropeArgs& a, cudaStream_t stream);

cudaError_t launch_kv_append(const void* k_new, const void* v_new,
                             const int32_t* slot_mapping, int64_t num_tokens,
                             void* k_pool, void* v_pool, int64_t num_slots,
                             int row_bytes, uint32_t* err,
                             cudaStream_t stream);

cudaError_t launch_split_merge(__nv_bfloat16* out, const float* partial_out,
                               const float* partial_lse,
                               const int32_t* context_lens, int num_seqs,
                               int num_q_heads, int partition_tokens,
                               int max_partitions, cudaStream_t stream);

struct PrefillArgs {
  __nv_bfloat16* out;            // [rows][Hq][D]
  const int32_t* query_start_loc;  // [B+1]
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint32_t* err;
  int max_blocks_per_seq;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int num_pages;
  int max_query_len;
  int64_t num_query_rows;
  float scale_log2;
  int page_shift;                // page_size = 16 << page_shift
  int group;                     // query heads per KV head: 1, 2, 4 or 8
  // Dispatch order: order[i] = seq * prefill_blocks(max_query_len, group) + block of
  // the i-th CTA group (costliest first), written by the ordering kernel
  // into caller workspace; nullptr = grid order.
  int32_t* order;
};

// A prefill CTA owns two MMA tiles of 128 rows = (128 / group) query rows x
// the group's heads, so 256 / group query rows (chunk positions).
constexpr int kPrefillTileRows = 128;
__host__ __device__ inline int prefill_rows_per_cta(int group) {
  return 2 * kPrefillTileRows / group;
}
__host__ __device__ inline int prefill_blocks(int max_query_len, int group) {
  const int rows = prefill_rows_per_cta(group);
  return (max_query_len + rows - 1) / rows;
}

// Launches the ordering kernel first when a.order is set.
cudaError_t launch_paged_prefill(const PrefillArgs& a, const CUtensorMap& tq,
                                 const CUtensorMap& tk, const CUtensorMap& tv,
                                 cudaStream_t stream);

// Attention of a chunk of rows per sequence (paged_chunk.cu, and for more than
// stream_rows rows paged_chunk_tile.cu).
struct ChunkEntry {              // work of the tile kernel, for every KV head
  int32_t seq, blk;              // sequence, block of 256 rows x heads
  int32_t tile0, tile1;          // range of key tiles
  int32_t part_base, part, parts;  // of a block cut along the keys
  int32_t pad;
};
struct ChunkPlan {
  int32_t entries;
  int32_t next;                  // unit (entry x KV head) to be taken next
  int32_t joins;                 // cut blocks
  int32_t failed;                // a wait of the tile kernel ran out (read
                                 // with `joins`)
};
struct ChunkArgs {
  __nv_bfloat16* out;            // [rows][Hq][D]
  const __nv_bfloat16* q;        // [rows][Hq][D]
  const int32_t* query_start_loc;  // [B+1]
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint32_t* err;
  int max_blocks_per_seq;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int num_pages;
  int max_query_len;
  int64_t num_query_rows;
  float scale_log2;
  int page_shift;                // page_size = 16 << page_shift
  int group_shift;               // query heads per KV head = 1 << group_shift
  // With a workspace: CTAs of the balanced grid (0: one CTA per KV head, row
  // block and sequence), which serves the sequences of up to stream_rows rows.
  int balanced_ctas;             // kChunkCtasPerSm per SM
  int stream_rows;
  int32_t* ws_counters;          // [balanced_ctas], zero between calls
  float* ws_parts;               // [balanced_ctas][2][kChunkPartFloats]
  // The tile kernel's part of the workspace (tile_ctas 0: not launched).
  int tile_ctas;
  ChunkPlan* plan;
  ChunkEntry* plan_entries;
  int4* plan_joins;              // cut blocks: sequence, block, part_base, parts
  float* tile_parts;             // [4 tile_ctas][kTilePartFloats]
};
constexpr int kMaxChunkSeqs = 1024;     // prefix sums live in shared memory
constexpr int kMinChunkBlocks = 16;     // 16-token blocks worth a CTA
constexpr int kChunkPartRows = 32;      // rows x heads per KV head
// m, l and the unscaled output of one part
constexpr int kChunkPartFloats = kChunkPartRows * (2 + 64);
constexpr int kChunkCtasPerSm = 3;     // at most
// m, l and the unscaled output of two query tiles of 128 rows
constexpr int kTilePartFloats = 2 * 128 * (2 + 64);
__host__ __device__ inline int chunk_tile_blocks(int max_query_len,
                                                 int group_shift) {
  return (int)((((int64_t)max_query_len << group_shift) + 255) / 256);
}

cudaError_t launch_paged_chunk(const ChunkArgs& a, const CUtensorMap& tk,
                               const CUtensorMap& tv, bool causal,
                               cudaStream_t stream);
// The plan kernel and the tile kernel.
cudaError_t launch_chunk_tiles(const ChunkArgs& a, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv,
                               bool causal, cudaStream_t stream);

}  // namespace tv
