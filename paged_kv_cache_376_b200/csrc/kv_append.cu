// KV append: scatter each new token's K and V rows into their page slots.
//
// "tiny-vllm：从零构建高性能LLM推理引擎的完整指南", sec. "推理流程：从Prefill到
// Decode": every generated token's K,V are computed and appended to the cache;
// "Tiny-vLLM 实战：用 C++/CUDA 手写高性能 LLM 推理引擎", sec. "内存池管理": a
// page holds page_size token rows of num_kv_heads x head_dim bf16 values.
// Slot s names row s of the pool viewed as [num_pages * page_size][row]
// (page s / page_size, offset s % page_size).  Negative slots are padding.
//
// The copy is bit-exact: one thread moves one 16-byte vector, so a token row
// of 1 KB (8 heads x 64 x bf16) is 64 fully coalesced vectors per tensor.
// The grid is a multiple of the SM count and strides over the work.  A
// second kernel rotates K by RoPE on the way (tv_kv_append_rope).
#include "tv_device.cuh"
#include "tv_kernels.h"

namespace tv {
namespace {

__global__ void __launch_bounds__(256)
    kv_append_kernel(const uint4* __restrict__ k_new,
                     const uint4* __restrict__ v_new,
                     const int32_t* __restrict__ slot_mapping,
                     int64_t num_tokens, uint4* __restrict__ k_pool,
                     uint4* __restrict__ v_pool, int64_t num_slots,
                     int row_vecs, uint32_t* err) {
  const int64_t per_token = 2 * (int64_t)row_vecs;  // K vectors then V
  const int64_t total = num_tokens * per_token;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per_token;
    const int r = (int)(i - t * per_token);
    const int64_t slot = slot_mapping[t];
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (r == 0) flag_error(err, DEVERR_BAD_SLOT);
      continue;
    }
    if (r < row_vecs) {
      k_pool[slot * row_vecs + r] = k_new[t * row_vecs + r];
    } else {
      const int c = r - row_vecs;
      v_pool[slot * row_vecs + c] = v_new[t * row_vecs + c];
    }
  }
}

// RoPE variant ("tiny-vllm：从零构建高性能LLM推理引擎的完整指南", sec. "Llama
// 3.2 1B架构拆解": the position enters K by a rotation; V is copied as is).
// A head of a K row is 8 vectors of 8 dimensions; vector u < 4 pairs with
// vector u + 4 (dimensions i and i + 32), so one work item moves such a pair
// (rotated) and the 8 V vectors are 8 more items: 12 items per head.
__global__ void __launch_bounds__(256)
    kv_append_rope_kernel(const uint4* __restrict__ k_new,
                          const uint4* __restrict__ v_new,
                          const int32_t* __restrict__ slot_mapping,
                          const int32_t* __restrict__ positions,
                          int64_t num_tokens, uint4* __restrict__ k_pool,
                          uint4* __restrict__ v_pool, int64_t num_slots,
                          int num_kv_heads, const float* __restrict__ cos_sin,
                          int max_position, uint32_t* err) {
  const int row_vecs = num_kv_heads * 8;
  const int64_t per_token = 12 * (int64_t)num_kv_heads;
  const int64_t total = num_tokens * per_token;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per_token;
    const int r = (int)(i - t * per_token);
    const int h = r / 12, u = r - 12 * h;
    const int64_t slot = slot_mapping[t];
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (r == 0) flag_error(err, DEVERR_BAD_SLOT);
      continue;
    }
    const int64_t src = t * row_vecs + h * 8;
    const int64_t dst = slot * row_vecs + h * 8;
    if (u < 4) {
      uint4 lo = k_new[src + u], hi = k_new[src + u + 4];
      const int pos = positions[t];
      if (pos >= 0 && pos < max_position) {
        float c8[8], s8[8];
        rope_load8(cos_sin, pos, 8 * u, c8, s8);
        rope_rotate8(lo, hi, c8, s8);
      } else if (r == 0) {
        flag_error(err, DEVERR_BAD_POSITION);
      }
      k_pool[dst + u] = lo;
      k_pool[dst + u + 4] = hi;
    } else {
      v_pool[dst + u - 4] = v_new[src + u - 4];
    }
  }
}

// RoPE by positions of several axes, on q and K.  Pair (i, i + 32) of every
// head turns by the angle of positions[pair_axis[i]] (time, height, width, ...
// of an image or video token), looked up in one cos/sin table; the arithmetic
// is that of kv_append_rope_kernel.
//
// Bound: bytes, 2 x (Hq + 2 Hkv) x 128 per token plus its angles.  One warp per
// token: lane i looks up pair i's angle once (its axis, its position, two table
// entries), the lanes exchange them by shuffles, and every lane turns the
// vector pair u = lane & 3 (dimensions 8u .. 8u + 7 with + 32) of heads
// lane >> 2, + 8, + 16, ... , so the angles are read once per token however
// many heads it has.  The first heads' vectors are loaded before the angles,
// whose two lookups depend on one another.  Two head vectors a lane in flight at
// 64 registers: 8192 tokens of 32 + 16 heads 16.7 us (6.1 TB/s; three at 80
// registers, fewer warps: 18.7), 64 tokens 4.2 us.
__global__ void __launch_bounds__(128, 8)
    kv_append_mrope_kernel(const MropeArgs a) {
  constexpr int kHeads = 2;   // heads of a lane in flight at once
  const int lane = threadIdx.x & 31;
  const int u = lane & 3;
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int axis = a.pair_axis[lane];
  const bool axis_ok = axis >= 0 && axis < a.num_axes;
  const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
  uint4 lo[kHeads], hi[kHeads];
  auto load = [&](int64_t t, int h0) {
#pragma unroll
    for (int n = 0; n < kHeads; ++n) {
      const int h = h0 + 8 * n;
      if (h >= heads) continue;
      const int hk = h - a.num_q_heads, hv = hk - a.num_kv_heads;
      const __nv_bfloat16* src =
          hk < 0   ? a.q + t * a.q_stride + h * 64
          : hv < 0 ? a.k_new + t * a.k_stride + hk * 64
                   : a.v_new + t * a.v_stride + hv * 64;
      lo[n] = reinterpret_cast<const uint4*>(src)[u];
      hi[n] = reinterpret_cast<const uint4*>(src)[u + 4];
    }
  };
  for (int64_t t = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
       t < a.num_tokens; t += stride) {
    const int64_t slot = a.slot_mapping[t];
    const int pos = axis_ok ? a.positions[axis * a.num_tokens + t] : -1;
    load(t, lane >> 2);
    if (slot < 0) continue;                  // padding
    const bool slot_ok = slot < a.num_slots;
    // a token turns as a whole or, with a bad position, not at all
    const bool turn = __all_sync(0xffffffffu, pos >= 0 && pos < a.max_position);
    if (lane == 0) {
      if (!slot_ok) flag_error(a.err, DEVERR_BAD_SLOT);
      if (!turn) flag_error(a.err, DEVERR_BAD_POSITION);
    }
    float cl = 1.f, sl = 0.f;
    if (turn) {
      cl = __ldg(a.cos_sin + (size_t)pos * 64 + lane);
      sl = __ldg(a.cos_sin + (size_t)pos * 64 + 32 + lane);
    }
    float c8[8], s8[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c8[k] = __shfl_sync(0xffffffffu, cl, 8 * u + k);
      s8[k] = __shfl_sync(0xffffffffu, sl, 8 * u + k);
    }
    for (int h0 = lane >> 2; h0 < heads; h0 += 8 * kHeads) {
      if (h0 >= 8 * kHeads) load(t, h0);
#pragma unroll
      for (int n = 0; n < kHeads; ++n) {
        const int h = h0 + 8 * n;
        if (h >= heads) continue;
        const int hk = h - a.num_q_heads, hv = hk - a.num_kv_heads;
        if (hk >= 0 && !slot_ok) continue;
        if (hv < 0 && turn) rope_rotate8(lo[n], hi[n], c8, s8);
        __nv_bfloat16* dst =
            hk < 0   ? a.q_out + (t * a.num_q_heads + h) * 64
            : hv < 0 ? a.k_pool + (slot * a.num_kv_heads + hk) * 64
                     : a.v_pool + (slot * a.num_kv_heads + hv) * 64;
        reinterpret_cast<uint4*>(dst)[u] = lo[n];
        reinterpret_cast<uint4*>(dst)[u + 4] = hi[n];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append_mrope(const MropeArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int64_t want = (a.num_tokens + 3) / 4;
  const int64_t cap = (int64_t)device_sm_count() * 64;
  kv_append_mrope_kernel<<<(int)(want < cap ? want : cap), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append_rope(const void* k_new, const void* v_new,
                                  const int32_t* slot_mapping,
                                  const int32_t* positions, int64_t num_tokens,
                                  void* k_pool, void* v_pool,
                                  int64_t num_slots, int num_kv_heads,
                                  const float* rope_cos_sin,
                                  int rope_max_position, uint32_t* err,
                                  cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  const int64_t total = num_tokens * 12 * num_kv_heads;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t want = (total + 255) / 256;
  const int64_t cap = (int64_t)sms * 8;
  const int blocks = (int)(want < cap ? want : cap);
  kv_append_rope_kernel<<<blocks, 256, 0, stream>>>(
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
      slot_mapping, positions, num_tokens, static_cast<uint4*>(k_pool),
      static_cast<uint4*>(v_pool), num_slots, num_kv_heads, rope_cos_sin,
      rope_max_position, err);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const void* k_new, const void* v_new,
                             const int32_t* slot_mapping, int64_t num_tokens,
                             void* k_pool, void* v_pool, int64_t num_slots,
                             int row_bytes, uint32_t* err,
                             cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  const int row_vecs = row_bytes / 16;
  const int64_t total = num_tokens * 2 * row_vecs;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t want = (total + 255) / 256;
  const int64_t cap = (int64_t)sms * 8;
  const int blocks = (int)(want < cap ? want : cap);
  kv_append_kernel<<<blocks, 256, 0, stream>>>(
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
      slot_mapping, num_tokens, static_cast<uint4*>(k_pool),
      static_cast<uint4*>(v_pool), num_slots, row_vecs, err);
  return cudaGetLastError();
}

}  // namespace tv
