// KV page pool on the device: free-page stack, per-page reference counts,
// on-demand allocation with copy-on-write of shared pages, fork and release.
//
// What it follows: "Tiny-vLLM 实战：用 C++/CUDA 手写高性能 LLM 推理引擎",
// sec. 内存池管理 (pages allocated when a request produces a new token,
// returned to the free pool when it ends, shared between requests for prefix
// caching; a free-page list is the pool's core structure), and
// "tiny-vllm：从零构建高性能LLM推理引擎的完整指南", sec. PagedAttention (pages
// allocated only when needed; sharing made safe by copy-on-write).
//
// B200 design.  The pool lives in device memory so a decode step (room for
// the new token, then the fused append + attention) runs without the host
// and can be captured in a CUDA graph.  The free list is an array stack
// (constant-time pop/push by index arithmetic instead of a pointer chase).
// The bookkeeping kernels run as one CTA of 1024 threads, one thread per
// sequence (B <= 1024), and take every decision with block-wide scans in a
// fixed order, so the pages a call hands out do not depend on thread timing:
//   * needs are reserved in batch order (exclusive scan), pops take
//     stack[top-1-offset-j];
//   * copy-on-write: a sequence writing into a partly filled page held by
//     r > 1 rows copies it first, except the last writer of that page in
//     batch order when all r holders write this step (that one keeps it);
//     the number of writers per page and the last one are found with
//     atomicAdd / atomicMax on two scratch arrays, both order-independent;
//   * released pages whose count reaches zero are pushed in ascending id
//     order (a scan over the whole pool).
// All of this is integer index work; pages are copied with 16-byte vectors.
#include <cstdint>

#include "tv_device.cuh"
#include "tv_kernels.h"

namespace tv {
namespace {

constexpr int kThreads = 1024;

struct PoolView {
  int32_t* top;
  int32_t* last_slots;   // slots written by the last append call
  int32_t* page_size;    // tokens per page, set by init (16 or 32)
  int32_t* stack;        // [num_pages]
  int32_t* ref;          // [num_pages]
  int32_t* cnt_app;      // [num_pages], zero between calls
  int32_t* last_app;     // [num_pages], zero between calls
  int32_t* grown;        // [kPoolMaxSeqs]: 1 = got its tokens in the last
                         // append call, 0 = did not (idle, unserved, flagged)
  int num_pages;
};

__host__ __device__ inline PoolView view(int32_t* state, int num_pages) {
  PoolView v;
  v.top = state + 0;
  v.last_slots = state + 2;
  v.page_size = state + 3;
  v.stack = state + 4;
  v.ref = v.stack + num_pages;
  v.cnt_app = v.ref + num_pages;
  v.last_app = v.cnt_app + num_pages;
  v.grown = v.last_app + num_pages;
  v.num_pages = num_pages;
  return v;
}

__device__ __forceinline__ int pages_for(int ctx, int ps) {
  return (ctx + ps - 1) / ps;
}

// Exclusive scan of one int per thread over the threads of the CTA (a
// multiple of 32, at most 1024); *total receives the sum.  `sh` holds 33
// ints.
__device__ int block_exclusive_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  __syncthreads();  // sh may still be read by a previous scan
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < (int)(blockDim.x >> 5) ? sh[lane] : 0;
    int wi = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, wi, off);
      if (lane >= off) wi += t;
    }
    sh[lane] = wi - w;                // exclusive prefix of warp totals
    if (lane == 31) sh[32] = wi;      // grand total
  }
  __syncthreads();
  const int res = sh[warp] + incl - v;
  *total = sh[32];
  return res;
}

// ---- init -------------------------------------------------------------------
__global__ void pool_clear_kernel(PoolView p) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.num_pages;
       i += gridDim.x * blockDim.x) {
    p.ref[i] = 0;
    p.cnt_app[i] = 0;
    p.last_app[i] = 0;
  }
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < kPoolMaxSeqs;
       i += gridDim.x * blockDim.x)
    p.grown[i] = 0;
}

__global__ void pool_count_refs_kernel(PoolView p, const int32_t* bt, int mb,
                                       const int32_t* ctx, int num_seqs,
                                       int kPS, uint32_t* err) {
  const int64_t total = (int64_t)num_seqs * mb;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int s = (int)(i / mb), b = (int)(i % mb);
    int c = ctx[s];
    if (c < 0 || c > mb * kPS) {
      if (b == 0) flag_error(err, DEVERR_BAD_CONTEXT);
      c = c < 0 ? 0 : mb * kPS;
    }
    if (b >= pages_for(c, kPS)) continue;
    const int page = bt[(size_t)s * mb + b];
    if (page < 0 || page >= p.num_pages) {
      flag_error(err, DEVERR_BAD_PAGE);
      continue;
    }
    atomicAdd(p.ref + page, 1);
  }
}

// stack = unreferenced pages in descending id order (a fresh pool pops 0, 1..)
__global__ void __launch_bounds__(kThreads, 1)
    pool_stack_kernel(PoolView p, int page_size) {
  __shared__ int sh[33];
  int base = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int page = p.num_pages - 1 - i;
    const int f = (i < p.num_pages && p.ref[page] == 0) ? 1 : 0;
    int tot;
    const int pos = block_exclusive_scan(f, sh, &tot);
    if (f) p.stack[base + pos] = page;
    base += tot;
  }
  if (threadIdx.x == 0) {
    *p.top = base;
    *p.last_slots = 0;
    *p.page_size = page_size;
  }
}

// ---- append slots -----------------------------------------------------------
// Room for n[s] new tokens at positions ctx .. ctx+n-1 of every sequence.
__global__ void __launch_bounds__(kThreads, 1)
    pool_append_kernel(PoolView p, int32_t* bt, int mb, int32_t* ctx,
                       const int32_t* n_new, int num_seqs,
                       int32_t* slot_mapping, uint8_t* k_pool,
                       uint8_t* v_pool, int row_bytes, int kPS,
                       uint32_t* err) {
  __shared__ int sh[33];
  __shared__ int job_old[kThreads], job_new[kThreads];
  const int s = threadIdx.x;
  const bool live = s < num_seqs;
  // The loads that do not depend on one another go out together (the kernel
  // is a chain of dependent round trips: context -> last page -> its
  // reference count -> free-stack pops); nothing below writes top or ref
  // before the scans.
  const int pool_ps = *p.page_size;
  const int top = *p.top;
  int c = live ? ctx[s] : 0;
  int n = live && n_new ? n_new[s] : 0;
  if (pool_ps != kPS) {   // pools of another page size: touch nothing
    if (threadIdx.x == 0) flag_error(err, DEVERR_BAD_SEQ);
    if (live) p.grown[s] = 0;
    return;
  }
  int part = -1, r = 0;
  if (live) {
    // decode steps (n_new == nullptr) add one token to every live sequence
    if (!n_new) n = c > 0 ? 1 : 0;
    if (n < 0) n = 0;
    if (c < 0 || c + n > mb * kPS) {
      flag_error(err, DEVERR_BAD_CONTEXT);
      n = 0;
    }
    if (n > 0 && c % kPS) {
      part = bt[(size_t)s * mb + c / kPS];
      if (part < 0 || part >= p.num_pages) {
        flag_error(err, DEVERR_BAD_PAGE);
        n = 0;
        part = -1;
      } else {
        atomicAdd(p.cnt_app + part, 1);
        atomicMax(p.last_app + part, s + 1);
        r = p.ref[part];
      }
    }
  }
  __syncthreads();
  // copy-on-write decision (see the file comment) and pages needed; the
  // writer counts are read only for a shared page
  bool cow = false;
  if (part >= 0 && r > 1)
    cow = !(p.cnt_app[part] == r && p.last_app[part] == s + 1);
  const int need =
      n > 0 ? (int)cow + pages_for(c + n, kPS) - pages_for(c, kPS) : 0;
  int total;
  const int off = block_exclusive_scan(need, sh, &total);
  const bool served = live && n > 0 && off + need <= top;
  if (live && n > 0 && !served) flag_error(err, DEVERR_POOL_EMPTY);
  // what a decode step launched next reads: only a sequence whose context
  // grew may append at its last position (any other would overwrite a
  // cached token there)
  if (live) p.grown[s] = served ? 1 : 0;
  int used;
  const int served_need = served ? need : 0;
  (void)block_exclusive_scan(served_need, sh, &used);
  int nslots;
  const int slot_off = block_exclusive_scan(served ? n : 0, sh, &nslots);

  // pops: stack[top-1-off], stack[top-2-off], ... (copy first)
  int job = -1;
  if (served) {
    int k = top - 1 - off;
    if (cow) {
      const int fresh = p.stack[k--];
      bt[(size_t)s * mb + c / kPS] = fresh;
      p.ref[fresh] = 1;
      atomicSub(p.ref + part, 1);
      job_old[s] = part;
      job_new[s] = fresh;
      job = s;
    }
    for (int b = pages_for(c, kPS); b < pages_for(c + n, kPS); ++b) {
      const int fresh = p.stack[k--];
      bt[(size_t)s * mb + b] = fresh;
      p.ref[fresh] = 1;
    }
    if (slot_mapping)
      for (int t = c; t < c + n; ++t)
        slot_mapping[slot_off + (t - c)] =
            bt[(size_t)s * mb + t / kPS] * kPS + t % kPS;
    ctx[s] = c + n;
  }
  // the scratch counters of every written page go back to zero
  __syncthreads();
  if (part >= 0) {
    p.cnt_app[part] = 0;
    p.last_app[part] = 0;
  }
  // copy-on-write copies: each job is one page of K and one of V
  int njobs;
  const int jpos = block_exclusive_scan(job >= 0 ? 1 : 0, sh, &njobs);
  __shared__ int jl_old[kThreads], jl_new[kThreads];
  if (job >= 0) {
    jl_old[jpos] = job_old[job];
    jl_new[jpos] = job_new[job];
  }
  __syncthreads();
  const int page_vec = kPS * row_bytes / 16;   // 16-byte vectors per page
  for (int j = 0; j < njobs; ++j) {
    const size_t src = (size_t)jl_old[j] * kPS * row_bytes;
    const size_t dst = (size_t)jl_new[j] * kPS * row_bytes;
    for (int v = threadIdx.x; v < page_vec; v += blockDim.x) {
      reinterpret_cast<uint4*>(k_pool + dst)[v] =
          reinterpret_cast<const uint4*>(k_pool + src)[v];
      reinterpret_cast<uint4*>(v_pool + dst)[v] =
          reinterpret_cast<const uint4*>(v_pool + src)[v];
    }
  }
  if (threadIdx.x == 0) {
    *p.top = top - used;
    *p.last_slots = nslots;
  }
}

// ---- fork ---------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads, 1)
    pool_fork_kernel(PoolView p, int32_t* bt, int mb, int32_t* ctx,
                     int num_seqs, const int32_t* src, const int32_t* dst,
                     int num_pairs, uint32_t* err) {
  const int kPS = *p.page_size;
  for (int i = 0; i < num_pairs; ++i) {
    const int a = src[i], b = dst[i];
    bool ok = a >= 0 && a < num_seqs && b >= 0 && b < num_seqs && a != b;
    int c = ok ? ctx[a] : 0;
    ok = ok && ctx[b] == 0 && c >= 0 && c <= mb * kPS;
    if (!ok) {
      if (threadIdx.x == 0) flag_error(err, DEVERR_BAD_SEQ);
      __syncthreads();
      continue;
    }
    const int np = pages_for(c, kPS);
    for (int k = threadIdx.x; k < mb; k += kThreads) {
      const int page = k < np ? bt[(size_t)a * mb + k] : -1;
      bt[(size_t)b * mb + k] = page;
      if (page >= 0 && page < p.num_pages) atomicAdd(p.ref + page, 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) ctx[b] = c;
    __syncthreads();
  }
}

// ---- release ------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads, 1)
    pool_release_kernel(PoolView p, int32_t* bt, int mb, int32_t* ctx,
                        int num_seqs, const int32_t* seqs, int num_release,
                        uint32_t* err) {
  constexpr int kList = 8192;   // freed pages sorted in shared memory
  __shared__ int sh[33];
  __shared__ int freed[kList];
  __shared__ int nfreed;
  const int kPS = *p.page_size;
  if (threadIdx.x == 0) nfreed = 0;
  __syncthreads();
  for (int i = 0; i < num_release; ++i) {
    const int s = seqs[i];
    if (s < 0 || s >= num_seqs) {
      if (threadIdx.x == 0) flag_error(err, DEVERR_BAD_SEQ);
      continue;
    }
    int c = ctx[s];
    c = c < 0 ? 0 : (c > mb * kPS ? mb * kPS : c);
    const int np = pages_for(c, kPS);
    for (int k = threadIdx.x; k < mb; k += kThreads) {
      if (k < np) {
        const int page = bt[(size_t)s * mb + k];
        if (page >= 0 && page < p.num_pages &&
            atomicSub(p.ref + page, 1) == 1) {
          p.last_app[page] = 1;   // freed in this call
          const int slot = atomicAdd(&nfreed, 1);
          if (slot < kList) freed[slot] = page;
        }
      }
      bt[(size_t)s * mb + k] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) ctx[s] = 0;
    __syncthreads();
  }
  // push the freed pages in ascending id order
  const int top = *p.top;
  const int n = nfreed;
  auto push = [&](int pos, int page) {
    // a consistent pool never overflows; a corrupted one is flagged
    if (top + pos < p.num_pages)
      p.stack[top + pos] = page;
    else
      flag_error(err, DEVERR_BAD_SEQ);
    p.last_app[page] = 0;
  };
  if (n <= kList) {
    // bitonic sort of the list, padded to a power of two
    int m = 1;
    while (m < n) m <<= 1;
    for (int i = n + threadIdx.x; i < m; i += kThreads) freed[i] = INT32_MAX;
    __syncthreads();
    for (int k = 2; k <= m; k <<= 1) {
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = threadIdx.x; i < m; i += kThreads) {
          const int ij = i ^ j;
          if (ij > i) {
            const int x = freed[i], y = freed[ij];
            if (((i & k) == 0) == (x > y)) {
              freed[i] = y;
              freed[ij] = x;
            }
          }
        }
        __syncthreads();
      }
    }
    for (int i = threadIdx.x; i < n; i += kThreads) push(i, freed[i]);
    if (threadIdx.x == 0) *p.top = min(top + n, p.num_pages);
    return;
  }
  // more than the list holds: scan the whole pool for the flags
  int base = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += kThreads) {
    const int page = i0 + threadIdx.x;
    const int f = (page < p.num_pages && p.last_app[page]) ? 1 : 0;
    int tot;
    const int pos = block_exclusive_scan(f, sh, &tot);
    if (f) push(base + pos, page);
    base += tot;
  }
  if (threadIdx.x == 0) *p.top = min(top + base, p.num_pages);
}

// ---- bitmaps of pages -----------------------------------------------------------
// Lists the set bits of words w0 .. w0 + nw - 1 in ascending order: emit(i, page)
// for the i-th, counted from `first`; returns the count behind the last.  One
// CTA of kThreads; a warp writes a word's pages side by side (one thread per
// word would scatter a CTA's stores over 32 lines each: 45 us instead of 4 for
// 18,000 pages).
constexpr int kWordChunk = 2 * kThreads;
struct BitList {
  uint32_t bits[kWordChunk];
  int base[kWordChunk];
  int sh[33];
};
template <typename Word, typename Emit>
__device__ __forceinline__ int list_bits(BitList& m, int words, int first,
                                         Word word, Emit emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int c0 = 0; c0 < words; c0 += kWordChunk) {
    const int w = c0 + 2 * threadIdx.x;
    const uint32_t b0 = w < words ? word(w) : 0u;
    const uint32_t b1 = w + 1 < words ? word(w + 1) : 0u;
    int total;
    const int pos = first + block_exclusive_scan(__popc(b0) + __popc(b1), m.sh,
                                                 &total);
    m.bits[2 * threadIdx.x] = b0;
    m.bits[2 * threadIdx.x + 1] = b1;
    m.base[2 * threadIdx.x] = pos;
    m.base[2 * threadIdx.x + 1] = pos + __popc(b0);
    __syncthreads();
    const int nw = min(kWordChunk, words - c0);
#pragma unroll 4
    for (int i = warp; i < nw; i += kThreads / 32) {
      const uint32_t b = m.bits[i];
      if ((b >> lane) & 1u)
        emit(m.base[i] + __popc(b & ((1u << lane) - 1)), 32 * (c0 + i) + lane);
    }
    first += total;
    __syncthreads();
  }
  return first;
}

// ---- truncate -----------------------------------------------------------------
// Sequence s keeps its first new_lens[s] tokens: the pages behind them lose a
// reference, and those that nobody holds any more go back on the stack in
// ascending id order, as in a release.
//
// Bound: latency (a few integers per dropped page; a chain of context -> entry
// -> count -> mark).  16 lanes per sequence, eight pages of each in flight; the
// freed pages are marked in a bitmap (one bit per page, in scratch words),
// whose order is the id order, so a scan over num_pages / 32 words by the CTA
// that ends last replaces a sort.
constexpr int kSeqLanes = 16;

__global__ void __launch_bounds__(kThreads, 1)
    pool_truncate_kernel(PoolView p, int32_t* bt, int mb, int32_t* ctx,
                         const int32_t* new_lens, int num_seqs,
                         uint32_t* err) {
  __shared__ BitList list;
  __shared__ bool last_cta;
  const int kPS = *p.page_size;
  const int top0 = *p.top;
  const int lane = threadIdx.x % kSeqLanes;
  const int s = (blockIdx.x * blockDim.x + threadIdx.x) / kSeqLanes;
  uint32_t* marks = reinterpret_cast<uint32_t*>(p.cnt_app);
  int c = 0, n = 0;
  if (s < num_seqs) {
    c = ctx[s];
    n = new_lens[s];
    if (c < 0 || c > mb * kPS || n < 0 || n > c) {
      if (lane == 0) flag_error(err, DEVERR_BAD_CONTEXT);
      c = n = -1;
    }
  }
  __syncwarp();   // every lane has read the context
  if (s < num_seqs && c >= 0) {
    int32_t* row = bt + (size_t)s * mb;
    const int end = pages_for(c, kPS);
    constexpr int kU = 8;
    for (int k0 = pages_for(n, kPS) + lane; k0 < end; k0 += kU * kSeqLanes) {
      int page[kU], left[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSeqLanes;
        page[u] = k < end ? row[k] : INT32_MAX;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSeqLanes;
        left[u] = 0;
        if (k >= end) continue;
        row[k] = -1;
        if (page[u] < 0 || page[u] >= p.num_pages)
          flag_error(err, DEVERR_BAD_PAGE);
        else
          left[u] = atomicSub(p.ref + page[u], 1);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (left[u] == 1) atomicOr(marks + (page[u] >> 5), 1u << (page[u] & 31));
    }
    if (lane == 0) ctx[s] = n;
  }
  __syncthreads();
  if (gridDim.x > 1) {
    // the CTA that ends last goes on (the count is a scratch word too)
    if (threadIdx.x == 0) {
      __threadfence();
      last_cta = atomicAdd(p.last_app, 1) == (int)gridDim.x - 1;
      if (last_cta) *p.last_app = 0;
      __threadfence();
    }
    __syncthreads();
    if (!last_cta) return;
  }
  const int top = list_bits(
      list, (p.num_pages + 31) / 32, top0,
      [&](int w) {
        const uint32_t b = __ldcg(marks + w);
        if (b) marks[w] = 0;
        return b;
      },
      [&](int pos, int page) {
        // a consistent pool never overflows; a corrupted one is flagged
        if (pos < p.num_pages) p.stack[pos] = page;
        else flag_error(err, DEVERR_BAD_SEQ);
      });
  if (threadIdx.x == 0) *p.top = min(top, p.num_pages);
}

// ---- compaction -----------------------------------------------------------------
// With U pages in use (count > 0), the i-th used page at or above U moves to
// the i-th free page below U; both lists are ascending and equally long.  Then
// the pages in use are exactly 0 .. U - 1 and the free stack is rebuilt as init
// leaves it.  This kernel (one CTA, latency-bound) plans: counts as bit words,
// sixteen words a warp in flight, their scan, the move lists and the stack.
constexpr int kHeldWords = 4096;   // bit words kept in shared memory

__global__ void __launch_bounds__(kThreads, 1)
    pool_compact_plan_kernel(PoolView p, int page_size, int32_t* move_src,
                             int32_t* move_dst, int32_t* num_moves,
                             uint32_t* err) {
  __shared__ BitList list;
  __shared__ uint32_t sh_held[kHeldWords];
  let_next_kernel_start();
  const int n = p.num_pages;
  const int words = (n + 31) / 32;
  if (*p.page_size != page_size) {   // pools of another page size
    if (threadIdx.x == 0) {
      flag_error(err, DEVERR_BAD_SEQ);
      *num_moves = 0;
    }
    return;
  }
  const bool on_chip = words <= kHeldWords;
  uint32_t* held =
      on_chip ? sh_held : reinterpret_cast<uint32_t*>(p.cnt_app);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int mine = 0;
  constexpr int kU = 16;
  for (int w0 = warp * kU; w0 < words; w0 += kU * (kThreads / 32)) {
    int r[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = 32 * (w0 + u) + lane;
      r[u] = i < n ? p.ref[i] : 0;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t b = __ballot_sync(0xffffffffu, r[u] > 0);
      if (lane == u && w0 + u < words) {
        held[w0 + u] = b;
        mine += __popc(b);
      }
    }
  }
  int used;
  (void)block_exclusive_scan(mine, list.sh, &used);   // its barriers order `held`
  // bits of word w whose page id is below `used`
  auto low = [&](int w) {
    const int k = used - 32 * w;
    return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
  };
  const int ns = list_bits(
      list, words, 0, [&](int w) { return held[w] & ~low(w); },
      [&](int i, int page) { move_src[i] = page; });
  list_bits(
      list, words, 0,
      [&](int w) {
        const uint32_t b = held[w];
        if (!on_chip) held[w] = 0;   // scratch goes back to zero
        return ~b & low(w);
      },
      [&](int i, int page) { move_dst[i] = page; });
  for (int i = threadIdx.x; i < n - used; i += kThreads)
    p.stack[i] = n - 1 - i;
  if (threadIdx.x == 0) {
    *p.top = n - used;
    *num_moves = ns;
  }
}

// Counts and block-table entries follow their pages, the entries by a binary
// search in the ascending list of moved pages (those below its first page did
// not move).
__device__ __forceinline__ void move_entries(int32_t* ref, int32_t* bt, int mb,
                                             const int32_t* ctx, int num_seqs,
                                             int kPS, const int32_t* move_src,
                                             const int32_t* move_dst, int n,
                                             int cta, int ctas,
                                             uint32_t* err) {
  const int first = n > 0 ? __ldcg(move_src) : 0;
  for (int i = cta * blockDim.x + threadIdx.x; i < n; i += ctas * blockDim.x) {
    const int a = __ldcg(move_src + i), b = __ldcg(move_dst + i);
    ref[b] = ref[a];
    ref[a] = 0;
  }
  const int64_t total = (int64_t)num_seqs * mb;
  for (int64_t i = cta * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)ctas * blockDim.x) {
    const int s = (int)(i / mb), b = (int)(i % mb);
    int c = ctx[s];
    if (c < 0 || c > mb * kPS) {
      if (b == 0) flag_error(err, DEVERR_BAD_CONTEXT);
      c = c < 0 ? 0 : mb * kPS;
    }
    if (n == 0 || b >= pages_for(c, kPS)) continue;
    const int page = bt[i];
    if (page < first) continue;
    int lo = 0, hi = n;             // first entry >= page
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(move_src + mid) < page) lo = mid + 1;
      else hi = mid;
    }
    if (lo < n && __ldcg(move_src + lo) == page) bt[i] = __ldcg(move_dst + lo);
  }
}

// Whole pages of K and V, src[i] to dst[i]: HBM-bound (2 x the bytes moved).
// A unit is 8 KB of one tensor: 256 threads x two 16-byte vectors, the next
// unit's page ids in flight beside them.
constexpr int kUnitVecs = 512;

__device__ __forceinline__ void copy_pages(uint4* k_pool, uint4* v_pool,
                                           int num_pages, int page_vecs,
                                           const int32_t* src,
                                           const int32_t* dst, int64_t n,
                                           int64_t cta, int64_t ctas,
                                           uint32_t* err) {
  const int per = (page_vecs + kUnitVecs - 1) / kUnitVecs;   // units of a page
  // unit = (pair, r), r < per: K, else V; a step of `ctas` units by addition
  // (a 64-bit division per unit costs as much as its copy)
  const int both = 2 * per;
  const int64_t pair_step = ctas / both;
  const int r_step = (int)(ctas % both);
  int64_t pair = cta / both;
  int r = (int)(cta % both);
  int a = 0, b = 0;
  if (pair < n) {
    a = __ldcg(src + pair);
    b = __ldcg(dst + pair);
  }
  while (pair < n) {
    const int from_page = a, to_page = b, unit = r;
    pair += pair_step;
    r += r_step;
    if (r >= both) {
      r -= both;
      ++pair;
    }
    if (pair < n) {
      a = __ldcg(src + pair);
      b = __ldcg(dst + pair);
    }
    if (from_page < 0 || from_page >= num_pages || to_page < 0 ||
        to_page >= num_pages) {
      if (threadIdx.x == 0 && unit == 0) flag_error(err, DEVERR_BAD_PAGE);
      continue;
    }
    uint4* pool = unit < per ? k_pool : v_pool;
    const int v0 =
        (unit < per ? unit : unit - per) * kUnitVecs + threadIdx.x;
    const uint4* from = pool + (size_t)from_page * page_vecs;
    uint4* to = pool + (size_t)to_page * page_vecs;
    uint4 x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (v0 + 256 * k < page_vecs) x[k] = __ldcs(from + v0 + 256 * k);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (v0 + 256 * k < page_vecs) __stcs(to + v0 + 256 * k, x[k]);
  }
}

__global__ void __launch_bounds__(256)
    page_copy_kernel(uint4* k_pool, uint4* v_pool, int num_pages,
                     int page_vecs, const int32_t* src, const int32_t* dst,
                     int64_t max_pairs, const int32_t* num_pairs,
                     uint32_t* err) {
  wait_for_last_kernel();   // the lists, and what wrote the pages
  int64_t n = max_pairs;
  if (num_pairs) {
    n = *num_pairs;
    n = n < 0 ? 0 : (n > max_pairs ? max_pairs : n);
  }
  copy_pages(k_pool, v_pool, num_pages, page_vecs, src, dst, n, blockIdx.x,
             gridDim.x, err);
}

// What the plan leaves to do, in one launch that starts beside the plan: the
// first table_ctas CTAs move counts and entries, the others copy pages.
__global__ void __launch_bounds__(256)
    pool_compact_move_kernel(int32_t* ref, int32_t* bt, int mb, const int32_t* ctx,
                             int num_seqs, int kPS, int table_ctas,
                             const int32_t* move_src, const int32_t* move_dst,
                             const int32_t* num_moves, uint4* k_pool,
                             uint4* v_pool, int num_pages, int page_vecs,
                             uint32_t* err) {
  let_next_kernel_start();
  wait_for_last_kernel();
  const int n = __ldcg(num_moves);
  if ((int)blockIdx.x < table_ctas)
    move_entries(ref, bt, mb, ctx, num_seqs, kPS, move_src, move_dst, n,
                 blockIdx.x, table_ctas, err);
  else
    copy_pages(k_pool, v_pool, num_pages, page_vecs, move_src, move_dst, n,
               blockIdx.x - table_ctas, gridDim.x - table_ctas, err);
}

// CTAs of a page copy: eight a SM are resident, more even the last wave out.
int copy_ctas(int64_t max_pairs, int page_vecs) {
  const int64_t want =
      max_pairs * 2 * ((page_vecs + kUnitVecs - 1) / kUnitVecs);
  const int64_t cap = (int64_t)device_sm_count() * 8;
  return (int)(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_pool_truncate(int32_t* state, int num_pages, int32_t* bt,
                                 int mb, int32_t* ctx, const int32_t* new_lens,
                                 int num_seqs, uint32_t* err,
                                 cudaStream_t stream) {
  constexpr int per = kThreads / kSeqLanes;
  pool_truncate_kernel<<<(num_seqs + per - 1) / per, kThreads, 0, stream>>>(
      view(state, num_pages), bt, mb, ctx, new_lens, num_seqs, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_compact(int32_t* state, int num_pages, int page_size,
                                int32_t* bt, int mb, const int32_t* ctx,
                                int num_seqs, int32_t* move_src,
                                int32_t* move_dst, int32_t* num_moves,
                                void* k_pool, void* v_pool, int row_bytes,
                                uint32_t* err, cudaStream_t stream) {
  pool_compact_plan_kernel<<<1, kThreads, 0, stream>>>(
      view(state, num_pages), page_size, move_src, move_dst, num_moves, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t want = ((int64_t)num_seqs * mb + 255) / 256 + 1;
  const int64_t cap = (int64_t)device_sm_count() * 2;
  const int table_ctas = (int)(want < cap ? want : cap);
  const int page_vecs = page_size * row_bytes / 16;
  const int ctas =
      table_ctas + (k_pool ? copy_ctas(num_pages / 2, page_vecs) : 0);
  return launch_kernel<pool_compact_move_kernel>(
      dim3(ctas), 256, 0, true, stream, view(state, num_pages).ref, bt, mb, ctx, num_seqs, page_size,
      table_ctas, (const int32_t*)move_src, (const int32_t*)move_dst,
      (const int32_t*)num_moves, static_cast<uint4*>(k_pool),
      static_cast<uint4*>(v_pool), num_pages, page_vecs, err);
}

cudaError_t launch_page_copy(void* k_pool, void* v_pool, int num_pages,
                             int page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t max_pairs,
                             const int32_t* num_pairs, uint32_t* err,
                             cudaStream_t stream) {
  if (max_pairs == 0) return cudaSuccess;
  const int page_vecs = page_bytes / 16;
  // (starts beside a compaction that it follows)
  return launch_kernel<page_copy_kernel>(
      dim3(copy_ctas(max_pairs, page_vecs)), 256, 0, true, stream,
      static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), num_pages,
      page_vecs, src, dst, max_pairs, num_pairs, err);
}

cudaError_t launch_pool_init(int32_t* state, int num_pages, int page_size,
                             const int32_t* bt, int mb, const int32_t* ctx,
                             int num_seqs, uint32_t* err,
                             cudaStream_t stream) {
  const PoolView p = view(state, num_pages);
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  pool_clear_kernel<<<sms, 256, 0, stream>>>(p);
  if (bt && num_seqs > 0)
    pool_count_refs_kernel<<<sms * 4, 256, 0, stream>>>(
        p, bt, mb, ctx, num_seqs, page_size, err);
  pool_stack_kernel<<<1, kThreads, 0, stream>>>(p, page_size);
  return cudaGetLastError();
}

cudaError_t launch_pool_append(int32_t* state, int num_pages, int page_size,
                               int32_t* bt, int mb, int32_t* ctx,
                               const int32_t* n_new, int num_seqs,
                               int32_t* slot_mapping, void* k_pool,
                               void* v_pool, int row_bytes, uint32_t* err,
                               cudaStream_t stream) {
  // one thread per sequence, whole warps (the scans' barriers are cheaper
  // over fewer warps)
  const int threads = num_seqs < 32 ? 32 : ((num_seqs + 31) / 32) * 32;
  pool_append_kernel<<<1, threads < kThreads ? threads : kThreads, 0, stream>>>(
      view(state, num_pages), bt, mb, ctx, n_new, num_seqs, slot_mapping,
      static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool),
      row_bytes, page_size, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_fork(int32_t* state, int num_pages, int32_t* bt,
                             int mb, int32_t* ctx, int num_seqs,
                             const int32_t* src, const int32_t* dst,
                             int num_pairs, uint32_t* err,
                             cudaStream_t stream) {
  pool_fork_kernel<<<1, kThreads, 0, stream>>>(view(state, num_pages), bt, mb,
                                               ctx, num_seqs, src, dst,
                                               num_pairs, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_release(int32_t* state, int num_pages, int32_t* bt,
                                int mb, int32_t* ctx, int num_seqs,
                                const int32_t* seqs, int num_release,
                                uint32_t* err, cudaStream_t stream) {
  pool_release_kernel<<<1, kThreads, 0, stream>>>(view(state, num_pages), bt,
                                                  mb, ctx, num_seqs, seqs,
                                                  num_release, err);
  return cudaGetLastError();
}

}  // namespace tv
