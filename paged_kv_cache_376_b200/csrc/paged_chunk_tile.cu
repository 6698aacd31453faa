// Chunk and cross attention of many rows per sequence on the tcgen05 tensor
// cores: the sequences whose rows x heads per KV head fill more than the 32
// rows of the streaming kernel (paged_chunk.cu).
//
// Mathematics: row r = (query row, head of the KV head's group) of sequence s,
//   S = scale q.K_j,  P_j = exp(S_j - m),  out = (sum_j P_j V_j) / sum_j P_j
// over the keys j that it sees (0 .. C - T + i, or all C), in tiles of 128
// keys with a running offset m that moves only when a tile's maximum exceeds
// it by more than 2^8 (then O and the sum are rescaled).
//
// What bounds it: 2 x 64 multiply-adds and one exponential per (row, key).
// Per SM and clock the tensor core does 4096 multiply-adds and the special
// function unit 16 exponentials, so a 128 x 128 tile costs 512 clocks of the
// one and 1024 of the other: the exponentials are the floor.
//
// Design.
//  * A plan kernel (one CTA) lists the work: (sequence, block of 256 rows),
//    cut along the keys where one block would hold an SM for more than half
//    of an SM's share, costliest first.  A resident grid of one CTA per SM
//    takes (entry, KV head) units from it in a fixed order, back and forth,
//    so the shares come out even and no CTA starts a long unit last.
//  * A CTA owns two 128-row query tiles (A, B) that share every K/V tile; the
//    tensor core works for one while the other's softmax runs.
//  * S and P have tensor-memory columns of their own: the softmax copies S
//    into registers at once and hands the columns back, so S of the next
//    key tile is computed during the exponentials of this one.  P never
//    goes through shared memory: P.V reads it from tensor memory.
//  * warp 0 loads (K/V ring of 4 tiles of 128 keys, 16 page boxes each; q,
//    double buffered, so the next unit's loads run ahead); warp 3 issues
//    S = Q K^T for both tiles, warps 1 / 2 issue O += P V of tile A / B
//    (three issuing threads, because issuing takes longer than the products);
//    warps 4-7 / 8-11 are the softmax of tile A / B, one row per thread.
//  * P enters the second product in bf16.  A weight's rounding (2^-9 of it)
//    averages out over the keys of a row, except where there are few: units
//    whose first row sees fewer than kExactKeys keys add P's remainder,
//    P - bf16(P), in a second pass over the tile.
//  * What a row does not see never reaches it: on the tiles that cross the
//    diagonal or the end, warp 0 zeroes the V rows behind the last key and
//    takes infinities and NaNs out of V; it notes per dim the first key
//    that held one, and rows that see that key get NaN there.
//  * A cut block leaves (m, l, O) per range in the workspace; the CTA that
//    completes its counter joins them in the order of the keys.
//  * Every wait is bounded (2 s).
#include "tv_device.cuh"
#include "tv_kernels.h"

namespace tv {
namespace {

constexpr int kD = 64;
constexpr int kPS = 16;
constexpr int kBM = 128;                  // rows of a query tile
constexpr int kBN = 128;                  // keys of a key tile
constexpr int kST = 4;                    // K/V ring depth
constexpr int kPages = kBN / kPS;         // 16-token boxes of a key tile
constexpr int kRowBytes = kD * 2;
constexpr int kTileBytes = kBN * kRowBytes;
constexpr int kPageBytes = kPS * kRowBytes;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kSCol = 0;                  // S of tile t: [128 t, +128)
constexpr int kPCol = 256;                // P of tile t: [256 + 64 t, +64)
constexpr int kOCol = 384;                // O of tile t: [384 + 64 t, +64)
constexpr float kLazy = 8.f;              // log2 of the growth allowed
constexpr int kExactKeys = 512;           // see the file comment
constexpr int kMinTiles = 4;              // key tiles worth a unit of their own

constexpr uint32_t kIdescQK = idesc_bf16_f32(kBM, kBN, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, kD, true);

// ---- plan -----------------------------------------------------------------------
// The key tiles of a block, from the rows it covers.
struct Block {
  int q_row;            // first query row in q / out
  int tb;               // query rows
  int first_limit;      // last key that the first row sees
  int key_end;          // keys that some row sees: [0, key_end)
};

template <bool kCausal>
__device__ __forceinline__ bool tile_block(const ChunkArgs& a, int seq,
                                           int blk, Block* b) {
  const int qs = a.query_start_loc[seq];
  const int T = a.query_start_loc[seq + 1] - qs;
  const int cap = a.max_blocks_per_seq * (kPS << a.page_shift);
  const int ctx = min(max(a.context_lens[seq], 0), cap);
  // what is out of range is flagged by the streaming kernel of this call
  if (T <= a.stream_rows || T > a.max_query_len || qs < 0 ||
      (int64_t)qs + T > a.num_query_rows || (kCausal && T > ctx))
    return false;
  const int rows = 2 * kBM >> a.group_shift;
  const int t0 = blk * rows;
  if (t0 >= T) return false;
  b->q_row = qs + t0;
  b->tb = min(rows, T - t0);
  b->first_limit = kCausal ? ctx - T + t0 : ctx - 1;
  b->key_end = kCausal ? b->first_limit + b->tb : ctx;
  return true;
}

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 4096;            // costs above share the top
constexpr int kPerThread = kBuckets / kPlanThreads;

template <bool kCausal>
__global__ void __launch_bounds__(kPlanThreads, 1)
    chunk_plan_kernel(const ChunkArgs a) {
  __shared__ int slot[kBuckets];          // histogram, then next free position
  __shared__ int warp_sum[32];
  __shared__ unsigned long long total;
  __shared__ int parts;
  const int nblk = chunk_tile_blocks(a.max_query_len, a.group_shift);
  const int n_items = a.num_seqs * nblk;
  for (int i = threadIdx.x; i < kBuckets; i += kPlanThreads) slot[i] = 0;
  if (threadIdx.x == 0) {
    total = 0;
    parts = 0;
  }
  __syncthreads();
  auto tiles_of = [&](int item, Block* b) {
    return tile_block<kCausal>(a, item / nblk, item % nblk, b)
               ? (b->key_end + kBN - 1) / kBN
               : -1;
  };
  Block b;
  long long mine = 0;
  for (int i = threadIdx.x; i < n_items; i += kPlanThreads)
    mine += max(0, tiles_of(i, &b));
  if (mine) atomicAdd(&total, (unsigned long long)mine);
  __syncthreads();
  // no unit longer than half an SM's share, none shorter than kMinTiles
  const long long share =
      ((long long)total * a.num_kv_heads + 2 * a.tile_ctas - 1) /
      (2 * a.tile_ctas);
  const long long longest = max(share, (long long)kMinTiles);
  auto cuts_of = [&](int n) {
    return n > longest ? (int)((n + longest - 1) / longest) : 1;
  };
  auto edge = [](int n, int k, int of) { return (int)((long long)n * k / of); };
  for (int i = threadIdx.x; i < n_items; i += kPlanThreads) {
    const int n = tiles_of(i, &b);
    if (n < 0) continue;
    const int of = cuts_of(n);
    for (int k = 0; k < of; ++k)
      atomicAdd(&slot[min(edge(n, k + 1, of) - edge(n, k, of), kBuckets - 1)],
                1);
  }
  __syncthreads();
  // thread t owns the costs kBuckets-1-4t down to ...-4t-3
  int own[kPerThread];
  int sum = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    own[k] = slot[kBuckets - 1 - (threadIdx.x * kPerThread + k)];
    sum += own[k];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += v;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  int start = incl - sum + (warp > 0 ? warp_sum[warp - 1] : 0);
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    slot[kBuckets - 1 - (threadIdx.x * kPerThread + k)] = start;
    start += own[k];
  }
  if (threadIdx.x == kPlanThreads - 1) a.plan->entries = start;
  __syncthreads();
  for (int i = threadIdx.x; i < n_items; i += kPlanThreads) {
    const int n = tiles_of(i, &b);
    if (n < 0) continue;
    const int of = cuts_of(n);
    const int base = of > 1 ? atomicAdd(&parts, of) : -1;
    for (int k = 0; k < of; ++k) {
      const int k0 = edge(n, k, of), k1 = edge(n, k + 1, of);
      ChunkEntry e;
      e.seq = i / nblk;
      e.blk = i % nblk;
      e.tile0 = k0;
      e.tile1 = k1;
      e.part_base = base;
      e.part = k;
      e.parts = of;
      e.pad = 0;
      a.plan_entries[atomicAdd(&slot[min(k1 - k0, kBuckets - 1)], 1)] = e;
    }
  }
}

// ---- tensor memory ------------------------------------------------------------------
// 128 consecutive columns of the warp's 32 lanes, one lane per thread; the
// wait sits in the same statement, so no use can be scheduled before it.
#define TV_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), \
    "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), \
    "=r"(r[i + 7])
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, "
      "%44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, "
      "%58, %59, %60, %61, %62, %63, %64, %65, %66, %67, %68, %69, %70, %71, "
      "%72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, "
      "%86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, "
      "%100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, "
      "%111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, "
      "%122, %123, %124, %125, %126, %127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : TV_R8(r, 0), TV_R8(r, 8), TV_R8(r, 16), TV_R8(r, 24), TV_R8(r, 32),
        TV_R8(r, 40), TV_R8(r, 48), TV_R8(r, 56), TV_R8(r, 64), TV_R8(r, 72),
        TV_R8(r, 80), TV_R8(r, 88), TV_R8(r, 96), TV_R8(r, 104),
        TV_R8(r, 112), TV_R8(r, 120)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}

// ---- the kernel ------------------------------------------------------------------------
struct TileSmem {
  alignas(1024) uint8_t q[2][2][kBM * kRowBytes];   // [unit parity][tile]
  alignas(1024) uint8_t k[kST][kTileBytes];
  alignas(1024) uint8_t v[kST][kTileBytes];
  alignas(8) uint64_t q_full[2];
  uint64_t q_empty[2];       // S issued and the unit's results written
  uint64_t kv_full[kST], kv_empty[kST];
  uint64_t v_ready[kST];     // V of an edge tile is clean
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2], o_free[2];
  uint64_t drain[3];
  uint32_t tmem_base;
  uint32_t bad_pages[kST];
  int32_t poison[2][kD];     // [unit parity]: first key with a non-finite V
  int32_t last[2];
};

// A unit: a plan entry for one KV head, and what follows from it.
struct Unit {
  ChunkEntry e;
  Block b;
  int kvh;
  int n[2];        // key tiles of query tile 0 / 1, from e.tile0 on
  int n_tiles;     // key tiles loaded
  int edge0;       // first key tile with a key that some row does not see
};

template <bool kCausal>
__device__ __forceinline__ bool unit_at(const ChunkArgs& a, int round,
                                        int n_units, Unit* u) {
  // back and forth over the sorted list
  const int g = gridDim.x;
  const int i = round * g + ((round & 1) ? g - 1 - (int)blockIdx.x
                                         : (int)blockIdx.x);
  if (i >= n_units) return false;
  u->e = a.plan_entries[i / a.num_kv_heads];
  u->kvh = i % a.num_kv_heads;
  tile_block<kCausal>(a, u->e.seq, u->e.blk, &u->b);
  const int per = kBM >> a.group_shift;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int rows = min(per, u->b.tb - t * per);
    const int keys = rows <= 0 ? 0
                     : kCausal ? u->b.first_limit + t * per + rows
                               : u->b.key_end;
    u->n[t] = max(0, min((keys + kBN - 1) / kBN, u->e.tile1) - u->e.tile0);
  }
  u->n_tiles = u->e.tile1 - u->e.tile0;
  u->edge0 = max(0, u->b.first_limit + 1) / kBN;
  return true;
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity));
}

// Rows [r0, 128) of a V tile that holds the keys key0 .. : rows behind the last
// key become zero, and non-finite elements of the others leave for zero after
// their key went into `poison` (all by one warp).
__device__ __forceinline__ void clean_v(uint8_t* v, int key0, int r0,
                                        int key_end, int32_t* poison,
                                        int lane) {
  for (int i = r0 * 8 + lane; i < kBN * 8; i += 32) {
    const int r = i >> 3;
    uint4* p = reinterpret_cast<uint4*>(v + i * 16);
    if (key0 + r >= key_end) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 u = *p;
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool any = false;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      any |= (w[k] & 0x7f80u) == 0x7f80u ||
             (w[k] & 0x7f800000u) == 0x7f800000u;
    if (!any) continue;
    const int d0 = ((i & 7) ^ (r & 7)) * 8;     // the slice is swizzled
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7f80u) == 0x7f80u) {
        atomicMin(poison + d0 + 2 * k, key0 + r);
        w[k] &= 0xffff0000u;
      }
      if ((w[k] & 0x7f800000u) == 0x7f800000u) {
        atomicMin(poison + d0 + 2 * k + 1, key0 + r);
        w[k] &= 0xffffu;
      }
    }
    *p = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool kCausal>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tile_kernel(const ChunkArgs a,
                      const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* base = smem_dyn + ((1024 - (smem_u32(smem_dyn) & 1023)) & 1023);
  auto& sm = *reinterpret_cast<TileSmem*>(base);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_units = a.plan->entries * a.num_kv_heads;
  if ((int)blockIdx.x >= n_units) return;
  const int per = kBM >> a.group_shift;     // query rows of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 1);
      mbar_init(smem_u32(&sm.q_empty[i]), 1 + 8);
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.s_free[i]), 4);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.o_done[i]), 1);
      mbar_init(smem_u32(&sm.o_free[i]), 4);
    }
    for (int i = 0; i < kST; ++i) {
      mbar_init(smem_u32(&sm.kv_full[i]), 1);
      mbar_init(smem_u32(&sm.kv_empty[i]), 3);   // three issuers
      mbar_init(smem_u32(&sm.v_ready[i]), 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&sm.drain[i]), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // Counters that run through all units of the CTA: `it` K/V tiles, `c` tile
  // passes of a query tile.  A barrier's n-th use (from 0) completes its phase
  // of parity n & 1.
  Unit u;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  }
  if (warp == 0) {
    // ======================= loads =============================================
    const int oob_row = (a.num_pages << a.page_shift) * kPS;   // reads as zeros
    const int pp = (lane >> 1) & (kPages - 1);
    const bool is_v = lane & 1;
    const CUtensorMap* tmap = is_v ? &tm_v : &tm_k;
    bool ok = true;
    uint32_t it = 0, v_uses = 0;
    for (int round = 0; ok && unit_at<kCausal>(a, round, n_units, &u);
         ++round) {
      const int ub = round & 1;
      if (round >= 2 && !wait_warp(&sm.q_empty[ub], ((round >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      sm.poison[ub][lane] = sm.poison[ub][lane + 32] = INT32_MAX;
      if (lane == 0) {
        const uint32_t qbar = smem_u32(&sm.q_full[ub]);
        mbar_arrive_expect_tx(qbar, 2 * kBM * kRowBytes);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          tma_load_3d(smem_u32(sm.q[ub][t]), &tm_q, 0,
                      u.kvh << a.group_shift, u.b.q_row + t * per, qbar);
      }
      const int n_pages = (u.b.key_end + kPS - 1) / kPS;
      const int32_t* bt =
          a.block_tables + (size_t)u.e.seq * a.max_blocks_per_seq;
      const uint32_t it0 = it;
      for (int j = 0; j < u.n_tiles; ++j, ++it) {
        const int st = it % kST;
        if (it >= kST && !wait_warp(&sm.kv_empty[st], (it / kST + 1) & 1)) {
          ok = false;
          break;
        }
        int y = oob_row;
        bool badp = false;
        if (lane < kPages) {       // lane p looks up page p of the tile
          const int lp = (u.e.tile0 + j) * kPages + lane;
          if (lp < n_pages) {
            const int pid = __ldg(bt + (lp >> a.page_shift));
            if (pid >= 0 && pid < a.num_pages)
              y = ((pid << a.page_shift) + (lp & ((1 << a.page_shift) - 1))) *
                  kPS;
            else
              badp = true;
          }
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, badp);
        const int row = __shfl_sync(0xffffffffu, y, pp);
        const uint32_t bar = smem_u32(&sm.kv_full[st]);
        if (lane == 0) {
          if (bad) flag_error(a.err, DEVERR_BAD_PAGE);
          sm.bad_pages[st] = bad;
          mbar_arrive_expect_tx(bar, 2 * kTileBytes);
        }
        __syncwarp();
        if (lane < 2 * kPages)
          tma_load_2d(smem_u32(is_v ? sm.v[st] : sm.k[st]) + pp * kPageBytes,
                      tmap, u.kvh * kD, row, bar);
      }
      // the edge tiles (at most three, the last of a block) once they are in
      for (int j = max(0, u.edge0 - u.e.tile0); ok && j < u.n_tiles; ++j) {
        const uint32_t i = it0 + j;
        const int st = i % kST;
        if (!wait_warp(&sm.kv_full[st], (i / kST) & 1)) {
          ok = false;
          break;
        }
        const int key0 = (u.e.tile0 + j) * kBN;
        clean_v(sm.v[st], key0, max(0, u.b.first_limit + 1 - key0),
                u.b.key_end, sm.poison[ub], lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.v_ready[st]));
        v_uses ^= 1u << st;
      }
    }
    if (!ok && lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
    // no copy may be in flight when the CTA ends (bounded waits; all of them
    // have landed unless a wait gave up)
    if (!ok)
      for (uint32_t i = it > kST ? it - kST : 0; i < it; ++i)
        mbar_wait(smem_u32(&sm.kv_full[i % kST]), (i / kST) & 1);
  } else if (warp < 4) {
    // ======================= MMA issuers =======================================
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0, v_uses = 0;
      uint32_t c[2] = {0, 0};
      for (int round = 0; ok && unit_at<kCausal>(a, round, n_units, &u);
           ++round) {
        if (warp == 3) {
          const int ub = round & 1;
          ok = mbar_wait(smem_u32(&sm.q_full[ub]), (round >> 1) & 1);
          for (int j = 0; ok && j < u.n_tiles; ++j, ++it) {
            const int st = it % kST;
            if (!mbar_wait(smem_u32(&sm.kv_full[st]), (it / kST) & 1)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (j >= u.n[t]) continue;
              // the softmax has taken the last S out of the columns
              if (c[t] > 0 &&
                  !mbar_wait(smem_u32(&sm.s_free[t]), (c[t] - 1) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t q_addr = smem_u32(sm.q[ub][t]);
              const uint32_t k_addr = smem_u32(sm.k[st]);
#pragma unroll
              for (int k = 0; k < kD / 16; ++k)
                tc_mma_bf16(tmem + kSCol + t * kBN,
                            smem_desc_sw128(q_addr + k * 32, 16, 1024),
                            smem_desc_sw128(k_addr + k * 32, 16, 1024),
                            kIdescQK, k > 0);
              tc_commit(smem_u32(&sm.s_full[t]));
              ++c[t];
            }
            if (!ok) break;
            tc_commit(smem_u32(&sm.kv_empty[st]));
          }
          if (ok) tc_commit(smem_u32(&sm.q_empty[ub]));
        } else {
          const int t = warp - 1;
          const int passes = u.b.first_limit + 1 < kExactKeys ? 2 : 1;
          if (u.n[t] > 0 && round > 0)   // the last unit's O has been read
            ok = mbar_wait(smem_u32(&sm.o_free[t]), (c[1] - 1) & 1);
          for (int j = 0; ok && j < u.n_tiles; ++j, ++it) {
            const int st = it % kST;
            if (!mbar_wait(smem_u32(&sm.kv_full[st]), (it / kST) & 1)) {
              ok = false;
              break;
            }
            if (u.e.tile0 + j >= u.edge0) {
              if (!mbar_wait(smem_u32(&sm.v_ready[st]), (v_uses >> st) & 1)) {
                ok = false;
                break;
              }
              v_uses ^= 1u << st;
            }
            if (j < u.n[t]) {
              const uint32_t v_addr = smem_u32(sm.v[st]);
              for (int p = 0; p < passes; ++p, ++c[0]) {
                if (!mbar_wait(smem_u32(&sm.p_full[t]), c[0] & 1)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kBN / 16; ++k)
                  // A = P: 16 keys are 8 columns; B = V, MN-major (head dim
                  // contiguous): 16 keys = 2 x 8 rows
                  tc_mma_bf16_ts(tmem + kOCol + t * kD,
                                 tmem + kPCol + t * (kBN / 2) + k * 8,
                                 smem_desc_sw128(v_addr + k * 16 * kRowBytes,
                                                 kTileBytes, 1024),
                                 kIdescPV, (j | p | k) != 0);
                tc_commit(smem_u32(&sm.o_done[t]));
              }
              if (!ok) break;
              tc_commit(smem_u32(&sm.kv_empty[st]));
            } else {
              mbar_arrive(smem_u32(&sm.kv_empty[st]));
            }
          }
          if (u.n[t] > 0) ++c[1];        // units with an O of this tile
        }
      }
      if (!ok) flag_error(a.err, DEVERR_TIMEOUT);
      // this thread's products finish before tensor memory is freed
      tc_commit(smem_u32(&sm.drain[warp - 1]));
      mbar_wait(smem_u32(&sm.drain[warp - 1]), 0);
    }
  } else {
    // ======================= softmax ===========================================
    const int t = (warp >> 2) - 1;           // query tile
    const int quarter = warp & 3;            // tensor-memory lane quarter
    const int r = quarter * 32 + lane;       // row of the tile
    const int qi = r >> a.group_shift;       // query row of the tile
    const int hh = r & ((1 << a.group_shift) - 1);
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kSCol + t * kBN;
    const uint32_t p_addr = tmem + lane_base + kPCol + t * (kBN / 2);
    const uint32_t o_addr = tmem + lane_base + kOCol + t * kD;
    const float cs = a.scale_log2;
    bool ok = true;
    uint32_t it = 0, v_uses = 0;
    uint32_t c = 0, cp = 0;                  // S tiles, P passes so far
    for (int round = 0; unit_at<kCausal>(a, round, n_units, &u); ++round) {
      const int ub = round & 1;
      const bool real = t * per + qi < u.b.tb;
      const int limit =
          kCausal ? u.b.first_limit + (real ? t * per + qi : u.b.tb - 1)
                  : u.b.key_end - 1;
      const int tile_limit = kCausal ? u.b.first_limit + t * per
                                     : u.b.key_end - 1;
      const bool exact = u.b.first_limit + 1 < kExactKeys;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < u.n_tiles; ++j, ++it) {
        const int st = it % kST;
        const uint32_t v_use = (v_uses >> st) & 1;
        const bool edge = u.e.tile0 + j >= u.edge0;
        if (edge) v_uses ^= 1u << st;
        if (j >= u.n[t] || !ok) continue;
        if (edge && !wait_warp(&sm.v_ready[st], v_use)) {
          ok = false;   // (orders the notes in `poison` before the result)
          continue;
        }
        const int key0 = (u.e.tile0 + j) * kBN;
        if (!wait_warp(&sm.s_full[t], c & 1)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        float s[kBN];
        tmem_ld128(s_addr, s);
        const uint32_t bad = sm.bad_pages[st];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_free[t]));
        ++c;
        if (bad != 0 || key0 + kBN - 1 > tile_limit) {
#pragma unroll
          for (int x = 0; x < kBN; ++x)
            if (key0 + x > limit || ((bad >> (x / kPS)) & 1u))
              s[x] = -INFINITY;
        }
        // ---- the tile's maximum; the offset moves when it grew by 2^8 -----------
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int x = 0; x < kBN; x += 4) {
          mx0 = fmax3(mx0, s[x], s[x + 1]);
          mx1 = fmax3(mx1, s[x + 2], s[x + 3]);
        }
        const float m_tile = fmaxf(mx0, mx1) * cs;   // scale > 0
        const bool grow = m_tile > m_run + kLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? m_tile : m_run;
          const float alpha = grow ? fast_exp2(m_run - m_new) : 1.f;
          l_run *= alpha;
          m_run = m_new;
          if (j > 0) {
            if (!wait_warp(&sm.o_done[t], (cp - 1) & 1)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            float o[64];
            tmem_ld64(o_addr, o);
#pragma unroll
            for (int d = 0; d < 64; ++d) o[d] *= alpha;
            tmem_st64(o_addr, o);
          }
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        // ---- exponentials, their sum, P in bf16 ----------------------------------
        const float2 cs2 = make_float2(cs, cs);
        const float2 nm2 = make_float2(-m_use, -m_use);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
        float hi[64];
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          const float2 x =
              __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), cs2, nm2);
          const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          if (e & 1) sum1 = __fadd2_rn(sum1, p);
          else sum0 = __fadd2_rn(sum0, p);
          const uint32_t h = pack_bf16x2(p.x, p.y);
          hi[e] = __uint_as_float(h);
          if (exact) {
            s[2 * e] = p.x - bf16_lo(h);
            s[2 * e + 1] = p.y - bf16_hi(h);
          }
        }
        l_run += (sum0.x + sum0.y) + (sum1.x + sum1.y);
        // P's columns are free once the last pass has read them
        if (cp > 0 && !wait_warp(&sm.o_done[t], (cp - 1) & 1)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        tmem_st64(p_addr, hi);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[t]));
        ++cp;
        if (exact) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            hi[e] = __uint_as_float(pack_bf16x2(s[2 * e], s[2 * e + 1]));
          if (!wait_warp(&sm.o_done[t], (cp - 1) & 1)) {
            ok = false;
            continue;
          }
          tc_fence_after();
          tmem_st64(p_addr, hi);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[t]));
          ++cp;
        }
      }

      // ---- the unit's result ------------------------------------------------------
      float o[64];
      if (u.n[t] > 0 && ok) ok = wait_warp(&sm.o_done[t], (cp - 1) & 1);
      if (u.n[t] > 0 && ok) {
        tc_fence_after();
        tmem_ld64(o_addr, o);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.o_free[t]));
      } else {
#pragma unroll
        for (int d = 0; d < 64; ++d) o[d] = 0.f;
        l_run = 0.f;
        m_run = -INFINITY;
      }
      if (u.e.tile1 > u.edge0) {     // the unit had edge tiles
#pragma unroll
        for (int d = 0; d < 64; ++d)
          if (sm.poison[ub][d] <= limit) o[d] = NAN;
      }
      bool write = real;
      if (u.e.parts > 1) {
        // leave (m, l, O); [dim / 4][row] float4, so that a warp's stores are
        // contiguous
        const size_t slot0 = (size_t)u.e.part_base * a.num_kv_heads + u.kvh;
        auto part = [&](int k) {
          return a.tile_parts +
                 (slot0 + (size_t)k * a.num_kv_heads) * kTilePartFloats +
                 t * (kTilePartFloats / 2);
        };
        float* mine = part(u.e.part);
        __stcg(mine + r, m_run);
        __stcg(mine + kBM + r, l_run);
        float4* dst = reinterpret_cast<float4*>(mine + 2 * kBM) + r;
#pragma unroll
        for (int d = 0; d < 16; ++d)
          __stcg(dst + d * kBM, make_float4(o[4 * d], o[4 * d + 1],
                                            o[4 * d + 2], o[4 * d + 3]));
        asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
        if ((threadIdx.x & 127) == 0) {
          int32_t* counter = a.tile_counters + 2 * slot0 + t;
          __threadfence();
          sm.last[t] = atomicAdd(counter, 1) == u.e.parts - 1;
          if (sm.last[t]) *counter = 0;
          __threadfence();
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
        write = real && sm.last[t];
        if (sm.last[t]) {
          m_run = -INFINITY;
          for (int k = 0; k < u.e.parts; ++k)
            m_run = fmaxf(m_run, __ldcg(part(k) + r));
          l_run = 0.f;
#pragma unroll
          for (int d = 0; d < 64; ++d) o[d] = 0.f;
          for (int k = 0; k < u.e.parts; ++k) {
            const float* p = part(k);
            const float mk = __ldcg(p + r);
            const float f = mk == m_run ? 1.f : fast_exp2(mk - m_run);
            l_run = fmaf(__ldcg(p + kBM + r), f, l_run);
            const float4* src =
                reinterpret_cast<const float4*>(p + 2 * kBM) + r;
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              const float4 x = __ldcg(src + d * kBM);
              o[4 * d] = fmaf(x.x, f, o[4 * d]);
              o[4 * d + 1] = fmaf(x.y, f, o[4 * d + 1]);
              o[4 * d + 2] = fmaf(x.z, f, o[4 * d + 2]);
              o[4 * d + 3] = fmaf(x.w, f, o[4 * d + 3]);
            }
          }
        }
      }
      if (write) {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;   // NaN stays
        uint4* dst = reinterpret_cast<uint4*>(
            a.out + ((size_t)(u.b.q_row + t * per + qi) * a.num_q_heads +
                     (u.kvh << a.group_shift) + hh) * kD);
#pragma unroll
        for (int k = 0; k < kD / 8; ++k)
          dst[k] = make_uint4(
              pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
              pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
              pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
              pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_empty[ub]));
    }
    if (!ok && lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

static_assert(sizeof(TileSmem) + 1024 <= 227 * 1024,
              "shared memory of the tile kernel");

template <bool kCausal>
cudaError_t launch(const ChunkArgs& a, const CUtensorMap& tq,
                   const CUtensorMap& tk, const CUtensorMap& tv,
                   cudaStream_t stream) {
  const int smem = sizeof(TileSmem) + 1024;
  auto kern = chunk_tile_kernel<kCausal>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_plan_kernel<kCausal><<<1, kPlanThreads, 0, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kern<<<a.tile_ctas, kThreads, smem, stream>>>(a, tq, tk, tv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_tiles(const ChunkArgs& a, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv,
                               bool causal, cudaStream_t stream) {
  return causal ? launch<true>(a, tq, tk, tv, stream)
                : launch<false>(a, tq, tk, tv, stream);
}

}  // namespace tv
