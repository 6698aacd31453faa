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
// Per SM and clock the tensor core does 4096 multiply-adds (here 2900: 46
// clocks for a product of N = 64) and the special function unit 16
// exponentials, so a 128 x 128 tile costs 768 (1080) clocks of the one, P V
// counted twice for P's two terms, and 1024 of the other.  What it takes longer
// is the softmax warps' own latency: two warps per scheduler are what tensor
// memory (S, P and O of two query tiles) and registers leave room for (four at
// 96 registers: slower, they spill).  32 decoder prompts over 1500 states: 185
// us (345 TFLOP/s, plan and launches included), 162 with P in bf16 alone; in the
// kernel the tensor pipe is at 35 %, the special function units at 47 %, the
// issue slots at 44 %.  16 prompts of 512 rows over 2048 keys: 237 us, 229 with
// tv_paged_prefill.  Every
// fourth pair of exponentials as a polynomial on the FMA units gains 1 % beside
// P's two terms (187.3 against 185.3 us) and was left out: a row's bits would
// depend on which way its neighbours' offsets send the warp.
//
// Design.
//  * A plan kernel (one CTA) lists the work: (sequence, block of 256 rows),
//    cut along the keys where one block would hold an SM for more than half
//    of an SM's share, costliest first.  A resident grid of one CTA per SM
//    takes (entry, KV head) units from it, the next one fetched while the
//    last one loads, so no SM starts a long unit when the others end.
//  * A CTA owns two 128-row query tiles that share every K/V tile of 128 keys;
//    the tensor core works for one while the other's softmax runs.
//  * A key tile is two halves of 64 keys.  P of a half takes the tensor-memory
//    columns of its S (P.V reads it from there, never through shared memory),
//    and a query tile has three such buffers: while one is exponentiated, S of
//    the next two is being computed or has been, and P.V of the last runs.
//  * warp 0 loads (K/V ring of 4 tiles of 128 keys, 16 page boxes each; q,
//    double buffered, so the next unit's loads run ahead); warp 3 issues
//    S = Q K^T, warps 1 / 2 issue O += P V of query tile 0 / 1 (three issuing
//    threads, because issuing takes longer than the products); warps 4-7 /
//    8-11 are the softmax of query tile 0 / 1, one row per thread.
//  * The softmax exponentiates against its offset as it stands and takes the
//    maximum beside it; only where a row's maximum grew by more than 2^8 (and
//    at a unit's first half) does it move the offset, rescale O and the sum
//    and exponentiate again.  A row's offset depends on its own scores alone,
//    and so do its bits.
//  * P enters the second product with 16 bits: bf16(P), and the remainder
//    P - bf16(P) in a second pass over the tile (a weight is off by at most
//    2^-16 from it, as in the prefill).
//  * What a row does not see never reaches it: on the tiles that cross the
//    diagonal or the end, warp 0 zeroes the V rows behind the last key and
//    takes infinities and NaNs out of V; it notes per dim the first key
//    that held one, and rows that see that key get NaN there.
//  * A cut block leaves (m, l, O) per range in the workspace; the streaming
//    kernel that follows joins them, in the order of the keys, with all its
//    warps (joined by one CTA each, one KV head's 80 and 197 rows over 53,287
//    and 28,329 tokens took 172 us, most of it the join; now 54).
//  * Every wait is bounded (2 s).
#include "tv_chunk.cuh"

namespace tv {
namespace {

constexpr int kD = 64;
constexpr int kPS = 16;
constexpr int kBM = 128;                  // rows of a query tile
constexpr int kBN = 128;                  // keys of a key tile
constexpr int kHalf = 64;                 // keys of a half tile
constexpr int kST = 4;                    // K/V ring depth
constexpr int kPages = kBN / kPS;         // 16-token boxes of a key tile
constexpr int kRowBytes = kD * 2;
constexpr int kTileBytes = kBN * kRowBytes;
constexpr int kPageBytes = kPS * kRowBytes;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kBuf = 3;                   // S/P buffers of a query tile
constexpr int kSCol = 0;                  // S, then P, in buffer b of query
                                          // tile t: [64 (3 t + b), +64)
constexpr int kOCol = 384;                // O of tile t: [384 + 64 t, +64)
constexpr float kLazy = 8.f;              // log2 of the growth allowed
constexpr int kMinTiles = 8;              // key tiles worth a unit of their own

constexpr uint32_t kIdescQK = idesc_bf16_f32(kBM, kHalf, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, kD, true);

// ---- plan -----------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = kPlanThreads;     // costs above share the top

template <bool kCausal>
__global__ void __launch_bounds__(kPlanThreads, 1)
    chunk_plan_kernel(const ChunkArgs a) {
  __shared__ int slot[kBuckets];          // histogram, then next free position
  __shared__ int warp_sum[32];
  __shared__ unsigned long long total;
  __shared__ int parts, joins;
  let_next_kernel_start();
  const int nblk = chunk_tile_blocks(a.max_query_len, a.group_shift);
  const int n_items = a.num_seqs * nblk;
  slot[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    total = 0;
    parts = 0;
    joins = 0;
  }
  auto tiles_of = [&](int item, TileBlock* b) {
    return tile_block<kCausal>(a, item / nblk, item % nblk, b)
               ? (b->key_end + kBN - 1) / kBN
               : -1;
  };
  // the thread's first item stays in registers for the further passes
  TileBlock b0{};
  const int n0 = (int)threadIdx.x < n_items ? tiles_of(threadIdx.x, &b0) : -1;
  auto again = [&](int item, TileBlock* b) {
    if (item == (int)threadIdx.x) {
      *b = b0;
      return n0;
    }
    return tiles_of(item, b);
  };
  TileBlock b;
  long long mine = max(0, n0);
  for (int i = threadIdx.x + kPlanThreads; i < n_items; i += kPlanThreads)
    mine += max(0, tiles_of(i, &b));
  __syncthreads();
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
  // key tiles, two thirds of them where there is one query tile
  const int per = kBM >> a.group_shift;
  auto cost = [&](const TileBlock& b, int n) {
    return min(b.tb > per ? 3 * n : 2 * n, kBuckets - 1);
  };
  auto edge = [](int n, int k, int of) { return (int)((long long)n * k / of); };
  for (int i = threadIdx.x; i < n_items; i += kPlanThreads) {
    const int n = again(i, &b);
    if (n < 0) continue;
    const int of = cuts_of(n);
    for (int k = 0; k < of; ++k)
      atomicAdd(&slot[cost(b, edge(n, k + 1, of) - edge(n, k, of))], 1);
  }
  __syncthreads();
  // thread t owns the cost kBuckets - 1 - t
  const int sum = slot[kBuckets - 1 - threadIdx.x];
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
  const int start = incl - sum + (warp > 0 ? warp_sum[warp - 1] : 0);
  slot[kBuckets - 1 - threadIdx.x] = start;
  if (threadIdx.x == kPlanThreads - 1) {
    a.plan->entries = start + sum;
    a.plan->next = a.tile_ctas;
    a.plan->failed = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_items; i += kPlanThreads) {
    const int n = again(i, &b);
    if (n < 0) continue;
    const int of = cuts_of(n);
    const int base = of > 1 ? atomicAdd(&parts, of) : -1;
    if (of > 1)
      a.plan_joins[atomicAdd(&joins, 1)] =
          make_int4(i / nblk, i % nblk, base, of);
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
      a.plan_entries[atomicAdd(&slot[cost(b, k1 - k0)], 1)] = e;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.plan->joins = joins;
}

// ---- the kernel ------------------------------------------------------------------------
// A unit: a plan entry for one KV head, and what follows from it.
struct Unit {
  ChunkEntry e;
  TileBlock b;
  int kvh;
  int n[2];        // halves of key tiles of query tile 0 / 1, from e.tile0 on
  int n_tiles;     // key tiles loaded
  int edge0;       // first key tile with a key that some row does not see
  int live;        // 0: no more units
};

struct TileSmem {
  alignas(1024) uint8_t q[2][2][kBM * kRowBytes];   // [unit parity][tile]
  alignas(1024) uint8_t k[kST][kTileBytes];
  alignas(1024) uint8_t v[kST][kTileBytes];
  alignas(8) uint64_t q_full[2];
  uint64_t q_empty[2];       // every other warp is done with the unit
  uint64_t unit_full[2];     // the unit is in `unit`
  uint64_t kv_full[kST], kv_empty[kST];
  uint64_t v_ready[kST];     // V of an edge tile is clean
  uint64_t s_full[2][kBuf], p_full[2][kBuf], o_done[2][kBuf];
  uint64_t o_free[2];                              // [query tile]
  uint64_t drain[3];
  uint32_t tmem_base;
  uint32_t bad_pages[kST];
  uint64_t clean[2];         // [unit parity]: `poison` is complete
  int32_t poison[2][kD];     // first key with a non-finite V
  int32_t poisoned[2];       // any of them
  int32_t bad_unit[2];       // a page of the unit so far was bad
  Unit unit[2];              // [unit parity]
};

// The S/P buffer of a half and the parity of this use of its barriers.
struct Turn {
  int b = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++b == kBuf) {
      b = 0;
      parity ^= 1;
    }
  }
};

template <bool kCausal>
__device__ __forceinline__ void unit_at(const ChunkArgs& a, int i, int n_units,
                                        Unit* u) {
  u->live = i < n_units;
  u->n_tiles = 0;
  if (!u->live) return;
  const int4* e =
      reinterpret_cast<const int4*>(a.plan_entries + i / a.num_kv_heads);
  const int4 e0 = __ldcg(e), e1 = __ldcg(e + 1);
  u->e = ChunkEntry{e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
  u->kvh = i % a.num_kv_heads;
  tile_block<kCausal>(a, u->e.seq, u->e.blk, &u->b);
  const int per = kBM >> a.group_shift;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int rows = min(per, u->b.tb - t * per);
    const int keys = rows <= 0 ? 0
                     : kCausal ? u->b.first_limit + t * per + rows
                               : u->b.key_end;
    u->n[t] = max(0, min((keys + kHalf - 1) / kHalf, 2 * u->e.tile1) -
                         2 * u->e.tile0);
  }
  u->n_tiles = u->e.tile1 - u->e.tile0;
  u->edge0 = max(0, u->b.first_limit + 1) / kBN;
}

// One thread of a converged warp; the compiler knows that there is one, and
// feeds the products' descriptors through uniform registers (the issue of four
// of them takes 194 clocks, under `lane == 0` 250; the tensor core needs 184).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Four products over 64 elements of K.  S = Q K^T: both operands K-major, 32
// bytes on per 16 elements.
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t q, uint32_t k,
                                         uint32_t desc_hi, uint32_t bar) {
#pragma unroll
  for (int i = 0; i < kD / 16; ++i)
    tc_mma_bf16(d, (uint64_t)desc_hi << 32 | (q + 2 * i),
                (uint64_t)desc_hi << 32 | (k + 2 * i), kIdescQK, i > 0);
  tc_commit(bar);
}
// O += P V: 16 keys are 8 columns of P, and 2 x 8 rows of V (MN-major).
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint32_t v,
                                         uint32_t desc_hi, bool accumulate) {
#pragma unroll
  for (int i = 0; i < kHalf / 16; ++i)
    tc_mma_bf16_ts(d, p + 8 * i,
                   (uint64_t)desc_hi << 32 | (v + (2 * i * 1024 >> 4)),
                   kIdescPV, accumulate || i > 0);
}

// A wait ran out: the kernel that follows then writes zeros.
__device__ __forceinline__ void give_up(const ChunkArgs& a) {
  flag_error(a.err, DEVERR_TIMEOUT);
  a.plan->failed = 1;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity));
}

// 32 columns of the warp's 32 lanes, one lane per thread; the registers hold
// them after tmem_wait32 (through which they are passed, so that no use is
// scheduled before it).
#define TV_OUT8(r, i)                                                     \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]),             \
      "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define TV_INOUT8(r, i)                                                   \
  "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),             \
      "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : TV_OUT8(r, 0), TV_OUT8(r, 8), TV_OUT8(r, 16), TV_OUT8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : TV_INOUT8(r, 0), TV_INOUT8(r, 8), TV_INOUT8(r, 16),
                 TV_INOUT8(r, 24)
               :
               : "memory");
}

// Stores without their wait: a thread's 32 registers, or the first 16 of 32.
#define TV_IN8(r, i)                                                    \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
      "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void tmem_put32(uint32_t taddr,
                                           const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
      "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      TV_IN8(r, 0), TV_IN8(r, 8), TV_IN8(r, 16), TV_IN8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr,
                                           const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      TV_IN8(r, 0), TV_IN8(r, 8)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : TV_OUT8(r, 0), TV_OUT8(r, 8)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr,
                                          const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Rows [r0, 128) of a V tile that holds the keys key0 .. : rows behind the last
// key become zero, and non-finite elements of the others leave for zero after
// their key went into `poison` (all by one warp).
__device__ __forceinline__ void clean_v(uint8_t* v, int key0, int r0,
                                        int key_end, int32_t* poison,
                                        int32_t* poisoned, int lane) {
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
    *poisoned = 1;
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
  let_next_kernel_start();
  const int per = kBM >> a.group_shift;     // query rows of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 1);
      mbar_init(smem_u32(&sm.q_empty[i]), 3 + 8);
      mbar_init(smem_u32(&sm.unit_full[i]), 1);
      mbar_init(smem_u32(&sm.clean[i]), 1);
      mbar_init(smem_u32(&sm.o_free[i]), 4);
      for (int k = 0; k < kBuf; ++k) {
        mbar_init(smem_u32(&sm.s_full[i][k]), 1);
        mbar_init(smem_u32(&sm.p_full[i][k]), 4);
        mbar_init(smem_u32(&sm.o_done[i][k]), 1);
      }
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
  wait_for_last_kernel();                   // the plan
  const int n_units = __ldcg(&a.plan->entries) * a.num_kv_heads;

  // `it` counts the K/V tiles of all units of the CTA, a Turn the halves of a
  // query tile.  A barrier's n-th use (from 0) completes its phase of parity
  // n & 1.
  if (warp == 0) {
    // ======================= loads =============================================
    const int oob_row = (a.num_pages << a.page_shift) * kPS;   // reads as zeros
    const int pp = (lane >> 1) & (kPages - 1);
    const bool is_v = lane & 1;
    const CUtensorMap* tmap = is_v ? &tm_v : &tm_k;
    bool ok = true;
    uint32_t it = 0;
    int q_loads = 0;
    int unit = blockIdx.x;
    for (int round = 0;; ++round) {
      const int ub = round & 1;
      if (round >= 2 && !wait_warp(&sm.q_empty[ub], ((round >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      Unit u;
      unit_at<kCausal>(a, unit, n_units, &u);
      if (lane == 0) {
        sm.unit[ub] = u;
        sm.poisoned[ub] = 0;
        sm.bad_unit[ub] = 0;
        mbar_arrive(smem_u32(&sm.unit_full[ub]));
      }
      if (!u.live) break;
      // the number after this one, fetched while this unit loads
      if (lane == 0) unit = atomicAdd(&a.plan->next, 1);
      sm.poison[ub][lane] = sm.poison[ub][lane + 32] = INT32_MAX;
      q_loads = round + 1;
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
      // first pool row of the pages of tiles j .. j + 3, one per lane: behind
      // the last page where a box reads zeros, -1 for a bad page
      auto page_rows = [&](int j) {
        const int lp = (u.e.tile0 + j) * kPages + lane;
        if (lp >= n_pages) return oob_row;
        const int pid = __ldg(bt + (lp >> a.page_shift));
        return pid >= 0 && pid < a.num_pages
                   ? ((pid << a.page_shift) +
                      (lp & ((1 << a.page_shift) - 1))) * kPS
                   : -1;
      };
      int rows = page_rows(0), rows_ahead = page_rows(4);
      for (int j = 0; j < u.n_tiles; ++j, ++it) {
        const int st = it % kST;
        if (it >= kST && !wait_warp(&sm.kv_empty[st], (it / kST + 1) & 1)) {
          ok = false;
          break;
        }
        if ((j & 3) == 0 && j > 0) {   // the next four tiles' pages
          rows = rows_ahead;
          rows_ahead = page_rows(j + 4);
        }
        const int src = (j & 3) * kPages;
        const int y = __shfl_sync(0xffffffffu, rows, src + pp);
        const uint32_t bad =
            (__ballot_sync(0xffffffffu, rows < 0) >> src) & 0xffu;
        const int row = y < 0 ? oob_row : y;
        const uint32_t bar = smem_u32(&sm.kv_full[st]);
        if (lane == 0) {
          if (bad) {
            flag_error(a.err, DEVERR_BAD_PAGE);
            sm.bad_unit[ub] = 1;
          }
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
                u.b.key_end, sm.poison[ub], &sm.poisoned[ub], lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.v_ready[st]));
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(smem_u32(&sm.clean[ub]));
      unit = __shfl_sync(0xffffffffu, unit, 0);
    }
    if (!ok && lane == 0) give_up(a);
    // no copy may be in flight when the CTA ends (bounded waits; all of them
    // have landed unless a wait gave up)
    if (!ok) {
      for (uint32_t i = it > kST ? it - kST : 0; i < it; ++i)
        mbar_wait(smem_u32(&sm.kv_full[i % kST]), (i / kST) & 1);
      for (int i = max(0, q_loads - 2); i < q_loads; ++i)
        mbar_wait(smem_u32(&sm.q_full[i & 1]), (i >> 1) & 1);
    }
  } else if (warp < 4) {
    // ======================= MMA issuers =======================================
    const bool leader = elect_one();
    // shared-memory descriptors: address >> 4 in the low word, strides and
    // layout in the high one (V: see smem_desc_sw128's leading offset)
    const uint64_t dq = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_u32(sm.v[0]), kTileBytes, 1024);
    const uint32_t hi_k = (uint32_t)(dk >> 32), hi_v = (uint32_t)(dv >> 32);
    bool ok = true;
    uint32_t it = 0, v_uses = 0;
    Turn turn[2];
    uint32_t results = 0;
    for (int round = 0;; ++round) {
      const int ub = round & 1;
      ok = wait_warp(&sm.unit_full[ub], (round >> 1) & 1);
      if (!ok || !sm.unit[ub].live) break;
      const Unit& u = sm.unit[ub];
      const int n_tiles = u.n_tiles;
      if (warp == 3) {
        const int n0 = u.n[0], n1 = u.n[1];
        ok = wait_warp(&sm.q_full[ub], (round >> 1) & 1);
        const uint32_t q_lo = (uint32_t)dq + ub * (2 * kBM * kRowBytes >> 4);
        for (int j = 0; ok && j < n_tiles; ++j, ++it) {
          const int st = it % kST;
          if (!wait_warp(&sm.kv_full[st], (it / kST) & 1)) {
            ok = false;
            break;
          }
          const uint32_t k_lo = (uint32_t)dk + st * (kTileBytes >> 4);
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || 2 * j + half >= (t ? n1 : n0)) continue;
              Turn& h = turn[t];
              // P.V of the buffer's last half has read it (true at first)
              if (!wait_warp(&sm.o_done[t][h.b], h.parity ^ 1)) {
                ok = false;
                continue;
              }
              tc_fence_after();
              if (leader)
                issue_qk(tmem + kSCol + (t * kBuf + h.b) * kHalf,
                         q_lo + t * (kBM * kRowBytes >> 4),
                         k_lo + half * (kHalf * kRowBytes >> 4), hi_k,
                         smem_u32(&sm.s_full[t][h.b]));
              __syncwarp();
              h.next();
            }
          if (!ok) break;
          if (leader) tc_commit(smem_u32(&sm.kv_empty[st]));
          __syncwarp();
        }
        if (!ok) break;
        if (leader) tc_commit(smem_u32(&sm.q_empty[ub]));
        __syncwarp();
      } else {
        const int t = warp - 1;
        Turn& h = turn[0];
        const int n = u.n[t];
        const int edge = u.edge0 - u.e.tile0;
        if (n > 0 && results > 0)   // the last unit's O has been read
          ok = wait_warp(&sm.o_free[t], (results - 1) & 1);
        for (int j = 0; ok && j < n_tiles; ++j, ++it) {
          const int st = it % kST;
          if (!wait_warp(&sm.kv_full[st], (it / kST) & 1)) {
            ok = false;
            break;
          }
          if (j >= edge) {
            if (!wait_warp(&sm.v_ready[st], (v_uses >> st) & 1)) {
              ok = false;
              break;
            }
            v_uses ^= 1u << st;
          }
          if (2 * j >= n) {
            if (leader) mbar_arrive(smem_u32(&sm.kv_empty[st]));
            __syncwarp();
            continue;
          }
          const uint32_t v_lo = (uint32_t)dv + st * (kTileBytes >> 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (2 * j + half >= n) continue;
            if (!ok || !wait_warp(&sm.p_full[t][h.b], h.parity)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (leader) {
              const uint32_t p_col = tmem + kSCol + (t * kBuf + h.b) * kHalf;
              const uint32_t v_half = v_lo + half * (kHalf * kRowBytes >> 4);
              issue_pv(tmem + kOCol + t * kD, p_col, v_half, hi_v,
                       (j | half) != 0);
              issue_pv(tmem + kOCol + t * kD, p_col + kHalf / 2, v_half, hi_v,
                       true);   // the remainder
              tc_commit(smem_u32(&sm.o_done[t][h.b]));
            }
            __syncwarp();
            h.next();
          }
          if (!ok) break;
          if (leader) tc_commit(smem_u32(&sm.kv_empty[st]));
          __syncwarp();
        }
        if (!ok) break;
        results += n > 0;
        if (leader) mbar_arrive(smem_u32(&sm.q_empty[ub]));
        __syncwarp();
      }
    }
    if (!ok && lane == 0) give_up(a);
    // this thread's products finish before tensor memory is freed
    if (leader) tc_commit(smem_u32(&sm.drain[warp - 1]));
    __syncwarp();
    mbar_wait(smem_u32(&sm.drain[warp - 1]), 0);
  } else {
    // ======================= softmax ===========================================
    const int t = (warp >> 2) - 1;           // query tile
    const int quarter = warp & 3;            // tensor-memory lane quarter
    const int r = quarter * 32 + lane;       // row of the tile
    const int qi = r >> a.group_shift;       // query row of the tile
    const int hh = r & ((1 << a.group_shift) - 1);
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kSCol + t * kBuf * kHalf;
    const uint32_t o_addr = tmem + lane_base + kOCol + t * kD;
    const float cs = a.scale_log2;
    const float2 cs2 = make_float2(cs, cs);
    bool ok = true;
    uint32_t it = 0;
    Turn h;
    // O holds every half handed over so far (there is one)
    auto o_ready = [&]() {
      const int b = h.b == 0 ? kBuf - 1 : h.b - 1;
      if (!wait_warp(&sm.o_done[t][b], h.b == 0 ? h.parity ^ 1 : h.parity))
        return false;
      tc_fence_after();
      return true;
    };
    for (int round = 0;; ++round) {
      const int ub = round & 1;
      if (!wait_warp(&sm.unit_full[ub], (round >> 1) & 1)) {
        ok = false;
        break;
      }
      const Unit& u = sm.unit[ub];
      if (!u.live) break;
      const int n_tiles = u.n_tiles, n = u.n[t], tile0 = u.e.tile0;
      const int tb = u.b.tb, first_limit = u.b.first_limit;
      const bool real = t * per + qi < tb;
      const int limit = kCausal
                            ? first_limit + (real ? t * per + qi : tb - 1)
                            : u.b.key_end - 1;
      const int tile_limit = kCausal ? first_limit + t * per : limit;
      float m_run = kNoOffset, l_run = 0.f;
      // ---- the halves: two loads of 32 columns, the second in flight while the
      //      first is exponentiated against the offset m_run as it stands, the
      //      maximum beside it.  Halves with hidden keys, the first of a unit
      //      and those where a row's maximum grew by 2^8 take the maximum
      //      first, move the offset (rescaling O and the sum) and exponentiate
      //      (again, from tensor memory: the first weights' remainders have
      //      taken the scores' registers).  The loop's scalar code is kept
      //      short: it costs as much time as the exponentials --------------------
      const int halves = ok ? n : 0;
      const int plain = (tile_limit + 1 - tile0 * kBN) / kHalf;
      volatile const int32_t* bad_unit = &sm.bad_unit[ub];
#pragma unroll 1
      for (int i = 0; i < halves; ++i) {
          if (!wait_warp(&sm.s_full[t][h.b], h.parity) ||
              TV_GIVE_UP(2, warp, i)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t buf = s_addr + h.b * kHalf;
          uint32_t x[32], y[32], hi[32];
          tmem_ld32(buf, x);
          tmem_wait32(x);
          tmem_ld32(buf + 32, y);
          bool again = i == 0 || i >= plain || *bad_unit;
          float2 sum = make_float2(0.f, 0.f);
          float mx[2] = {-INFINITY, -INFINITY};
          float m_use = m_run;
          auto scaled = [&](const uint32_t (&z)[32], int e) {
            return __ffma2_rn(make_float2(__uint_as_float(z[2 * e]),
                                          __uint_as_float(z[2 * e + 1])),
                              cs2, make_float2(-m_use, -m_use));
          };
          auto maximum = [&](const uint32_t (&z)[32], int e) {
            mx[e & 1] = fmax3(mx[e & 1], __uint_as_float(z[2 * e]),
                              __uint_as_float(z[2 * e + 1]));
          };
          // a pair's weights in two bf16 terms, the remainder in place of the
          // scores
          auto split = [&](float2 w, int e, uint32_t& z) {
            hi[e] = pack_bf16x2(w.x, w.y);
            const float2 rest =
                __ffma2_rn(make_float2(bf16_lo(hi[e]), bf16_hi(hi[e])),
                           make_float2(-1.f, -1.f), w);
            z = pack_bf16x2(rest.x, rest.y);
          };
          const bool quick_half = !again;
          if (__builtin_expect(quick_half, 1)) {
            auto quick = [&](uint32_t (&z)[32], int base) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 v = scaled(z, e);
                const float2 w = make_float2(fast_exp2(v.x), fast_exp2(v.y));
                maximum(z, e);
                sum = __fadd2_rn(sum, w);
                split(w, base + e, z[e]);
              }
            };
            quick(x, 0);
            tmem_wait32(y);
            quick(y, 16);
          } else {
            tmem_wait32(y);
            const uint32_t bad =
                (sm.bad_pages[(it + (i >> 1)) % kST] >> (4 * (i & 1))) & 15u;
            const int key0 = tile0 * kBN + i * kHalf;
            if (bad != 0 || key0 + kHalf - 1 > tile_limit) {
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (key0 + k > limit || ((bad >> (k / kPS)) & 1u))
                  x[k] = 0xff800000u;   // -inf
                if (key0 + 32 + k > limit || ((bad >> (2 + k / kPS)) & 1u))
                  y[k] = 0xff800000u;
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              maximum(x, e);
              maximum(y, e);
            }
          }
          const float m_half = fmaxf(mx[0], mx[1]) * cs;   // scale > 0
          const bool grow = m_half > m_run + kLazy;
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
            again = true;
            const float alpha = grow ? fast_exp2(m_run - m_half) : 1.f;
            m_run = grow ? m_half : m_run;
            l_run *= alpha;
            if (i > 0) {
              if (!o_ready()) {
                ok = false;
                break;
              }
#pragma unroll 1
              for (int d0 = 0; d0 < kD; d0 += 16) {
                uint32_t o[16];
                tmem_ld16(o_addr + d0, o);
#pragma unroll
                for (int d = 0; d < 16; ++d)
                  o[d] = __float_as_uint(__uint_as_float(o[d]) * alpha);
                tmem_st16(o_addr + d0, o);
              }
            }
          }
          if (__builtin_expect(again, 0)) {
            if (quick_half) {   // the scores have given way to remainders
              tmem_ld32(buf, x);
              tmem_ld32(buf + 32, y);
              tmem_wait32(x);
              tmem_wait32(y);
            }
            m_use = m_run;
            sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 v = e < 16 ? scaled(x, e) : scaled(y, e - 16);
              const float2 w = make_float2(fast_exp2(v.x), fast_exp2(v.y));
              sum = __fadd2_rn(sum, w);
              split(w, e, e < 16 ? x[e] : y[e - 16]);
            }
          }
          l_run += sum.x + sum.y;
          // P takes the place of S (the remainder behind it)
          tmem_put32(buf, hi);
          tmem_put16(buf + 32, x);
          tmem_put16(buf + 48, y);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[t][h.b]));
          h.next();
      }
      it += n_tiles;

      // ---- the unit's result, 32 dims at a time ------------------------------------
      if (n > 0 && ok) ok = o_ready();
      if (!wait_warp(&sm.clean[ub], (round >> 1) & 1)) ok = false;
      const bool any = n > 0 && ok;
      if (!any) {
        m_run = kNoOffset;
        l_run = 0.f;
      }
      const bool poisoned = sm.poisoned[ub] != 0;
      const int parts = u.e.parts;
      // a part: m, l, then O as [dim / 4][row] float4, so that a warp's
      // accesses are contiguous
      float* part =
          a.tile_parts +
          ((size_t)(u.e.part_base + u.e.part) * a.num_kv_heads + u.kvh) *
              kTilePartFloats +
          t * (kTilePartFloats / 2);
      uint4* dst = reinterpret_cast<uint4*>(
          a.out + ((size_t)(u.b.q_row + t * per + qi) * a.num_q_heads +
                   (u.kvh << a.group_shift) + hh) * kD);
      auto write32 = [&](const float (&o)[32], int d0, float inv) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[d0 / 8 + k] = make_uint4(
              pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
              pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
              pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
              pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      };
#pragma unroll 1
      for (int d0 = 0; d0 < kD; d0 += 32) {
        float o[32];
        if (any) {
          uint32_t x[32];
          tmem_ld32(o_addr + d0, x);
          tmem_wait32(x);
#pragma unroll
          for (int d = 0; d < 32; ++d) o[d] = __uint_as_float(x[d]);
        } else {
#pragma unroll
          for (int d = 0; d < 32; ++d) o[d] = 0.f;
        }
        if (poisoned) {
#pragma unroll
          for (int d = 0; d < 32; ++d)
            if (sm.poison[ub][d0 + d] <= limit) o[d] = NAN;
        }
        if (parts > 1) {
          float4* to = reinterpret_cast<float4*>(part + 2 * kBM) +
                       d0 / 4 * kBM + r;
#pragma unroll
          for (int d = 0; d < 8; ++d)
            __stcg(to + d * kBM, make_float4(o[4 * d], o[4 * d + 1],
                                             o[4 * d + 2], o[4 * d + 3]));
        } else if (real) {
          write32(o, d0, l_run == 0.f ? 0.f : 1.f / l_run);   // NaN stays
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.o_free[t]));
      }
      if (parts > 1) {
        __stcg(part + r, m_run);
        __stcg(part + kBM + r, l_run);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_empty[ub]));
    }
    if (!ok && lane == 0) give_up(a);
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
  cudaError_t e = launch_kernel<chunk_plan_kernel<kCausal>>(
      dim3(1), kPlanThreads, 0, false, stream, a);
  if (e != cudaSuccess) return e;
  return launch_kernel<chunk_tile_kernel<kCausal>>(
      dim3(a.tile_ctas), kThreads, sizeof(TileSmem) + 1024, true, stream, a,
      tq, tk, tv);
}

}  // namespace

cudaError_t launch_chunk_tiles(const ChunkArgs& a, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv,
                               bool causal, cudaStream_t stream) {
  return causal ? launch<true>(a, tq, tk, tv, stream)
                : launch<false>(a, tq, tk, tv, stream);
}

}  // namespace tv
