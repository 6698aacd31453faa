// Attention of a chunk of new rows per sequence over the paged cache, causal
// or over every key, for row counts too small for a 128-row MMA tile.
//
// Mathematics: sequence s has T query rows and C cached keys.  Row i, head h:
//   out = sum_j softmax_j(scale q.K_j) V_j  over the keys j it sees, which
//   are 0 .. C - T + i (causal chunk) or all C (cross attention).
// The softmax is online: a running maximum m and sum l per row, O rescaled
// when m moves.
//
// What bounds it: a sequence's K and V are read once for up to 32 rows x heads
// per KV head, and that stream from HBM is the floor.  Up to 16 rows it is also
// the bound (8 x 131072 tokens, 16 rows: 326 to 343 us on two GPUs, 6.6 to 6.3
// TB/s, about the rate of a copy).
// With 32 (64 x 2048 tokens: 70 us, where the stream takes 41) neither the
// stream, the tensor pipe (36 %) nor the issue slots (38 %) are full: chains of
// products, exponentials and products on 2.5 warps per scheduler, and 2.7
// sequences a CTA to combine or to leave a part of; what each of them takes was
// not measured.
//
// Design.  Every warp works on pages of its own, which reach it through a
// private ring of TMA boxes (16 tokens x 128 B of K and of V, 128-byte
// swizzle), so no warp waits for another before a sequence's rows are combined.
// A row of the product is one (query row, head of the KV head's group) pair,
// row r = query row r / G, head r % G, 16 * MB rows per block.  Per page a
// warp forms S = Q K^T and O += P V with m16n8k16 bf16 products and fp32
// accumulators: with at least 16 rows, rows in the M dimension put P's
// accumulator fragment where the next product wants its A operand, so P needs
// no shuffles (the decode kernels, with at most 8 rows, put tokens in M
// instead).  Two kernels share this step: one CTA per (KV head, block of rows,
// sequence), for calls without a workspace, and a balanced grid.
//
// P enters the second product with 16 bits, as in the decode and the prefill:
// bf16(P), and the remainder P - bf16(P) in a second product over the same V
// fragments (a weight is then off by at most 2^-16; bf16(P) alone would be by
// 2^-8, which shows where few keys carry a row).
#include "tv_chunk.cuh"
#include "tv_decode.cuh"

namespace tv {
namespace {

constexpr int kD = 64;
constexpr int kPS = 16;          // tokens per TMA box
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;       // boxes of K and V in flight per warp
constexpr int kRowBytes = kD * 2;
constexpr int kSliceBytes = kPS * kRowBytes;
constexpr int kStageBytes = 2 * kSliceBytes;
constexpr float kLazy = 8.f;     // log2 of the growth the running sums allow

template <int kW>
struct ChunkRing {
  alignas(1024) uint8_t slot[kW][kStages][kStageBytes];
  alignas(8) uint64_t full[kW][kStages];
  uint64_t empty[kW][kStages];
};

// Per-warp results of 16 rows, handed to the combine (rows padded so that the
// lanes of a fragment hit different banks).
template <int kW>
struct ChunkCombine {
  float m[kW][16];
  float l[kW][16];
  alignas(16) float acc[kW][16][kD + 8];
};

// The rows of one sequence that a CTA works on, and the keys they see.
struct ChunkRows {
  int q_row;          // first query row in q / out
  int tb;             // query rows
  int first_limit;    // last key that the first row sees
  int key_end;        // keys that some row sees: [0, key_end)
};

// A weight of zero does not hide an infinity or a NaN in V.  On a page of
// which some rows of the block see a token that others do not, such elements
// leave the V slice (for zero) and go straight into the sums of the rows that
// see them; any positive weight gives the same non-finite sum.
template <int MB>
__device__ __forceinline__ void part_visible_nonfinite(
    uint8_t* vbase, int tok0, int first_limit, int lane,
    const int (&limit)[MB][2], float (&acc)[MB][8][4]) {
  bool any = false;
#pragma unroll
  for (int e = lane; e < kPS * 8; e += 32) {
    const uint4 u = *reinterpret_cast<const uint4*>(vbase + e * 16);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      any |= (w[k] & 0x7f80u) == 0x7f80u ||
             (w[k] & 0x7f800000u) == 0x7f800000u;
  }
  if (!__any_sync(0xffffffffu, any)) return;
  const int c = lane & 3;
  for (int r = max(0, first_limit + 1 - tok0); r < kPS; ++r)
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          vbase + r * kRowBytes + ((d ^ (r & 7)) << 4) + 4 * c);
      const float x = bf16_lo(w), y = bf16_hi(w);
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (tok0 + r <= limit[b][e]) {
            if (!isfinite(x)) acc[b][d][2 * e] += x;
            if (!isfinite(y)) acc[b][d][2 * e + 1] += y;
          }
    }
  __syncwarp();
  uint32_t* words = reinterpret_cast<uint32_t*>(vbase);
  for (int r = max(0, first_limit + 1 - tok0); r < kPS; ++r) {
    uint32_t w = words[r * 32 + lane];
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    words[r * 32 + lane] = w;
  }
  __syncwarp();
}

// What a warp holds of 16 MB rows: q, the running offset and sum of each row
// and the accumulators.  Lane 4g + c owns rows g and g + 8 of each 16-row
// block, and in the accumulators dims 8d + 2c, +1 of them.
template <int MB, bool kCausal>
struct WarpRows {
  uint32_t qa[MB][4][4];
  int limit[MB][2];      // last key that the row sees
  float m[MB][2], l[MB][2], acc[MB][8][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      m[b][0] = m[b][1] = kNoOffset;
      l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][n][e] = 0.f;
    }
  }

  // As the A operand of S = Q K^T a lane holds dims 16k + 2c, +1 and + 8.
  __device__ __forceinline__ void load(const ChunkArgs& a, const ChunkRows& w,
                                       int kvh, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const int G = 1 << a.group_shift;
    const int rows = w.tb << a.group_shift;
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * b + g + 8 * e;
        const bool real = r < rows;
        const int t = real ? r >> a.group_shift : w.tb - 1;
        const int h = r & (G - 1);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            a.q + ((size_t)(w.q_row + t) * a.num_q_heads + kvh * G + h) * kD);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          qa[b][k][e] = real ? __ldg(src + 8 * k + c) : 0u;
          qa[b][k][e + 2] = real ? __ldg(src + 8 * k + c + 4) : 0u;
        }
        limit[b][e] = kCausal ? w.first_limit + t : w.key_end - 1;
      }
  }

  // One 16-token page that lies in a ring slot: tokens tok0 .. tok0 + 15.  True
  // when it wrote into the slot.
  __device__ __forceinline__ bool page(uint8_t* kbase, int tok0, bool page_ok,
                                       const ChunkRows& w,
                                       const uint32_t (&koff)[4],
                                       const uint32_t (&voff)[4], float sl,
                                       int lane) {
    const int c = lane & 3;
    uint8_t* vbase = kbase + kSliceBytes;
    // warp-uniform: every row sees every token of the page
    const bool full_page = page_ok && tok0 + kPS - 1 <= w.first_limit;
    if (!page_ok || tok0 + kPS > w.key_end) {
      // tokens that no row of the block sees (stale slots may hold NaN, and
      // 0 * NaN would reach the sum) and bad pages: zero V rows
#pragma unroll
      for (int e = lane; e < kPS * 8; e += 32) {
        const int r = e >> 3;
        if (!(page_ok && tok0 + r < w.key_end))
          *reinterpret_cast<uint4*>(vbase + r * kRowBytes + (e & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    if (kCausal && page_ok && !full_page)
      part_visible_nonfinite(vbase, tok0, w.first_limit, lane, limit, acc);
    const uint32_t kb = smem_u32(kbase), vb = smem_u32(vbase);

    // ---- S = Q K^T: 16 MB rows x 16 tokens ----------------------------------
    float s[MB][2][4];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t kf[4];
      ldsm_x4(kb + koff[k], kf);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        mma_bf16_16816(s[b][0], qa[b][k], kf[0], kf[1]);
        mma_bf16_16816(s[b][1], qa[b][k], kf[2], kf[3]);
      }
    }
    // ---- weights against the offsets as they stand, in bf16 and already in
    //      A-operand order.  Where a score exceeds its row's offset by 2^kLazy
    //      (any offset gives the same acc / l), and on pages with hidden
    //      tokens, the row's maximum is taken, its offset moved and the
    //      weights are done again; the check is off the path to the
    //      exponentials, and needs no exchange between lanes -----------------
    uint32_t ph[MB][4], pl[MB][4];    // and the weights' remainders
    auto weight = [&](int b, int n, int e, int k) {
      return fast_exp2(fmaf(s[b][n][2 * e + k], sl, -m[b][e]));
    };
    auto split = [&](int b, int i, float p0, float p1) {
      const uint32_t h = pack_bf16x2(p0, p1);
      ph[b][i] = h;
      const float2 rest =
          __ffma2_rn(make_float2(bf16_lo(h), bf16_hi(h)),
                     make_float2(-1.f, -1.f), make_float2(p0, p1));
      pl[b][i] = pack_bf16x2(rest.x, rest.y);
    };
    float top = -INFINITY, ls[MB][2];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ls[b][e] = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          // (kNoOffset, no finite score seen yet, makes the exponential of a
          // finite score infinite: done again)
          const float x0 = fmaf(s[b][n][2 * e], sl, -m[b][e]);
          const float x1 = fmaf(s[b][n][2 * e + 1], sl, -m[b][e]);
          top = fmax3(top, x0, x1);
          const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
          ls[b][e] += p0 + p1;
          split(b, 2 * n + e, p0, p1);
        }
      }
    if (!full_page || __any_sync(0xffffffffu, top > kLazy)) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int tok = tok0 + 8 * n + 2 * c + k;
              if (!(page_ok && tok <= limit[b][e]))
                s[b][n][2 * e + k] = -INFINITY;
              x = fmaxf(x, s[b][n][2 * e + k]);
            }
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          x *= sl;                    // scale > 0: the maximum commutes with it
          // a row's offset depends on its own scores alone, so a row gives
          // the same result whatever stands in the rows beside it
          if (x > m[b][e] + kLazy) {
            const float f = fast_exp2(m[b][e] - x);
            m[b][e] = x;
            l[b][e] *= f;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              acc[b][d][2 * e] *= f;
              acc[b][d][2 * e + 1] *= f;
            }
          }
          ls[b][e] = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = weight(b, n, e, 0), p1 = weight(b, n, e, 1);
            ls[b][e] += p0 + p1;
            split(b, 2 * n + e, p0, p1);
          }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      l[b][0] += ls[b][0];
      l[b][1] += ls[b][1];
    }

    // ---- O += P V --------------------------------------------------------------
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t vf[4];
      ldsm_x4_trans(vb + voff[t], vf);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        mma_bf16_16816(acc[b][2 * t], ph[b], vf[0], vf[1]);
        mma_bf16_16816(acc[b][2 * t + 1], ph[b], vf[2], vf[3]);
        mma_bf16_16816(acc[b][2 * t], pl[b], vf[0], vf[1]);
        mma_bf16_16816(acc[b][2 * t + 1], pl[b], vf[2], vf[3]);
      }
    }
    return !full_page;
  }

  // The quads hold a row's sum in four parts.
  __device__ __forceinline__ void finish_sums() {
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], 1);
        l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], 2);
      }
  }

  template <int kW>
  __device__ __forceinline__ void put(ChunkCombine<kW>& cb, int b, int warp,
                                      int lane) const {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<float2*>(&cb.acc[warp][r][8 * d + 2 * c]) =
            make_float2(acc[b][d][2 * e], acc[b][d][2 * e + 1]);
      if (c == 0) {
        cb.m[warp][r] = m[b][e];
        cb.l[warp][r] = l[b][e];
      }
    }
  }
};

// Joins partial results (offset m, sum l, unscaled output) of 8 dims of one
// row, dims 4k .. 4k + 3 and 32 + 4k .. : any common offset gives the same
// ratio, and the order of the parts is fixed.
struct Joined {
  float M = -INFINITY, L = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
  bool lost = false;    // a part of it ran out of time: zeros
  __device__ __forceinline__ void add(float m, float l, float4 u, float4 v) {
    lost |= m != m;     // (an offset is NaN only as this mark)
    // equal offsets first: -inf (no finite score) must not become NaN
    const float f = m == M ? 1.f : fast_exp2(m - M);
    L = fmaf(l, f, L);
    x.x = fmaf(u.x, f, x.x);
    x.y = fmaf(u.y, f, x.y);
    x.z = fmaf(u.z, f, x.z);
    x.w = fmaf(u.w, f, x.w);
    y.x = fmaf(v.x, f, y.x);
    y.y = fmaf(v.y, f, y.y);
    y.z = fmaf(v.z, f, y.z);
    y.w = fmaf(v.w, f, y.w);
  }
  // a larger offset for what was added so far
  __device__ __forceinline__ void raise(float m) {
    const float f = m == M ? 1.f : fast_exp2(M - m);
    M = m;
    L *= f;
    x = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    y = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
  }
  __device__ __forceinline__ void write(__nv_bfloat16* row, int k) const {
    const float inv = L == 0.f ? 0.f : 1.f / L;   // NaN scores stay NaN
    uint2 lo = make_uint2(pack_bf16x2(x.x * inv, x.y * inv),
                          pack_bf16x2(x.z * inv, x.w * inv));
    uint2 hi = make_uint2(pack_bf16x2(y.x * inv, y.y * inv),
                          pack_bf16x2(y.z * inv, y.w * inv));
    if (lost) lo = hi = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(row + 4 * k) = lo;
    *reinterpret_cast<uint2*>(row + 32 + 4 * k) = hi;
  }
  __device__ __forceinline__ float mark() const { return lost ? NAN : M; }
};

template <int kW>
__device__ __forceinline__ Joined join_warps(const ChunkCombine<kW>& cb, int r,
                                             int k) {
  Joined j;
#pragma unroll
  for (int w = 0; w < kW; ++w) j.M = fmaxf(j.M, cb.m[w][r]);
#pragma unroll
  for (int w = 0; w < kW; ++w)
    j.add(cb.m[w][r], cb.l[w][r],
          *reinterpret_cast<const float4*>(&cb.acc[w][r][4 * k]),
          *reinterpret_cast<const float4*>(&cb.acc[w][r][32 + 4 * k]));
  return j;
}

// Row r of a CTA's rows in the output.
__device__ __forceinline__ __nv_bfloat16* out_row(const ChunkArgs& a,
                                                  int q_row, int kvh, int r) {
  return a.out + ((size_t)(q_row + (r >> a.group_shift)) * a.num_q_heads +
                  (kvh << a.group_shift) + (r & ((1 << a.group_shift) - 1))) *
                     kD;
}

// ldmatrix row addresses inside a swizzled 2 KB slice (16-byte chunk j of row r
// at chunk j ^ (r & 7)).  K: (rows 0-7 | 8-15) x (chunk 2k | 2k + 1), V
// (transposed): (chunk 2t | 2t + 1) x (rows 0-7 | 8-15).
__device__ __forceinline__ void slice_offsets(int lane, uint32_t (&koff)[4],
                                              uint32_t (&voff)[4]) {
  const int mi = lane >> 3, r7 = lane & 7;
  const int kr = r7 + 8 * (mi >> 1), vr = r7 + 8 * (mi & 1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    koff[k] = kr * kRowBytes + (((2 * k + (mi & 1)) ^ r7) << 4);
    voff[k] = vr * kRowBytes + (((2 * k + (mi >> 1)) ^ r7) << 4);
  }
}

// Pool block (16 rows) of 16-token block `b` of a sequence, -1 when its
// block-table entry is not a page of the pool.
__device__ __forceinline__ int pool_block(const ChunkArgs& a, int seq, int b) {
  const int page = __ldg(a.block_tables + (size_t)seq * a.max_blocks_per_seq +
                         (b >> a.page_shift));
  return page >= 0 && page < a.num_pages
             ? (page << a.page_shift) + (b & ((1 << a.page_shift) - 1))
             : -1;
}

// Fills a ring slot; a bad page (-1) is flagged and block 0 loaded in its
// place (its tokens are masked and its V rows zeroed before use).
__device__ __forceinline__ void issue_block(const ChunkArgs& a,
                                            const CUtensorMap* tm_k,
                                            const CUtensorMap* tm_v, int x,
                                            int block, uint32_t dst,
                                            uint32_t bar, uint64_t policy) {
  if (block < 0) flag_error(a.err, DEVERR_BAD_PAGE);
  const int y = (block < 0 ? 0 : block) * kPS;
  mbar_arrive_expect_tx(bar, kStageBytes);
  tma_load_2d_hint(dst, tm_k, x, y, bar, policy);
  tma_load_2d_hint(dst + kSliceBytes, tm_v, x, y, bar, policy);
}

// Rows and context of a sequence as the call may use them; flags what is out
// of range when `report`.  False when the sequence has no rows to serve.
template <bool kCausal>
__device__ __forceinline__ bool sequence_rows(const ChunkArgs& a, int seq,
                                              bool report, int* qs, int* T,
                                              int* ctx) {
  *qs = a.query_start_loc[seq];
  *T = a.query_start_loc[seq + 1] - *qs;
  *ctx = a.context_lens[seq];
  const int cap = a.max_blocks_per_seq * (kPS << a.page_shift);
  if (*ctx < 0 || *ctx > cap) {
    if (report) flag_error(a.err, DEVERR_BAD_CONTEXT);
    *ctx = *ctx < 0 ? 0 : cap;
  }
  if (*T < 0 || *T > a.max_query_len || *qs < 0 ||
      (int64_t)*qs + *T > a.num_query_rows || (kCausal && *T > *ctx)) {
    if (report) flag_error(a.err, DEVERR_BAD_QUERY);
    return false;
  }
  return *T > 0;
}

// ---- one CTA per (KV head, block of rows, sequence) -----------------------------
// Without a workspace, or with more sequences than the balanced kernel's
// prefix sums hold.
template <int MB, bool kCausal>
__global__ void __launch_bounds__(kThreads, 3)
    paged_chunk_kernel(const ChunkArgs a,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v) {
  static_assert(sizeof(ChunkCombine<kWarps>) <= sizeof(ChunkRing<kWarps>::slot),
                "the combine buffer must fit in the ring");
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem_raw = smem_dyn + ((1024 - (smem_u32(smem_dyn) & 1023)) & 1023);
  auto& sm = *reinterpret_cast<ChunkRing<kWarps>*>(smem_raw);

  const int kvh = blockIdx.x;
  const int seq = blockIdx.y;
  const int blk = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int per_block = (16 * MB) >> a.group_shift;   // query rows

  int qs, T, ctx;
  if (!sequence_rows<kCausal>(a, seq, threadIdx.x == 0 && blk == 0 && kvh == 0,
                              &qs, &T, &ctx))
    return;
  const int t0 = blk * per_block;   // first query row
  if (t0 >= T) return;
  ChunkRows w;
  w.q_row = qs + t0;
  w.tb = min(per_block, T - t0);
  w.first_limit = kCausal ? ctx - T + t0 : ctx - 1;
  w.key_end = kCausal ? w.first_limit + w.tb : ctx;
  const int n_pages = (w.key_end + kPS - 1) / kPS;
  const int my_n = n_pages > warp ? (n_pages - warp + kWarps - 1) / kWarps : 0;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&sm.full[warp][s]), 1);
    fence_mbar_init();
  }
  __syncwarp();

  // this warp's 16-token blocks, 32 per batch, one per lane
  auto load_blocks = [&](int batch) -> int {
    const int i = batch * 32 + lane;
    return i < my_n ? pool_block(a, seq, warp + kWarps * i) : -1;
  };
  const uint64_t policy = l2_policy_evict_first();
  auto issue = [&](int block, int stage) {
    issue_block(a, &tm_k, &tm_v, kvh * kD, block,
                smem_u32(&sm.slot[warp][stage][0]),
                smem_u32(&sm.full[warp][stage]), policy);
  };
  int cur = load_blocks(0), next = load_blocks(1);
#pragma unroll
  for (int j = 0; j < kStages; ++j) {
    const int block = __shfl_sync(0xffffffffu, cur, j);
    if (lane == 0 && j < my_n) issue(block, j);
  }

  WarpRows<MB, kCausal> rows;
  rows.load(a, w, kvh, lane);
  rows.clear();
  uint32_t koff[4], voff[4];
  slice_offsets(lane, koff, voff);

  bool failed = false;
  int issued = min(my_n, kStages);
  int i = 0;
  for (; i < my_n; ++i) {
    const int stage = i % kStages;
    if ((i & 31) == 0 && i > 0) {
      cur = next;
      next = load_blocks((i >> 5) + 1);
    }
    const bool page_ok = __shfl_sync(0xffffffffu, cur, i & 31) >= 0;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[warp][stage]),
                                           (i / kStages) & 1)) ||
        TV_GIVE_UP(0, warp, i)) {
      failed = true;
      break;
    }
    // ---- hand the slot back to the TMA unit (plain writes into it are ordered
    //      before the copies that follow) -----------------------------------------
    if (rows.page(&sm.slot[warp][stage][0], (warp + kWarps * i) * kPS, page_ok,
                  w, koff, voff, a.scale_log2, lane))
      fence_proxy_async_smem();
    __syncwarp();
    const int j = i + kStages;
    const int src = ((j >> 5) == (i >> 5)) ? cur : next;
    const int block = __shfl_sync(0xffffffffu, src, j & 31);
    if (j < my_n) {
      if (lane == 0) issue(block, stage);
      ++issued;
    }
  }
  if (failed) {
    // let the copies in flight land (bounded)
    if (lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
    for (int k = i; k < issued; ++k)
      mbar_wait(smem_u32(&sm.full[warp][k % kStages]), (k / kStages) & 1);
  }
  // the rows need every warp's keys: without one warp's they are zeros
  if (__syncthreads_or(failed)) rows.clear();

  // ---- combine the four warps, 16 rows at a time, and write -----------------------
  rows.finish_sums();
  auto& cb = *reinterpret_cast<ChunkCombine<kWarps>*>(smem_raw);
  const int n_rows = w.tb << a.group_shift;
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    if (16 * b >= n_rows) break;
    __syncthreads();   // every warp is done with its ring, or the last rows
    rows.put(cb, b, warp, lane);
    __syncthreads();
    const int row = 16 * b + (threadIdx.x >> 3);
    if (row < n_rows)
      join_warps(cb, threadIdx.x >> 3, threadIdx.x & 7)
          .write(out_row(a, w.q_row, kvh, row), threadIdx.x & 7);
  }
}

// ---- balanced over the whole grid ------------------------------------------------
// The blocks of 16 tokens of all sequences (those with up to 16 MB rows per KV
// head), laid end to end, are cut into equal ranges, one per group of Hkv
// CTAs; CTA h of a group streams KV head h of the range, so the heads of a
// page are read at about the same time.  The grid is what is resident, so no
// last wave runs half empty whatever the lengths, and a long context is spread
// over as many SMs as it needs.  A boundary closer than kSnap blocks to the
// end of a sequence moves there, so short sequences are never cut.
//
// A sequence inside one range is written directly.  One that is cut leaves a
// part (m, l, unscaled output) per range in the workspace and counts up the
// counter of the first boundary inside it; the CTA that completes the count joins the parts, in the order of
// the ranges (results do not depend on timing), and sets the counter back to
// zero.  No CTA waits for another.
//
// W warps compute, block x0 + w + W i the i-th of warp w; one more looks the
// blocks up and issues the loads into their rings.  The rings run across
// sequence ends: the loads of the next sequence are in flight while the last
// one's warps are combined.  (With each warp issuing its own loads, that took
// it 72 us instead of 64 for 64 x 2048 tokens, 32 rows, when P still had one
// term.)  Measured against one CTA per sequence and KV head, in a graph: 32 rows,
// 64 x 2048 tokens 68 us and 75 (512 CTAs on 444 places); 16 rows, 8 x 131072: 319
// and 1196; one row, 8 x 16384: 49 and 143.  Where sequences x KV heads fill the
// GPU evenly it loses: one row, 64 x 2048 tokens 51 and 44, 64 x 375-1500 states
// of 16 KV heads 45 and 39.  Every call with a workspace takes it all the same
// (lengths are on the device, where a rule could not choose the launch); a caller
// that knows them passes no workspace.
constexpr int kSnap = 4;
// A sub-core's 16,384 registers hold three warps of 32 rows (168 each) or four
// of 16 rows (128) nearly without spills.  Measured with one term of P, W x CTAs
// an SM: 32 rows, 64 x 2048 tokens, 5 x 2 64.8 us, 3 x 3 66.6; 16 rows,
// 8 x 131072 tokens, 4 x 3 322 us, 5 x 2 329, 3 x 3 333.
__host__ __device__ constexpr int compute_warps(int mb) {
  return mb == 1 ? 4 : 5;
}
__host__ __device__ constexpr int ctas_per_sm(int mb) {
  return mb == 1 ? kChunkCtasPerSm : 2;
}

template <int kW>
struct BalancedSmem {
  ChunkRing<kW> ring;
  ChunkCombine<kW> cb;
  int32_t warp_total[kW + 1];
  int32_t items;
  int32_t last[2];
  int32_t failed;              // a warp's wait ran out
  uint32_t bad[kW][kStages];   // the slot's block was no page
  int32_t pre[kMaxChunkSeqs + 1];
};

// The CTA's range of blocks, from the prefix sums in shared memory.
struct BlockLine {
  const int32_t* pre;
  int B, W, NG;
  __device__ __forceinline__ int seq_of(int x) const {   // pre[s] <= x < pre[s+1]
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ int raw(int g) const {
    return W < 1 << 20 ? (int)((uint32_t)g * (uint32_t)W / (uint32_t)NG)
                       : (int)((int64_t)g * W / NG);
  }
  // first block of group g's range: moved to a close sequence end
  __device__ __forceinline__ int cut(int g) const {
    const int y = raw(g);
    if (y >= W) return W;
    const int s = seq_of(y);
    if (y - pre[s] < kSnap) return pre[s];
    if (pre[s + 1] - y < kSnap) return pre[s + 1];
    return y;
  }
};

template <int kW>
__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kW * 32) : "memory");
}

// Joins the parts of the blocks that the tile kernel cut along the keys: a warp
// takes 8 dims of 32 rows (a lane each) of one query tile and KV head.
template <bool kCausal>
__device__ __forceinline__ void join_tiles(const ChunkArgs& a, int warp,
                                           int warps, int lane) {
  const int Hkv = a.num_kv_heads;
  const int2 end = __ldcg(reinterpret_cast<const int2*>(&a.plan->joins));
  if (end.y) {
    // a wait of the tile kernel ran out, and units may have been left: the rows
    // of all its sequences are zeros
    for (int s = warp; s < a.num_seqs; s += warps) {
      TileBlock b;
      if (!tile_block<kCausal>(a, s, 0, &b)) continue;
      const int64_t n =
          (int64_t)(a.query_start_loc[s + 1] - b.q_row) * a.num_q_heads * 8;
      uint4* row = reinterpret_cast<uint4*>(
          a.out + (size_t)b.q_row * a.num_q_heads * kD);
      for (int64_t i = lane; i < n; i += 32) row[i] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int tasks = end.x * Hkv * 2 * 4 * 8;
  for (int i = warp; i < tasks; i += warps) {
    const int dims = i & 7, quarter = (i >> 3) & 3, t = (i >> 5) & 1;
    const int kvh = (i >> 6) % Hkv;
    const int4 e = __ldcg(a.plan_joins + (i >> 6) / Hkv);
    TileBlock b;
    tile_block<kCausal>(a, e.x, e.y, &b);
    const int r = quarter * 32 + lane;           // row of the query tile
    const int row = t * 128 + r;                 // row of the block
    const float* part0 = a.tile_parts +
                         ((size_t)e.z * Hkv + kvh) * kTilePartFloats +
                         t * (kTilePartFloats / 2);
    const size_t step = (size_t)Hkv * kTilePartFloats;
    Joined j;
    for (int k0 = 0; k0 < e.w; k0 += 8) {
      float m8[8], l8[8];
      float4 x8[8], y8[8];
      float top = j.M;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        m8[q] = -INFINITY;
        l8[q] = 0.f;
        x8[q] = y8[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + q < e.w) {
          const float* p = part0 + (k0 + q) * step;
          const float4* v = reinterpret_cast<const float4*>(p + 256) +
                            2 * dims * 128 + r;
          m8[q] = __ldcg(p + r);
          l8[q] = __ldcg(p + 128 + r);
          x8[q] = __ldcg(v);
          y8[q] = __ldcg(v + 128);
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) top = fmaxf(top, m8[q]);
      j.raise(top);
#pragma unroll
      for (int q = 0; q < 8; ++q) j.add(m8[q], l8[q], x8[q], y8[q]);
    }
    if (row < b.tb << a.group_shift) {
      const float inv = j.L == 0.f ? 0.f : 1.f / j.L;   // NaN scores stay NaN
      *reinterpret_cast<uint4*>(out_row(a, b.q_row, kvh, row) + 8 * dims) =
          make_uint4(pack_bf16x2(j.x.x * inv, j.x.y * inv),
                     pack_bf16x2(j.x.z * inv, j.x.w * inv),
                     pack_bf16x2(j.y.x * inv, j.y.y * inv),
                     pack_bf16x2(j.y.z * inv, j.y.w * inv));
    }
  }
}

template <int MB, bool kCausal>
__global__ void __launch_bounds__((compute_warps(MB) + 1) * 32,
                                  ctas_per_sm(MB))
    balanced_chunk_kernel(const ChunkArgs a,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kW = compute_warps(MB);
  constexpr int kBalancedThreads = (kW + 1) * 32;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem_raw = smem_dyn + ((1024 - (smem_u32(smem_dyn) & 1023)) & 1023);
  auto& sm = *reinterpret_cast<BalancedSmem<kW>*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.num_seqs;
  const int Hkv = a.num_kv_heads;

  // ---- blocks per sequence, exclusive prefix in shared memory ------------------
  if (threadIdx.x == 0) sm.items = sm.failed = 0;
  if (lane == 0 && warp < kW) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.ring.full[warp][s]), 1);
      mbar_init(smem_u32(&sm.ring.empty[warp][s]), 1);
    }
    fence_mbar_init();
  }
  // thread t sums the sequences t * per .. + per - 1
  const int per = (B + kBalancedThreads - 1) / kBalancedThreads;
  const int s0 = min(B, (int)threadIdx.x * per), s1 = min(B, s0 + per);
  int own = 0, live_seqs = 0;
  for (int s = s0; s < s1; ++s) {
    int qs, T, ctx;
    const bool live = sequence_rows<kCausal>(a, s, blockIdx.x == 0, &qs, &T,
                                             &ctx) &&
                      T <= a.stream_rows;
    // a sequence without keys keeps one block, not loaded, for its zero rows
    const int n = live ? max(1, (ctx + kPS - 1) / kPS) : 0;
    sm.pre[s] = n;
    own += n;
    live_seqs += live;
  }
  int incl = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) sm.warp_total[warp] = incl;
  __syncthreads();
  if (live_seqs) atomicAdd(&sm.items, live_seqs);
  int run = incl - own;
  for (int v = 0; v < warp; ++v) run += sm.warp_total[v];
  for (int s = s0; s < s1; ++s) {
    const int n = sm.pre[s];
    sm.pre[s] = run;
    run += n;
  }
  if (threadIdx.x == kBalancedThreads - 1) sm.pre[B] = run;
  __syncthreads();

  // ---- this CTA's range ----------------------------------------------------------
  BlockLine line;
  line.pre = sm.pre;
  line.B = B;
  line.W = sm.pre[B];
  // A range worth a CTA: more parts of one sequence shorten its ranges but are
  // joined by one CTA, so ranges grow with the root of the whole (one KV head, 31
  // and 47 rows over 90,063 and 42,422 tokens: 242 us with up to 375 parts of 16
  // blocks joined thread by thread, now 60).
  const int least = min(64, max(kMinChunkBlocks, (int)(0.6f * sqrtf(line.W))));
  line.NG = min((int)gridDim.x / Hkv, max(line.W / least, sm.items));
  const int W = line.W, NG = line.NG;
  const int grp = blockIdx.x / Hkv;
  const int head = blockIdx.x - grp * Hkv;
  const int x0 = grp < NG ? line.cut(grp) : 0;
  const int x1 = grp < NG ? line.cut(grp + 1) : 0;
  const int steps = (x1 - x0 + kW - 1) / kW;

  if (warp == kW) {
    // ======================= loads =============================================
    // Lane 2 w + v issues K (v = 0) or V of warp w's block; the blocks of as many
    // steps as fit are looked up one per lane.
    constexpr int kLook = 32 / kW;
    const int w = lane >> 1;
    const bool is_v = lane & 1;
    const bool issuer = lane < 2 * kW;
    const uint64_t policy = l2_policy_evict_first();
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    auto look_up = [&](int step) -> int {
      const int x = x0 + step * kW + lane;
      if (lane >= kLook * kW || x >= x1) return -2;
      const int s = line.seq_of(x);
      // (a sequence without keys has nothing to look up: block 0)
      return a.context_lens[s] > 0 ? pool_block(a, s, x - sm.pre[s]) : 0;
    };
    int blocks = look_up(0), ahead = look_up(kLook);
    int in_look = 0;
    bool ok = true;
    int i = 0;
    for (; i < steps; ++i) {
      if (in_look == kLook) {
        in_look = 0;
        blocks = ahead;
        ahead = look_up(i + kLook);
      }
      const int block = __shfl_sync(0xffffffffu, blocks,
                                    in_look * kW + (issuer ? w : 0));
      ++in_look;
      const int stage = i % kStages;
      const bool mine = issuer && block != -2;
      const bool ready =
          !mine || i < kStages ||
          mbar_wait(smem_u32(&sm.ring.empty[w][stage]), (i / kStages + 1) & 1);
      if (!__all_sync(0xffffffffu, ready)) {
        ok = false;
        break;
      }
      if (mine) {
        const uint32_t bar = smem_u32(&sm.ring.full[w][stage]);
        if (!is_v) {
          // a bad page is flagged and block 0 loaded in its place
          if (block < 0) flag_error(a.err, DEVERR_BAD_PAGE);
          sm.bad[w][stage] = block < 0;
          mbar_arrive_expect_tx(bar, kStageBytes);
        }
        tma_load_2d_hint(smem_u32(&sm.ring.slot[w][stage][0]) +
                             (is_v ? kSliceBytes : 0),
                         tm, head * kD, max(block, 0) * kPS, bar, policy);
      }
    }
    if (!ok) {
      if (lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
      // the copies in flight land before the CTA ends (bounded)
      if (issuer && !is_v)
        for (int k = max(0, i - kStages); k < i; ++k)
          if (x0 + k * kW + w < x1)
            mbar_wait(smem_u32(&sm.ring.full[w][k % kStages]),
                      (k / kStages) & 1);
    }
  } else if (x0 < x1) {
    // ======================= products ==========================================
    uint32_t koff[4], voff[4];
    slice_offsets(lane, koff, voff);
    WarpRows<MB, kCausal> rows;
    bool failed = false;
    int stage = 0;
    uint32_t parity = 0;
    int x = x0 + warp;                  // the warp's next block
    int seq = line.seq_of(x0);
    int next_qs, next_T, next_ctx;
    sequence_rows<kCausal>(a, seq, false, &next_qs, &next_T, &next_ctx);
    ChunkRows w;
    auto set_rows = [&]() {
      w.q_row = next_qs;
      w.tb = next_T;
      w.first_limit = kCausal ? next_ctx - next_T : next_ctx - 1;
      w.key_end = next_ctx;
    };
    set_rows();
    rows.load(a, w, head, lane);
    // Parts of the groups that a cut sequence is spread over: group g0 - 1 + k's
    // is part k.
    struct Parts {
      int g0, n;
    };
    auto first_inside = [&](int s) {  // first group with a boundary inside it
      return (int)(((int64_t)(sm.pre[s] + kSnap) * NG + W - 1) / W);
    };
    auto parts_of = [&](int s) {
      const int z1 = sm.pre[s + 1] - kSnap;
      const int g0 = first_inside(s);
      const int g1 = (int)(((int64_t)(z1 + 1) * NG + W - 1) / W) - 1;
      return Parts{g0, g1 - g0 + 2};
    };
    // A boundary lies inside one sequence, so its group's word is that
    // sequence's own, and there is one per CTA for any batch.
    auto counter_of = [&](int s) {
      return a.ws_counters + first_inside(s) * Hkv + head;
    };
    const int r16 = threadIdx.x >> 3, k8 = threadIdx.x & 7;
    int cut_seq[2] = {-1, -1};        // the cut sequences of the range's ends
    int counted[2] = {0, 0};          // thread 0: their counters before its own
    for (int p0 = x0; p0 < x1;) {
      const int base = sm.pre[seq];
      const int end = min(x1, sm.pre[seq + 1]);
      const int q_row = w.q_row, n_rows = w.tb << a.group_shift;
      int next_seq = seq;
      if (end < x1) {   // the next sequence's rows, and its q into the cache
        do ++next_seq; while (sm.pre[next_seq + 1] <= end);
        sequence_rows<kCausal>(a, next_seq, false, &next_qs, &next_T,
                               &next_ctx);
        if (warp == 0 && lane < next_T << a.group_shift)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(
              a.q + ((size_t)(next_qs + (lane >> a.group_shift)) *
                         a.num_q_heads + (head << a.group_shift) +
                     (lane & ((1 << a.group_shift) - 1))) * kD));
      }
      rows.clear();
      for (; x < end && !failed; x += kW) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait(smem_u32(&sm.ring.full[warp][stage]),
                                  parity)) ||
            TV_GIVE_UP(1, warp, x - x0)) {
          failed = true;
          break;
        }
        if (rows.page(&sm.ring.slot[warp][stage][0], (x - base) * kPS,
                      sm.bad[warp][stage] == 0, w, koff, voff, a.scale_log2,
                      lane))
          fence_proxy_async_smem();   // plain writes, before the next copy
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.ring.empty[warp][stage]));
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
      if (failed) sm.failed = 1;
      if (end < x1) {   // the next q, in flight during the combine
        set_rows();
        rows.load(a, w, head, lane);
      }

      // ---- combine the warps; write, or leave a part --------------------------------
      rows.finish_sums();
      const bool whole = p0 == base && end == sm.pre[seq + 1];
      const int slot = p0 == x0 ? 0 : 1;
      bool lost = false;
      float* part =
          a.ws_parts + ((size_t)blockIdx.x * 2 + slot) * kChunkPartFloats;
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        if (16 * b >= n_rows) break;
        compute_barrier<kW>();   // the last rows have been read
        // the rows need every warp's keys: without one warp's, here or in a
        // part of theirs elsewhere, they are zeros
        if (b == 0) lost = *(volatile int32_t*)&sm.failed != 0;
        if (lost) rows.clear();
        rows.put(sm.cb, b, warp, lane);
        compute_barrier<kW>();
        const int row = 16 * b + r16;
        if (r16 >= 16 || row >= n_rows) continue;
        const Joined j = join_warps(sm.cb, r16, k8);
        if (whole) {
          j.write(out_row(a, q_row, head, row), k8);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + 2 * kChunkPartRows +
                                                  row * kD + 4 * k8);
          __stcg(dst, j.x);
          __stcg(dst + 8, j.y);
          if (k8 == 0) {
            __stcg(part + row, lost ? NAN : j.M);
            __stcg(part + kChunkPartRows + row, j.L);
          }
        }
      }
      if (!whole) {
        // count the part; what the count says is looked at when the range is done
        cut_seq[slot] = seq;
        compute_barrier<kW>();
        if (threadIdx.x == 0) {
          __threadfence();   // the CTA's part, ordered by the barrier
          counted[slot] = atomicAdd(counter_of(seq), 1);
        }
      }
      p0 = end;
      seq = next_seq;
    }

    // ---- cut sequences whose last part was this CTA's: join the parts ----------------
    if (cut_seq[0] >= 0 || cut_seq[1] >= 0) {
      if (threadIdx.x == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sm.last[e] =
              cut_seq[e] >= 0 && counted[e] == parts_of(cut_seq[e]).n - 1;
        __threadfence();
      }
      compute_barrier<kW>();
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        if (!sm.last[e]) continue;
        const int s = cut_seq[e];
        const Parts parts = parts_of(s);
        const bool first0 = line.cut(parts.g0 - 1) == sm.pre[s];
        auto part_of = [&](int k) {
          return a.ws_parts +
                 ((size_t)((parts.g0 - 1 + k) * Hkv + head) * 2 +
                  (k == 0 && !first0 ? 1 : 0)) *
                     kChunkPartFloats;
        };
        int qs, T, ctx;
        sequence_rows<kCausal>(a, s, false, &qs, &T, &ctx);
        // a few parts: a thread joins 8 dims of its rows
        const bool few = parts.n <= 8;
        for (int row = r16; few && row < T << a.group_shift; row += kW * 4) {
          Joined j;
#pragma unroll 4
          for (int k = 0; k < parts.n; ++k)
            j.M = fmaxf(j.M, __ldcg(part_of(k) + row));
#pragma unroll 4
          for (int k = 0; k < parts.n; ++k) {
            const float* q = part_of(k);
            const float4* v = reinterpret_cast<const float4*>(
                q + 2 * kChunkPartRows + row * kD + 4 * k8);
            j.add(__ldcg(q + row), __ldcg(q + kChunkPartRows + row),
                  __ldcg(v), __ldcg(v + 8));
          }
          j.write(out_row(a, qs, head, row), k8);
        }
        // many: warp w joins parts w, w + kW, ... of 4 rows at a time (eight of
        // them in flight), then the warps' results as after a range
        const int jr = lane >> 3;
        for (int row0 = 0; !few && row0 < T << a.group_shift; row0 += 16) {
#pragma unroll 1
          for (int g = 0; g < 16; g += 4) {
            const int row = min(row0 + g + jr, kChunkPartRows - 1);
            Joined j;
            for (int k0 = warp; k0 < parts.n; k0 += 8 * kW) {
              float m8[8], l8[8];
              float4 x8[8], y8[8];
              float top = j.M;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int k = k0 + e * kW;
                m8[e] = -INFINITY;
                l8[e] = 0.f;
                x8[e] = y8[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < parts.n) {
                  const float* q = part_of(k);
                  const float4* v = reinterpret_cast<const float4*>(
                      q + 2 * kChunkPartRows + row * kD + 4 * k8);
                  m8[e] = __ldcg(q + row);
                  l8[e] = __ldcg(q + kChunkPartRows + row);
                  x8[e] = __ldcg(v);
                  y8[e] = __ldcg(v + 8);
                }
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) top = fmaxf(top, m8[e]);
              j.raise(top);
#pragma unroll
              for (int e = 0; e < 8; ++e) j.add(m8[e], l8[e], x8[e], y8[e]);
            }
            if (k8 == 0) {
              sm.cb.m[warp][g + jr] = j.mark();
              sm.cb.l[warp][g + jr] = j.L;
            }
            float* acc = sm.cb.acc[warp][g + jr];
            *reinterpret_cast<float4*>(acc + 4 * k8) = j.x;
            *reinterpret_cast<float4*>(acc + 32 + 4 * k8) = j.y;
          }
          compute_barrier<kW>();
          if (r16 < 16 && row0 + r16 < T << a.group_shift)
            join_warps(sm.cb, r16, k8)
                .write(out_row(a, qs, head, row0 + r16), k8);
          compute_barrier<kW>();
        }
        if (threadIdx.x == 0) *counter_of(s) = 0;
      }
    }
    if (failed && lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
  }
  // the rows of the tile kernel are written when this kernel ends
  if (a.tile_ctas) {
    wait_for_last_kernel();
    join_tiles<kCausal>(a, blockIdx.x * (kBalancedThreads / 32) + warp,
                        gridDim.x * (kBalancedThreads / 32), lane);
  }
}

template <int MB>
constexpr bool fits() {
  return ctas_per_sm(MB) *
             (sizeof(BalancedSmem<compute_warps(MB)>) + 1024 + 1024) <=
         228 * 1024;
}
static_assert(fits<1>() && fits<2>(),
              "the CTAs of an SM must fit in its shared memory");

template <int MB, bool kCausal>
cudaError_t launch_mb(const ChunkArgs& a, const CUtensorMap& tk,
                      const CUtensorMap& tv, cudaStream_t stream) {
  // behind the tile kernel it fills the SMs that run out of tiles
  if (a.balanced_ctas)
    return launch_kernel<balanced_chunk_kernel<MB, kCausal>>(
        dim3(a.balanced_ctas / kChunkCtasPerSm * ctas_per_sm(MB)),
        (compute_warps(MB) + 1) * 32,
        sizeof(BalancedSmem<compute_warps(MB)>) + 1024,
        a.tile_ctas > 0, stream, a, tk, tv);
  const int per = (16 * MB) >> a.group_shift;
  return launch_kernel<paged_chunk_kernel<MB, kCausal>>(
      dim3(a.num_kv_heads, a.num_seqs, (a.max_query_len + per - 1) / per),
      kThreads, sizeof(ChunkRing<kWarps>) + 1024, false, stream, a, tk, tv);
}

}  // namespace

cudaError_t launch_paged_chunk(const ChunkArgs& a, const CUtensorMap& tk,
                               const CUtensorMap& tv, bool causal,
                               cudaStream_t stream) {
  const int64_t rows = (int64_t)a.max_query_len << a.group_shift;
  if (rows <= 16)
    return causal ? launch_mb<1, true>(a, tk, tv, stream)
                  : launch_mb<1, false>(a, tk, tv, stream);
  return causal ? launch_mb<2, true>(a, tk, tv, stream)
                : launch_mb<2, false>(a, tk, tv, stream);
}

}  // namespace tv
