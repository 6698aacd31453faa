// Attention of a chunk of new rows per sequence over the paged cache, causal
// or over every key, for row counts too small for a 128-row MMA tile.
//
// Mathematics: sequence s has T query rows and C cached keys.  Row i, head h:
//   out = sum_j softmax_j(scale q.K_j) V_j  over the keys j it sees, which
//   are 0 .. C - T + i (causal chunk) or all C (cross attention).
// The softmax is online: a running maximum m and sum l per row, O rescaled
// when m moves.
//
// What bounds it: a sequence's K and V are read once for all of its rows, so
// up to about 64 rows x heads per KV head the work is the HBM stream.
//
// Design.  One CTA of 4 warps per (KV head, block of rows, sequence); every
// warp streams its own pages w, w + 4, ... through a private ring of TMA
// boxes (16 tokens x 128 B of K and of V, 128-byte swizzle), so no warp waits
// for another before the final combine.  A row of the product is one (query
// row, head of the KV head's group) pair, row r = query row r / G, head
// r % G, 16 * MB rows per block.  Per page a warp forms S = Q K^T and
// O += P V with m16n8k16 bf16 products and fp32 accumulators: with at least
// 16 rows, rows in the M dimension put P's accumulator fragment where the
// next product wants its A operand, so P needs no shuffles (the decode
// kernels, with at most 8 rows, put tokens in M instead).  P enters as two
// bf16 terms, as in the decode and the prefill, because one term's 8 bits
// are too few for rows that see few keys.
#include "tv_decode.cuh"
#include "tv_device.cuh"
#include "tv_kernels.h"

namespace tv {
namespace {

constexpr int kD = 64;
constexpr int kPS = 16;          // tokens per TMA box
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRowBytes = kD * 2;
constexpr int kSliceBytes = kPS * kRowBytes;
constexpr int kStageBytes = 2 * kSliceBytes;
constexpr float kLazy = 8.f;     // log2 of the growth the running sums allow

template <int MB, int kStages>
struct ChunkSmem {
  alignas(1024) uint8_t ring[kWarps][kStages][kStageBytes];
  alignas(8) uint64_t full[kWarps][kStages];
};

template <int MB>
struct ChunkCombine {   // per-warp results handed to the final combine
  float m[kWarps][16 * MB];
  float l[kWarps][16 * MB];
  float acc[kWarps][16 * MB][kD];
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

template <int MB, int kStages, bool kCausal>
__global__ void __launch_bounds__(kThreads, MB == 1 ? 4 : 3)
    paged_chunk_kernel(const ChunkArgs a,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kRows = 16 * MB;
  static_assert(sizeof(ChunkCombine<MB>) <=
                    sizeof(ChunkSmem<MB, kStages>::ring),
                "combine buffer must fit in the ring");
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem_raw = smem_dyn + ((1024 - (smem_u32(smem_dyn) & 1023)) & 1023);
  auto& sm = *reinterpret_cast<ChunkSmem<MB, kStages>*>(smem_raw);

  const int kvh = blockIdx.x;
  const int seq = blockIdx.y;
  const int blk = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = 1 << a.group_shift;

  // ---- rows and keys of this CTA ---------------------------------------------
  const int qs = a.query_start_loc[seq];
  const int T = a.query_start_loc[seq + 1] - qs;
  int ctx = a.context_lens[seq];
  const int t0 = blk * (kRows >> a.group_shift);   // first query row
  const int ctx_cap = a.max_blocks_per_seq * (kPS << a.page_shift);
  const bool head_cta = threadIdx.x == 0 && blk == 0 && kvh == 0;
  if (ctx < 0 || ctx > ctx_cap) {
    if (head_cta) flag_error(a.err, DEVERR_BAD_CONTEXT);
    ctx = ctx < 0 ? 0 : ctx_cap;
  }
  if (T < 0 || T > a.max_query_len || qs < 0 ||
      (int64_t)qs + T > a.num_query_rows || (kCausal && T > ctx)) {
    if (head_cta) flag_error(a.err, DEVERR_BAD_QUERY);
    return;
  }
  if (t0 >= T) return;
  const int tb = min(kRows >> a.group_shift, T - t0);   // query rows here
  const int rows = tb << a.group_shift;
  const int first_limit = kCausal ? ctx - T + t0 : ctx - 1;  // row 0's last key
  const int key_end = kCausal ? first_limit + tb : ctx;
  const int n_pages = (key_end + kPS - 1) / kPS;
  const int my_n = n_pages > warp ? (n_pages - warp + kWarps - 1) / kWarps : 0;
  const int32_t* bt = a.block_tables + (size_t)seq * a.max_blocks_per_seq;
  const int sub_mask = (1 << a.page_shift) - 1;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&sm.full[warp][s]), 1);
    fence_mbar_init();
  }
  __syncwarp();

  // Pool blocks of this warp's 16-token blocks, 32 per batch, one per lane
  // (-1 when the block-table entry is not a page of the pool).
  auto load_pids = [&](int batch) -> int {
    const int i = batch * 32 + lane;
    if (i >= my_n) return -1;
    const int b = warp + kWarps * i;
    const int page = __ldg(bt + (b >> a.page_shift));
    return page >= 0 && page < a.num_pages
               ? (page << a.page_shift) + (b & sub_mask) : -1;
  };
  const uint64_t policy = l2_policy_evict_first();
  auto issue = [&](int pid, int stage) {
    if (pid < 0) flag_error(a.err, DEVERR_BAD_PAGE);
    const int y = (pid < 0 ? 0 : pid) * kPS;
    const uint32_t bar = smem_u32(&sm.full[warp][stage]);
    const uint32_t dst = smem_u32(&sm.ring[warp][stage][0]);
    mbar_arrive_expect_tx(bar, kStageBytes);
    tma_load_2d_hint(dst, &tm_k, kvh * kD, y, bar, policy);
    tma_load_2d_hint(dst + kSliceBytes, &tm_v, kvh * kD, y, bar, policy);
  };
  int pid_cur = load_pids(0), pid_next = load_pids(1);
#pragma unroll
  for (int j = 0; j < kStages; ++j) {
    const int pid = __shfl_sync(0xffffffffu, pid_cur, j);
    if (lane == 0 && j < my_n) issue(pid, j);
  }

  // ---- fragments ---------------------------------------------------------------
  // Lane 4g + c.  Rows g and g + 8 of each 16-row block are the lane's; as
  // the A operand of S = Q K^T it holds dims 16k + 2c, +1 and + 8 of them.
  const int g = lane >> 2;
  const int c = lane & 3;
  uint32_t qa[MB][4][4];
  int limit[MB][2];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 16 * b + g + 8 * e;
      const bool real = r < rows;
      const int t = r >> a.group_shift, h = r & (G - 1);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          a.q + ((size_t)(qs + t0 + (real ? t : 0)) * a.num_q_heads +
                 kvh * G + (real ? h : 0)) * kD);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        qa[b][k][e] = real ? __ldg(src + 8 * k + c) : 0u;
        qa[b][k][e + 2] = real ? __ldg(src + 8 * k + c + 4) : 0u;
      }
      limit[b][e] = kCausal ? first_limit + (real ? t : tb - 1) : ctx - 1;
    }
  }
  // ldmatrix row addresses inside a swizzled 2 KB slice (16-byte chunk j of
  // row r at chunk j ^ (r & 7)).  K: (rows 0-7 | 8-15) x (chunk 2k | 2k + 1),
  // V (transposed): (chunk 2t | 2t + 1) x (rows 0-7 | 8-15).
  uint32_t koff[4], voff[4];
  {
    const int mi = lane >> 3, r7 = lane & 7;
    const int kr = r7 + 8 * (mi >> 1), vr = r7 + 8 * (mi & 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      koff[k] = kr * kRowBytes + (((2 * k + (mi & 1)) ^ r7) << 4);
      voff[k] = vr * kRowBytes + (((2 * k + (mi >> 1)) ^ r7) << 4);
    }
  }

  float m[MB][2], l[MB][2], acc[MB][8][4];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    m[b][0] = m[b][1] = -INFINITY;
    l[b][0] = l[b][1] = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[b][n][e] = 0.f;
  }
  const float sl = a.scale_log2;

  bool failed = false;
  int issued = min(my_n, kStages);
  int i = 0;
  for (; i < my_n; ++i) {
    const int stage = i % kStages;
    if ((i & 31) == 0 && i > 0) {
      pid_cur = pid_next;
      pid_next = load_pids((i >> 5) + 1);
    }
    const bool page_ok = __shfl_sync(0xffffffffu, pid_cur, i & 31) >= 0;
    const int tok0 = (warp + kWarps * i) * kPS;
    // warp-uniform: every row sees every token of the page
    const bool full_page = page_ok && tok0 + kPS - 1 <= first_limit;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[warp][stage]),
                                           (i / kStages) & 1))) {
      failed = true;
      break;
    }
    uint8_t* kbase = &sm.ring[warp][stage][0];
    uint8_t* vbase = kbase + kSliceBytes;
    if (!page_ok || tok0 + kPS > key_end) {
      // tokens that no row of the block sees (stale slots may hold NaN, and
      // 0 * NaN would reach the sum) and bad pages: zero V rows
#pragma unroll
      for (int e = lane; e < kPS * 8; e += 32) {
        const int r = e >> 3;
        if (!(page_ok && tok0 + r < key_end))
          *reinterpret_cast<uint4*>(vbase + r * kRowBytes + (e & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    if (kCausal && page_ok && !full_page)
      part_visible_nonfinite(vbase, tok0, first_limit, lane, limit, acc);
    const uint32_t kb = smem_u32(kbase), vb = smem_u32(vbase);

    // ---- S = Q K^T: 16 MB rows x 16 tokens ------------------------------------
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
    if (!full_page) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = tok0 + 8 * n + 2 * c + (e & 1);
            if (!(page_ok && tok <= limit[b][e >> 1])) s[b][n][e] = -INFINITY;
          }
    }

    // ---- online softmax; the offset moves only when a page's maximum exceeds
    //      it by 2^kLazy (any offset gives the same acc / l) ------------------
    float pm[MB][2];
    bool grow = false;
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(s[b][0][2 * e], s[b][0][2 * e + 1]),
                        fmaxf(s[b][1][2 * e], s[b][1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        pm[b][e] = x * sl;          // scale > 0: the maximum commutes with it
        grow |= pm[b][e] > m[b][e] + kLazy;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a row's offset depends on its own scores alone, so a row gives
          // the same result whatever stands in the rows beside it
          if (!(pm[b][e] > m[b][e] + kLazy)) continue;
          const float n = pm[b][e];
          const float f = fast_exp2(m[b][e] - n);
          m[b][e] = n;
          l[b][e] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            acc[b][d][2 * e] *= f;
            acc[b][d][2 * e + 1] *= f;
          }
        }
    }
    // P as two bf16 terms (hi + lo, ~16 bits), already in A-operand order
    uint32_t ph[MB][4], pl[MB][4];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mu = m[b][e] == -INFINITY ? 0.f : m[b][e];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = fast_exp2(fmaf(s[b][n][2 * e], sl, -mu));
          const float p1 = fast_exp2(fmaf(s[b][n][2 * e + 1], sl, -mu));
          l[b][e] += p0 + p1;
          const uint32_t h = pack_bf16x2(p0, p1);
          ph[b][2 * n + e] = h;
          pl[b][2 * n + e] = pack_bf16x2(p0 - bf16_lo(h), p1 - bf16_hi(h));
        }
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

    // ---- hand the slot back to the TMA unit ------------------------------------
    fence_proxy_async_smem();
    __syncwarp();
    const int j = i + kStages;
    const int src = ((j >> 5) == (i >> 5)) ? pid_cur : pid_next;
    const int pid_j = __shfl_sync(0xffffffffu, src, j & 31);
    if (j < my_n) {
      if (lane == 0) issue(pid_j, stage);
      ++issued;
    }
  }
  if (failed) {
    // let the copies in flight land (bounded), then an empty result
    if (lane == 0) flag_error(a.err, DEVERR_TIMEOUT);
    for (int k = i; k < issued; ++k)
      mbar_wait(smem_u32(&sm.full[warp][k % kStages]), (k / kStages) & 1);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[b][e] = -INFINITY;
        l[b][e] = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[b][d][2 * e] = acc[b][d][2 * e + 1] = 0.f;
      }
  }

  // ---- combine the four warps and write -----------------------------------------
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], 1);
      l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], 2);
    }
  __syncthreads();   // every warp is done with its ring
  auto& cb = *reinterpret_cast<ChunkCombine<MB>*>(smem_raw);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 16 * b + g + 8 * e;
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<float2*>(&cb.acc[warp][r][8 * d + 2 * c]) =
            make_float2(acc[b][d][2 * e], acc[b][d][2 * e + 1]);
      if (c == 0) {
        cb.m[warp][r] = m[b][e];
        cb.l[warp][r] = l[b][e];
      }
    }
  __syncthreads();
  for (int o = threadIdx.x; o < rows * (kD / 2); o += kThreads) {
    const int r = o / (kD / 2), d = 2 * (o % (kD / 2));
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cb.m[w][r]);
    float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // equal offsets first: -inf (no finite score) must not become NaN
      const float f = cb.m[w][r] == M ? 1.f : fast_exp2(cb.m[w][r] - M);
      const float2 v = *reinterpret_cast<const float2*>(&cb.acc[w][r][d]);
      L = fmaf(cb.l[w][r], f, L);
      x = fmaf(v.x, f, x);
      y = fmaf(v.y, f, y);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;   // NaN scores stay NaN
    const size_t row = (size_t)(qs + t0 + (r >> a.group_shift)) *
                           a.num_q_heads + kvh * G + (r & (G - 1));
    *reinterpret_cast<uint32_t*>(a.out + row * kD + d) =
        pack_bf16x2(x * inv, y * inv);
  }
}

template <int MB, bool kCausal>
cudaError_t launch_mb(const ChunkArgs& a, const CUtensorMap& tk,
                      const CUtensorMap& tv, cudaStream_t stream) {
  constexpr int kStages = 3;
  auto kern = paged_chunk_kernel<MB, kStages, kCausal>;
  const int smem = sizeof(ChunkSmem<MB, kStages>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int per = (16 * MB) >> a.group_shift;
  dim3 grid(a.num_kv_heads, a.num_seqs, (a.max_query_len + per - 1) / per);
  kern<<<grid, kThreads, smem, stream>>>(a, tk, tv);
  return cudaGetLastError();
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
