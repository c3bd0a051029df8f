// ssd_kv4_attn.cuh -- attention over a 4-bit paged cache: one kernel for the dense pass of n_cand
// candidates (verify; n_cand = 1 is plain decoding) and for the draft over a list of selected tokens,
// and one for the tokens' criticality.
//
// Mathematics, per (request, KV head) unit with R = G * n_cand query rows, x_rt = scale * q_r . k_t:
//   out_r = sum_t exp(x_rt) v_t / sum_t exp(x_rt) over the tokens row r sees, lse_r = log sum_t exp(x_rt),
//   crit_t = sum_r exp(x_rt - lse_r)   (SparseSpec §4.1: criticality summed over the group's heads and
//   the verify positions).
// One pass over K and V keeps a running reference m_r (a past maximum), the sum of exp2(x - m) and
// the weighted sum of V, all in fp32.
//
// Bound: 9 bits per (K, V) element pair stored, 144 bytes per token of a head at d = 128, so HBM bounds
// small R; the f16 tensor-core rate of mma.sync (1024 multiply-adds per clock and SM) bounds R > 20.
//
// Layout of the work.  A warp takes tiles of 32 tokens and computes, on the tensor cores,
//   S^T [32 tokens x 8 NT rows] = K Q^T   and   O^T [d x 8 NT rows] += V^T P^T,
// so that the cache is the A operand of both products and the few query rows the narrow N side (M = 16
// rows of queries would be mostly padding).  Codes go from shared memory to A fragments in registers:
// a lane reads 16 bytes of a token's K row and 8 of a V row, converts pairs of codes to f16 and
// multiplies them by their scale (exact, see ssd_kv4.cuh).  Which d a lane's fragment column stands for
// is free for K as long as Q is laid out alike, and for V it only permutes the output rows, so both
// reads are contiguous.  P^T is S^T's fragment transposed (movmatrix).
#pragma once

#include "ssd_kv4.cuh"
#include "ssd_sm100.cuh"

namespace ssd {

constexpr int kKv4Tile = 32;         // tokens per warp tile
constexpr int kKv4Warps = 8;
constexpr int kKv4MaxBlocks = 1024;  // bound of the grid (sizes the workspace)
constexpr int kKv4MaxNT = 4;         // query rows are taken 8 NT <= 32 at a time
constexpr float kKv4Slack = 8.f;     // the reference moves when a logit exceeds it by this (log2)
constexpr float kKv4Lift = 6.f;      // probabilities are carried times 2^6: at most 2^14 in f16

struct Kv4AttnArgs {
  KVView kv;
  const void *q;
  int q_f32, out_f32;
  int h_q, G, R, n_c, n_chunk;
  float scale_log2;       // scale * log2(e) * k_scale
  float v_scale;
  const int32_t *idx;     // draft: token lists [batch][h_kv][k_max]
  const int32_t *cnt;
  int k_max;
  void *out;
  float *lse;
  float *part_o, *part_ml;
  unsigned *counters;
  float *scores;
  int64_t scores_stride;
  const float *lse_in;    // criticality pass
  int n_units;            // batch * h_kv * n_chunk
  unsigned *status;
};

// Position within a group of 8 tokens that row (or column) k of a fragment stands for: K fragments
// read rows k = 0..7, V fragments columns 2c and 2c + 1; with the lowest bit flipped for odd k / 2 the
// tokens read together fall in different halves of a 128-byte line for both.
__device__ __forceinline__ int kv4_sigma(int k) { return (k & 6) | ((k ^ (k >> 1)) & 1); }

template <int D>
struct Kv4Smem {
  static constexpr int kCb = kv4_code_bytes(D), kSb = kv4_scale_bytes(D);
  static constexpr int kHalf = kKv4Tile * (kCb + kSb);  // K or V part of a tile
  static constexpr int kStage = 2 * kHalf;
};

template <int D, int NT, int QS, int NST>
constexpr int kv4_smem_bytes() {
  // ring, query fragments, per-row logit factors and the warps' references and sums, barriers
  return kKv4Warps * NST * Kv4Smem<D>::kStage + NT * 8 * D * 2 * QS + NT * 8 * 4 + 2 * kKv4Warps * NT * 8 * 4 +
         kKv4Warps * NST * 8 + 64;
}

// Tiles of a unit; a unit without tokens has one empty tile, whose rows come out as 0 and -inf.
template <bool LIST>
__device__ __forceinline__ int kv4_tiles(const Kv4AttnArgs &a, int u) {
  int n;
  if (LIST) {
    n = a.cnt[u];
    n = n < 0 ? 0 : (n > a.k_max ? a.k_max : n);
  } else {
    n = a.kv.seq_lens[u / (a.kv.h_kv * a.n_chunk)];
    n = n < 0 ? 0 : (n > a.kv.max_seq_len ? a.kv.max_seq_len : n);
  }
  return n > 0 ? cdiv(n, kKv4Tile) : 1;
}

// Position of this block in the list of all units' tiles: the tiles are dealt out in equal contiguous
// ranges, whatever the lengths.  Returns false when the block has none.
struct Kv4Range {
  int64_t x, x1, per;  // next tile, end, tiles per block
  int u, off;          // unit and tile inside it of x
};
template <bool LIST>
__device__ __forceinline__ bool kv4_range(const Kv4AttnArgs &a, Kv4Range &r, int64_t *s_scan /* [kKv4Warps + 3] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_thread = cdiv(a.n_units, kKv4Warps * 32);
  const int u0 = min(a.n_units, tid * per_thread), u1 = min(a.n_units, u0 + per_thread);
  int64_t sum = 0;
  for (int u = u0; u < u1; ++u) sum += kv4_tiles<LIST>(a, u);
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kKv4Warps; ++w) {
    const int64_t v = s_scan[w];
    if (w < warp) base += v;
    total += v;
  }
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kKv4Warps) per = kKv4Warps;  // a tile for every warp before another block is used
  const int64_t x0 = per * blockIdx.x;
  if (x0 >= total) return false;
  const int64_t excl = base + inc - sum;
  if (x0 >= excl && x0 < excl + sum) {
    int64_t e = excl;
    int u = u0;
    for (;; ++u) {
      const int n = kv4_tiles<LIST>(a, u);
      if (x0 < e + n) break;
      e += n;
    }
    s_scan[kKv4Warps] = u;
    s_scan[kKv4Warps + 1] = x0 - e;
  }
  __syncthreads();
  r.x = x0, r.x1 = min(total, x0 + per), r.per = per;
  r.u = (int)s_scan[kKv4Warps], r.off = (int)s_scan[kKv4Warps + 1];
  return true;
}

// Loads of one warp's tiles into its ring.  Dense tiles come by bulk copies (one per page, or part of a
// large page, and K or V: codes and scales of a page's head are contiguous), counted on an mbarrier;
// list tiles by 16- and 8-byte (d = 64: 4-byte) cp.async, one group per tile.
template <int D, bool LIST, bool K_ONLY>
struct Kv4Loader {
  using S = Kv4Smem<D>;
  const Kv4AttnArgs &a;
  const char *base;        // pool
  const int32_t *table;
  const int32_t *list;
  int g, L, n;             // head, request length, tokens of the unit (list entries, or L)
  int64_t slab;            // bytes of a (page, K|V, head) block
  int cs, log2_cs;         // tokens of a page inside a tile

  __device__ __forceinline__ Kv4Loader(const Kv4AttnArgs &args) : a(args) {
    base = static_cast<const char *>(a.kv.pool);
    slab = (int64_t)a.kv.page_size * (S::kCb + S::kSb);
    cs = LIST ? kKv4Tile : min(a.kv.page_size, kKv4Tile);
    log2_cs = LIST ? 5 : min(a.kv.log2_ps, 5);
  }
  __device__ __forceinline__ void unit(int b, int head, int len, int count, const int32_t *lst) {
    table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
    g = head, L = len, n = count, list = lst;
  }
  __device__ __forceinline__ void load(int tile, uint32_t dst, uint32_t bar, int lane) const {
    const int t0 = tile * kKv4Tile, nv = min(kKv4Tile, n - t0);
    if (!LIST) {
      constexpr int KV = K_ONLY ? 1 : 2;
      const bool sub = a.kv.page_size > kKv4Tile;
      const int chunks = nv > 0 ? (nv + cs - 1) >> log2_cs : 0;
      // Lane -> (page of the tile, K or V), or for a part of a large page (K or V, codes or scales).
      const int which = K_ONLY ? 0 : lane & 1;
      const int j = K_ONLY ? lane : lane >> 1;
      const bool mine = nv > 0 && j < (sub ? 2 : chunks);
      bool ok = false;
      const char *src = nullptr;
      uint32_t to = 0, bytes = 0;
      if (mine) {
        const int32_t p = __ldg(table + (t0 >> a.kv.log2_ps) + (sub ? 0 : j));
        ok = p >= 0 && (int64_t)p < a.kv.num_pages;
        src = base + (((int64_t)p * 2 + which) * a.kv.h_kv + g) * slab;
        to = dst + which * S::kHalf;
        if (sub) {
          const int s0 = t0 & (a.kv.page_size - 1);
          src += j ? (int64_t)a.kv.page_size * S::kCb + s0 * S::kSb : (int64_t)s0 * S::kCb;
          to += j ? kKv4Tile * S::kCb : 0;
          bytes = kKv4Tile * (j ? S::kSb : S::kCb);
        } else {
          bytes = cs * (S::kCb + S::kSb);
          to += j * bytes;
        }
        if (!ok) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
      }
      const unsigned good = __ballot_sync(0xffffffffu, mine && ok), bad = __ballot_sync(0xffffffffu, mine && !ok);
      const uint32_t total = sub ? (good ? (uint32_t)(KV * S::kHalf) : 0u) : __popc(good) * (uint32_t)(cs * (S::kCb + S::kSb));
      if (bad) {  // the rows of a page outside the pool read as zeros
        if (mine && !ok)
          for (uint32_t o = 0; o < bytes; o += 16) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(to + o), "r"(0) : "memory");
        sm100::fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) sm100::mbar_arrive_expect_tx(bar, total);
      __syncwarp();
      if (mine && ok) sm100::bulk_load(to, src, bytes, bar);
    } else {
      // Each lane resolves one list entry; then 16-byte pieces of the rows go out, lane after lane.
      int64_t row = -1;  // byte offset of the entry's (page, K, head) block
      int slot = 0;
      if (lane < nv) {
        const int t = __ldg(list + t0 + lane);
        if (t < 0 || t >= L) {
          atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
        } else {
          const int32_t p = __ldg(table + (t >> a.kv.log2_ps));
          if (p < 0 || (int64_t)p >= a.kv.num_pages) {
            atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
          } else {
            row = ((int64_t)p * 2 * a.kv.h_kv + g) * slab;
            slot = t & (a.kv.page_size - 1);
          }
        }
      }
      const int64_t v_off = a.kv.h_kv * slab;
      constexpr int CPR = S::kCb / 16;  // 16-byte pieces of a row's codes
#pragma unroll
      for (int i = 0; i < CPR; ++i) {
        const int e = i * 32 + lane, tok = e / CPR, c = e % CPR;
        const int64_t rw = __shfl_sync(0xffffffffu, row, tok);
        const int sl = __shfl_sync(0xffffffffu, slot, tok);
        if (tok < nv) {
          const char *src = base + (rw >= 0 ? rw + sl * S::kCb + c * 16 : 0);
          cp_async16(dst + tok * S::kCb + c * 16, src, rw >= 0 ? 16 : 0);
          cp_async16(dst + S::kHalf + tok * S::kCb + c * 16, src + (rw >= 0 ? v_off : 0), rw >= 0 ? 16 : 0);
        }
      }
      if (lane < nv) {
        const char *src = base + (row >= 0 ? row + (int64_t)a.kv.page_size * S::kCb + slot * S::kSb : 0);
        const uint32_t to = dst + kKv4Tile * S::kCb + lane * S::kSb;
        const int nb = row >= 0 ? S::kSb : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(to), "l"(src), "n"(S::kSb), "r"(nb) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(to + S::kHalf), "l"(src + (row >= 0 ? v_off : 0)), "n"(S::kSb), "r"(nb)
                     : "memory");
      }
    }
  }
};

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t &x, uint32_t &y) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// S^T of one half tile (16 tokens): c[nt] holds rows (tokens) sigma(r), 8 + sigma(r), columns (query rows)
// 8 nt + 2c, +1 for lane 4r + c.  `codes` / `scales` point at the half's first tokens; its second eight
// tokens lie code_step / scale_step bytes on.
template <int D, int NT, int QS>
__device__ __forceinline__ void kv4_qk(float (&c)[NT][4], uint32_t codes, uint32_t scales, int code_step, int scale_step,
                                       uint32_t qfrag, int lane) {
  using S = Kv4Smem<D>;
  const int r = lane >> 2, col = lane & 3, tok = kv4_sigma(r);
  constexpr int W = D / 32;  // words of a lane's share of a row
  uint32_t lo[W], hi[W];
  const uint32_t ka = codes + tok * S::kCb + col * (S::kCb / 4);
  if (D == 128) {
    lds128(ka, *reinterpret_cast<uint32_t(*)[4]>(&lo));
    lds128(ka + code_step, *reinterpret_cast<uint32_t(*)[4]>(&hi));
  } else {
    lds64(ka, lo[0], lo[1]);
    lds64(ka + code_step, hi[0], hi[1]);
  }
  uint32_t sl, sh;  // scale of the lane's groups as f16: low half first group
  if (D == 128) {
    sl = e4m3x2_to_f16x2(lds16(scales + tok * S::kSb + col * 2));
    sh = e4m3x2_to_f16x2(lds16(scales + scale_step + tok * S::kSb + col * 2));
  } else {
    sl = e4m3x2_to_f16x2(lds8(scales + tok * S::kSb + col) * 0x101u);
    sh = e4m3x2_to_f16x2(lds8(scales + scale_step + tok * S::kSb + col) * 0x101u);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 4; ++k) c[nt][k] = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint32_t fl[4], fh[4];
    e2m1_to_f16x2(lo[w], fl);
    e2m1_to_f16x2(hi[w], fh);
    const uint32_t pl = D == 128 ? __byte_perm(sl, 0, w < W / 2 ? 0x1010 : 0x3232) : sl;
    const uint32_t ph = D == 128 ? __byte_perm(sh, 0, w < W / 2 ? 0x1010 : 0x3232) : sh;
#pragma unroll
    for (int k = 0; k < 4; ++k) fl[k] = mul_f16x2(fl[k], pl), fh[k] = mul_f16x2(fh[k], ph);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int j = 2 * w + s;
#pragma unroll
      for (int qs = 0; qs < QS; ++qs)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b0, b1;
          lds64(qfrag + (((qs * NT + nt) * (D / 16) + j) * 32 + lane) * 8, b0, b1);
          mma_f16(c[nt], fl[2 * s], fh[2 * s], fl[2 * s + 1], fh[2 * s + 1], b0, b1);
        }
    }
  }
}

// Query rows [r0, r0 + rows) of (request b, head g) as B fragments in shared memory, and per row the
// factor that turns a product into a log2-domain logit.  A row is scaled by a power of two so that its
// largest value lies in [2^13, 2^14): f16 then holds bf16 values exactly down to 2^-28 of the row's
// largest, and fp32 values as the sum of two f16 (QS = 2).
template <int D, int NT, int QS>
__device__ __forceinline__ void kv4_stage_q(const Kv4AttnArgs &a, int b, int g, int r0, int rows, char *qf, float *s_sl) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int V = D / 32;  // elements per lane
  for (int r = warp; r < NT * 8; r += kKv4Warps) {
    float x[V];
    float mx = 0.f;
    if (r < rows) {
      const int rr = r0 + r, i = rr / a.G, h = g * a.G + rr % a.G;
      const int64_t off = (((int64_t)b * a.n_c + i) * a.h_q + h) * D + lane * V;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[k] = QS == 2 ? __ldg(static_cast<const float *>(a.q) + off + k)
                       : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[off + k]);
        mx = fmaxf(mx, fabsf(x[k]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = 0.f;
    }
    mx = warp_max(mx);
    const int e = (int)(__float_as_uint(mx) >> 23) - 127;  // floor(log2 mx); 128 for inf
    const int up = (mx == 0.f || e == 128) ? 0 : min(13 - e, 126);
    const float f = __uint_as_float((uint32_t)(127 + up) << 23);
    if (lane == 0) s_sl[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
    // element d of row 8 nt + rr sits in step j = (d % (D/4)) / 4 of lane 4 rr + d / (D/4)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int d = lane * V + k, col = d / (D / 4), j = (d % (D / 4)) / 4, pos = d & 3;
      const float v = x[k] * f;
      const __half h = __float2half_rn(v);
      const int at = (((r >> 3) * (D / 16) + j) * 32 + (r & 7) * 4 + col) * 4 + pos;
      reinterpret_cast<__half *>(qf)[at] = h;
      if (QS == 2) reinterpret_cast<__half *>(qf)[NT * (D / 16) * 32 * 4 + at] = __float2half_rn(v - __half2float(h));
    }
  }
}

__device__ __forceinline__ void kv4_write4(const Kv4AttnArgs &a, int64_t elem, const float4 &v) {
  if (a.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + elem) = v;
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + elem) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// PS = 2 carries a probability as the sum of two f16 (22 bits) for fp32 outputs; PS = 1 rounds it to f16
// (2^-12 relative) for bf16 outputs, whose own rounding is 2^-9.
template <int D, int NT, int QS, int PS, int NST, int BPS, bool LIST>
__global__ void __launch_bounds__(kKv4Warps * 32, BPS) kv4_attn_kernel(Kv4AttnArgs a) {
  using S = Kv4Smem<D>;
  constexpr int MT = D / 16;
  constexpr int ROWS = NT * 8;
  extern __shared__ __align__(128) char smem[];
  char *ring = smem;
  char *qf = ring + kKv4Warps * NST * S::kStage;
  float *s_sl = reinterpret_cast<float *>(qf + ROWS * D * 2 * QS);
  float *s_m = s_sl + ROWS, *s_l = s_m + kKv4Warps * ROWS;
  const uint32_t bars = smem_u32(s_l + kKv4Warps * ROWS);
  __shared__ int64_t s_scan[kKv4Warps + 3];
  __shared__ int s_abort, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, col = lane & 3;
  if (tid == 0) s_abort = 0;
  if (tid < kKv4Warps * NST) sm100::mbar_init(bars + tid * 8, 1);
  sm100::mbar_init_fence();
  __syncthreads();
  pdl_wait();
  Kv4Range rg;
  if (!kv4_range<LIST>(a, rg, s_scan)) return;
  if (blockIdx.x == 0) {  // lengths out of range are clamped; say so once
    for (int b = tid; b < a.kv.batch; b += kKv4Warps * 32) effective_len(a.kv, b, LIST ? 0 : a.n_c, a.status);
    if (LIST)
      for (int u = tid; u < a.n_units; u += kKv4Warps * 32)
        if (a.cnt[u] < 0 || a.cnt[u] > a.k_max) atomicOr(a.status, (unsigned)SSD_FAULT_KMAX);
  }
  const uint32_t my_ring = smem_u32(ring) + warp * NST * S::kStage;
  const uint32_t my_bars = bars + warp * NST * 8;
  const uint32_t qfrag = smem_u32(qf);
  Kv4Loader<D, LIST, false> ld(a);
  // Offsets of the four groups of eight tokens of a tile (page blocks carry their scales inside).
  int coff[4], soff[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (8 * k) >> ld.log2_cs;
    coff[k] = 8 * k * S::kCb + c * ld.cs * S::kSb;
    soff[k] = 8 * k * S::kSb + (c + 1) * ld.cs * S::kCb;
  }
  int issued = 0, used = 0;  // tiles of this warp so far: ring position and barrier phase

  while (rg.x < rg.x1) {
    const int u = rg.u, b = u / (a.kv.h_kv * a.n_chunk), g = (u / a.n_chunk) % a.kv.h_kv, r0 = (u % a.n_chunk) * ROWS;
    const int rows = min(ROWS, a.R - r0);
    const int n_tiles = kv4_tiles<LIST>(a, u);
    const int seg0 = rg.off, seg1 = seg0 + (int)min((int64_t)(n_tiles - rg.off), rg.x1 - rg.x);
    const int L = min(max(a.kv.seq_lens[b], 0), a.kv.max_seq_len);
    const int count = LIST ? min(max(a.cnt[u], 0), a.k_max) : L;
    ld.unit(b, g, L, count, LIST ? a.idx + (int64_t)u * a.k_max : nullptr);
    // First tiles on their way, then the queries.
    int next = seg0 + warp;
#pragma unroll
    for (int s = 0; s < NST; ++s) {
      if (next < seg1) {
        const int st = issued % NST;
        ld.load(next, my_ring + st * S::kStage, my_bars + st * 8, lane);
        ++issued;
        next += kKv4Warps;
      }
      if (LIST) cp_async_commit();
    }
    kv4_stage_q<D, NT, QS>(a, b, g, r0, rows, qf, s_sl);
    __syncthreads();
    float sl[NT][2], m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) sl[nt][k] = s_sl[8 * nt + 2 * col + k], m[nt][k] = -1e30f, l[nt][k] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;

    for (int tile = seg0 + warp; tile < seg1; tile += kKv4Warps) {
      const int st = used % NST;
      if (LIST) {
        cp_async_wait<NST - 1>();
        __syncwarp();
      } else if (!sm100::mbar_wait(my_bars + st * 8, (used / NST) & 1, &s_abort)) {
        atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
      }
      const uint32_t kt = my_ring + st * S::kStage, vt = kt + S::kHalf;
      const int t0 = tile * kKv4Tile;
      float c[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        kv4_qk<D, NT, QS>(c[h], kt + coff[2 * h], kt + soff[2 * h], coff[2 * h + 1] - coff[2 * h],
                          soff[2 * h + 1] - soff[2 * h], qfrag, lane);
      const bool edge = LIST ? t0 + kKv4Tile > count : t0 + kKv4Tile > L - a.n_c + 1;
      float top = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x0 = c[0][nt][k] * sl[nt][k & 1], x1 = c[1][nt][k] * sl[nt][k & 1];
          if (edge) {
            const int lim = LIST ? count : min(L, L - a.n_c + 1 + (r0 + 8 * nt + 2 * col + (k & 1)) / a.G);
            const int t = t0 + kv4_sigma(r) + (k >> 1) * 8;
            if (t >= lim) x0 = -INFINITY;
            if (t + 16 >= lim) x1 = -INFINITY;
          }
          c[0][nt][k] = x0, c[1][nt][k] = x1;
          top = fmaxf(top, fmaxf(x0, x1) - m[nt][k & 1]);
        }
      if (__any_sync(0xffffffffu, top > kKv4Slack)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = fmaxf(fmaxf(c[0][nt][k], c[0][nt][k + 2]), fmaxf(c[1][nt][k], c[1][nt][k + 2]));
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = fmaxf(mx, m[nt][k]);
            const float f = fast_exp2(m[nt][k] - mx);
            m[nt][k] = mx;
            l[nt][k] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][nt][k] *= f, o[i][nt][k + 2] *= f;
          }
      }
      uint32_t p[2][NT][2], pl[2][NT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = fast_exp2(c[h][nt][k] - (m[nt][k & 1] - kKv4Lift));
            l[nt][k & 1] += e[k];
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 hi = __floats2half2_rn(e[2 * k], e[2 * k + 1]);
            p[h][nt][k] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&hi));
            if (PS == 2) {
              const float2 back = __half22float2(hi);
              pl[h][nt][k] = movmatrix_trans(pack_half(e[2 * k] - back.x, e[2 * k + 1] - back.y));
            }
          }
        }
      // O^T += V^T P^T, 16 tokens a step.  A lane reads its d / 8 elements of four tokens and pairs the codes
      // of two tokens in a byte, so that each conversion gives a fragment register.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int W = D / 64;
        uint32_t w[4][W], sc[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t cb = vt + coff[2 * h + k] + r * (4 * W), sb = vt + soff[2 * h + k] + (D == 128 ? r : r >> 1);
          const int ta = kv4_sigma(2 * col), tb = ta ^ 1;
          if (W == 2) {
            lds64(cb + ta * S::kCb, w[2 * k][0], w[2 * k][W - 1]);
            lds64(cb + tb * S::kCb, w[2 * k + 1][0], w[2 * k + 1][W - 1]);
          } else {
            w[2 * k][0] = lds32(cb + ta * S::kCb);
            w[2 * k + 1][0] = lds32(cb + tb * S::kCb);
          }
          uint32_t sa = lds8(sb + ta * S::kSb), sbb = lds8(sb + tb * S::kSb);
          if (edge) {  // tokens past the end: whatever their slots hold counts as 0
            const int t = t0 + 16 * h + 8 * k;
            if (t + ta >= count) sa = 0;
            if (t + tb >= count) sbb = 0;
          }
          sc[k] = e4m3x2_to_f16x2(sa | (sbb << 8));
        }
#pragma unroll
        for (int x = 0; x < W; ++x) {
          uint32_t f[4][4];
          e2m1_to_f16x2((w[0][x] & 0x0f0f0f0fu) | ((w[1][x] << 4) & 0xf0f0f0f0u), f[0]);
          e2m1_to_f16x2(((w[0][x] >> 4) & 0x0f0f0f0fu) | (w[1][x] & 0xf0f0f0f0u), f[1]);
          e2m1_to_f16x2((w[2][x] & 0x0f0f0f0fu) | ((w[3][x] << 4) & 0xf0f0f0f0u), f[2]);
          e2m1_to_f16x2(((w[2][x] >> 4) & 0x0f0f0f0fu) | (w[3][x] & 0xf0f0f0f0u), f[3]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t a0 = mul_f16x2(f[0][y], sc[0]), a1 = mul_f16x2(f[1][y], sc[0]), a2 = mul_f16x2(f[2][y], sc[1]),
                           a3 = mul_f16x2(f[3][y], sc[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(o[4 * x + y][nt], a0, a1, a2, a3, p[h][nt][0], p[h][nt][1]);
              if (PS == 2) mma_f16(o[4 * x + y][nt], a0, a1, a2, a3, pl[h][nt][0], pl[h][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      ++used;
      if (next < seg1) {
        const int ns = issued % NST;
        ld.load(next, my_ring + ns * S::kStage, my_bars + ns * 8, lane);
        ++issued;
        next += kKv4Warps;
      }
      if (LIST) cp_async_commit();
    }

    // Sums of the lanes of a query row, then of the warps: the ring is free now and takes their O.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], s);
        if (r == 0) s_m[warp * ROWS + 8 * nt + 2 * col + k] = m[nt][k], s_l[warp * ROWS + 8 * nt + 2 * col + k] = l[nt][k];
      }
    __syncthreads();
    const int nw = min(kKv4Warps, seg1 - seg0);
    float *acc = reinterpret_cast<float *>(ring);  // [warp][row][d], 16-byte pieces of a row permuted
    if (warp < nw) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int q = 8 * nt + 2 * col + k;
          float M = -1e30f;
          for (int w = 0; w < nw; ++w) M = fmaxf(M, s_m[w * ROWS + q]);
          const float f = fast_exp2(m[nt][k] - M);
          float *dst = acc + (int64_t)(warp * ROWS + q) * D;
#pragma unroll
          for (int i = 0; i < MT; i += 2) {
            const int piece = r * (MT / 2) + i / 2;  // d = 2 MT r + 2 i ..
            reinterpret_cast<float4 *>(dst)[piece ^ (r >> 1) ^ col] =
                make_float4(o[i][nt][k] * f, o[i][nt][k + 2] * f, o[i + 1][nt][k] * f, o[i + 1][nt][k + 2] * f);
          }
        }
    }
    __syncthreads();
    const int64_t ua = rg.x - rg.off;  // the unit's tiles are ua .. ua + n_tiles - 1 of all
    const int blk0 = (int)(ua / rg.per), blk1 = (int)((ua + n_tiles - 1) / rg.per);
    const bool whole = blk0 == blk1;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (rg.x == rg.per * blockIdx.x ? 0 : 1);
    for (int e = tid; e < rows * (D / 4); e += kKv4Warps * 32) {
      const int q = e / (D / 4), piece = e % (D / 4), rr = piece / (MT / 2);
      float M = -1e30f, Z = 0.f;
      for (int w = 0; w < nw; ++w) M = fmaxf(M, s_m[w * ROWS + q]);
      for (int w = 0; w < nw; ++w) Z += s_l[w * ROWS + q] * fast_exp2(s_m[w * ROWS + q] - M);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < nw; ++w) {
        const float4 x = reinterpret_cast<const float4 *>(acc + (int64_t)(w * ROWS + q) * D)[piece ^ (rr >> 1) ^ ((q >> 1) & 3)];
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      if (whole) {
        const int gr = r0 + q;
        const int64_t row = ((int64_t)b * a.n_c + gr / a.G) * a.h_q + g * a.G + gr % a.G;
        const float f = Z == 0.f ? 0.f : a.v_scale / Z;
        kv4_write4(a, row * D + piece * 4, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        if (piece == 0 && a.lse) a.lse[row] = Z == 0.f ? -INFINITY : (M - kKv4Lift + __log2f(Z)) * kLn2;
      } else {
        __stcg(reinterpret_cast<float4 *>(a.part_o + (slot * ROWS + q) * D) + piece, v);
        if (piece == 0) __stcg(reinterpret_cast<float2 *>(a.part_ml) + slot * ROWS + q, make_float2(M, Z));
      }
    }
    if (!whole) {
      // The last block of the unit to arrive joins the partial results, in the blocks' order.
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned n = (unsigned)(blk1 - blk0 + 1);
        const unsigned old = atomicAdd(a.counters + blk0, 1u);
        s_last = old == n - 1;
        if (s_last) a.counters[blk0] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int n = blk1 - blk0 + 1;
        // Only the first block can hold the unit's start behind another unit's tiles.
        const int64_t slot0 = (int64_t)blk0 * 2 + (ua == rg.per * blk0 ? 0 : 1);
        for (int e = tid; e < rows * (D / 4); e += kKv4Warps * 32) {
          const int q = e / (D / 4), piece = e % (D / 4);
          const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + q;
          float M = -1e30f;
          for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(ml + (k ? (int64_t)(blk0 + k) * 2 : slot0) * ROWS).x);
          float Z = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < n; ++k) {
            const int64_t sk = (k ? (int64_t)(blk0 + k) * 2 : slot0) * ROWS;
            const float2 w = __ldcg(ml + sk);
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.part_o + (sk + q) * D) + piece);
            const float f = fast_exp2(w.x - M);
            Z += w.y * f;
            v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
          }
          const int gr = r0 + q;
          const int64_t row = ((int64_t)b * a.n_c + gr / a.G) * a.h_q + g * a.G + gr % a.G;
          const float f = Z == 0.f ? 0.f : a.v_scale / Z;
          kv4_write4(a, row * D + piece * 4, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
          if (piece == 0 && a.lse) a.lse[row] = Z == 0.f ? -INFINITY : (M - kKv4Lift + __log2f(Z)) * kLn2;
        }
      }
    }
    if (!LIST) sm100::fence_proxy_async_smem();  // the ring goes back to the bulk copies
    __syncthreads();
    rg.x += seg1 - seg0;
    rg.u = u + 1;
    rg.off = 0;
  }
}

// Criticality: a second pass over K alone recomputes the logits and sums exp(x - lse) over the rows.
// (Keeping them from the first pass would cost 2 R bytes per token each way, more than K's 72 for R > 18,
// and a rounding to f16.)
template <int D, int NT, int QS, int NST, int BPS>
__global__ void __launch_bounds__(kKv4Warps * 32, BPS) kv4_crit_kernel(Kv4AttnArgs a) {
  using S = Kv4Smem<D>;
  constexpr int ROWS = NT * 8;
  extern __shared__ __align__(128) char smem[];
  char *ring = smem;
  char *qf = ring + kKv4Warps * NST * S::kHalf;
  float *s_sl = reinterpret_cast<float *>(qf + 2 * ROWS * D * 2 * QS);  // two chunks of rows at most
  float *s_lse = s_sl + 2 * ROWS;
  const uint32_t bars = smem_u32(s_lse + 2 * ROWS);
  __shared__ int64_t s_scan[kKv4Warps + 3];
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, col = lane & 3;
  if (tid == 0) s_abort = 0;
  if (tid < kKv4Warps * NST) sm100::mbar_init(bars + tid * 8, 1);
  sm100::mbar_init_fence();
  __syncthreads();
  pdl_wait();
  Kv4Range rg;
  if (!kv4_range<false>(a, rg, s_scan)) return;
  const uint32_t my_ring = smem_u32(ring) + warp * NST * S::kHalf;
  const uint32_t my_bars = bars + warp * NST * 8;
  Kv4Loader<D, false, true> ld(a);
  int coff[4], soff[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (8 * k) >> ld.log2_cs;
    coff[k] = 8 * k * S::kCb + c * ld.cs * S::kSb;
    soff[k] = 8 * k * S::kSb + (c + 1) * ld.cs * S::kCb;
  }
  const int n_chunk = cdiv(a.R, ROWS);
  int issued = 0, used = 0;
  while (rg.x < rg.x1) {
    const int u = rg.u, b = u / a.kv.h_kv, g = u % a.kv.h_kv;
    const int n_tiles = kv4_tiles<false>(a, u);
    const int seg0 = rg.off, seg1 = seg0 + (int)min((int64_t)(n_tiles - rg.off), rg.x1 - rg.x);
    const int L = min(max(a.kv.seq_lens[b], 0), a.kv.max_seq_len);
    ld.unit(b, g, L, L, nullptr);
    int next = seg0 + warp;
#pragma unroll
    for (int s = 0; s < NST; ++s)
      if (next < seg1) {
        const int st = issued % NST;
        ld.load(next, my_ring + st * S::kHalf, my_bars + st * 8, lane);
        ++issued;
        next += kKv4Warps;
      }
    for (int ch = 0; ch < n_chunk; ++ch)
      kv4_stage_q<D, NT, QS>(a, b, g, ch * ROWS, min(ROWS, a.R - ch * ROWS), qf + ch * ROWS * D * 2 * QS, s_sl + ch * ROWS);
    for (int q = tid; q < n_chunk * ROWS; q += kKv4Warps * 32) {
      float v = INFINITY;  // rows that see nothing, and the padding: exp(x - inf) = 0
      if (q < a.R) {
        v = a.lse_in[((int64_t)b * a.n_c + q / a.G) * a.h_q + g * a.G + q % a.G];
        v = v == -INFINITY ? INFINITY : v * kLog2e;
      }
      s_lse[q] = v;
    }
    __syncthreads();
    for (int tile = seg0 + warp; tile < seg1; tile += kKv4Warps) {
      const int st = used % NST;
      if (!sm100::mbar_wait(my_bars + st * 8, (used / NST) & 1, &s_abort)) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
      const uint32_t kt = my_ring + st * S::kHalf;
      const int t0 = tile * kKv4Tile;
      const bool edge = t0 + kKv4Tile > L - a.n_c + 1;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int ch = 0; ch < n_chunk; ++ch) {
        const uint32_t qfrag = smem_u32(qf) + ch * ROWS * D * 2 * QS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float c[NT][4];
          kv4_qk<D, NT, QS>(c, kt + coff[2 * h], kt + soff[2 * h], coff[2 * h + 1] - coff[2 * h], soff[2 * h + 1] - soff[2 * h],
                            qfrag, lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int q = ch * ROWS + 8 * nt + 2 * col + (k & 1);
              float e = fast_exp2(fmaf(c[nt][k], s_sl[q], -s_lse[q]));
              if (edge && t0 + 16 * h + (k >> 1) * 8 + kv4_sigma(r) >= min(L, L - a.n_c + 1 + q / a.G)) e = 0.f;
              sum[2 * h + (k >> 1)] += q < a.R ? e : 0.f;
            }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
      }
      // lane 4r + col stores the token of row r in eight-token group col
      const float v = col == 0 ? sum[0] : col == 1 ? sum[1] : col == 2 ? sum[2] : sum[3];
      const int t = t0 + 8 * col + kv4_sigma(r);
      if (t < L) a.scores[(int64_t)u * a.scores_stride + t] = v;
      __syncwarp();
      ++used;
      if (next < seg1) {
        const int ns = issued % NST;
        ld.load(next, my_ring + ns * S::kHalf, my_bars + ns * 8, lane);
        ++issued;
        next += kKv4Warps;
      }
    }
    __syncthreads();
    rg.x += seg1 - seg0;
    rg.u = u + 1;
    rg.off = 0;
  }
}

}  // namespace ssd

// ---- launches -------------------------------------------------------------------------------
#include "ssd_host.h"

namespace ssd {

// Blocks per SM and ring depth by the rows of a pass, from registers (the O accumulators take 32 NT a
// lane) and shared memory (the ring also holds the warps' O at a segment's end: NT * 32 KB at d = 128).
template <int NT>
struct Kv4Tune {
  static constexpr int kBlocks = NT == 1 ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 3 : 4;
};

template <int D, int NT, int QS, int PS, bool LIST>
int kv4_launch_attn(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr int NST = Kv4Tune<NT>::kStages, BPS = Kv4Tune<NT>::kBlocks;
  static_assert(kKv4Warps * NST * Kv4Smem<D>::kStage >= kKv4Warps * NT * 8 * D * 4, "the ring holds the warps' O");
  constexpr int smem = kv4_smem_bytes<D, NT, QS, NST>();
  constexpr auto kernel = kv4_attn_kernel<D, NT, QS, PS, NST, BPS, LIST>;
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  return launch(kernel, dim3(grid), dim3(kKv4Warps * 32), smem, st, LIST ? "kv4_attn_kernel (draft)" : "kv4_attn_kernel", a);
}

template <int D, int NT, bool LIST>
int kv4_attn_types(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  if (a.q_f32) return kv4_launch_attn<D, NT, 2, 2, LIST>(a, grid, st);
  if (a.out_f32) return kv4_launch_attn<D, NT, 1, 2, LIST>(a, grid, st);
  return kv4_launch_attn<D, NT, 1, 1, LIST>(a, grid, st);
}

template <int D, int NT, int QS>
int kv4_launch_crit(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr int NST = 4, BPS = 2;
  constexpr int smem = kKv4Warps * NST * Kv4Smem<D>::kHalf + 2 * NT * 8 * D * 2 * QS + 4 * NT * 8 * 4 + kKv4Warps * NST * 8 + 64;
  constexpr auto kernel = kv4_crit_kernel<D, NT, QS, NST, BPS>;
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  return launch(kernel, dim3(grid), dim3(kKv4Warps * 32), smem, st, "kv4_crit_kernel", a);
}

}  // namespace ssd
