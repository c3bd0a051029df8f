// ssd_kv4_attn.cuh -- attention over a 4-bit paged cache: one kernel for the dense pass of n_cand
// candidates (verify; n_cand = 1 is plain decoding) and for the draft over a list of selected tokens,
// and one for the tokens' criticality.
//
// Mathematics, per (request, KV head) unit with R = G * n_cand query rows, x_rt = scale * q_r . k_t:
//   out_r = sum_t exp(x_rt) v_t / sum_t exp(x_rt) over the tokens row r sees, lse_r = log sum_t exp(x_rt),
//   crit_t = sum_r exp(x_rt - lse_r)   (SparseSpec §4.1: criticality summed over the group's heads and
//   the verify positions).
// One pass over K and V keeps a running reference m_r (a past maximum, in log2 units), the sum l_r of exp2(x - m) and
// the weighted sum of V, all in fp32; the criticality takes exp2(x - m_r) / l_r.
//
// Bound: 9 bits per (K, V) element pair stored, 144 bytes per token of a head at d = 128, so HBM bounds
// small R; the f16 tensor-core rate of mma.sync (1024 multiply-adds per clock and SM) bounds R > 20.
//
// Layout of the work.  A warp takes tiles of 32 tokens and computes, on the tensor cores,
//   S^T [32 tokens x 8 NT rows] = K Q^T   and   O^T [d x 8 NT rows] += V^T P^T,
// so that the cache is the A operand of both products and the few query rows the narrow N side (M = 16
// rows of queries would be mostly padding).  Codes go from shared memory to A fragments in registers: pairs
// of codes are converted to f16 and multiplied by their scale (exact, see ssd_kv4.cuh).  Which d a lane's
// fragment column stands for is free for K as long as Q is laid out alike, and for V it only permutes the
// output rows, so a lane reads consecutive bytes of both.  P^T is S^T's fragment transposed (movmatrix).
//
// What bounds it: its steady loop takes 185 clocks a tile and SM, what HBM takes to deliver one (195), at about
// 600 instructions, 256 of them the conversions; the rest is the start (5 us), merges and joins where
// blocks change units (4 us each), and blocks ending apart.  8 heads of d = 128, 4 rows each, bf16 outputs: 32 requests of
// 2048 to 8192 tokens 48 us (59 % of the measured HBM rate), 128 such requests 154 us (73 %), 8 of 65536 tokens
// 114 us (78 %).  With more rows the O accumulators leave room for few warps, and the kernel of ssd_kv4_tc.cuh
// takes over at d = 128.
#pragma once

#include "ssd_kv4.cuh"

namespace ssd {

constexpr int kKv4Tile = 32;         // tokens per warp tile
constexpr int kKv4MaxBlocks = 1024;  // bound of the grid (sizes the workspace)
constexpr int kKv4MaxNT = 4;         // query rows are taken 8 NT <= 32 at a time
// A row's reference m is the largest logit (log2) seen when it last moved, less the lift; it moves again when a logit
// exceeds it by the slack.  exp2(x - m), at least 2^lift where the largest is, goes to the tensor cores in f16, which
// holds 11 bits down to 2^-14 and steps of 2^-24 below.
//   bf16 outputs (one f16): 2^-12 relative down to 2^-20 of the largest, 2^-31 of it absolute below.
//   fp32 outputs (two f16): 22 bits down to 2^-13 of the largest, 2^-35 of it absolute below: n tokens that far down may
//     take n 2^-35 off a row's weight; fp32 sums of n / 128 terms take as much.  (With a lift of 6, 131072 tokens of
//     2^-31 each were lost altogether: 5.6e-5 of the outputs.)  The slack stays below f16's 2^16.  Each reference that
//     moves costs a pass over O: lifts of 6, 9, 10, 11, 13 took 99.5, 101.5, 101.5, 103.5, 124 us for 32 requests of
//     2048 to 8192 tokens, 8 heads, d = 64, 32 rows, and 99.5, 99.5, 99.5, 100.5, 107 for d = 128, 20 rows (L2 flushed).
constexpr float kv4_lift(int ps) { return ps == 2 ? 10.f : 6.f; }
constexpr float kv4_slack(int ps) { return ps == 2 ? 15.75f : 14.f; }

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
  float2 *fin;            // per query row: its reference and 1 / sum, for the criticality pass; or NULL
  int n_units;            // batch * h_kv * n_chunk
  int join_blocks;        // tcgen05: blocks whose parts kv4_join_kernel joins, or 0: the last block of a unit does
  unsigned *status;
};

// Position within a group of 8 tokens that row (or column) k of a fragment stands for: rows 2i and 2i + 1 of
// K (a line of shared memory holds two) stay together, columns 0, 2, 4, 6 of V differ mod 4, so that both
// reads touch every bank once.
__device__ __forceinline__ int kv4_sigma(int k) { return k ^ (((k >> 1) ^ (k >> 2)) & 1); }

// A tile in shared memory: codes of K and of V, scales of K and of V.
template <int D>
struct Kv4Smem {
  static constexpr int kCb = kv4_code_bytes(D), kSb = kv4_scale_bytes(D);
  static constexpr int kV = kKv4Tile * kCb, kKs = 2 * kV, kVs = kKs + kKv4Tile * kSb;  // offsets
  static constexpr int kStage = kVs + kKv4Tile * kSb;
  // Criticality pass: K alone.
  static constexpr int kCritScales = kV, kCritStage = kV + kKv4Tile * kSb;
  // Byte of 16-byte piece c of token t's codes: at d = 128 a 128-byte line holds two tokens, and odd lines have
  // their pieces permuted, against bank conflicts.
  static __device__ __forceinline__ int piece(int t, int c) {
    return D == 128 ? (t >> 1) * 128 + ((((t & 1) * 4 + c) ^ ((t >> 1 & 1) * 2)) << 4) : t * 32 + c * 16;
  }
};

// Whether the warps' O have a place of their own at a segment's end, so that the next segment's tiles are on their
// way meanwhile; otherwise they go to the ring.
constexpr bool kv4_ahead(int nt) { return nt == 1; }
constexpr bool kv4_own_o(int nt, int ps) { return kv4_ahead(nt) || ps == 2; }

// For fp32 outputs a warp's O leaves the tensor cores' accumulators every so many of its tiles, to be added up in shared
// memory: mma.sync adds with truncation, one-sided.  Parts of 65536 tokens, relative 2-norm off the 64-bit result
// (normal V | positive V): 2.0e-5 | 4.4e-5 without, 1.3e-6 | 1.5e-6 every 16 tiles, 0.8e-6 | 0.7e-6 every 8; a plain
// fp32 computation 1.0e-6 | 0.2e-6.  32 requests of 2048 to 8192 tokens, 8 heads, d = 128 with 4 rows, d = 64 with 20 and
// 32 (L2 flushed): 58.5, 81, 99.5 us without, 60.5, 81, 99.5 every 16, 59.5, 81, 101.5 every 8.
constexpr int kKv4Flush = 16;

template <int D, int NT, int QS, int PS, int NW, int NST>
constexpr int kv4_smem_bytes() {
  // ring, the warps' O, query fragments, per-row logit factors, the warps' references and sums
  return NW * NST * Kv4Smem<D>::kStage + (kv4_own_o(NT, PS) ? NW * NT * 8 * D * 4 : 0) + NT * 8 * D * 2 * QS + NT * 8 * 4 +
         2 * NW * NT * 8 * 4;
}

// Tiles of a unit; a unit without tokens has one empty tile, whose rows come out as 0 and -inf.
template <bool LIST, int TILE = kKv4Tile>
__device__ __forceinline__ int kv4_tiles(const Kv4AttnArgs &a, int u) {
  int n;
  if (LIST) {
    n = a.cnt[u];
    n = n < 0 ? 0 : (n > a.k_max ? a.k_max : n);
  } else {
    n = a.kv.seq_lens[u / (a.kv.h_kv * a.n_chunk)];
    n = n < 0 ? 0 : (n > a.kv.max_seq_len ? a.kv.max_seq_len : n);
  }
  return n > 0 ? cdiv(n, TILE) : 1;
}

// Dealing out the units' tiles to blocks.  All units stand in one line, each with a lead before its own tiles:
// about what starting, merging and writing a unit costs, in tiles.  Blocks take equal contiguous stretches of the
// line.  A boundary inside a lead, or at most kKv4Snap tiles from a unit's start or end, moves there: a unit cut in
// two costs a join as well.  (Without leads, a block whose stretch held many short units ran twice as long as the
// others: 128 requests of 1 to 2048 tokens, 8 heads of 128, one query row a head: 143 us against 85 with them; the
// same with 5 candidates: 292 against 148.)
template <int TILE>
constexpr int kKv4Lead = TILE == kKv4Tile ? 16 : 6;  // 4 us of a block's time
template <int TILE>
constexpr int kKv4Snap = TILE == kKv4Tile ? 4 : 0;  // (20: decode 48.8 us against 47.5)
struct Kv4Range {
  int64_t x, x1, per;  // place of the unit u in the line, the block's end, a stretch's length
  int u, off;          // next unit, and its first tile of this block
};
// Blocks that hold parts of the unit of n tiles at place x: `first` and `more` blocks after it.  The unit's start
// is stored in the first one's second slot, other parts in their block's first one.
template <int TILE>
struct Kv4Parts {
  int first, more;
  __device__ __forceinline__ Kv4Parts(const Kv4Range &r, int64_t x, int n) {
    constexpr int lead = kKv4Lead<TILE>;
    first = (int)((x + lead + kKv4Snap<TILE>) / r.per);
    more = max(0, (int)((x + lead + n - kKv4Snap<TILE> + r.per - 1) / r.per) - 1 - first);
  }
  __device__ __forceinline__ int64_t slot(int k) const { return k ? (int64_t)(first + k) * 2 : (int64_t)first * 2 + 1; }
};
// Length of a block's stretch of the line.  least: a tile for every warp before another block is used.
__device__ __forceinline__ int64_t kv4_per(int64_t total, int blocks, int least) {
  const int64_t per = (total + blocks - 1) / blocks;
  return per < least ? least : per;
}
// Returns false when the block has no tile.
template <bool LIST, int NW, int TILE = kKv4Tile, int MIN = NW>
__device__ __forceinline__ bool kv4_range(const Kv4AttnArgs &a, Kv4Range &r, int64_t *s_scan /* [NW + 4] */) {
  constexpr int LEAD = kKv4Lead<TILE>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_thread = cdiv(a.n_units, NW * 32);
  const int u0 = min(a.n_units, tid * per_thread), u1 = min(a.n_units, u0 + per_thread);
  int64_t sum = 0;
  for (int u = u0; u < u1; ++u) sum += kv4_tiles<LIST, TILE>(a, u) + LEAD;
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
  for (int w = 0; w < NW; ++w) {
    const int64_t v = s_scan[w];
    if (w < warp) base += v;
    total += v;
  }
  const int64_t per = r.per = kv4_per(total, gridDim.x, MIN);
  const int64_t excl = base + inc - sum;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t y = per * ((int64_t)blockIdx.x + k);
    if (y >= total && tid == 0) s_scan[NW + 2 * k] = total;
    if (y >= excl && y < excl + sum) {
      int64_t e = excl;
      int u = u0, n;
      for (;; ++u) {
        n = kv4_tiles<LIST, TILE>(a, u) + LEAD;
        if (y < e + n) break;
        e += n;
      }
      const bool down = y - e <= LEAD + kKv4Snap<TILE>, up = !down && e + n - y <= kKv4Snap<TILE>;
      s_scan[NW + 2 * k] = down ? e : up ? e + n : y;
      if (k == 0) s_scan[NW + 1] = (int64_t)(u + up) << 32 | (uint32_t)(down || up ? 0 : (int)(y - e) - LEAD);
    }
  }
  __syncthreads();
  r.x = s_scan[NW], r.x1 = s_scan[NW + 2];
  if (r.x >= r.x1) return false;
  r.u = (int)(s_scan[NW + 1] >> 32), r.off = (int)(uint32_t)s_scan[NW + 1];
  if (r.off) r.x -= r.off + LEAD;
  return true;
}
// End of the block's tiles of the unit at r, which has n; and the step to the next unit.
template <int TILE = kKv4Tile>
__device__ __forceinline__ int kv4_range_end(const Kv4Range &r, int n) {
  return (int)min((int64_t)n, r.x1 - r.x - kKv4Lead<TILE>);
}
template <int TILE = kKv4Tile>
__device__ __forceinline__ void kv4_range_next(Kv4Range &r, int n) {
  r.x += n + kKv4Lead<TILE>, r.u += 1, r.off = 0;
}

// Loads of one warp's tiles into its ring, by 16-byte cp.async, one group per tile.  (A page's rows of one head
// are 1152 bytes at page size 16 and d = 128: bulk copies of that size took about 200 clocks each to issue.)
template <int D>
struct Kv4Loader {
  using S = Kv4Smem<D>;
  static constexpr int CPR = S::kCb / 16;  // 16-byte pieces of a row's codes
  const Kv4AttnArgs &a;
  const char *head;     // the head's K block of page 0
  const int32_t *table, *list;
  int L, n;             // request length, tokens of the unit (list entries, or L)
  int log2_cs;          // log2 of the tokens of a page inside a tile
  uint32_t page_bytes;  // of all heads' K and V blocks
  uint32_t v_off;       // from a head's K block to its V block
  uint32_t lane_to;     // this lane's piece of the first rows, in a tile

  __device__ __forceinline__ Kv4Loader(const Kv4AttnArgs &args) : a(args) {
    const int lane = threadIdx.x & 31;
    log2_cs = min(a.kv.log2_ps, 5);
    v_off = (uint32_t)a.kv.h_kv * a.kv.page_size * (S::kCb + S::kSb);
    page_bytes = 2 * v_off;
    lane_to = S::piece(lane / CPR, lane % CPR);
  }
  __device__ __forceinline__ void unit(int b, int g, int len, int count, const int32_t *lst) {
    table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
    head = static_cast<const char *>(a.kv.pool) + (uint32_t)g * a.kv.page_size * (S::kCb + S::kSb);
    L = len, n = count, list = lst;
  }
  __device__ __forceinline__ bool in_pool(int32_t p) const { return p >= 0 && (int64_t)p < a.kv.num_pages; }

  // Dense tiles.  peek(): the id of the tile's page `lane` (0 where the tile has none), fetched a tile ahead of
  // load(), because the latency would otherwise stall the warp between two tiles.  Slots behind the
  // request's end are copied as they are (its last page) or from page 0 (pages that it does not have):
  // nothing uses them.
  __device__ __forceinline__ int32_t peek(int tile, int lane) const {
    const int at = tile * kKv4Tile + (lane << log2_cs);
    return lane < (kKv4Tile >> log2_cs) && at < n ? table[at >> a.kv.log2_ps] : 0;
  }
  // The codes of G consecutive tokens of a page are G * kCb consecutive bytes.
  template <int G, bool K_ONLY>
  __device__ __forceinline__ void codes(int t0, int32_t pid, uint32_t dst, int lane) const {
    constexpr int R = 32 / CPR;  // rows that a warp copies at once
#pragma unroll
    for (int i = 0; i < kKv4Tile / G; ++i) {
      const int32_t p = __shfl_sync(0xffffffffu, pid, (G * i) >> log2_cs);
      const char *src = head + (uint64_t)(uint32_t)p * page_bytes + ((t0 + G * i) & (a.kv.page_size - 1)) * S::kCb + lane * 16;
#pragma unroll
      for (int k = 0; k < G; k += R) {
        if (G < R && lane >= G * CPR) break;
        const uint32_t to = dst + lane_to + (G * i + k) * S::kCb;
        cp_async16(to, src + k * S::kCb, 16);
        if (!K_ONLY) cp_async16(to + S::kV, src + v_off + k * S::kCb, 16);
      }
    }
  }
  template <bool K_ONLY>
  __device__ __forceinline__ void load(int tile, int32_t pid, uint32_t dst, int lane) const {
    constexpr int scales = K_ONLY ? S::kCritScales : S::kKs;
    const int t0 = tile * kKv4Tile;
    const bool ok = in_pool(pid);
    const unsigned bad = __ballot_sync(0xffffffffu, !ok);
    if (!ok) pid = 0;
    if (log2_cs >= 4)
      codes<16, K_ONLY>(t0, pid, dst, lane);
    else
      codes<8, K_ONLY>(t0, pid, dst, lane);
    // Scales: TPC tokens to a piece; the first lanes K's, the next V's.
    constexpr int TPC = 16 / S::kSb, N = kKv4Tile / TPC;
    const int which = lane / N, t = lane % N * TPC;
    const int32_t p = __shfl_sync(0xffffffffu, pid, t >> log2_cs);
    const char *src = head + (uint64_t)(uint32_t)p * page_bytes + which * v_off + (uint32_t)a.kv.page_size * S::kCb +
                      ((t0 + t) & (a.kv.page_size - 1)) * S::kSb;
    if (which < (K_ONLY ? 1 : 2)) cp_async16(dst + scales + lane * 16, src, 16);
    if (bad) {
      // Pages outside the pool: scales of 0 make their rows zeros.
      if (!ok) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
      if (bad >> (lane >> log2_cs) & 1)
        for (int k = 0; k < (K_ONLY ? 1 : 2) * kKv4Tile * S::kSb; k += kKv4Tile * S::kSb)
          for (int j = 0; j < S::kSb; j += 4)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + scales + k + lane * S::kSb + j), "r"(0) : "memory");
      __syncwarp();
    }
  }

  // List tiles: each lane resolves one entry, then pieces of the rows go out.  An entry that is not there reads
  // as zeros.
  __device__ __forceinline__ int32_t peek_list(int tile, int lane) const {
    return tile * kKv4Tile + lane < n ? list[tile * kKv4Tile + lane] : -1;
  }
  __device__ __forceinline__ void load_list(int tile, int32_t token, uint32_t dst, int lane) const {
    const char *row = nullptr, *scales = head;  // the entry's codes and scales in the head's K block
    if (tile * kKv4Tile + lane < n) {
      if (token < 0 || token >= L) {
        atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
      } else {
        const int32_t p = table[token >> a.kv.log2_ps];
        if (in_pool(p)) {
          const int slot = token & (a.kv.page_size - 1);
          row = head + (uint64_t)(uint32_t)p * page_bytes + slot * S::kCb;
          scales = head + (uint64_t)(uint32_t)p * page_bytes + (uint32_t)a.kv.page_size * S::kCb + slot * S::kSb;
        } else {
          atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < CPR; ++i) {
      constexpr int R = 32 / CPR;
      const char *rw =
          reinterpret_cast<const char *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), i * R + lane / CPR));
      const char *src = rw ? rw + lane % CPR * 16 : head;
      const int nb = rw ? 16 : 0;
      const uint32_t to = dst + lane_to + i * R * S::kCb;
      cp_async16(to, src, nb);
      cp_async16(to + S::kV, src + (rw ? v_off : 0), nb);
    }
    const int nb = row ? S::kSb : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst + S::kKs + lane * S::kSb), "l"(scales), "n"(S::kSb), "r"(nb)
                 : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst + S::kVs + lane * S::kSb), "l"(scales + (row ? v_off : 0)),
                 "n"(S::kSb), "r"(nb)
                 : "memory");
  }
};

// S^T of a tile: c[h][nt] holds rows (tokens) 16 h + sigma(r) and + 8, columns (query rows) 8 nt + 2c, + 1 for
// lane 4r + c.  `codes`, `scales`: the tile's K.
template <int D, int NT, int QS>
__device__ __forceinline__ void kv4_qk(float (&c)[2][NT][4], const char *codes, const char *scales, const char *qf, int lane) {
  using S = Kv4Smem<D>;
  const int r = lane >> 2, col = lane & 3, tok = kv4_sigma(r);
  constexpr int W = D / 32;  // words of a lane's share of a row
  uint32_t w[4][W], sc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const char *sa = scales + (8 * k + tok) * S::kSb;
    if (D == 128) {
      const uint4 v = *reinterpret_cast<const uint4 *>(codes + S::piece(tok, col) + 8 * k * S::kCb);
      w[k][0] = v.x, w[k][1] = v.y, w[k][W - 2] = v.z, w[k][W - 1] = v.w;
      sc[k] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(sa + col * 2));  // the lane's two groups
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(codes + (8 * k + tok) * S::kCb + col * 8);
      w[k][0] = v.x, w[k][1] = v.y;
      sc[k] = e4m3x2_to_f16x2(*reinterpret_cast<const uint8_t *>(sa + col) * 0x101u);  // its one group, twice
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) c[h][nt][k] = 0.f;
#pragma unroll
  for (int x = 0; x < W; ++x) {
    uint32_t f[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      e2m1_to_f16x2(w[k][x], f[k]);
      const uint32_t s = D == 128 ? __byte_perm(sc[k], 0, x < W / 2 ? 0x1010 : 0x3232) : sc[k];
#pragma unroll
      for (int y = 0; y < 4; ++y) f[k][y] = mul_f16x2(f[k][y], s);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int qs = 0; qs < QS; ++qs)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = reinterpret_cast<const uint2 *>(qf)[((qs * NT + nt) * (D / 16) + 2 * x + y) * 32 + lane];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_f16(c[h][nt], f[2 * h][2 * y], f[2 * h + 1][2 * y], f[2 * h][2 * y + 1], f[2 * h + 1][2 * y + 1], q.x, q.y);
        }
  }
}

// Query rows [r0, r0 + rows) of (request b, head g) as B fragments in shared memory, and per row the
// factor that turns a product into a log2-domain logit.  A row is scaled by a power of two so that its
// largest value lies in [2^13, 2^14): f16 then holds bf16 values exactly down to 2^-28 of the row's
// largest, and fp32 values as the sum of two f16 (QS = 2).
//
// fetch() starts the loads (before the tiles' loads queue up behind each other), store() does the rest.
template <int D, int NT, int QS, int NW>
struct Kv4Queries {
  static constexpr int V = D / 32;  // elements per lane
  static constexpr int N = cdiv(NT * 8, NW);
  float xs[N][V];

  __device__ __forceinline__ void fetch(const Kv4AttnArgs &a, int b, int g, int r0, int rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = warp + n * NW;
#pragma unroll
      for (int k = 0; k < V; ++k) xs[n][k] = 0.f;
      if (r < rows) {
        const int rr = r0 + r, i = rr / a.G, h = g * a.G + rr % a.G;
        const int64_t off = (((int64_t)b * a.n_c + i) * a.h_q + h) * D + lane * V;
#pragma unroll
        for (int k = 0; k < V; ++k)
          xs[n][k] = QS == 2 ? static_cast<const float *>(a.q)[off + k]
                             : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[off + k]);
      }
    }
  }
  __device__ __forceinline__ void store(const Kv4AttnArgs &a, char *qf, float *s_sl) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = warp + n * NW;
      if (r >= NT * 8) break;
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) mx = fmaxf(mx, fabsf(xs[n][k]));
      mx = warp_max(mx);
      const int e = (int)(__float_as_uint(mx) >> 23) - 127;  // floor(log2 mx); 128 for inf
      const int up = (mx == 0.f || e == 128) ? 0 : min(13 - e, 126);
      const float f = __uint_as_float((uint32_t)(127 + up) << 23);
      if (lane == 0) s_sl[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
      // element d of row 8 nt + rr sits in step j = (d % (D/4)) / 4 of lane 4 rr + d / (D/4)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int d = lane * V + k, col = d / (D / 4), j = (d % (D / 4)) / 4, pos = d & 3;
        const float v = xs[n][k] * f;
        const __half h = __float2half_rn(v);
        const int at = (((r >> 3) * (D / 16) + j) * 32 + (r & 7) * 4 + col) * 4 + pos;
        reinterpret_cast<__half *>(qf)[at] = h;
        if (QS == 2) reinterpret_cast<__half *>(qf)[NT * (D / 16) * 32 * 4 + at] = __float2half_rn(v - __half2float(h));
      }
    }
  }
};

__device__ __forceinline__ void kv4_write4(const Kv4AttnArgs &a, int64_t elem, const float4 &v) {
  if (a.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + elem) = v;
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + elem) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// A row's log-sum-exp from its reference M and the sum Z of exp2(x - M).  The criticality pass takes M and 1 / Z
// themselves: exp2(x - M) / Z is off by 1e-7, exp(x - lse) by lse's own rounding, up to 1e-6.
__device__ __forceinline__ void kv4_row_done(const Kv4AttnArgs &a, int64_t row, float M, float Z) {
  if (a.lse) a.lse[row] = Z == 0.f ? -INFINITY : (M + log2f(Z)) * kLn2;
  if (a.fin) a.fin[row] = Z == 0.f ? make_float2(INFINITY, 0.f) : make_float2(M, 1.f / Z);
}

// Counts a block in, after a barrier of the threads that wrote its part: releases those writes, and lets the last
// block's threads (after a barrier) see the others'.
__device__ __forceinline__ unsigned kv4_arrive(unsigned *counter) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

// Joins the `parts` partial results of a unit's pass, in the blocks' order: part k lies in rows row_of_part(k) .. of
// part_o / part_ml.  NT threads (whole warps), `sync` their barrier; s_M, s_F, s_Z: `rows` floats each.  Several loads
// are kept on their way: a part's load behind the last one's took 0.7 us each.
template <int D, int NT, typename PartRow, typename OutRow, typename Sync>
__device__ __forceinline__ void kv4_join(const Kv4AttnArgs &a, int parts, int rows, int tid, float *s_M, float *s_F, float *s_Z,
                                         PartRow part, OutRow row_of, Sync sync) {
  const int lane = tid & 31, warp = tid >> 5;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  if (parts <= 8) {  // every thread loads all it needs at once
    for (int e = tid; e < rows * (D / 4); e += NT) {
      const int q = e / (D / 4), piece = e % (D / 4);
      float4 y[8];
      float2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = make_float4(0.f, 0.f, 0.f, 0.f), v[j] = make_float2(-1e30f, 0.f);
        if (j < parts) {
          const int64_t at = part(j) + q;
          v[j] = __ldcg(ml + at);
          y[j] = __ldcg(reinterpret_cast<const float4 *>(a.part_o) + at * (D / 4) + piece);
        }
      }
      float M = v[0].x, Z = 0.f;
#pragma unroll
      for (int j = 1; j < 8; ++j) M = fmaxf(M, v[j].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = fast_exp2(v[j].x - M);
        Z = fmaf(v[j].y, f, Z);
        acc.x = fmaf(y[j].x, f, acc.x), acc.y = fmaf(y[j].y, f, acc.y), acc.z = fmaf(y[j].z, f, acc.z), acc.w = fmaf(y[j].w, f, acc.w);
      }
      const float f = Z == 0.f ? 0.f : a.v_scale / Z;
      kv4_write4(a, row_of(q) * D + piece * 4, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
      if (piece == 0) kv4_row_done(a, row_of(q), M, Z);
    }
    return;
  }
  constexpr int U = 4;  // rows of a warp at once
  for (int q0 = warp; q0 < rows; q0 += U * (NT / 32)) {
    float2 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int q = q0 + j * (NT / 32);
      v[j] = q < rows && lane < parts ? __ldcg(ml + part(lane) + q) : make_float2(-1e30f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int q = q0 + j * (NT / 32);
      if (q >= rows) break;
      float M = v[j].x;
      for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, __ldcg(ml + part(k) + q).x);
      M = warp_max(M);
      float Z = v[j].y * fast_exp2(v[j].x - M);
      for (int k = lane + 32; k < parts; k += 32) {
        const float2 w = __ldcg(ml + part(k) + q);
        Z += w.y * fast_exp2(w.x - M);
      }
      Z = warp_sum(Z);
      if (lane == 0) {
        s_M[q] = M;
        s_F[q] = Z == 0.f ? 0.f : a.v_scale / Z;
        s_Z[q] = Z;
      }
    }
  }
  sync();
  for (int e = tid; e < rows * (D / 4); e += NT) {
    const int q = e / (D / 4), piece = e % (D / 4);
    const float M = s_M[q];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += 8) {
      float4 y[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = make_float4(0.f, 0.f, 0.f, 0.f), w[j] = -INFINITY;
        if (k0 + j < parts) {
          const int64_t at = part(k0 + j) + q;
          y[j] = __ldcg(reinterpret_cast<const float4 *>(a.part_o) + at * (D / 4) + piece);
          w[j] = __ldcg(ml + at).x;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = fast_exp2(w[j] - M);
        acc.x = fmaf(y[j].x, f, acc.x), acc.y = fmaf(y[j].y, f, acc.y), acc.z = fmaf(y[j].z, f, acc.z), acc.w = fmaf(y[j].w, f, acc.w);
      }
    }
    const float f = s_F[q];
    kv4_write4(a, row_of(q) * D + piece * 4, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
    if (piece == 0) kv4_row_done(a, row_of(q), M, s_Z[q]);
  }
}

// PS = 2 carries a probability as the sum of two f16 for fp32 outputs; PS = 1 rounds it to f16 for bf16 outputs, whose
// own rounding is 2^-9.
template <int D, int NT, int QS, int PS, int NW, int NST, int BPS, bool LIST>
__global__ void __launch_bounds__(NW * 32, BPS) kv4_attn_kernel(Kv4AttnArgs a) {
  using S = Kv4Smem<D>;
  constexpr int MT = D / 16;  // fragments of 16 d
  constexpr int ROWS = NT * 8;
  constexpr int PIECES = D / 4;  // 16-byte pieces of a row of O
  constexpr bool AHEAD = kv4_ahead(NT), OWN_O = kv4_own_o(NT, PS);
  constexpr float kLift = kv4_lift(PS), kSlack = kv4_slack(PS);
  extern __shared__ __align__(128) char smem[];
  char *ring = smem;
  char *qf = ring + NW * NST * S::kStage + (OWN_O ? NW * ROWS * D * 4 : 0);
  float *s_sl = reinterpret_cast<float *>(qf + ROWS * D * 2 * QS);
  float *s_m = s_sl + ROWS, *s_l = s_m + NW * ROWS;
  float *acc = reinterpret_cast<float *>(OWN_O ? ring + NW * NST * S::kStage : ring);  // [warp][row][d], pieces of a row permuted
  __shared__ int64_t s_scan[NW + 4];
  __shared__ int s_last;
  __shared__ float s_join[3 * ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, col = lane & 3;
  pdl_wait();
  if (blockIdx.x == 0) {  // lengths out of range are clamped; say so once
    for (int b = tid; b < a.kv.batch; b += NW * 32) effective_len(a.kv, b, LIST ? 0 : a.n_c, a.status);
    if (LIST)
      for (int u = tid; u < a.n_units; u += NW * 32)
        if (a.cnt[u] < 0 || a.cnt[u] > a.k_max) atomicOr(a.status, (unsigned)SSD_FAULT_KMAX);
  }
  Kv4Range rg;
  if (!kv4_range<LIST, NW>(a, rg, s_scan)) return;
  const char *my_tiles = ring + warp * NST * S::kStage;
  const uint32_t my_ring = smem_u32(my_tiles);
  Kv4Loader<D> ld(a);
  Kv4Queries<D, NT, QS, NW> qs;
  int issued = 0, used = 0;  // the warp's ring positions
  int next = 0, end = 0;     // the warp's next tile to load, and the end of its segment
  int32_t seen = -1;
  auto peek = [&](int tile) { return LIST ? ld.peek_list(tile, lane) : ld.peek(tile, lane); };
  auto issue = [&](bool look) {
    if (next < end) {
      const int32_t now = seen;
      if (look && next + NW < end) seen = peek(next + NW);
      if (LIST)
        ld.load_list(next, now, my_ring + issued * S::kStage, lane);
      else
        ld.template load<false>(next, now, my_ring + issued * S::kStage, lane);
      issued = issued + 1 == NST ? 0 : issued + 1;
      next += NW;
    }
    cp_async_commit();
  };
  // The segment at rg: its queries and first tiles on their way.
  struct Seg {
    int u, b, g, r0, rows, n_tiles, t0, t1, L, count;
  };
  auto begin = [&]() {
    Seg s;
    s.u = rg.u, s.b = s.u / (a.kv.h_kv * a.n_chunk), s.g = (s.u / a.n_chunk) % a.kv.h_kv, s.r0 = (s.u % a.n_chunk) * ROWS;
    s.rows = min(ROWS, a.R - s.r0);
    s.n_tiles = kv4_tiles<LIST>(a, s.u);
    s.t0 = rg.off, s.t1 = kv4_range_end(rg, s.n_tiles);
    s.L = min(max(a.kv.seq_lens[s.b], 0), a.kv.max_seq_len);
    s.count = LIST ? min(max(a.cnt[s.u], 0), a.k_max) : s.L;
    ld.unit(s.b, s.g, s.L, s.count, LIST ? a.idx + (int64_t)s.u * a.k_max : nullptr);
    qs.fetch(a, s.b, s.g, s.r0, s.rows);
    next = s.t0 + warp, end = s.t1;
    // The first tiles' pages at once, then their loads.
    int32_t first[NST];
#pragma unroll
    for (int k = 0; k < NST; ++k) first[k] = next + k * NW < end ? peek(next + k * NW) : -1;
#pragma unroll 1
    for (int k = 0; k < NST; ++k) {
      seen = first[0];
#pragma unroll
      for (int j = 0; j + 1 < NST; ++j) first[j] = first[j + 1];
      issue(k + 1 == NST);
    }
    return s;
  };

  Seg sg = begin();
  for (;;) {
    const int b = sg.b, g = sg.g, r0 = sg.r0, rows = sg.rows, n_tiles = sg.n_tiles, seg0 = sg.t0, seg1 = sg.t1, L = sg.L, count = sg.count;
    const int64_t place = rg.x;
    qs.store(a, qf, s_sl);
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
    // The lane's 16-byte pieces of its warp's O in shared memory, of columns 8 nt + 2 col + k and rows 4 r .. of i, i + 1.
    auto piece_of = [&](int nt, int k, int i) {
      return reinterpret_cast<float4 *>(acc) + (warp * ROWS + 8 * nt + 2 * col + k) * PIECES +
             ((r * (MT / 2) + i / 2) ^ (r >> 1) ^ col);
    };
    int held = 0;          // PS = 2: tiles whose products the accumulators hold
    bool flushed = false;  // and whether there are earlier ones' in shared memory

    for (int tile = seg0 + warp; tile < seg1; tile += NW) {
      cp_async_wait<NST - 1>();
      __syncwarp();
      const char *st = my_tiles + used * S::kStage;
      const int t0 = tile * kKv4Tile;
      const bool edge = LIST ? t0 + kKv4Tile > count : t0 + kKv4Tile > L - a.n_c + 1;
      float c[2][NT][4], x[2][NT][4];
      kv4_qk<D, NT, QS>(c, st, st + S::kKs, qf, lane);
      // x = logit (log2) - reference; -inf where a row does not see the token.
      auto visible = [&](int h, int nt, int k) {
        const int lim = LIST ? count : min(L, L - a.n_c + 1 + (r0 + 8 * nt + 2 * col + (k & 1)) / a.G);
        return t0 + 16 * h + (k >> 1) * 8 + kv4_sigma(r) < lim;
      };
      auto logits = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[h][nt][k] = fmaf(c[h][nt][k], sl[nt][k & 1], -m[nt][k & 1]);
        if (edge) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!visible(h, nt, k)) x[h][nt][k] = -INFINITY;
        }
      };
      logits();
      float top = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, x[h][nt][k]);
      if (__any_sync(0xffffffffu, top > kSlack)) {
        // The references move to the tile's largest logits; O and the sums follow.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = k; j < 4; j += 2)
                if (!edge || visible(h, nt, j)) mx = fmaxf(mx, c[h][nt][j] * sl[nt][k]);
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = fmaxf(mx, m[nt][k] + kLift);
            const float f = fast_exp2(m[nt][k] + kLift - mx);
            m[nt][k] = mx - kLift;
            l[nt][k] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][nt][k] *= f, o[i][nt][k + 2] *= f;
            if (PS == 2 && flushed) {
#pragma unroll
              for (int i = 0; i < MT; i += 2) {
                const float4 y = *piece_of(nt, k, i);
                *piece_of(nt, k, i) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
              }
            }
          }
        logits();
      }
      uint32_t p[2][NT][2], pl[2][NT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = fast_exp2(x[h][nt][k]);
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
      // O^T += V^T P^T, 16 tokens a step.  A lane reads its d / 8 elements of four tokens and pairs the codes of two
      // tokens in a byte, so that each conversion gives a fragment register.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int W = D / 64;
        uint32_t w[4][W], sc[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int g8 = 16 * h + 8 * k, ta = kv4_sigma(2 * col), tb = ta ^ 1;  // the eight tokens, the lane's two
          const char *vb = st + S::kV + g8 * S::kCb;
          if (W == 2) {
            const uint2 va = *reinterpret_cast<const uint2 *>(vb + S::piece(ta, r >> 1) + (r & 1) * 8);
            const uint2 vc = *reinterpret_cast<const uint2 *>(vb + S::piece(tb, r >> 1) + (r & 1) * 8);
            w[2 * k][0] = va.x, w[2 * k][W - 1] = va.y;
            w[2 * k + 1][0] = vc.x, w[2 * k + 1][W - 1] = vc.y;
          } else {
            w[2 * k][0] = *reinterpret_cast<const uint32_t *>(vb + ta * S::kCb + r * 4);
            w[2 * k + 1][0] = *reinterpret_cast<const uint32_t *>(vb + tb * S::kCb + r * 4);
          }
          const char *sb = st + S::kVs + g8 * S::kSb + (D == 128 ? r : r >> 1);
          uint32_t sa = *reinterpret_cast<const uint8_t *>(sb + ta * S::kSb), sbb = *reinterpret_cast<const uint8_t *>(sb + tb * S::kSb);
          if (edge) {  // tokens past the end: whatever their slots hold counts as 0
            if (t0 + g8 + ta >= count) sa = 0;
            if (t0 + g8 + tb >= count) sbb = 0;
          }
          sc[k] = e4m3x2_to_f16x2(sa | (sbb << 8));
        }
#pragma unroll
        for (int y = 0; y < W; ++y) {
          uint32_t f[4][4];
          e2m1_to_f16x2((w[0][y] & 0x0f0f0f0fu) | ((w[1][y] << 4) & 0xf0f0f0f0u), f[0]);
          e2m1_to_f16x2(((w[0][y] >> 4) & 0x0f0f0f0fu) | (w[1][y] & 0xf0f0f0f0u), f[1]);
          e2m1_to_f16x2((w[2][y] & 0x0f0f0f0fu) | ((w[3][y] << 4) & 0xf0f0f0f0u), f[2]);
          e2m1_to_f16x2(((w[2][y] >> 4) & 0x0f0f0f0fu) | (w[3][y] & 0xf0f0f0f0u), f[3]);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t a0 = mul_f16x2(f[0][z], sc[0]), a1 = mul_f16x2(f[1][z], sc[0]), a2 = mul_f16x2(f[2][z], sc[1]),
                           a3 = mul_f16x2(f[3][z], sc[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(o[4 * y + z][nt], a0, a1, a2, a3, p[h][nt][0], p[h][nt][1]);
              if (PS == 2) mma_f16(o[4 * y + z][nt], a0, a1, a2, a3, pl[h][nt][0], pl[h][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      used = used + 1 == NST ? 0 : used + 1;
      issue(true);
      if (PS == 2 && ++held == kKv4Flush) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < MT; i += 2) {
              float4 y = flushed ? *piece_of(nt, k, i) : make_float4(0.f, 0.f, 0.f, 0.f);
              y.x += o[i][nt][k], y.y += o[i][nt][k + 2], y.z += o[i + 1][nt][k], y.w += o[i + 1][nt][k + 2];
              *piece_of(nt, k, i) = y;
              o[i][nt][k] = o[i][nt][k + 2] = o[i + 1][nt][k] = o[i + 1][nt][k + 2] = 0.f;
            }
        held = 0, flushed = true;
      }
    }
    kv4_range_next(rg, n_tiles);
    const bool more = rg.x < rg.x1;
    if (!more) pdl_trigger();
    if (AHEAD && more) sg = begin();

    // Sums of the lanes of a query row, then of the warps.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], s);
        if (r == 0) s_m[warp * ROWS + 8 * nt + 2 * col + k] = m[nt][k], s_l[warp * ROWS + 8 * nt + 2 * col + k] = l[nt][k];
      }
    __syncthreads();
    const int nw = min(NW, seg1 - seg0);           // warps that had a tile
    if (warp < nw) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int q = 8 * nt + 2 * col + k;
          float M = -1e30f;
#pragma unroll
          for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * ROWS + q]);
          const float f = fast_exp2(m[nt][k] - M);
#pragma unroll
          for (int i = 0; i < MT; i += 2) {
            float4 y = make_float4(o[i][nt][k], o[i][nt][k + 2], o[i + 1][nt][k], o[i + 1][nt][k + 2]);
            if (PS == 2 && flushed) {
              const float4 z = *piece_of(nt, k, i);
              y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            *piece_of(nt, k, i) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
          }
        }
    }
    __syncthreads();
    const Kv4Parts<kKv4Tile> parts(rg, place, n_tiles);
    const bool whole = parts.more == 0;
    const int64_t slot = parts.slot((int)blockIdx.x - parts.first);
    auto row_of = [&](int q) {
      const int rr = r0 + q;
      return ((int64_t)b * a.n_c + rr / a.G) * a.h_q + g * a.G + rr % a.G;
    };
    for (int e = tid; e < rows * PIECES; e += NW * 32) {
      const int q = e / PIECES, piece = e % PIECES, rr = piece / (MT / 2);
      float M = -1e30f, Z = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * ROWS + q]);  // (a warp without a tile: -1e30 and 0)
#pragma unroll
      for (int w = 0; w < NW; ++w) Z += s_l[w * ROWS + q] * fast_exp2(s_m[w * ROWS + q] - M);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w >= nw) break;
        const float4 y = reinterpret_cast<const float4 *>(acc)[(w * ROWS + q) * PIECES + (piece ^ (rr >> 1) ^ ((q >> 1) & 3))];
        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      }
      if (whole) {
        const int64_t row = row_of(q);
        const float f = Z == 0.f ? 0.f : a.v_scale / Z;
        kv4_write4(a, row * D + piece * 4, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        if (piece == 0) kv4_row_done(a, row, M, Z);
      } else {
        __stcg(reinterpret_cast<float4 *>(a.part_o + (slot * ROWS + q) * D) + piece, v);
        if (piece == 0) __stcg(reinterpret_cast<float2 *>(a.part_ml) + slot * ROWS + q, make_float2(M, Z));
      }
    }
    if (!whole) {
      // The last block of the unit to arrive joins the partial results.
      __syncthreads();
      if (tid == 0) {
        s_last = kv4_arrive(a.counters + parts.first) == (unsigned)parts.more;
        if (s_last) a.counters[parts.first] = 0;
      }
      __syncthreads();
      if (s_last)
        kv4_join<D, NW * 32>(
            a, parts.more + 1, rows, tid, s_join, s_join + ROWS, s_join + 2 * ROWS,
            [&](int k) { return parts.slot(k) * ROWS; }, row_of, [] { __syncthreads(); });
    }
    if (!more) break;
    __syncthreads();
    if (!AHEAD) sg = begin();
  }
}

// Criticality: a second pass over K alone recomputes the logits and sums exp2(x - m) / l over the rows, from each row's
// reference and 1 / sum.  (Keeping them from the first pass would cost 2 R bytes per token each way, more than K's 36
// for R > 9, and a rounding to f16.)
// d = 64 (at d = 128 kv4_crit_tc_kernel takes all calls).
template <int NT, int QS, int NW, int NST, int BPS>
__global__ void __launch_bounds__(NW * 32, BPS) kv4_crit_kernel(Kv4AttnArgs a) {
  constexpr int D = 64;
  using S = Kv4Smem<D>;
  constexpr int ROWS = NT * 8;
  extern __shared__ __align__(128) char smem[];
  char *ring = smem;
  char *qf = ring + NW * NST * S::kCritStage;
  float *s_sl = reinterpret_cast<float *>(qf + 2 * ROWS * D * 2 * QS);  // two chunks of rows at most
  float *s_ref = s_sl + 2 * ROWS, *s_inv = s_ref + 2 * ROWS;
  __shared__ int64_t s_scan[NW + 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, col = lane & 3;
  // Everything but a.fin was written before the attention kernel ran, which waited for it and only then let
  // this one start; a.fin is waited for below.
  Kv4Range rg;
  if (!kv4_range<false, NW>(a, rg, s_scan)) {
    pdl_wait();
    return;
  }
  const char *my_tiles = ring + warp * NST * S::kCritStage;
  const uint32_t my_ring = smem_u32(my_tiles);
  Kv4Loader<D> ld(a);
  const int n_chunk = cdiv(a.R, ROWS);
  int issued = 0, used = 0;
  while (rg.x < rg.x1) {
    const int u = rg.u, b = u / a.kv.h_kv, g = u % a.kv.h_kv;
    const int n_tiles = kv4_tiles<false>(a, u);
    const int seg0 = rg.off, seg1 = kv4_range_end(rg, n_tiles);
    const int L = min(max(a.kv.seq_lens[b], 0), a.kv.max_seq_len);
    ld.unit(b, g, L, L, nullptr);
    int next = seg0 + warp;
    int32_t seen = next < seg1 ? ld.peek(next, lane) : -1;
    auto issue = [&]() {
      if (next < seg1) {
        const int32_t now = seen;
        if (next + NW < seg1) seen = ld.peek(next + NW, lane);
        ld.template load<true>(next, now, my_ring + issued * S::kCritStage, lane);
        issued = issued + 1 == NST ? 0 : issued + 1;
        next += NW;
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < NST; ++s) issue();
    for (int ch = 0; ch < n_chunk; ++ch) {
      Kv4Queries<D, NT, QS, NW> qs;
      qs.fetch(a, b, g, ch * ROWS, min(ROWS, a.R - ch * ROWS));
      qs.store(a, qf + ch * ROWS * D * 2 * QS, s_sl + ch * ROWS);
    }
    pdl_wait();
    for (int q = tid; q < n_chunk * ROWS; q += NW * 32) {
      float2 v = make_float2(INFINITY, 0.f);  // the padding, as rows that see nothing: exp2(x - inf) = 0
      if (q < a.R) v = a.fin[((int64_t)b * a.n_c + q / a.G) * a.h_q + g * a.G + q % a.G];
      s_ref[q] = v.x, s_inv[q] = v.y;
    }
    __syncthreads();
    for (int tile = seg0 + warp; tile < seg1; tile += NW) {
      cp_async_wait<NST - 1>();
      __syncwarp();
      const char *kt = my_tiles + used * S::kCritStage;
      const int t0 = tile * kKv4Tile;
      const bool edge = t0 + kKv4Tile > L - a.n_c + 1;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int ch = 0; ch < n_chunk; ++ch) {
        float c[2][NT][4];
        kv4_qk<D, NT, QS>(c, kt, kt + S::kCritScales, qf + ch * ROWS * D * 2 * QS, lane);
        const float *fac = s_sl + ch * ROWS + 2 * col, *off = s_ref + ch * ROWS + 2 * col, *inv = s_inv + ch * ROWS + 2 * col;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2 *>(fac + 8 * nt), z = *reinterpret_cast<const float2 *>(off + 8 * nt);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[h][nt][k] = fmaf(c[h][nt][k], k & 1 ? f.y : f.x, -(k & 1 ? z.y : z.x));
        }
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int lim = min(L, L - a.n_c + 1 + (ch * ROWS + 8 * nt + 2 * col + (k & 1)) / a.G);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (t0 + 16 * h + (k >> 1) * 8 + kv4_sigma(r) >= lim) c[h][nt][k] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2 *>(inv + 8 * nt);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[2 * h + (k >> 1)] = fmaf(fast_exp2(c[h][nt][k]), k & 1 ? f.y : f.x, sum[2 * h + (k >> 1)]);
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
      used = used + 1 == NST ? 0 : used + 1;
      issue();
    }
    __syncthreads();
    kv4_range_next(rg, n_tiles);
  }
}

}  // namespace ssd

// ---- launches -------------------------------------------------------------------------------
#include "ssd_host.h"

namespace ssd {

// Warps and blocks per SM, and ring depth, by the rows of a pass: registers bound the warps (the O accumulators take
// 32 NT a lane at d = 128, 16 NT at d = 64), and the ring also holds the warps' O at a segment's end.  d = 64, 32
// requests of 2048 to 8192 tokens, 8 heads: 16 rows 44 us with two blocks of 8 warps, 52 with one; 20 rows 65 with 8
// warps, 62 with 12, 60 with two blocks of 8, which spill and take 16.5 us instead of 15 for a short request; 32
// rows 76 with 8 warps, 84 with 12, 106 with two blocks of 8; 4 rows 34.4 with two blocks, 36.5 with three.
template <int D, int NT>
struct Kv4Tune {
  static constexpr int kWarps = D == 64 && NT == 3 ? 12 : 8;
  static constexpr int kBlocks = NT == 1 || (D == 64 && NT == 2) ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 2 : NT == 2 ? 3 : 4;
};
constexpr int kKv4CritWarps = 8, kKv4CritBlocks = 2, kKv4CritStages = 4;

template <int D, int NT, int QS, int PS, bool LIST>
int kv4_launch_attn(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr int NST = Kv4Tune<D, NT>::kStages, BPS = Kv4Tune<D, NT>::kBlocks, NW = Kv4Tune<D, NT>::kWarps;
  static_assert(kv4_own_o(NT, PS) || NST * Kv4Smem<D>::kStage >= NT * 8 * D * 4, "the ring holds the warps' O");
  constexpr int smem = kv4_smem_bytes<D, NT, QS, PS, NW, NST>();
  static_assert(smem * BPS + BPS * 1024 + 2048 <= 227 * 1024, "the blocks of an SM fit");
  constexpr auto kernel = kv4_attn_kernel<D, NT, QS, PS, NW, NST, BPS, LIST>;
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  return launch(kernel, dim3(grid), dim3(NW * 32), smem, st, LIST ? "kv4_attn_kernel (draft)" : "kv4_attn_kernel", a);
}

template <int D, int NT, bool LIST>
int kv4_attn_types(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  if (a.q_f32) return kv4_launch_attn<D, NT, 2, 2, LIST>(a, grid, st);
  if (a.out_f32) return kv4_launch_attn<D, NT, 1, 2, LIST>(a, grid, st);
  return kv4_launch_attn<D, NT, 1, 1, LIST>(a, grid, st);
}

template <int NT, int QS>
int kv4_launch_crit(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr int NW = kKv4CritWarps, NST = kKv4CritStages, BPS = kKv4CritBlocks;
  constexpr int smem = NW * NST * Kv4Smem<64>::kCritStage + 2 * NT * 8 * 64 * 2 * QS + 6 * NT * 8 * 4;
  constexpr auto kernel = kv4_crit_kernel<NT, QS, NW, NST, BPS>;
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  return launch(kernel, dim3(grid), dim3(NW * 32), smem, st, "kv4_crit_kernel", a);
}

}  // namespace ssd
