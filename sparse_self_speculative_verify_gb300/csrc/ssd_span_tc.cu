// ssd_span_tc.cu -- span attention over bf16 caches on the 5th-generation tensor cores (tcgen05, TMA, tensor memory).
//
// Up to 128 query rows of a (request, KV head) are the M side of both products, a row per lane of tensor memory:
//   S [128 rows x 128 tokens] = Q K^T      (both from shared memory)
//   O [128 rows x D]         += P V        (P from tensor memory, in the place of S; V as it lies, token-major)
// so that a row's softmax belongs to one thread.  A block runs two such streams, which take turns on the tensor cores: while
// one's softmax runs, the other's products do.
//   WIDE (n queries of more than 128 rows, whatever a request's own number): the streams are two tiles of rows and share every tile
//   of K and V;
//   else both streams have the same rows and take K / V tiles in turn, their O joined at a segment's end.
// Roles: warps 0-3 and 4-7 the softmax of a stream (and its O), warp 8 loads Q and K, warp 11 V (TMA boxes of up to 16 tokens
// of a page, 128-byte swizzle), warps 9 and 10 issue a stream's products.
//
// Softmax.  A row's reference follows its maximum only when that has grown by 2^8, so that O is seldom rescaled; sums, O and
// references are fp32.  P is rounded to bf16 for the second product (half a step, 2^-8 of each term, whose signs differ: 0.0023
// of the outputs' 2-norm beside the output type's own 0.0017); the row's sum takes the unrounded P.
//
// What bounds it, one GB300, 8 heads of 128 (us a call, launch and join included):
//   decoding, 128 requests of 8192 tokens: HBM, 612 (7.0 TB/s of K and V);
//   trees of 16 nodes, 4 heads a group (64 rows), 32 requests of 2048 to 8192 tokens: HBM, 106 to 116 by the draw (5.9 TB/s);
//   trees of up to 64 nodes, 5 heads a group (3 tiles of rows), 8 requests of 16384 to 65536: 290 to 376 by the draw, the
//     tensor cores half busy, 3.6 TB/s: groups of 256 rows read K and V for themselves, S of a stream's next tile waits for the
//     softmax and O += P V of this one (P lies in S's place), and a last group of up to 128 rows has one stream alone;
//   4 chunks of up to 4096 prompt tokens, window 2048: 320 to 382 by the draw, 1.33 PFLOP/s, as above; whole prompts 1.36;
//   one window of 1024 tokens for each of 32 requests: 35, start and the units' ends around 20 us of HBM; one request: 11 to 14.
//
// Work.  A unit is one (request, KV head, group of as many queries as a block holds).  The units' tiles lie end to end and are
// cut into equal shares, one per block (one block per SM); a cut close to a unit's border moves there.  A unit that several
// blocks share leaves partial results, joined by span_join_kernel.  (Groups of the same head read K and V for themselves: at
// 256 rows a tile takes longer on the tensor cores than from memory.  Blocks that walked the groups of a head side by side,
// to read it once, had to do the same work: 8 requests of 33 to 64 nodes with 5 heads a group took 488 us.)
#include "ssd_sm100.cuh"
#include "ssd_sm100_pairs.cuh"
#include "ssd_span.h"

namespace ssd {
using namespace sm100;

constexpr int kSpanTile = 128;          // tokens of a tile, rows of a stream
constexpr int kSpanThreads = 12 * 32;
constexpr int kSpanProducer = 8, kSpanMma = 9, kSpanLoadV = 11;
constexpr int kSpanMaxBatch = 1024;     // requests of a launch (their sizes lie in shared memory)
constexpr int kSpanOverhead = 1;        // what starting and ending a unit costs, in tiles
constexpr int kSpanSnap = 3;            // a cut this close to a unit's border moves there
// Units of more than kSpanWhole tiles are cut; shorter ones where equal shares save more than kSpanJoin tiles, what leaving
// parts and joining them costs.  (32 requests, 8 heads, 10 tiles: whole 34.9 us, cut 37.5; 100 requests: 87.6 and 84.4; one of
// 6 tiles: 14.6 and 15.9, of 8: 15 and 14; of 64 requests of up to 12 tiles each their own number, 60 and 63.3.)
constexpr int kSpanWhole = 12, kSpanJoin = 5;
// Least share of a block: one request of 1000 tokens, 64 rows, 15.5 us with 4 and 13.5 with 3; 8000 tokens, 256 rows, 28.3 and 30.1.
constexpr int kSpanLeast = 3, kSpanLeastWide = 4;
// Every part of a unit has tiles: a cut inside lies behind the overhead, and two of one unit are a share apart.
static_assert(kSpanSnap > kSpanOverhead && kSpanLeast >= 1 && kSpanLeastWide >= 1, "parts without tiles");
constexpr float kSpanLazy = 8.f;        // a row's reference moves when a score exceeds it by this (log2)

struct SpanPlan {
  int n_groups;          // row groups of a unit
  int row_nodes;         // queries of a stream's tile
  int nodes;             // of a group
  int blocks, least;     // shares, at most; the least cost of one
  int box;               // tokens of a copy: of a page, at most 16
  int split;             // whether units are cut; else shares end at their borders and nothing is left to join
  int32_t *cut_unit;     // [blocks]: the unit that a block's share begins inside of, or -1
  float *o, *lse;        // [blocks][2][D / 4][rows of a block][4], [blocks][2][rows] (log2)
};

struct SpanSeg {
  int b, g, rg;       // request, KV head, row group
  int k0, k1;         // tiles of the unit
  int part;           // -1: the whole unit; else the slot of its results
  int c;              // the request's queries
  SpanTiles st;
};
// Segments handed from the producer to the other warps.  A slot is written again once every warp that reads it has arrived: the loads
// of V, the products, and the softmax of both streams, of which a WIDE block's second passes over segments without rows for it
// and is held back by nothing else there.
constexpr int kSpanRing = 8;

template <int D, bool WIDE>
struct SpanCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kSpanTile * D * 2;
  static constexpr int kGroup = 1024 * kPanels;  // bytes of 8 tokens: panel after panel of 8 x 128 bytes
  // Slots of K and of V: V is held through the softmax.  (D = 128: all of the shared memory.)
  static constexpr int kSlotsK = D == 128 ? 2 : 4, kSlotsV = D == 128 ? (WIDE ? 3 : 2) : 4;
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kSlotsK * kTileBytes, kMisc = kV + kSlotsV * kTileBytes;
  static constexpr int kBars = 2 * (kSlotsK + kSlotsV) + 16 + 2 * kSpanRing;
  static constexpr int kReaders = 8 + 1 + (WIDE ? 1 : 2);  // warps that read a segment
  // barriers, segments, the streams' maxima and sums
  static constexpr int kSmem = kMisc + kBars * 8 + kSpanRing * (int)sizeof(SpanSeg) + (WIDE ? 0 : 512 * 4) + 1024;
  // before the first copy, in the slots: the requests' prefix, size, length and queries
  static_assert((kSlotsK + kSlotsV) * kTileBytes >= (4 * kSpanMaxBatch + 1) * 4, "sizes");
  static constexpr int kRows = WIDE ? 256 : 128;
  static constexpr int kColO = 256;  // tensor memory: S (P) of the streams, O of the streams
};

// The segments of a block, in order.  (Costs of a launch fit 31 bits: span_tc cuts the batch so.)
struct SpanWalk {
  const SpanArgs &a;
  const SpanPlan &pl;
  // Until the first segment: prefix of the requests' costs; cost of a KV head's groups.
  const int *pre, *size, *len, *cnt;
  int pos, end, u0, u1;       // of the share; the unit at pos
  int b, g, rg;
  int L, c, next_L, next_c;   // of request b, of the one behind it
  bool inside;                // the share begins inside a unit

  __device__ SpanWalk(const SpanArgs &a_, const SpanPlan &p_, const int *pre_, const int *size_, const int *len_, const int *cnt_)
      : a(a_), pl(p_), pre(pre_), size(size_), len(len_), cnt(cnt_), u0(0), u1(0), b(0), g(0), rg(0) {
    if (pl.n_groups == 1) {  // both ends at once, by even and odd lanes
      const int x = cut(blockIdx.x + (threadIdx.x & 1));
      pos = __shfl_sync(0xffffffffu, x, 0);
      end = __shfl_sync(0xffffffffu, x, 1);
      u0 = __shfl_sync(0xffffffffu, u0, 0);
      u1 = __shfl_sync(0xffffffffu, u1, 0);
      b = __shfl_sync(0xffffffffu, b, 0);
      g = __shfl_sync(0xffffffffu, g, 0);
    } else {
      end = cut(blockIdx.x + 1);
      pos = cut(blockIdx.x);
    }
    inside = pos > u0 && pos < u1;
    L = len[b], c = cnt[b];
    look_ahead();
  }
  __device__ void look_ahead() {
    if (b + 1 < a.kv.batch) span_sizes(a, b + 1, false, next_L, next_c);
  }
  __device__ SpanTiles tiles_of(int len_, int cnt_, int group) const {
    return span_tiles<kSpanTile>(a, len_, cnt_, group * pl.nodes, group * pl.nodes + pl.nodes - 1, pl.box);
  }
  // What group `group` of a request costs, in tiles.
  __device__ int cost(int len_, int cnt_, int group) const {
    const int n = tiles_of(len_, cnt_, group).n_tiles;
    return n ? n + kSpanOverhead : 0;
  }
  // Sets the unit that position x < pre[batch] lies in (by a converged warp where a unit has groups of its own).
  __device__ void locate(int x) {
    int lo = 0, hi = a.kv.batch;  // pre[lo] <= x < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    b = lo;
    const unsigned sz = size[lo], rem = x - pre[lo];
    g = rem / sz;
    u0 = pre[lo] + g * sz;
    u1 = u0 + sz;
    if (pl.n_groups == 1) return;
    const int lane = threadIdx.x & 31;
    int at = u0;
    for (int r0 = 0;; r0 += 32) {  // 32 groups at a time
      const int mine = r0 + lane < pl.n_groups ? cost(len[b], cnt[b], r0 + lane) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const unsigned past = __ballot_sync(0xffffffffu, at + incl > x);
      if (past || r0 + 32 >= pl.n_groups) {
        const int w = past ? __ffs(past) - 1 : 31;
        rg = r0 + w;
        u1 = at + __shfl_sync(0xffffffffu, incl, w);
        u0 = u1 - __shfl_sync(0xffffffffu, mine, w);
        return;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // Where block t's share begins; sets the unit there, or the one that ends there.
  __device__ int cut(int t) {
    const unsigned total = pre[a.kv.batch], n = min((unsigned)pl.blocks, max(1u, total / pl.least));
    if (t >= (int)n || total == 0) return total;
    const unsigned per = total / n, x = per * t + (total - per * n) * t / n;
    locate(x);
    if (!pl.split) return 2 * ((int)x - u0) < u1 - u0 ? u0 : u1;
    return (int)x - u0 < kSpanSnap ? u0 : u1 - (int)x < kSpanSnap ? u1 : (int)x;
  }
  __device__ int unit() const { return (b * a.kv.h_kv + g) * pl.n_groups + rg; }
  __device__ bool next(SpanSeg &s) {
    if (pos >= end) return false;
    if (pos >= u1) {  // the next unit that costs something
      u0 = u1;
      do {
        if (++rg * pl.nodes >= c) {  // (groups behind the queries cost nothing)
          rg = 0;
          if (++g >= a.kv.h_kv) {
            g = 0;
            do {  // a request that sees something
              ++b;
              L = next_L, c = next_c;
              look_ahead();
            } while (L == 0 || c == 0);
          }
        }
        u1 = u0 + cost(L, c, rg);
      } while (u1 == u0);
    }
    s.b = b;
    s.g = g;
    s.rg = rg;
    s.c = c;
    s.st = tiles_of(L, c, rg);
    const int stop = min(u1, end);
    s.k0 = min(max(0, pos - u0 - kSpanOverhead), s.st.n_tiles);
    s.k1 = stop == u1 ? s.st.n_tiles : min(max(0, stop - u0 - kSpanOverhead), s.st.n_tiles);
    s.part = pos == u0 && stop == u1 ? -1 : (int)blockIdx.x * 2 + (pos == u0);
    pos = stop;
    return true;
  }
};

// 16 columns of this thread's lane of tensor memory, a register each.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 x 8 pieces of 16 bytes, lane i of eight with row i: afterwards lane i has column i.
__device__ __forceinline__ void span_transpose(uint4 (&v)[8], int i) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    const bool upper = (i & s) != 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (p & s) continue;
      uint4 out = upper ? v[p] : v[p + s], in;
      in.x = __shfl_xor_sync(0xffffffffu, out.x, s), in.y = __shfl_xor_sync(0xffffffffu, out.y, s);
      in.z = __shfl_xor_sync(0xffffffffu, out.z, s), in.w = __shfl_xor_sync(0xffffffffu, out.w, s);
      if (upper) v[p] = in; else v[p + s] = in;
    }
  }
}

template <int V>
struct SpanInt {
  static constexpr int value = V;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kSpanThreads, 1)
    span_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap, SpanArgs a, SpanPlan pl) {
  using C = SpanCfg<D, WIDE>;
  constexpr int NK = C::kSlotsK, NV = C::kSlotsV;
  extern __shared__ __align__(1024) char smem_raw[];
  char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.kv.batch, h_kv = a.kv.h_kv, ps = a.kv.page_size;

  // K and V slots' full / empty, Q buffers' full / empty, the streams' S full, P's halves full, O done, drain
  const uint32_t bars = sbase + C::kMisc;
  const uint32_t k_full = bars, k_empty = k_full + 8 * NK, v_full = k_empty + 8 * NK, v_empty = v_full + 8 * NV;
  const uint32_t q_full = v_empty + 8 * NV, q_empty = q_full + 16, s_full = q_empty + 16, p_full = s_full + 16, o_done = p_full + 32,
                 drained = o_done + 16, group = drained + 16, seg_full = group + 8, seg_empty = seg_full + 8 * kSpanRing;
  SpanSeg *ring = reinterpret_cast<SpanSeg *>(sm + C::kMisc + C::kBars * 8);
  float *s_m = reinterpret_cast<float *>(ring + kSpanRing);  // [maxima, sums][stream][row]
  int *pre = reinterpret_cast<int *>(sm + C::kK), *s_size = pre + kSpanMaxBatch + 1, *s_len = s_size + kSpanMaxBatch, *s_cnt = s_len + kSpanMaxBatch;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_scan[kSpanThreads / 32];

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < NK; ++i) mbar_init(k_full + 8 * i, 1), mbar_init(k_empty + 8 * i, 1);
    for (int i = 0; i < NV; ++i) mbar_init(v_full + 8 * i, 1), mbar_init(v_empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1), mbar_init(q_empty + 8 * i, WIDE ? 1 : 8);
      mbar_init(s_full + 8 * i, 1), mbar_init(p_full + 8 * i, 4), mbar_init(p_full + 16 + 8 * i, 4), mbar_init(o_done + 8 * i, 1), mbar_init(drained + 8 * i, 1);
    }
    mbar_init(group, 8);
    for (int i = 0; i < kSpanRing; ++i) mbar_init(seg_full + 8 * i, 1), mbar_init(seg_empty + 8 * i, C::kReaders);
    mbar_init_fence();
  }
  if (warp == kSpanMma) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  if (warp == kSpanProducer && lane == 0) {
    tma_prefetch_desc(&kvmap);
    tma_prefetch_desc(&qmap);
  }
  pdl_wait();

  // Sizes of the requests; the costs of their units; the prefix of the requests' costs.
  for (int b = tid; b < B; b += kSpanThreads) {
    int L, c;
    span_sizes(a, b, blockIdx.x == 0, L, c);
    s_len[b] = L, s_cnt[b] = c;
    const int n = pl.n_groups == 1 ? span_tiles<kSpanTile>(a, L, c, 0, pl.nodes - 1, pl.box).n_tiles : 0;
    s_size[b] = n ? n + kSpanOverhead : 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (pl.n_groups > 1) {
    for (unsigned e = tid; e < (unsigned)B * pl.n_groups; e += kSpanThreads) {
      const int b = (int)(e / pl.n_groups), group = (int)(e - (unsigned)b * pl.n_groups);
      const int n = span_tiles<kSpanTile>(a, s_len[b], s_cnt[b], group * pl.nodes, group * pl.nodes + pl.nodes - 1, pl.box).n_tiles;
      if (n == 0) continue;
      atomicAdd(s_size + b, n + kSpanOverhead);
    }
    __syncthreads();
  }
  {
    constexpr int CH = cdiv(kSpanMaxBatch, kSpanThreads);
    int mine[CH], sum = 0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int b = tid * CH + k;
      mine[k] = b < B ? h_kv * s_size[b] : 0;
      sum += mine[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int off = incl - sum;
    for (int w = 0; w < warp; ++w) off += s_scan[w];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int b = tid * CH + k;
      if (b < B) pre[b] = off;
      off += mine[k];
      if (b == B - 1) pre[B] = off;
    }
    fence_proxy_async_smem();  // before the copies into this place
    __syncthreads();
  }
  const uint32_t tm = s_tmem;
  volatile int *abort = &s_abort;

  const int row_nodes = pl.row_nodes;
  // Segment j of the block, once the producer has published it; nullptr behind the last one (and where a wait ran out).
  auto segment = [&](int j) -> const SpanSeg * {
    const bool ok = mbar_wait(seg_full + 8 * (j % kSpanRing), (j / kSpanRing) & 1, abort);
    const SpanSeg *x = ring + j % kSpanRing;
    return __all_sync(0xffffffffu, ok) && x->b >= 0 ? x : nullptr;
  };
  // This warp is done with segment j's slot.
  auto release = [&](int j) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + 8 * (j % kSpanRing));
  };
  // Whether stream 1 of a WIDE block has rows in a segment.
  auto second = [&](const SpanSeg &x) { return x.rg * pl.nodes + row_nodes < x.c; };

  // Registers: 256 x 208 + 128 x 88 are the launch's 384 x 168.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kSpanProducer || warp == kSpanLoadV) {
      // ---------------------------------------------------------------- loads
      const int box_rows = pl.box, boxes = kSpanTile / box_rows;
      const uint64_t pol = a.parents && pl.n_groups == 1 ? policy_evict_first() : policy_evict_normal();
      const int oob = (int)((int64_t)a.kv.num_pages * 2 * h_kv * ps / 8);
      bool ok = true;
      // Page of lane's box of tile k, INT32_MIN where nothing of it is seen.
      auto page_of = [&](const SpanSeg &s, int k) -> int32_t {
        const int t = s.st.token(k * kSpanTile + lane * box_rows);
        const bool seen = lane < boxes && t < s.st.hi && (t < s.st.sink || t + box_rows > s.st.lo);
        return seen ? a.kv.page_table[(int64_t)s.b * a.kv.max_pages + (t >> a.kv.log2_ps)] : INT32_MIN;
      };
      // K (w = 0) or V of the block's tile f, tile k of segment s.
      auto load_tile = [&](const SpanSeg &s, int k, int32_t pid, uint32_t f, int w) {
        const uint32_t slots = w ? NV : NK, slot = f % slots, full = (w ? v_full : k_full) + 8 * slot;
        ok = __all_sync(0xffffffffu, ok & mbar_wait((w ? v_empty : k_empty) + 8 * slot, ((f / slots) & 1) ^ 1, abort));
        if (!ok) return;
        const int t = s.st.token(k * kSpanTile + lane * box_rows);
        const bool page_ok = pid >= 0 && (int64_t)pid < a.kv.num_pages;
        if (w == 0 && pid != INT32_MIN && !page_ok) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
        const int row8 = page_ok ? (int)((((int64_t)pid * 2 * h_kv + (w ? h_kv : 0) + s.g) * ps + (t & (ps - 1))) >> 3) : oob;
        if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
        __syncwarp();
        if (lane < boxes)
          tma_load_4d(sbase + (w ? C::kV : C::kK) + slot * C::kTileBytes + (lane * box_rows >> 3) * C::kGroup, &kvmap, 0, 0, 0, row8, full, pol);
        __syncwarp();
      };
      uint32_t f = 0;
      if (warp == kSpanLoadV) {
        const SpanSeg *sp;
        for (int j = 0; ok && (sp = segment(j)); ++j) {
          const SpanSeg seg = *sp;
          release(j);
          int32_t pid = page_of(seg, seg.k0);
          for (int k = seg.k0; ok && k < seg.k1; ++k, ++f) {
            const int32_t next = k + 1 < seg.k1 ? page_of(seg, k + 1) : 0;
            load_tile(seg, k, pid, f, 1);
            pid = next;
          }
        }
        if (!ok) {  // every copy in flight lands before the block's memory is released
          volatile int never = 0;
          for (uint32_t i = f > (uint32_t)NV ? f - NV : 0; i < f; ++i) mbar_wait(v_full + 8 * (i % NV), (i / NV) & 1, &never, 200000000ll);
        }
      } else {
        SpanWalk walk(a, pl, pre, s_size, s_len, s_cnt);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) pl.cut_unit[blockIdx.x] = walk.inside ? walk.unit() : -1;
        uint32_t q_uses[2] = {0, 0};
        int j = 0;  // segments so far
        auto load_q = [&](const SpanSeg &s) {
#pragma unroll
          for (int w = 0; w < (WIDE ? 2 : 1); ++w) {
            const int buf = WIDE ? w : j & 1;
            if (WIDE && w && !second(s)) continue;
            ok = __all_sync(0xffffffffu, ok & mbar_wait(q_empty + 8 * buf, (q_uses[buf] & 1) ^ 1, abort));
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(q_full + 8 * buf, row_nodes * a.G * D * 2);
              for (int p = 0; p < C::kPanels; ++p)
                tma_load_4d(sbase + C::kQ + buf * C::kTileBytes + p * (kSpanTile * 128), &qmap, p * 64, s.g * a.G, s.rg * pl.nodes + w * row_nodes,
                            s.b, q_full + 8 * buf);
            }
            __syncwarp();
            ++q_uses[buf];
          }
          ++j;
        };
        // Publishes the next segment, nullptr behind the last one (and where a wait ran out).
        int published = 0;
        auto next_segment = [&]() -> const SpanSeg * {
          if (published >= kSpanRing) {
            ok = __all_sync(0xffffffffu, ok & mbar_wait(seg_empty + 8 * (published % kSpanRing), (published / kSpanRing & 1) ^ 1, abort));
            if (!ok) return nullptr;
          }
          SpanSeg x;
          const bool more = walk.next(x);
          SpanSeg *to = ring + published % kSpanRing;
          if (!more) x.b = -1;
          if (lane == 0) {
            *to = x;
            mbar_arrive(seg_full + 8 * (published % kSpanRing));
          }
          __syncwarp();
          ++published;
          return more ? to : nullptr;
        };
        const SpanSeg *seg = next_segment();
        int k = 0;
        int32_t pid = 0;
        if (seg) {
          k = seg->k0;
          pid = page_of(*seg, k);
          load_q(*seg);
        }
        while (seg && ok) {
          // What follows, its page ids on their way.
          const SpanSeg *ns = seg;
          int nk = k + 1;
          const bool turn = nk == seg->k1;
          if (turn) {
            load_tile(*seg, k, pid, f, 0);
            ns = next_segment();
            nk = ns ? ns->k0 : 0;
          }
          const int32_t npid = ns ? page_of(*ns, nk) : 0;
          if (!turn) load_tile(*seg, k, pid, f, 0);
          if (turn && ns) load_q(*ns);
          ++f;
          seg = ns;
          k = nk;
          pid = npid;
        }
        pdl_trigger();
        if (!ok) {
          volatile int never = 0;
          for (uint32_t i = f > (uint32_t)NK ? f - NK : 0; i < f; ++i) mbar_wait(k_full + 8 * (i % NK), (i / NK) & 1, &never, 200000000ll);
        }
      }
      __syncwarp();
    } else if (warp == kSpanMma || warp == kSpanMma + 1) {
      // ---------------------------------------------------------------- products
      // WIDE: warp 9 issues for both streams in turn, O += P V of a tile and at once S of the next, so that one stream's
      // softmax always has the other's products beside it (issued by two warps they fell into step, and the tensor cores idled
      // during both softmaxes).  Else a warp per stream, which waits for its own tiles only.
      const int mine = warp - kSpanMma;
      const uint32_t id_qk = idesc_bf16_f32(128, 128, 0, 0), id_pv = idesc_bf16_f32(128, D, 0, 1);
      // One elected lane of a converged warp issues, so that the operands stay warp-uniform: from a lane chosen by its number an
      // instruction took 95 clocks.
      const uint64_t qd = smem_desc(sbase + C::kQ, 16, 1024), kd = smem_desc(sbase + C::kK, 16, C::kGroup), vd = smem_desc(sbase + C::kV, 1024, C::kGroup);
      const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
      auto issue_qk = [&](int s, int buf, int slot, bool free_k, bool free_q) {
        const uint64_t q = qd + (uint64_t)(buf * C::kTileBytes >> 4), k = kd + (uint64_t)(slot * C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmu + s * 128, q + (uint64_t)(((kk >> 2) * (kSpanTile * 128) + (kk & 3) * 32) >> 4),
                        k + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_qk, kk > 0 ? 1u : 0u);
          mma_commit(s_full + 8 * s);
          if (free_k) mma_commit(k_empty + 8 * slot);
          if (free_q) mma_commit(q_empty + 8 * buf);
        }
        __syncwarp();
      };
      // O += P V of stream s's tile n, a half of the tokens as soon as its half of P is there.
      auto issue_pv = [&](int s, uint32_t n, int slot, bool first, bool free_v) {
        const uint64_t v = vd + (uint64_t)(slot * C::kTileBytes >> 4);
        const uint32_t acc = first ? 0u : 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mbar_wait(p_full + 16 * h + 8 * s, n & 1, abort);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_bf16_ts(tmu + C::kColO + s * 128, tmu + s * 128 + kk * 8, v + (uint64_t)((kk * 2 * C::kGroup) >> 4), id_pv, kk > 0 ? 1u : acc);
            if (h) {
              mma_commit(o_done + 8 * s);
              if (free_v) mma_commit(v_empty + 8 * slot);
            }
          }
          __syncwarp();
        }
      };
      // Rows of V that nobody sees may hold anything, and 0 times it has to be 0: the places from `end` on and those in [from, to).
      auto clear_unseen = [&](int end, int from, int to, int t0, int slot) {
        if (t0 + kSpanTile <= end && (t0 + kSpanTile <= from || t0 >= to || from >= to)) return;
        constexpr int CPR = D / 8;  // 16-byte pieces of a row
        char *v = sm + C::kV + slot * C::kTileBytes;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        auto rows = [&](int r0, int r1) {  // at most a group's
          const int c = lane % CPR;
#pragma unroll 1
          for (int r = r0 + lane / CPR; r < r1; r += 32 / CPR)
            *reinterpret_cast<uint4 *>(v + (r >> 3) * C::kGroup + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) = zero;
        };
        auto range = [&](int r0, int r1) {
          if (r0 >= r1) return;
          const int g0 = (r0 + 7) & ~7, g1 = r1 & ~7;
          if (g0 > g1) return rows(r0, r1);
          rows(r0, g0);
          uint4 *at = reinterpret_cast<uint4 *>(v + (g0 >> 3) * C::kGroup) + lane;  // whole groups lie together
          for (int g = g0; g < g1; g += 8, at += C::kGroup / 16)
#pragma unroll
            for (int e = 0; e < C::kGroup / 512; ++e) at[32 * e] = zero;
          rows(g1, r1);
        };
        range(max(0, end - t0), kSpanTile);
        range(max(0, from - t0), min(kSpanTile, to - t0));
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint32_t f = 0;  // tiles of the block
      if (WIDE && mine == 0) {
        uint32_t n[2] = {0, 0}, q_uses[2] = {0, 0};
        const SpanSeg *sp;
        for (int j = 0; (sp = segment(j)); ++j) {
          const SpanSeg seg = *sp;
          release(j);
          const int streams = second(seg) ? 2 : 1;
          mbar_wait(k_full + 8 * (f % NK), (f / NK) & 1, abort);
          for (int s = 0; s < streams; ++s) {
            mbar_wait(q_full + 8 * s, q_uses[s]++ & 1, abort);
            tc_fence_after();
            issue_qk(s, s, f % NK, s == streams - 1, seg.k1 - seg.k0 == 1);
          }
          for (int k = seg.k0; k < seg.k1; ++k, ++f) {
            const int slot = f % NV, nslot = (f + 1) % NK;
            mbar_wait(v_full + 8 * slot, (f / NV) & 1, abort);
            clear_unseen(seg.st.hi + seg.st.off, seg.st.sink, seg.st.lo + seg.st.off, k * kSpanTile, slot);
            for (int s = 0; s < streams; ++s) {
              issue_pv(s, n[s]++, slot, k == seg.k0, s == streams - 1);
              if (k + 1 < seg.k1) {
                if (s == 0) {
                  mbar_wait(k_full + 8 * nslot, ((f + 1) / NK) & 1, abort);
                  tc_fence_after();
                }
                issue_qk(s, s, nslot, s == streams - 1, k + 2 == seg.k1);
              }
            }
          }
        }
      }
      if (!WIDE) {
        const int s = mine;
        uint32_t n = 0;
        const SpanSeg *sp;
        for (int j = 0; (sp = segment(j)); ++j) {
          const SpanSeg seg = *sp;
          release(j);
          mbar_wait(q_full + 8 * (j & 1), (j >> 1) & 1, abort);
          bool first = true;
          for (int k = seg.k0; k < seg.k1; ++k, ++f) {
            if ((f & 1) != (uint32_t)s) continue;
            const int slot = f % NV;
            mbar_wait(k_full + 8 * (f % NK), (f / NK) & 1, abort);
            tc_fence_after();
            issue_qk(s, j & 1, f % NK, true, false);
            mbar_wait(v_full + 8 * slot, (f / NV) & 1, abort);
            clear_unseen(seg.st.hi + seg.st.off, seg.st.sink, seg.st.lo + seg.st.off, k * kSpanTile, slot);
            issue_pv(s, n++, slot, first, true);
            first = false;
          }
        }
      }
      if (elect_one()) mma_commit(drained + 8 * mine);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(drained + 8 * mine, 0, &never);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------------------------------------------------------- softmax, O
    // Rows that see nothing; a request's are shared by every B-th block.
    for (int b = blockIdx.x % B; b < B; b += gridDim.x) {
      int L, c;
      span_sizes(a, b, false, L, c);
      const int below = min(max(0, c - L), c);  // queries [0, below) and [c, n)
      const int rows = below + a.n - c, sharers = max(1, cdiv((int)gridDim.x - b, B));
      for (int64_t e = (blockIdx.x / B) * 256 + tid; e < (int64_t)rows * a.h_q * (D / 8); e += sharers * 256) {
        const int64_t r = e / (D / 8);
        const int i0 = (int)(r / a.h_q), i = i0 < below ? i0 : c + i0 - below;
        const int64_t at = ((int64_t)b * a.n + i) * a.h_q + r % a.h_q;
        reinterpret_cast<uint4 *>(a.out)[at * (D / 8) + e % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (a.lse && e % (D / 8) == 0) a.lse[at] = -INFINITY;
      }
    }
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t col_s = tm + s * 128 + lanes, col_o = tm + C::kColO + s * 128 + lanes;
    const int node = row / a.G;  // of the stream's tile
    uint32_t f = 0, n = 0, syncs = 0;
    // Arrive and wait of both streams' warps.
    auto sync_streams = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(group);
      mbar_wait(group, syncs++ & 1, abort);
    };
    const SpanSeg *sp;
    for (int j = 0; (sp = segment(j)); ++j) {
      const SpanSeg &seg = *sp;
      if (WIDE && s && !second(seg)) {
        release(j);
        continue;
      }
      const int i = seg.rg * pl.nodes + (WIDE ? s * row_nodes : 0) + node;
      const bool valid = node < row_nodes && i < seg.c && seg.st.base + i >= 0;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int64_t at = ((int64_t)seg.b * a.n + i) * a.h_q + seg.g * a.G + (row - node * a.G);
      const int64_t prow = (int64_t)seg.part * C::kRows + (WIDE ? s * 128 : 0) + row;
      const int32_t *parents = a.parents ? a.parents + (int64_t)seg.b * a.n : nullptr;
      // The places [all_from, all_to) and [0, sink) hold tokens that every row of the group sees.
      const int i_first = max(seg.rg * pl.nodes, -seg.st.base), i_last = min(seg.rg * pl.nodes + pl.nodes, seg.c) - 1;
      const int all_to = a.parents ? max(seg.st.base, 0) : seg.st.base + i_first + 1 + seg.st.off;
      const int all_from = a.parents ? 0 : max(0, seg.st.base + i_last - a.window + 1) + seg.st.off;
      float mref = -INFINITY, l = 0.f;
      bool have = false;  // O holds something
      for (int k = seg.k0; k < seg.k1; ++k, ++f) {
        if (!WIDE && (f & 1) != (uint32_t)s) continue;
        mbar_wait(s_full + 8 * s, n & 1, abort);
        tc_fence_after();
        if (warp_valid) {
          float x[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(col_s + 32 * q, x + 32 * q);
          tmem_ld_wait();
          const int t0 = k * kSpanTile, t1 = t0 + kSpanTile;  // places
          if (t1 > all_to || !(t0 >= all_from || t1 <= a.sink)) {
            uint32_t m[4] = {~0u, ~0u, ~0u, ~0u};  // (rows without a query: anything)
            if (valid) span_mask<4>(a, parents, seg.st.base, seg.st.off, i, t0, a.status, m);
#pragma unroll
            for (int w = 0; w < 4; ++w)  // (most words of a border's tile are whole for the warp)
              if (__any_sync(0xffffffffu, m[w] != 0xffffffffu)) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[32 * w + e] = (m[w] >> e & 1u) ? x[32 * w + e] : -INFINITY;
              }
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = x[q];
#pragma unroll
          for (int e = 4; e < 124; e += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = fmaxf(fmaxf(mx[q], x[e + q]), x[e + 4 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], x[124 + q]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
          const bool need = valid && top > mref + kSpanLazy;
          if (__any_sync(0xffffffffu, need)) {
            const float f2 = need ? fast_exp2(mref - top) : 1.f;
            if (have) {
              mbar_wait(o_done + 8 * s, (n - 1) & 1, abort);
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float o[32];
                tmem_ld32(col_o + 32 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f2;
                tmem_st32(col_o + 32 * q, o);
              }
            }
            l *= f2;
            if (need) mref = top;
          }
          const float ref = mref == -INFINITY ? 0.f : mref;
          const uint64_t sl2 = pack2(a.scale_log2, a.scale_log2), ref2 = pack2(-ref, -ref);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float y0, y1;
              unpack2(fma2(pack2(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), sl2, ref2), y0, y1);
              y0 = fast_exp2(y0);
              y1 = fast_exp2(y1);
              sum[e & 1] = add2(sum[e & 1], pack2(y0, y1));
              p[e] = pack_bf16(y0, y1);
            }
            tmem_st16(col_s + 16 * q, p);
            if (q == 1) {
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_full + 8 * s);
            }
          }
          float l0, l1;
          unpack2(add2(sum[0], sum[1]), l0, l1);
          l += l0 + l1;
          tmem_st_wait();
          tc_fence_before();
        } else if (lane == 0) {
          mbar_arrive(p_full + 8 * s);
        }
        have = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 + 8 * s);
        ++n;
      }
      // The segment's end.
      if (have) {
        mbar_wait(o_done + 8 * s, (n - 1) & 1, abort);
        tc_fence_after();
      }
      const bool part = seg.part >= 0;
      // Columns [c0, c0 + 16) of the row: to the output, or to the part's slot as [4 columns][row].
      auto put = [&](const float *o, int c0) {
        if (!valid) return;
        if (part) {
          float4 *to = reinterpret_cast<float4 *>(pl.o) + ((int64_t)seg.part * (D / 4) + c0 / 4) * C::kRows + (WIDE ? s * 128 : 0) + row;
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e * C::kRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + c0);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            to[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]), pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                               pack_bf16(o[8 * e + 6], o[8 * e + 7]));
        }
      };
      if constexpr (WIDE) {
        const float f = 1.f / l;
        if (warp_valid && part) {
#pragma unroll 2
          for (int q = 0; q < D / 32; ++q) {
            float o[32];
            tmem_ld32(col_o + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            put(o, 32 * q);
            put(o + 16, 32 * q + 16);
          }
        } else if (warp_valid) {
          // Eight lanes exchange 16-byte pieces of their rows so that a store covers 128 bytes of four rows (16 bytes of 32
          // rows took 7300 clocks a segment).
          const int mine = lane & 7;
          const unsigned good = __ballot_sync(0xffffffffu, valid);
          __nv_bfloat16 *rows[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) rows[k] = static_cast<__nv_bfloat16 *>(a.out) + __shfl_sync(0xffffffffu, at, (lane & 24) + k) * D + mine * 8;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 64) {
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float o[32];
              tmem_ld32(col_o + c0 + 32 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[4 * q + e] = make_uint4(pack_bf16(o[8 * e] * f, o[8 * e + 1] * f), pack_bf16(o[8 * e + 2] * f, o[8 * e + 3] * f),
                                          pack_bf16(o[8 * e + 4] * f, o[8 * e + 5] * f), pack_bf16(o[8 * e + 6] * f, o[8 * e + 7] * f));
            }
            span_transpose(v, mine);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (good >> ((lane & 24) + k) & 1) *reinterpret_cast<uint4 *>(rows[k] + c0) = v[k];
          }
        }
      } else {
        // Each stream ends half of the columns and passes its share of the others on through the segment's Q buffer, whose
        // products are done by then: in one step, or with more than 64 rows in two.
        float *boxes = reinterpret_cast<float *>(sm + C::kQ + (j & 1) * C::kTileBytes);
        s_m[s * 128 + row] = have ? mref : -INFINITY;
        s_m[256 + s * 128 + row] = have ? l : 0.f;
        sync_streams();
        const float m_two = s_m[(1 - s) * 128 + row], m = fmaxf(s_m[s * 128 + row], m_two), ref = m == -INFINITY ? 0.f : m;
        float f0 = have ? fast_exp2(mref - ref) : 0.f, f1 = fast_exp2(m_two - ref);
        l = (have ? l : 0.f) * f0 + s_m[256 + (1 - s) * 128 + row] * f1;
        mref = m;
        const float f = 1.f / l;
        f0 *= f, f1 *= f;
        auto end = [&](auto rows_of_box, auto steps) {
          constexpr int RB = decltype(rows_of_box)::value, STEPS = decltype(steps)::value, W = D / 2 / STEPS;
          float *mine = boxes + s * RB * W, *theirs = boxes + (1 - s) * RB * W;
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += W) {
            if (warp_valid) {
              float o[W];
              if (have) {
#pragma unroll
                for (int e = 0; e < W; e += 16) tmem_ld16(col_o + (1 - s) * (D / 2) + c0 + e, o + e);
                tmem_ld_wait();
              }
#pragma unroll
              for (int e = 0; e < W; ++e) mine[e * RB + row] = have ? o[e] : 0.f;
            }
            fence_proxy_async_smem();  // before the next queries' copies
            sync_streams();
            if (warp_valid)
#pragma unroll 1
              for (int e0 = 0; e0 < W; e0 += 16) {
                float o[16];
                if (have) {
                  tmem_ld16(col_o + s * (D / 2) + c0 + e0, o);
                  tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = (have ? o[e] * f0 : 0.f) + theirs[(e0 + e) * RB + row] * f1;
                put(o, s * (D / 2) + c0 + e0);
              }
            if (STEPS > 1) sync_streams();
          }
        };
        if (row_nodes * a.G <= 64)
          end(SpanInt<64>{}, SpanInt<1>{});
        else
          end(SpanInt<128>{}, SpanInt<2>{});
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + 8 * (j & 1));
      }
      if (valid && (WIDE || s == 0)) {
        const float lse2 = mref + log2f(l);
        if (part)
          pl.lse[prow] = lse2;
        else if (a.lse)
          a.lse[at] = lse2 * kLn2;
      }
      tc_fence_before();
      release(j);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && s_abort) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
  if (warp == kSpanMma) tmem_dealloc(tm, 512);
}

// Joins the parts of the units that blocks share: weights 2^(lse - max) over their sum.  Blocks (block, 32 rows; a warp per
// D / 8 columns): the one of the first that begins inside a unit has that unit; its parts are slot 1 of the block before and
// slot 0 of every block that begins inside it.  What bounds it: latency, three loads that wait for one another, and its launch:
// 2 to 4 us of a call.  (The last block to arrive joining the parts in the attention kernel took 47 us where this takes 43.)
template <int D, bool WIDE>
__global__ void __launch_bounds__(256) span_join_kernel(SpanArgs a, SpanPlan pl) {
  using C = SpanCfg<D, WIDE>;
  constexpr int COLS = D / 8, U = 4;  // columns of a warp, parts in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x, r = blockIdx.y * 32 + lane;
  pdl_wait();
  pdl_trigger();
  // Lane i: what block first - 1 + i begins inside.
  const int seen = first - 1 + lane, cut = seen >= 0 && seen < pl.blocks ? pl.cut_unit[seen] : -1;
  const int unit = __shfl_sync(0xffffffffu, cut, 1);
  if (unit < 0 || __shfl_sync(0xffffffffu, cut, 0) == unit) return;
  unsigned others = ~(__ballot_sync(0xffffffffu, cut == unit) | 1u);
  int parts = others ? __ffs(others) - 1 : 32;
  for (int t0 = first + 31; !others; t0 += 32) {
    others = ~__ballot_sync(0xffffffffu, t0 + lane < pl.blocks && pl.cut_unit[t0 + lane] == unit);
    parts += others ? __ffs(others) - 1 : 32;
  }
  const int rg = unit % pl.n_groups, bg = unit / pl.n_groups, b = bg / a.kv.h_kv, g = bg % a.kv.h_kv;
  int L, c;
  span_sizes(a, b, false, L, c);
  const int s = r >> 7, node = (r & 127) / a.G, i = rg * pl.nodes + s * pl.row_nodes + node;
  float m = -INFINITY, z = 0.f, o[COLS] = {};
  for (int k0 = 0; k0 < parts; k0 += U) {
    float lse[U];
    float4 v[U][COLS / 4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t slot = (int64_t)(first - 1 + k0 + k) * 2 + (k0 + k == 0);
      lse[k] = -INFINITY;
      if (k0 + k >= parts) continue;
      lse[k] = pl.lse[slot * C::kRows + r];
      const float4 *src = reinterpret_cast<const float4 *>(pl.o) + (slot * (D / 4) + warp * (COLS / 4)) * C::kRows + r;
#pragma unroll
      for (int e = 0; e < COLS / 4; ++e) v[k][e] = src[e * C::kRows];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < U; ++k) top = fmaxf(top, lse[k]);
    const float ref = top == -INFINITY ? 0.f : top, f = fast_exp2(m - ref);
    m = top;
    z *= f;
#pragma unroll
    for (int e = 0; e < COLS; ++e) o[e] *= f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float w = fast_exp2(lse[k] - ref);
      if (w == 0.f) continue;  // a part that this row sees nothing of left no O
      z += w;
#pragma unroll
      for (int e = 0; e < COLS / 4; ++e) {
        o[4 * e] = fmaf(w, v[k][e].x, o[4 * e]), o[4 * e + 1] = fmaf(w, v[k][e].y, o[4 * e + 1]);
        o[4 * e + 2] = fmaf(w, v[k][e].z, o[4 * e + 2]), o[4 * e + 3] = fmaf(w, v[k][e].w, o[4 * e + 3]);
      }
    }
  }
  if (node >= pl.row_nodes || i >= c || L - c + i < 0) return;
  const int64_t at = ((int64_t)b * a.n + i) * a.h_q + g * a.G + ((r & 127) - node * a.G);
  const float f = 1.f / z;
  uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + warp * COLS);
#pragma unroll
  for (int e = 0; e < COLS / 8; ++e)
    dst[e] = make_uint4(pack_bf16(o[8 * e] * f, o[8 * e + 1] * f), pack_bf16(o[8 * e + 2] * f, o[8 * e + 3] * f),
                        pack_bf16(o[8 * e + 4] * f, o[8 * e + 5] * f), pack_bf16(o[8 * e + 6] * f, o[8 * e + 7] * f));
  if (a.lse && warp == 0) a.lse[at] = (m + log2f(z)) * kLn2;
}

// ------------------------------------------------------------------------------------------------
// Host side.
// ------------------------------------------------------------------------------------------------

// The driver's tensor-map encoder, looked up once; nullptr where it has none.
static decltype(&cuTensorMapEncodeTiled) span_encoder() {
  static decltype(&cuTensorMapEncodeTiled) const found = [] {
    void *at = nullptr;
    cudaDriverEntryPointQueryResult how = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &how) != cudaSuccess) cudaGetLastError();
    return how == cudaDriverEntryPointSuccess ? reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(at) : nullptr;
  }();
  return found;
}

bool span_tc_takes(const ssd_paged_kv *kv) {
  return kv->dtype == SSD_DTYPE_BF16 && kv->page_size >= 8 && kv->h_kv <= 4096 && (int64_t)kv->num_pages * 2 * kv->h_kv * kv->page_size / 8 < (int64_t)1 << 31;
}

static bool span_wide(const SpanArgs &a) { return a.n > kSpanTile / a.G; }

// Tiles of a unit's group, at most.
static int64_t span_most_tiles(const ssd_paged_kv *kv, const SpanArgs &a, const SpanPlan &p) {
  const int64_t all = cdiv(kv->max_seq_len, kSpanTile), most = cdiv64((int64_t)a.sink + a.window + p.nodes + 2 * p.box, kSpanTile);
  return all < most ? all : most;
}

static SpanPlan span_plan(const ssd_paged_kv *kv, const SpanArgs &a) {
  SpanPlan p = {};
  const int streams = span_wide(a) ? 2 : 1;
  p.row_nodes = a.n < kSpanTile / a.G ? a.n : kSpanTile / a.G;
  p.nodes = streams * p.row_nodes;
  p.n_groups = cdiv(a.n, p.nodes);
  p.blocks = sm_count();
  p.least = span_wide(a) ? kSpanLeastWide : kSpanLeast;
  p.box = kv->page_size < 16 ? kv->page_size : 16;
  const int64_t unit = span_most_tiles(kv, a, p) + kSpanOverhead, units = (int64_t)kv->batch * kv->h_kv * p.n_groups;
  const int64_t share = units * unit / p.blocks, longest = cdiv64(units, p.blocks) * unit;
  p.split = unit - kSpanOverhead > kSpanWhole || longest > (share > p.least ? share : p.least) + kSpanJoin;
  return p;
}

static size_t span_carve(const ssd_paged_kv *kv, SpanPlan &p, bool wide, void *ws) {
  Carver c(ws);
  c.take<char>(kCounterBytes);
  const size_t rows = (size_t)p.blocks * 2 * (wide ? 256 : 128);
  p.cut_unit = c.take<int32_t>(p.blocks);
  p.o = c.take<float>(rows * kv->d);
  p.lse = c.take<float>(rows);
  return c.off;
}

size_t span_tc_workspace(const ssd_paged_kv *kv, const SpanArgs &a) {
  SpanPlan p = span_plan(kv, a);
  return span_carve(kv, p, span_wide(a), nullptr);
}

template <int D, bool WIDE>
static int span_tc_launch(const CUtensorMap &kvmap, const CUtensorMap &qmap, const SpanArgs &a, const SpanPlan &p, cudaStream_t st) {
  constexpr auto kernel = span_tc_kernel<D, WIDE>;
  constexpr int smem = SpanCfg<D, WIDE>::kSmem;
  static_assert(smem <= 227 * 1024, "a block's shared memory");
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  if ((rc = launch(kernel, dim3(p.blocks), dim3(kSpanThreads), smem, st, "span_tc_kernel", kvmap, qmap, a, p)) || !p.split) return rc;
  const int rows = (WIDE ? 128 : 0) + p.row_nodes * a.G;  // (stream 1's behind 128 of stream 0's)
  return launch(span_join_kernel<D, WIDE>, dim3(p.blocks, cdiv(rows, 32)), dim3(256), 0, st, "span_join_kernel", a, p);
}

int span_tc(const ssd_paged_kv *kv, const SpanArgs &args, void *workspace, cudaStream_t st) {
  const auto enc = span_encoder();
  if (!enc) return fail(SSD_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const bool wide = span_wide(args);
  const int d = kv->d, panels = d / 64;
  SpanPlan p = span_plan(kv, args);
  span_carve(kv, p, wide, workspace);
  // K / V rows as (64 columns, row of 8, panel, group of 8 rows): a box lands as [group][panel][8 rows x 128 B].
  CUtensorMap kvmap, qmap;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)panels, (cuuint64_t)kv->num_pages * 2 * kv->h_kv * kv->page_size / 8};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, 128, (cuuint64_t)d * 16};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)panels, (cuuint32_t)p.box / 8};
  CUresult r = enc(&kvmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(kv->pool), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SSD_ERR_CUDA, "cuTensorMapEncodeTiled (KV pool) failed (%d)", (int)r);
  // Requests of a launch: their sizes fit shared memory, and their costs 31 bits.
  const int64_t one = kv->h_kv * p.n_groups * (span_most_tiles(kv, args, p) + kSpanOverhead);
  if (one >= (int64_t)1 << 31) return fail(SSD_ERR_UNSUPPORTED, "span attention: %d queries of %d heads over %d tokens", args.n, args.h_q, kv->max_seq_len);
  const int slice = (int)(((int64_t)1 << 31) / (one + 1) < kSpanMaxBatch ? ((int64_t)1 << 31) / (one + 1) : kSpanMaxBatch);
  for (int b0 = 0; b0 < kv->batch; b0 += slice) {
    SpanArgs a = args;
    a.kv.batch = kv->batch - b0 < slice ? kv->batch - b0 : slice;
    a.kv.page_table += (int64_t)b0 * kv->max_pages;
    a.kv.seq_lens += b0;
    const int64_t rows = (int64_t)b0 * a.n * a.h_q;
    a.q = static_cast<const char *>(a.q) + rows * d * 2;
    a.out = static_cast<char *>(a.out) + rows * d * 2;
    if (a.lse) a.lse += rows;
    if (a.parents) a.parents += (int64_t)b0 * a.n;
    if (a.counts) a.counts += b0;
    // Queries [B][n][h_q][d]: a box holds a panel of the group's heads of a stream's queries; queries past n read as zeros.
    const cuuint64_t qdims[4] = {(cuuint64_t)d, (cuuint64_t)a.h_q, (cuuint64_t)a.n, (cuuint64_t)a.kv.batch};
    const cuuint64_t qstrides[3] = {(cuuint64_t)d * 2, (cuuint64_t)a.h_q * d * 2, (cuuint64_t)a.n * a.h_q * d * 2};
    const cuuint32_t qbox[4] = {64, (cuuint32_t)a.G, (cuuint32_t)p.row_nodes, 1};
    r = enc(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(a.q), qdims, qstrides, qbox, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SSD_ERR_CUDA, "cuTensorMapEncodeTiled (queries) failed (%d)", (int)r);
    const int rc = d == 128 ? (wide ? span_tc_launch<128, true>(kvmap, qmap, a, p, st) : span_tc_launch<128, false>(kvmap, qmap, a, p, st))
                            : (wide ? span_tc_launch<64, true>(kvmap, qmap, a, p, st) : span_tc_launch<64, false>(kvmap, qmap, a, p, st));
    if (rc) return rc;
  }
  return SSD_OK;
}

}  // namespace ssd
