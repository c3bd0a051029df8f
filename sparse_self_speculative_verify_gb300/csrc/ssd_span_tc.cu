// ssd_span_tc.cu -- span attention over bf16 caches on the 5th-generation tensor cores (tcgen05, TMA, tensor memory).
//
// Up to 128 query rows of a (request, KV head) are the M side of both products, a row per lane of tensor memory:
//   S [128 rows x 128 tokens] = Q K^T      (both from shared memory)
//   O [128 rows x D]         += P V        (P from tensor memory, in the place of S; V as it lies, token-major)
// so that a row's softmax belongs to one thread.  A block runs two such streams, which take turns on the tensor cores: while
// one's softmax runs, the other's products do.
//   WIDE (more than 128 rows): the streams are two tiles of rows and share every tile of K and V;
//   else both streams have the same rows and take K / V tiles in turn, their O joined at a segment's end.
// Roles: warps 0-3 and 4-7 the softmax of a stream (and its O), warp 8 loads (one TMA box per page, 128-byte swizzle),
// warps 9 and 10 issue a stream's products.
//
// Work.  A unit is one (request, KV head); its rows are split into n_groups groups of one block's rows.  n_groups blocks
// form a team, one group each, that walks the same tokens side by side, so that K and V come from memory once and from L2
// for the others.  The units' tiles lie end to end and are cut into equal shares, one per team; a cut close to a unit's
// border moves there.  A unit that several teams share leaves partial results, joined by span_join_kernel.  Where there
// are many units with few tiles each (prompts with a window), blocks take whole (unit, group) items instead.
#include "ssd_sm100.cuh"
#include "ssd_span.h"
#include "ssd_tma.h"

namespace ssd {
using namespace sm100;

constexpr int kSpanTile = 128;          // tokens of a tile, rows of a stream
constexpr int kSpanThreads = 11 * 32;
constexpr int kSpanProducer = 8, kSpanMma = 9;
constexpr int kSpanMaxBatch = 1024;     // requests of a launch (their sizes lie in shared memory)
constexpr int kSpanOverhead = 1;        // what starting and ending a unit costs, in tiles
constexpr int kSpanSnap = 3;            // a cut this close to a unit's border moves there
constexpr int kSpanMinShare = 4;        // least share of a team
constexpr float kSpanLazy = 8.f;        // a row's reference moves when a score exceeds it by this (log2)

struct SpanPlan {
  int n_groups, nodes;   // row groups of a unit, queries of a group
  int teams;             // 0: items
  int64_t items;
  int32_t *cut_unit;     // [teams]: the unit that team t's share begins inside of, or -1
  float *o, *lse;        // [teams][2][n_groups][rows of a block][D], ... (log2)
};

template <int D, bool WIDE>
struct SpanCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kSpanTile * D * 2;
  static constexpr int kGroup = 1024 * kPanels;  // bytes of 8 tokens: panel after panel of 8 x 128 bytes
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes, kMisc = kV + kStages * kTileBytes;
  static constexpr int kBars = 4 * kStages + 16;
  // barriers, the requests' prefix, length, queries and tiles, the streams' maxima and sums
  static constexpr int kSmem = kMisc + kBars * 8 + (kSpanMaxBatch + 1) * 8 + 3 * kSpanMaxBatch * 4 + 4 * 128 * 4 + 1024;
  static constexpr int kRows = WIDE ? 256 : 128;
  static constexpr int kColO = 256;  // tensor memory: S (P) of the streams, O of the streams
};

struct SpanSeg {
  int b, g, rg;       // request, KV head, row group
  int k0, k1;         // tiles of the unit
  int part;           // -1: the whole unit; else the slot of its results
  SpanTiles st;
  int L, c;
};

// The segments of a block, in order; every role walks them by itself.
struct SpanWalk {
  const SpanArgs &a;
  const SpanPlan &pl;
  const int64_t *pre;
  const int *len, *cnt, *tiles;
  int64_t pos, end, start, item;
  int b, team;

  __device__ SpanWalk(const SpanArgs &a_, const SpanPlan &p_, const int64_t *pre_, const int *len_, const int *cnt_, const int *tiles_)
      : a(a_), pl(p_), pre(pre_), len(len_), cnt(cnt_), tiles(tiles_), b(0) {
    item = blockIdx.x;
    team = pl.teams ? blockIdx.x / pl.n_groups : 0;
    if (pl.teams) {
      start = pos = cut(team);
      end = cut(team + 1);
      if (pos < end) b = find(pos);
    }
  }
  // The request that position x < pre[batch] lies in.
  __device__ int find(int64_t x) {
    int lo = 0, hi = a.kv.batch;  // pre[lo] <= x < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
  // Where team t's share begins.
  __device__ int64_t cut(int t) {
    const int64_t total = pre[a.kv.batch];
    const int64_t n = min((int64_t)pl.teams, max((int64_t)1, total / kSpanMinShare));
    if (t >= n) return total;
    if (total == 0) return 0;
    const int64_t x = total * t / n;
    const int lo = find(x);
    const unsigned size = tiles[lo] + kSpanOverhead, off = (unsigned)(x - pre[lo]) % size;
    if (off < kSpanSnap) return x - off;
    return size - off < kSpanSnap ? x - off + size : x;
  }
  // The unit that the share begins inside of, or -1.
  __device__ int begins_inside() {
    if (start >= pre[a.kv.batch]) return -1;
    const int at = find(start);
    const unsigned size = tiles[at] + kSpanOverhead, off = (unsigned)(start - pre[at]);
    return off % size ? at * a.kv.h_kv + (int)(off / size) : -1;
  }
  __device__ void fill(SpanSeg &s) {
    s.L = len[s.b];
    s.c = cnt[s.b];
    s.st = span_tiles<kSpanTile>(a, s.L, s.c, s.rg * pl.nodes, s.rg * pl.nodes + pl.nodes - 1);
  }
  __device__ bool next(SpanSeg &s) {
    if (!pl.teams) {
      if (item >= pl.items) return false;
      const int64_t bg = item / pl.n_groups;
      s.rg = pl.n_groups - 1 - (int)(item - bg * pl.n_groups);  // the last queries see most
      s.b = (int)(bg / a.kv.h_kv);
      s.g = (int)(bg - (int64_t)s.b * a.kv.h_kv);
      item += gridDim.x;
      fill(s);
      s.k0 = 0;
      s.k1 = s.st.n_tiles;
      s.part = -1;
      return true;
    }
    if (pos >= end) return false;
    while (pre[b + 1] <= pos) ++b;
    const unsigned size = tiles[b] + kSpanOverhead, rem = (unsigned)(pos - pre[b]);
    s.b = b;
    s.g = (int)(rem / size);
    s.rg = blockIdx.x % pl.n_groups;
    const int64_t u0 = pre[b] + (int64_t)s.g * size, u1 = u0 + size, stop = min(u1, end);
    fill(s);
    s.k0 = min(max(0, (int)(pos - u0) - kSpanOverhead), s.st.n_tiles);
    s.k1 = stop == u1 ? s.st.n_tiles : min(max(0, (int)(stop - u0) - kSpanOverhead), s.st.n_tiles);
    s.part = pos == u0 && stop == u1 ? -1 : (team * 2 + (pos == u0)) * pl.n_groups + s.rg;
    pos = stop;
    return true;
  }
};

// D columns of 32 of a lane of O, times f, to dst.
template <int D, typename T>
__device__ __forceinline__ void span_store32(T *dst, const float *v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      *reinterpret_cast<uint4 *>(dst + i) = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]), pack_bf16(v[i + 4], v[i + 5]),
                                                       pack_bf16(v[i + 6], v[i + 7]));
  }
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kSpanThreads, 1)
    span_tc_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap, SpanArgs a, SpanPlan pl) {
  using C = SpanCfg<D, WIDE>;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) char smem_raw[];
  char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.kv.batch, h_kv = a.kv.h_kv, ps = a.kv.page_size;

  // K and V slots' full / empty, Q buffers' full / empty, the streams' S full, P full, O done, drain
  const uint32_t bars = sbase + C::kMisc;
  const uint32_t k_full = bars, k_empty = k_full + 8 * NS, v_full = k_empty + 8 * NS, v_empty = v_full + 8 * NS;
  const uint32_t q_full = v_empty + 8 * NS, q_empty = q_full + 16, s_full = q_empty + 16, p_full = s_full + 16, o_done = p_full + 16,
                 drained = o_done + 16;
  int64_t *pre = reinterpret_cast<int64_t *>(sm + C::kMisc + C::kBars * 8);
  int *s_len = reinterpret_cast<int *>(pre + kSpanMaxBatch + 1), *s_cnt = s_len + kSpanMaxBatch, *s_tiles = s_cnt + kSpanMaxBatch;
  float *s_m = reinterpret_cast<float *>(s_tiles + kSpanMaxBatch), *s_l = s_m + 256;  // [stream][row]
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int64_t s_scan[kSpanThreads / 32];

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full + 8 * i, 1), mbar_init(v_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, WIDE ? 2 : 1), mbar_init(v_empty + 8 * i, WIDE ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1), mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1), mbar_init(p_full + 8 * i, 4), mbar_init(o_done + 8 * i, 1), mbar_init(drained + 8 * i, 1);
    }
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

  // Sizes of the requests, and the prefix of their units' costs.
  {
    constexpr int CH = cdiv(kSpanMaxBatch, kSpanThreads);
    int64_t mine[CH], sum = 0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int b = tid * CH + k;
      mine[k] = 0;
      if (b < B) {
        int L, c;
        span_sizes(a, b, blockIdx.x == 0, L, c);
        int most = 0;
        if (pl.teams)
          for (int rg = 0; rg < pl.n_groups; ++rg)
            most = max(most, span_tiles<kSpanTile>(a, L, c, rg * pl.nodes, rg * pl.nodes + pl.nodes - 1).n_tiles);
        s_len[b] = L, s_cnt[b] = c, s_tiles[b] = most;
        mine[k] = most ? (int64_t)h_kv * (most + kSpanOverhead) : 0;
      }
      sum += mine[k];
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t off = incl - sum;
    for (int w = 0; w < warp; ++w) off += s_scan[w];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int b = tid * CH + k;
      if (b < B) pre[b] = off;
      off += mine[k];
      if (b == B - 1) pre[B] = off;
    }
    __syncthreads();
  }
  const uint32_t tm = s_tmem;
  volatile int *abort = &s_abort;

  // Rows that see nothing.
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    const int c = s_cnt[b], below = min(max(0, c - s_len[b]), c);  // queries [0, below) and [c, n)
    const int rows = below + a.n - c;
    for (int64_t e = tid; e < (int64_t)rows * a.h_q * (D / 8); e += kSpanThreads) {
      const int64_t r = e / (D / 8);
      const int i0 = (int)(r / a.h_q), i = i0 < below ? i0 : c + i0 - below;
      const int64_t at = ((int64_t)b * a.n + i) * a.h_q + r % a.h_q;
      reinterpret_cast<uint4 *>(a.out)[at * (D / 8) + e % (D / 8)] = make_uint4(0, 0, 0, 0);
      if (a.lse && e % (D / 8) == 0) a.lse[at] = -INFINITY;
    }
  }

  SpanWalk walk(a, pl, pre, s_len, s_cnt, s_tiles);
  SpanSeg seg;
  const int row_nodes = kSpanTile / a.G;  // queries of a stream's tile

  if (warp == kSpanProducer) {
    // ---------------------------------------------------------------- loads
    if (pl.teams && blockIdx.x % pl.n_groups == 0) {
      const int u = walk.begins_inside();
      if (lane == 0) pl.cut_unit[walk.team] = u;
    }
    const int box_rows = min(ps, kSpanTile), boxes = kSpanTile / box_rows;
    const uint64_t pol = pl.teams && pl.n_groups == 1 ? policy_evict_first() : policy_evict_normal();
    const int oob = (int)((int64_t)a.kv.num_pages * 2 * h_kv * ps / 8);
    uint32_t f = 0;  // tiles so far
    int j = 0;       // segments so far
    auto next_seg = [&](SpanSeg &s) {  // the next one with tiles
      for (;;) {
        if (!walk.next(s)) return false;
        if (s.k0 < s.k1) return true;
      }
    };
    // The group of 8 rows that lane's box of tile k starts at (K), or where nothing of it is seen `oob`.
    auto page_of = [&](const SpanSeg &s, int k) -> int32_t {
      const int t = s.st.tile(k) * kSpanTile + lane * box_rows;
      const bool seen = lane < boxes && t < s.st.hi && (t < s.st.sink || t + box_rows > s.st.lo);
      return seen ? a.kv.page_table[(int64_t)s.b * a.kv.max_pages + (t >> a.kv.log2_ps)] : INT32_MIN;
    };
    bool more = next_seg(seg);
    int k = seg.k0;
    int32_t pid = more ? page_of(seg, k) : 0;
    bool ok = true;
    while (more && ok) {
      if (k == seg.k0) {
        const int i0 = seg.rg * pl.nodes;
#pragma unroll
        for (int s = 0; s < (WIDE ? 2 : 1); ++s) {
          const int buf = WIDE ? s : j & 1, use = WIDE ? j : j >> 1;
          ok &= mbar_wait(q_empty + 8 * buf, (use & 1) ^ 1, abort);
          if (__all_sync(0xffffffffu, ok) && lane == 0) {
            mbar_arrive_expect_tx(q_full + 8 * buf, row_nodes * a.G * D * 2);
            for (int p = 0; p < C::kPanels; ++p)
              tma_load_4d(sbase + C::kQ + buf * C::kTileBytes + p * (kSpanTile * 128), &qmap, p * 64, seg.g * a.G, i0 + s * row_nodes, seg.b,
                          q_full + 8 * buf);
          }
          __syncwarp();
        }
        ++j;
      }
      // What follows, its page ids on their way.
      SpanSeg ns = seg;
      int nk = k + 1;
      bool nmore = true;
      if (nk == seg.k1) {
        nmore = next_seg(ns);
        nk = ns.k0;
      }
      const int32_t npid = nmore ? page_of(ns, nk) : 0;
      const int t = seg.st.tile(k) * kSpanTile + lane * box_rows;
      const bool page_ok = pid >= 0 && (int64_t)pid < a.kv.num_pages;
      if (pid != INT32_MIN && !page_ok) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
      const int row8 = page_ok ? (int)((((int64_t)pid * 2 * h_kv + seg.g) * ps + (t & (ps - 1))) >> 3) : oob;
      const int slot = f % NS;
      const uint32_t use = f / NS;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t full = (w ? v_full : k_full) + 8 * slot;
        ok &= mbar_wait((w ? v_empty : k_empty) + 8 * slot, (use & 1) ^ 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
          __syncwarp();
          if (lane < boxes)
            tma_load_4d(sbase + (w ? C::kV : C::kK) + slot * C::kTileBytes + (lane * box_rows >> 3) * C::kGroup, &kvmap, 0, 0, 0,
                        page_ok ? row8 + (w ? h_kv * ps >> 3 : 0) : oob, full, pol);
          __syncwarp();
        }
      }
      ++f;
      seg = ns;
      k = nk;
      pid = npid;
      more = nmore;
    }
    pdl_trigger();
    if (!ok && lane == 0) {  // every copy in flight lands before the block's memory is released
      volatile int never = 0;
      for (uint32_t i = f > (uint32_t)NS ? f - NS : 0; i < f; ++i) {
        mbar_wait(k_full + 8 * (i % NS), (i / NS) & 1, &never, 200000000ll);
        mbar_wait(v_full + 8 * (i % NS), (i / NS) & 1, &never, 200000000ll);
      }
    }
    __syncwarp();
  } else if (warp >= kSpanMma) {
    // ---------------------------------------------------------------- products
    const int s = warp - kSpanMma;
    const uint32_t id_qk = idesc_bf16_f32(128, 128, 0, 0), id_pv = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t col_s = tm + s * 128, col_o = tm + C::kColO + s * 128;
    uint32_t f = 0, n = 0;  // tiles of the block, of this stream
    int j = 0;
    while (walk.next(seg)) {
      if (seg.k0 >= seg.k1) continue;
      const int buf = WIDE ? s : j & 1, use = WIDE ? j : j >> 1;
      mbar_wait(q_full + 8 * buf, use & 1, abort);
      const uint64_t qd = smem_desc(sbase + C::kQ + buf * C::kTileBytes, 16, 1024);
      bool first = true;
      for (int k = seg.k0; k < seg.k1; ++k, ++f) {
        if (!WIDE && (f & 1) != (uint32_t)s) continue;
        const int slot = f % NS;
        const uint32_t ph = (f / NS) & 1;
        mbar_wait(k_full + 8 * slot, ph, abort);
        tc_fence_after();
        if (lane == 0 && !*abort) {
          const uint64_t kd = smem_desc(sbase + C::kK + slot * C::kTileBytes, 16, C::kGroup);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(col_s, qd + (uint64_t)(((kk >> 2) * (kSpanTile * 128) + (kk & 3) * 32) >> 4),
                        kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_qk, kk > 0);
          mma_commit(s_full + 8 * s);
          mma_commit(k_empty + 8 * slot);
          if (WIDE && k == seg.k1 - 1) mma_commit(q_empty + 8 * s);
        }
        __syncwarp();
        mbar_wait(v_full + 8 * slot, ph, abort);
        // Rows of V that nobody sees may hold anything, and 0 times it has to be 0.
        const int t0 = seg.st.tile(k) * kSpanTile, t1 = t0 + kSpanTile;
        if (t1 > seg.st.hi || !(t1 <= seg.st.sink || t0 >= seg.st.lo || seg.st.sink >= seg.st.lo)) {
          constexpr int CPR = D / 8;  // 16-byte pieces of a row
          for (int r = lane / CPR; r < kSpanTile; r += 32 / CPR) {
            const int c = lane % CPR;
            if (!seg.st.seen(t0 + r))
              *reinterpret_cast<uint4 *>(sm + C::kV + slot * C::kTileBytes + (r >> 3) * C::kGroup + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        mbar_wait(p_full + 8 * s, n & 1, abort);
        tc_fence_after();
        if (lane == 0 && !*abort) {
          const uint64_t vd = smem_desc(sbase + C::kV + slot * C::kTileBytes, 1024, C::kGroup);
#pragma unroll
          for (int kk = 0; kk < kSpanTile / 16; ++kk)
            mma_bf16_ts(col_o, col_s + kk * 8, vd + (uint64_t)((kk * 2 * C::kGroup) >> 4), id_pv, !first || kk > 0);
          mma_commit(o_done + 8 * s);
          mma_commit(v_empty + 8 * slot);
        }
        __syncwarp();
        first = false;
        ++n;
      }
      ++j;
    }
    if (lane == 0) {
      mma_commit(drained + 8 * s);
      volatile int never = 0;
      mbar_wait(drained + 8 * s, 0, &never);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax, O
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t col_s = tm + s * 128 + lanes, col_o = tm + C::kColO + s * 128 + lanes;
    const int node = row / a.G;  // of the stream's tile
    uint32_t f = 0, n = 0;
    int j = 0;
    while (walk.next(seg)) {
      const int i = seg.rg * pl.nodes + (WIDE ? s * row_nodes : 0) + node;
      const bool valid = node < row_nodes && i < seg.c && seg.st.base + i >= 0;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int64_t at = ((int64_t)seg.b * a.n + i) * a.h_q + seg.g * a.G + (row - node * a.G);
      const int64_t prow = (int64_t)seg.part * C::kRows + (WIDE ? s * 128 : 0) + row;
      if (seg.k0 >= seg.k1) {
        if (seg.part >= 0 && valid && (WIDE || s == 0)) pl.lse[prow] = -INFINITY;
        continue;
      }
      const int32_t *parents = a.parents ? a.parents + (int64_t)seg.b * a.n : nullptr;
      // Tokens [0, all_to) and, behind lo_all, up to it are seen by every row of the group.
      const int i_first = max(seg.rg * pl.nodes, -seg.st.base), i_last = min(seg.rg * pl.nodes + pl.nodes, seg.c) - 1;
      const int all_to = a.parents ? max(seg.st.base, 0) : seg.st.base + i_first + 1;
      const int all_from = a.parents ? 0 : max(0, seg.st.base + i_last - a.window + 1);
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
          const int t0 = seg.st.tile(k) * kSpanTile, t1 = t0 + kSpanTile;
          if (t1 > all_to || !(t0 >= all_from || t1 <= a.sink)) {
            uint32_t m[4] = {0u, 0u, 0u, 0u};
            if (valid) span_mask<4>(a, parents, seg.st.base, i, t0, a.status, m);
#pragma unroll
            for (int e = 0; e < 128; ++e) x[e] = (m[e >> 5] >> (e & 31) & 1u) ? x[e] : -INFINITY;
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = x[q];
#pragma unroll
          for (int e = 4; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], x[e]);
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
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 128; ++e) {
            x[e] = fast_exp2(fmaf(x[e], a.scale_log2, -ref));
            sum[e & 3] += x[e];
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = __uint_as_float(pack_bf16(x[64 * q + 2 * e], x[64 * q + 2 * e + 1]));
            tmem_st32(col_s + 32 * q, p);
          }
          tmem_st_wait();
        }
        have = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * s);
        ++n;
      }
      // The segment's end.
      if (have) {
        mbar_wait(o_done + 8 * s, (n - 1) & 1, abort);
        tc_fence_after();
      }
      float scale = 1.f, lse2;
      if constexpr (!WIDE) {
        s_m[s * 128 + row] = have ? mref : -INFINITY;
        s_l[s * 128 + row] = have ? l : 0.f;
        named_sync(1, 256);
        const float m0 = s_m[row], m1 = s_m[128 + row], m = fmaxf(m0, m1), ref = m == -INFINITY ? 0.f : m;
        const float f0 = fast_exp2(m0 - ref), f1 = fast_exp2(m1 - ref);
        l = s_l[row] * f0 + s_l[128 + row] * f1;
        scale = s ? f1 : f0;
        mref = m;
      }
      lse2 = mref + log2f(l);
      scale *= 1.f / l;
      const bool part = seg.part >= 0;
      if constexpr (WIDE) {
        if (warp_valid) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            float o[32];
            tmem_ld32(col_o + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= scale;
            if (valid && part) span_store32<D>(pl.o + prow * D + 32 * q, o);
            if (valid && !part) span_store32<D>(static_cast<__nv_bfloat16 *>(a.out) + at * D + 32 * q, o);
          }
        }
      } else {
        // Stream 1's share goes through the segment's Q buffer, whose products are done, half of the columns at a time.
        float *box = reinterpret_cast<float *>(sm + C::kQ + (j & 1) * C::kTileBytes);
#pragma unroll 1
        for (int hcol = 0; hcol < D; hcol += D / 2) {
          if (s == 1 && warp_valid) {
#pragma unroll 1
            for (int q = 0; q < D / 64; ++q) {
              float o[32];
              tmem_ld32(col_o + hcol + 32 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) box[(32 * q + e) * 128 + row] = have ? o[e] * scale : 0.f;
            }
            fence_proxy_async_smem();  // before the next queries' copies
          }
          named_sync(1, 256);
          if (s == 0 && warp_valid) {
#pragma unroll 1
            for (int q = 0; q < D / 64; ++q) {
              float o[32];
              tmem_ld32(col_o + hcol + 32 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = (have ? o[e] * scale : 0.f) + box[(32 * q + e) * 128 + row];
              if (valid && part) span_store32<D>(pl.o + prow * D + hcol + 32 * q, o);
              if (valid && !part) span_store32<D>(static_cast<__nv_bfloat16 *>(a.out) + at * D + hcol + 32 * q, o);
            }
          }
          named_sync(1, 256);
        }
        if (tid == 0) mbar_arrive(q_empty + 8 * (j & 1));
      }
      if (valid && (WIDE || s == 0)) {
        if (part)
          pl.lse[prow] = lse2;
        else if (a.lse)
          a.lse[at] = lse2 * kLn2;
      }
      tc_fence_before();
      ++j;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && s_abort) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
  if (warp == kSpanMma) tmem_dealloc(tm, 512);
}

// Joins the parts of the units that teams share.  Blocks (team, group, eight rows): the one of the first team that begins inside
// a unit has that unit; its parts are the team before's slot 1 and slot 0 of every team that begins inside it.
template <int D, bool WIDE>
__global__ void __launch_bounds__(256) span_join_kernel(SpanArgs a, SpanPlan pl) {
  using C = SpanCfg<D, WIDE>;
  const int lane = threadIdx.x & 31, team = blockIdx.x, rg = blockIdx.y, r = blockIdx.z * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const int unit = pl.cut_unit[team];
  if (unit < 0 || (team > 0 && pl.cut_unit[team - 1] == unit)) return;
  int parts = 1;  // the team before's, and those that follow
  for (int t0 = team;; t0 += 32) {
    const bool same = t0 + lane < pl.teams && pl.cut_unit[t0 + lane] == unit;
    const unsigned m = __ballot_sync(0xffffffffu, same);
    parts += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
    if (m != 0xffffffffu) break;
  }
  const int b = unit / a.kv.h_kv, g = unit % a.kv.h_kv;
  int L, c;
  span_sizes(a, b, false, L, c);
  const int row_nodes = kSpanTile / a.G, s = r >> 7, node = (r & 127) / a.G;
  const int i = rg * pl.nodes + s * row_nodes + node;
  if (node >= row_nodes || i >= c || i >= (rg + 1) * pl.nodes || L - c + i < 0) return;
  const int64_t at = ((int64_t)b * a.n + i) * a.h_q + g * a.G + ((r & 127) - node * a.G);
  auto row_of = [&](int k) { return ((int64_t)(k ? (team + k - 1) * 2 : (team - 1) * 2 + 1) * pl.n_groups + rg) * C::kRows + r; };
  float m = -INFINITY;
  for (int k = lane; k < parts; k += 32) m = fmaxf(m, pl.lse[row_of(k)]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  constexpr int PER = D / 32;
  float o[PER] = {}, z = 0.f;
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const float w = k0 + lane < parts ? fast_exp2(pl.lse[row_of(k0 + lane)] - ref) : 0.f;
    z += w;
    const int n = min(32, parts - k0);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      if (wk == 0.f) continue;  // a part without tiles left no O
      const float *src = pl.o + row_of(k0 + k) * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        o[0] = fmaf(wk, v.x, o[0]), o[1] = fmaf(wk, v.y, o[1]), o[2] = fmaf(wk, v.z, o[2]), o[3] = fmaf(wk, v.w, o[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] = fmaf(wk, v.x, o[0]), o[1] = fmaf(wk, v.y, o[1]);
      }
    }
  }
  z = warp_sum(z);
  const float f = 1.f / z;
  uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + lane * PER);
  if constexpr (PER == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
  else
    *dst = pack_bf16(o[0] * f, o[1] * f);
  if (a.lse && lane == 0) a.lse[at] = (m + log2f(z)) * kLn2;
}

// ------------------------------------------------------------------------------------------------
// Host side.
// ------------------------------------------------------------------------------------------------

bool span_tc_takes(const ssd_paged_kv *kv) {
  return kv->dtype == SSD_DTYPE_BF16 && kv->page_size >= 8 && kv->h_kv <= 4096 && (int64_t)kv->num_pages * 2 * kv->h_kv * kv->page_size / 8 < (int64_t)1 << 31;
}

static bool span_wide(const SpanArgs &a) { return a.n > kSpanTile / a.G; }

static SpanPlan span_plan(const ssd_paged_kv *kv, const SpanArgs &a) {
  SpanPlan p = {};
  p.nodes = (span_wide(a) ? 2 : 1) * (kSpanTile / a.G);
  p.n_groups = cdiv(a.n, p.nodes);
  const int sms = sm_count(), batch = kv->batch < kSpanMaxBatch ? kv->batch : kSpanMaxBatch;
  p.items = (int64_t)batch * kv->h_kv * p.n_groups;
  // Shares while the units would not fill the SMs about twice, and for trees, whose units are long; teams have to fit.
  const bool shares = p.n_groups <= sms && (a.parents || a.window == kSpanAll || p.n_groups == 1 || p.items < 2 * sms);
  p.teams = shares ? sms / p.n_groups : 0;
  return p;
}

static size_t span_carve(const ssd_paged_kv *kv, SpanPlan &p, bool wide, void *ws) {
  Carver c(ws);
  c.take<char>(kCounterBytes);
  if (p.teams) {
    const size_t rows = (size_t)p.teams * 2 * p.n_groups * (wide ? 256 : 128);
    p.cut_unit = c.take<int32_t>(p.teams);
    p.o = c.take<float>(rows * kv->d);
    p.lse = c.take<float>(rows);
  }
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
  const int64_t items = (int64_t)a.kv.batch * a.kv.h_kv * p.n_groups;
  const int grid = p.teams ? p.teams * p.n_groups : (int)(items < sm_count() ? items : sm_count());
  if ((rc = launch(kernel, dim3(grid), dim3(kSpanThreads), smem, st, "span_tc_kernel", kvmap, qmap, a, p)) || p.teams < 2) return rc;
  const int rows = WIDE ? 256 : a.n * a.G;
  return launch(span_join_kernel<D, WIDE>, dim3(p.teams, p.n_groups, cdiv(rows, 8)), dim3(256), 0, st, "span_join_kernel", a, p);
}

int span_tc(const ssd_paged_kv *kv, const SpanArgs &args, void *workspace, cudaStream_t st) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(SSD_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const bool wide = span_wide(args);
  const int d = kv->d, panels = d / 64, box_rows = kv->page_size < kSpanTile ? kv->page_size : kSpanTile;
  SpanPlan p = span_plan(kv, args);
  span_carve(kv, p, wide, workspace);
  // K / V rows as (64 columns, row of 8, panel, group of 8 rows): a box lands as [group][panel][8 rows x 128 B].
  CUtensorMap kvmap, qmap;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)panels, (cuuint64_t)kv->num_pages * 2 * kv->h_kv * kv->page_size / 8};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, 128, (cuuint64_t)d * 16};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)panels, (cuuint32_t)box_rows / 8};
  CUresult r = enc(&kvmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(kv->pool), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SSD_ERR_CUDA, "cuTensorMapEncodeTiled (KV pool) failed (%d)", (int)r);
  for (int b0 = 0; b0 < kv->batch; b0 += kSpanMaxBatch) {
    SpanArgs a = args;
    a.kv.batch = kv->batch - b0 < kSpanMaxBatch ? kv->batch - b0 : kSpanMaxBatch;
    a.kv.page_table += (int64_t)b0 * kv->max_pages;
    a.kv.seq_lens += b0;
    const int64_t rows = (int64_t)b0 * a.n * a.h_q;
    a.q = static_cast<const char *>(a.q) + rows * d * 2;
    a.out = static_cast<char *>(a.out) + rows * d * 2;
    if (a.lse) a.lse += rows;
    if (a.parents) a.parents += (int64_t)b0 * a.n;
    if (a.counts) a.counts += b0;
    p.items = (int64_t)a.kv.batch * kv->h_kv * p.n_groups;
    // Queries [B][n][h_q][d]: a box holds a panel of the group's heads of a stream's queries; queries past n read as zeros.
    const cuuint64_t qdims[4] = {(cuuint64_t)d, (cuuint64_t)a.h_q, (cuuint64_t)a.n, (cuuint64_t)a.kv.batch};
    const cuuint64_t qstrides[3] = {(cuuint64_t)d * 2, (cuuint64_t)a.h_q * d * 2, (cuuint64_t)a.n * a.h_q * d * 2};
    const cuuint32_t qbox[4] = {64, (cuuint32_t)a.G, (cuuint32_t)(kSpanTile / a.G), 1};
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
