// ssd_pages.cu -- pages of a paged cache shared, taken, given back and compacted on the device.
//
// The only state beside a cache's page table and lengths is one reference count per page: a page is free
// when its count is 0, and taking a page always takes the lowest free index, so the outcome of every call
// is a function of its inputs.  The calls move whole rows of bytes and work on 16-, 32- and 4-bit caches.
//
// SpecSA ("SpecSA：融合推测解码与稀疏注意力的高效LLM推理框架"), "branch handling": branches of a request
// share the KV of their common tokens.  SparseSpec §4.1: the tokens a verify selects are the ones kept.
#include "ssd_cache.h"
#include "ssd_kv4.cuh"

#include <type_traits>

namespace ssd {

// A row of bytes per (page, K|V, head, token): `wide` bytes at slot * wide of the block and, for a 4-bit
// cache, `thin` bytes behind all the wide parts.
struct RowShape {
  int wide, thin;
};
static RowShape row_shape(const ssd_paged_kv *kv) {
  if (kv->dtype == SSD_DTYPE_NVFP4) return {kv4_code_bytes(kv->d), kv4_scale_bytes(kv->d)};
  return {kv->d * (kv->dtype == SSD_DTYPE_BF16 ? 2 : 4), 0};
}

// ---- fork -----------------------------------------------------------------------------------
constexpr int kForkThreads = 256;

// One block per pair.  dst's row becomes a copy of the first ceil(L / page_size) entries of src's.  Pairs
// of one call must not touch each other's rows: whatever a pair reads no other pair writes.
__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(KVView kv, int32_t *table, int32_t *seq_lens, int32_t *refs,
                                                               const int32_t *src, const int32_t *dst, int n,
                                                               unsigned *status) {
  const int i = blockIdx.x, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int s = src[i], d = dst[i];
  bool ok = s >= 0 && s < kv.batch && d >= 0 && d < kv.batch;
  for (int j = tid; j < n && ok; j += kForkThreads) ok = dst[j] != s && !(j < i && dst[j] == d);
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(status, (unsigned)SSD_FAULT_INDEX);
    return;
  }
  const int L = seq_lens[s];
  if (L < 0 || L > kv.max_seq_len) {
    if (tid == 0) atomicOr(status, (unsigned)SSD_FAULT_SEQLEN);
    return;
  }
  const int np = (L + kv.page_size - 1) >> kv.log2_ps;
  const int32_t *from = table + (int64_t)s * kv.max_pages;
  int32_t *to = table + (int64_t)d * kv.max_pages;
  // Every page of src held by somebody, and dst's row empty.  Four entries in flight per thread: the loads'
  // latency is what the call costs (448 rows of up to 1024 pages: 10 us with one).
  constexpr int U = 4;
  for (int j0 = tid; j0 < kv.max_pages; j0 += U * kForkThreads) {
    int32_t p[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * kForkThreads;
      p[k] = j < np ? from[j] : 0;
      if (j < kv.max_pages) ok &= to[j] < 0;
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (j0 + k * kForkThreads < np) ok &= p[k] >= 0 && (int64_t)p[k] < kv.num_pages && refs[p[k]] > 0;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(status, (unsigned)SSD_FAULT_PAGE);
    return;
  }
  for (int j0 = tid; j0 < np; j0 += U * kForkThreads) {
    int32_t p[U];
#pragma unroll
    for (int k = 0; k < U; ++k) p[k] = j0 + k * kForkThreads < np ? from[j0 + k * kForkThreads] : -1;
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (p[k] >= 0) to[j0 + k * kForkThreads] = p[k], atomicAdd(refs + p[k], 1);
  }
  if (tid == 0) seq_lens[d] = L;
}

// ---- release --------------------------------------------------------------------------------
constexpr int kReleaseThreads = 256;

// One block per request: entries behind the kept tokens leave the row, and their pages lose a holder.
__global__ void __launch_bounds__(kReleaseThreads) kv_release_kernel(KVView kv, int32_t *table, int32_t *seq_lens,
                                                                     int32_t *refs, const int32_t *keep, unsigned *status) {
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int k = keep[b];
  if (k < 0) return;
  int32_t *row = table + (int64_t)b * kv.max_pages;
  for (int64_t j = ((int64_t)k + kv.page_size - 1) / kv.page_size + tid; j < kv.max_pages; j += kReleaseThreads) {
    const int32_t p = row[j];
    if (p < 0) continue;
    row[j] = -1;
    // A count never goes below 0, whatever the table says.
    if ((int64_t)p >= kv.num_pages) {
      atomicOr(status, (unsigned)SSD_FAULT_PAGE);
    } else if (atomicSub(refs + p, 1) <= 0) {
      atomicAdd(refs + p, 1);
      atomicOr(status, (unsigned)SSD_FAULT_PAGE);
    }
  }
  if (tid == 0) {
    const int L = seq_lens[b];
    if (L < 0 || L > kv.max_seq_len)
      atomicOr(status, (unsigned)SSD_FAULT_SEQLEN);
    else if (k < L)
      seq_lens[b] = k;
  }
}

// ---- reserve --------------------------------------------------------------------------------
constexpr int kResThreads = 1024;
constexpr int kResFew = 4;  // up to so many affected pages a request has a thread, above a warp

// Per page of the pool, valid for the pages that requests of the call hold and ask for.
struct PageAsk {
  int refs;    // its count before the call
  int asked;   // requests of the call that hold it and want to write it
  int lowest;  // the first of them
  int pad;
};
struct ReserveArgs {
  KVView kv;
  int32_t *table;
  int32_t *refs;
  const int32_t *counts;
  PageAsk *ask;     // [num_pages]
  int4 *row;        // [batch]: {first affected page index, their number (-1: request skipped), pages to take, sum of those before}
  int32_t *fresh;   // [num_pages]: the free pages handed out, ascending
  int4 *copies;     // [batch]: {old page, new page, live slots, 0}; slots 0: nothing to copy
  unsigned *status;
};

// Inclusive sum of v over the block's threads in order; s_warp: 32 values.  total: the block's.  64 bits: the pages that
// a table's rows ask for may be more than 2^31.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int64_t base = warp ? s_warp[warp - 1] : 0;
  total = s_warp[31];
  __syncthreads();
  return base + inc;
}

// One block.  A request needs a page for every page index that its tokens L .. L + n - 1 touch: where it has
// none, and where it holds one together with others.  If all holders of a page ask, the first of them keeps
// it.  Phases, with the whole block in step: what is asked of every page; how many new pages a request
// needs; the first free pages of the pool; hand them out.  If they do not suffice nothing is changed.
// LPR lanes share a request: bound by the latency of a dozen dependent loads, so a thread per request
// (all requests at once) where they need a page or two, a warp for long prompts.
template <int LPR>
__device__ __forceinline__ void reserve_rows(const ReserveArgs &a, int64_t *s_warp) {
  const int tid = threadIdx.x, gl = tid % LPR, grp = tid / LPR;
  constexpr int kGroups = kResThreads / LPR;
  const KVView &kv = a.kv;
  const unsigned gmask = LPR == 32 ? 0xffffffffu : 1u << (tid & 31);
  // Whether a request can be served at all, and its pages' counts before the call.
  for (int b = grp; b < kv.batch; b += kGroups) {
    const int4 r = a.row[b];
    const int32_t *row = a.table + (int64_t)b * kv.max_pages;
    bool ok = true;
    for (int i = gl; i < r.y; i += LPR) {
      const int32_t p = row[r.x + i];
      if (p < 0) {
        ok &= !(i == 0 && r.z);  // the page of live tokens is missing
      } else if ((int64_t)p >= kv.num_pages) {
        ok = false;
      } else {
        const int rc = a.refs[p];
        ok &= rc > 0;
        a.ask[p] = PageAsk{rc, 0, 0x7fffffff, 0};
      }
    }
    if (LPR > 1) ok = __all_sync(gmask, ok);
    if (!ok && gl == 0) {
      atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
      a.row[b].y = -1;
    }
  }
  __syncthreads();
  // Who asks for a page that it shares.
  for (int b = grp; b < kv.batch; b += kGroups) {
    const int4 r = a.row[b];
    const int32_t *row = a.table + (int64_t)b * kv.max_pages;
    for (int i = gl; i < r.y; i += LPR) {
      const int32_t p = row[r.x + i];
      if (p < 0 || a.ask[p].refs == 1) continue;
      atomicAdd(&a.ask[p].asked, 1);
      atomicMin(&a.ask[p].lowest, b);
    }
  }
  __syncthreads();
  auto takes = [&](int b, int32_t p) {
    if (p < 0) return true;
    const PageAsk k = a.ask[p];
    return !(k.refs == 1 || (k.asked == k.refs && k.lowest == b));
  };
  for (int b = grp; b < kv.batch; b += kGroups) {
    const int4 r = a.row[b];
    const int32_t *row = a.table + (int64_t)b * kv.max_pages;
    int c = 0;
    for (int i = gl; i < r.y; i += LPR) c += takes(b, row[r.x + i]);
    if (LPR > 1) c = __reduce_add_sync(gmask, c);
    if (gl == 0) {
      a.row[b].z = c;
      a.copies[b] = make_int4(0, 0, 0, 0);
    }
  }
  __syncthreads();
  // Sums over the requests, in their order.
  int64_t total = 0;
  for (int b0 = 0; b0 < kv.batch; b0 += kResThreads) {
    const int b = b0 + tid, v = b < kv.batch ? a.row[b].z : 0;
    int64_t part;
    const int64_t inc = block_scan(v, s_warp, part);
    if (b < kv.batch) a.row[b].w = (int)(total + inc - v);  // read only where the total is at most num_pages
    total += part;
  }
  if (total > kv.num_pages) {  // whatever the counts say
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_NOPAGE);
    return;
  }
  // The first `total` free pages, 16 counts a thread and step.
  int64_t found = 0;
  const bool vec = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  for (int64_t p0 = 0; p0 < kv.num_pages && found < total; p0 += kResThreads * 16) {
    const int64_t p = p0 + tid * 16;
    unsigned free = 0;
    if (vec && p + 16 <= kv.num_pages) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int4 v = *reinterpret_cast<const int4 *>(a.refs + p + 4 * k);
        free |= (unsigned)((v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3) << (4 * k);
      }
    } else {
      for (int k = 0; k < 16; ++k)
        if (p + k < kv.num_pages && a.refs[p + k] == 0) free |= 1u << k;
    }
    const int mine = __popc(free);
    int64_t part;
    int64_t at = found + block_scan(mine, s_warp, part) - mine;
    for (; free && at < total; free &= free - 1) a.fresh[at++] = (int32_t)(p + __ffs(free) - 1);
    found += part;
  }
  __syncthreads();
  if (found < total) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_NOPAGE);
    return;
  }
  for (int b = grp; b < kv.batch; b += kGroups) {
    const int4 r = a.row[b];
    if (r.z == 0) continue;
    int32_t *row = a.table + (int64_t)b * kv.max_pages;
    const int live = kv.seq_lens[b] & (kv.page_size - 1);
    int at = r.w;
    for (int i0 = 0; i0 < r.y; i0 += LPR) {
      const int i = i0 + gl;
      const int32_t p = i < r.y ? row[r.x + i] : -1;
      const bool t = i < r.y && takes(b, p);
      const unsigned m = LPR > 1 ? __ballot_sync(gmask, t) : (unsigned)t;
      if (t) {
        const int32_t f = a.fresh[at + (LPR > 1 ? __popc(m & ((1u << gl) - 1)) : 0)];
        row[r.x + i] = f;
        a.refs[f] = 1;
        if (p >= 0) {
          atomicSub(a.refs + p, 1);
          if (i == 0 && live) a.copies[b] = make_int4(p, f, live, 0);
        }
      }
      at += __popc(m);
    }
  }
}

__global__ void __launch_bounds__(kResThreads) kv_reserve_kernel(ReserveArgs a) {
  __shared__ int64_t s_warp[32];
  pdl_wait();
  bool many = false;
  for (int b = threadIdx.x; b < a.kv.batch; b += kResThreads) {
    const int L = a.kv.seq_lens[b], n = a.counts[b];
    int4 r = make_int4(0, 0, 0, 0);
    if (L < 0 || n < 0 || (int64_t)L + n > a.kv.max_seq_len) {
      atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    } else if (n > 0) {
      r.x = L >> a.kv.log2_ps;
      r.y = ((L + n - 1) >> a.kv.log2_ps) + 1 - r.x;
      r.z = L & (a.kv.page_size - 1);
    }
    many |= r.y > kResFew;
    a.row[b] = r;
  }
  if (__syncthreads_or(many))
    reserve_rows<32>(a, s_warp);
  else
    reserve_rows<1>(a, s_warp);
}

constexpr int kMoveThreads = 256;
constexpr int kMoveParts = kMoveThreads / 32;

// The live slots of shared last pages into the pages that replace them.  Block (x, b): parts (K or V of a head)
// [8 x, 8 x + 8) of row b, a warp each, so that hundreds of rows are one wave of blocks.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(char *pool, const int4 *copies, int page_size, int h_kv,
                                                               RowShape rs) {
  pdl_trigger();
  pdl_wait();
  const int4 c = copies[blockIdx.y];
  const int part = blockIdx.x * kMoveParts + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c.z == 0 || part >= 2 * h_kv) return;
  const int64_t block_bytes = (int64_t)page_size * (rs.wide + rs.thin);
  const char *src = pool + ((int64_t)c.x * 2 * h_kv + part) * block_bytes;
  char *dst = pool + ((int64_t)c.y * 2 * h_kv + part) * block_bytes;
  constexpr int U = 4;  // pieces in flight per thread
  const int n = c.z * (rs.wide / 16);  // (up to 2^24 tokens of 512 bytes)
#pragma unroll 1
  for (int e0 = lane; e0 < n; e0 += 32 * U) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (e0 + 32 * k < n) v[k] = reinterpret_cast<const uint4 *>(src)[e0 + 32 * k];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (e0 + 32 * k < n) reinterpret_cast<uint4 *>(dst)[e0 + 32 * k] = v[k];
  }
  const int64_t thin0 = (int64_t)page_size * rs.wide;
  for (int e = lane; e < c.z * rs.thin / 4; e += 32)
    reinterpret_cast<uint32_t *>(dst + thin0)[e] = reinterpret_cast<const uint32_t *>(src + thin0)[e];
}

// ---- compact --------------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactTokens = kCompactThreads;  // list entries per block at most

struct CompactArgs {
  KVView from, to;
  char *to_pool;
  int32_t *to_lens;
  const int32_t *to_refs;
  const int32_t *src, *dst, *idx, *cnt;
  int n, k_max, tokens;  // tokens: list entries per block
  bool same;  // one cache, or two with the same lengths: a row read must not be one that is written
  RowShape rs;
  unsigned *status;
};

// Block (x, g, i): list entries [x * a.tokens, ...) of head g of pair i.  Addresses first, one entry per thread,
// then 16-byte pieces of the rows.  What a block needs before its first row is loaded in two steps (all that hangs on
// i alone, then lengths and page ids).
//
// Bound: HBM, in the 64 bytes it moves at a time.  A 4-bit row of 72 bytes lies in two places and costs two such
// pieces: 8 lists of 13107 out of 131072 tokens, 8 heads, take 71 us for 438 MB of traffic (0.91 of the measured
// rate) where the rows alone are 242 MB; 32 lists of 410 bf16 rows 12.2 us for 67 MB (0.81).
__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(CompactArgs a) {
  const int i = blockIdx.z, g = blockIdx.y, j0 = blockIdx.x * a.tokens, tid = threadIdx.x, j = j0 + tid;
  const int h = a.from.h_kv;
  __shared__ int64_t s_from[kCompactTokens], s_to[kCompactTokens];  // K block of the entry, or -1
  __shared__ int s_slots[kCompactTokens];
  pdl_trigger();
  pdl_wait();
  const bool entry = tid < a.tokens && j < a.k_max;
  const int t = entry ? a.idx[((int64_t)i * h + g) * a.k_max + j] : -1;
  const int s = a.src[i], d = a.dst[i], count = a.cnt[(int64_t)i * h];
  bool same_count = count >= 0 && count <= a.k_max;
  for (int k = tid; k < h; k += kCompactThreads) same_count &= a.cnt[(int64_t)i * h + k] == count;
  bool ok = s >= 0 && s < a.from.batch && d >= 0 && d < a.to.batch;
  for (int k = tid; k < a.n && ok; k += kCompactThreads) ok = !(k < i && a.dst[k] == d) && !(a.same && a.src[k] == d);
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
    return;
  }
  if (!__syncthreads_and(same_count)) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_KMAX);
    return;
  }
  const int nj = min(a.tokens, count - j0);
  const bool mine = tid < nj && count <= a.to.max_seq_len, in_table = mine && t >= 0 && t < a.from.max_seq_len;
  const int L = a.from.seq_lens[s];
  const int32_t pf = in_table ? a.from.page_table[(int64_t)s * a.from.max_pages + (t >> a.from.log2_ps)] : -1;
  const int32_t pt = mine ? a.to.page_table[(int64_t)d * a.to.max_pages + (j >> a.to.log2_ps)] : -1;
  if (L < 0 || L > a.from.max_seq_len || count > a.to.max_seq_len) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    return;
  }
  if (tid == 0 && j0 == 0 && g == 0) a.to_lens[d] = count;
  const int64_t fb = (int64_t)a.from.page_size * (a.rs.wide + a.rs.thin), tb = (int64_t)a.to.page_size * (a.rs.wide + a.rs.thin);
  if (mine) {
    int64_t f = -1, to = -1;
    if (t < 0 || t >= L)
      atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
    else if (pf < 0 || (int64_t)pf >= a.from.num_pages)
      atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
    else
      f = ((int64_t)pf * 2 * h + g) * fb;
    if (pt < 0 || (int64_t)pt >= a.to.num_pages || (a.to_refs && a.to_refs[pt] != 1))
      atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
    else
      to = ((int64_t)pt * 2 * h + g) * tb;
    s_from[tid] = f, s_to[tid] = to;
    s_slots[tid] = t & (a.from.page_size - 1);
  }
  __syncthreads();
  // Pieces of 16 bytes, four loads on their way per thread; then a 4-bit cache's scales in words.
  const char *from = static_cast<const char *>(a.from.pool);
  const int64_t fv = h * fb, tv = h * tb;
  auto copy = [&](auto *tag, int width, int64_t at_from, int64_t at_to) {
    using V = typename std::remove_pointer<decltype(tag)>::type;
    const int sh = 31 - __clz(width / (int)sizeof(V));  // log2 of the pieces of a row (widths are powers of two)
    const int total = nj << (sh + 1);
    constexpr int U = 4;
    for (int e0 = tid; e0 < total; e0 += U * kCompactThreads) {
      V v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int e = e0 + k * kCompactThreads, c = e & ((1 << sh) - 1), which = (e >> sh) & 1, j = e >> (sh + 1);
        v[k] = V{};
        if (e < total && s_from[j] >= 0) v[k] = reinterpret_cast<const V *>(from + s_from[j] + (which ? fv : 0) + at_from + (int64_t)s_slots[j] * width)[c];
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int e = e0 + k * kCompactThreads, c = e & ((1 << sh) - 1), which = (e >> sh) & 1, j = e >> (sh + 1);
        if (e < total && s_to[j] >= 0)
          reinterpret_cast<V *>(a.to_pool + s_to[j] + (which ? tv : 0) + at_to + (int64_t)((j0 + j) & (a.to.page_size - 1)) * width)[c] = v[k];
      }
    }
  };
  copy(static_cast<uint4 *>(nullptr), a.rs.wide, 0, 0);
  if (a.rs.thin) copy(static_cast<uint32_t *>(nullptr), a.rs.thin, (int64_t)a.from.page_size * a.rs.wide, (int64_t)a.to.page_size * a.rs.wide);
}

static int page_checks(const ssd_paged_kv *kv, KVView *v, const int32_t *refs, const char *who) {
  int rc = validate_cache(kv, v, who, kCache16Or32 | kCacheNvfp4);
  if (rc) return rc;
  if (!refs) return fail(SSD_ERR_INVALID_ARG, "%s: page_refs must be non-NULL", who);
  if (kv->num_pages > 0x7fffffff) return fail(SSD_ERR_UNSUPPORTED, "%s: num_pages above 2^31 - 1", who);
  return SSD_OK;
}

}  // namespace ssd

using namespace ssd;

extern "C" int ssd_kv_fork(const ssd_paged_kv *kv, int32_t *page_refs, const int32_t *src, const int32_t *dst, int n,
                           ssd_stream_t stream) {
  const char *who = "ssd_kv_fork";
  KVView v;
  int rc = page_checks(kv, &v, page_refs, who);
  if (rc) return rc;
  if (n < 0) return fail(SSD_ERR_INVALID_ARG, "%s: n %d < 0", who, n);
  if (n == 0) return SSD_OK;
  if (!src || !dst) return fail(SSD_ERR_INVALID_ARG, "%s: src and dst must be non-NULL", who);
  unsigned *status = device_status();
  if (!status) return SSD_ERR_CUDA;
  return launch(kv_fork_kernel, dim3(n), dim3(kForkThreads), 0, reinterpret_cast<cudaStream_t>(stream), "kv_fork_kernel", v,
                const_cast<int32_t *>(kv->page_table), const_cast<int32_t *>(kv->seq_lens), page_refs, src, dst, n, status);
}

extern "C" int ssd_kv_release(const ssd_paged_kv *kv, int32_t *page_refs, const int32_t *keep, ssd_stream_t stream) {
  const char *who = "ssd_kv_release";
  KVView v;
  int rc = page_checks(kv, &v, page_refs, who);
  if (rc) return rc;
  if (kv->batch == 0) return SSD_OK;
  if (!keep) return fail(SSD_ERR_INVALID_ARG, "%s: keep must be non-NULL", who);
  unsigned *status = device_status();
  if (!status) return SSD_ERR_CUDA;
  return launch(kv_release_kernel, dim3(kv->batch), dim3(kReleaseThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                "kv_release_kernel", v, const_cast<int32_t *>(kv->page_table), const_cast<int32_t *>(kv->seq_lens), page_refs,
                keep, status);
}

static size_t reserve_layout(const ssd_paged_kv *kv, ReserveArgs *a, void *ws) {
  Carver c(ws);
  c.off = kCounterBytes;
  PageAsk *ask = c.take<PageAsk>((size_t)kv->num_pages);
  int32_t *fresh = c.take<int32_t>((size_t)kv->num_pages);
  int4 *copies = c.take<int4>((size_t)kv->batch);
  int4 *row = c.take<int4>((size_t)kv->batch);
  if (a) a->ask = ask, a->fresh = fresh, a->copies = copies, a->row = row;
  return c.off;
}

extern "C" size_t ssd_kv_reserve_workspace_bytes(const ssd_paged_kv *kv) {
  if (!kv || kv->num_pages <= 0 || kv->batch < 0) return 0;
  return reserve_layout(kv, nullptr, nullptr);
}

extern "C" int ssd_kv_reserve(const ssd_paged_kv *kv, int32_t *page_refs, const int32_t *counts, void *workspace,
                              size_t workspace_bytes, ssd_stream_t stream) {
  const char *who = "ssd_kv_reserve";
  ReserveArgs a{};
  int rc = page_checks(kv, &a.kv, page_refs, who);
  if (rc) return rc;
  if (kv->batch > 65535) return fail(SSD_ERR_UNSUPPORTED, "%s: batch above 65535", who);
  if (!counts && kv->batch > 0) return fail(SSD_ERR_INVALID_ARG, "%s: counts must be non-NULL", who);
  const size_t need = ssd_kv_reserve_workspace_bytes(kv);
  if (!workspace || workspace_bytes < need)
    return fail(SSD_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", who, workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(SSD_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  if (kv->batch == 0) return SSD_OK;
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  reserve_layout(kv, &a, workspace);
  a.table = const_cast<int32_t *>(kv->page_table);
  a.refs = page_refs;
  a.counts = counts;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((rc = launch(kv_reserve_kernel, dim3(1), dim3(kResThreads), 0, st, "kv_reserve_kernel", a))) return rc;
  return launch(kv_move_kernel, dim3(cdiv(2 * kv->h_kv, kMoveParts), kv->batch), dim3(kMoveThreads), 0, st, "kv_move_kernel",
                static_cast<char *>(const_cast<void *>(kv->pool)), a.copies, kv->page_size, kv->h_kv, row_shape(kv));
}

extern "C" int ssd_kv_compact(const ssd_paged_kv *kv, const ssd_paged_kv *to, const int32_t *to_refs, const int32_t *src,
                              const int32_t *dst, int n, const int32_t *idx, int k_max, const int32_t *cnt,
                              ssd_stream_t stream) {
  const char *who = "ssd_kv_compact";
  CompactArgs a{};
  int rc = validate_cache(kv, &a.from, who, kCache16Or32 | kCacheNvfp4);
  if (rc || (rc = validate_cache(to, &a.to, who, kCache16Or32 | kCacheNvfp4))) return rc;
  if (kv->dtype != to->dtype || kv->h_kv != to->h_kv || kv->d != to->d)
    return fail(SSD_ERR_INVALID_ARG, "%s: the two caches differ in dtype, h_kv or d", who);
  if (n < 0 || k_max < 0) return fail(SSD_ERR_INVALID_ARG, "%s: n and k_max must be >= 0", who);
  if (k_max > kMaxList) return fail(SSD_ERR_UNSUPPORTED, "%s: k_max above 2^24", who);
  if (n > 65535 || kv->h_kv > 65535) return fail(SSD_ERR_UNSUPPORTED, "%s: n or h_kv above 65535", who);
  if (n == 0) return SSD_OK;
  if (!src || !dst || !cnt || (!idx && k_max > 0)) return fail(SSD_ERR_INVALID_ARG, "%s: src, dst, idx and cnt must be non-NULL", who);
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  a.to_pool = static_cast<char *>(const_cast<void *>(to->pool));
  a.to_lens = const_cast<int32_t *>(to->seq_lens);
  a.to_refs = to_refs;
  a.src = src, a.dst = dst, a.idx = idx, a.cnt = cnt, a.n = n, a.k_max = k_max;
  a.same = kv->page_table == to->page_table || kv->seq_lens == to->seq_lens;
  a.rs = row_shape(kv);
  // Half as many entries per block while that leaves SMs without work.
  const int k = k_max > 0 ? k_max : 1;
  a.tokens = (int64_t)cdiv(k, kCompactTokens) * kv->h_kv * n < (int64_t)sm_count() * 8 ? kCompactTokens / 2 : kCompactTokens;
  return launch(kv_compact_kernel, dim3(cdiv(k, a.tokens), kv->h_kv, n), dim3(kCompactThreads), 0,
                reinterpret_cast<cudaStream_t>(stream), "kv_compact_kernel", a);
}
