// ssd_span.cuh -- attention of a request's last tokens ("span" attention): what the tree and the window form share.
//
// Query i of request b sits at position p = base + i, base = L_b - n_b.  Its tokens are a range [0, sink) and a range that
// ends with p: from p - window + 1 on for a window; for a tree from 0 on (window = kSpanAll) up to base, and behind it the
// ancestors of node i.  The rows of a KV head are (query, head of its group): row r = i * G + h.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

constexpr int kSpanAll = 1 << 30;      // a window that no length reaches
constexpr int kSpanMaxNodes = 512;     // nodes of a tree
constexpr int kSpanMaxTreeRows = 8192; // rows of a tree per KV head
constexpr int kSpanMaxGroup = 128;     // query heads per KV head

struct SpanArgs {
  KVView kv;
  const void *q;
  void *out;
  float *lse;
  const int32_t *parents;  // [batch][n]: a tree; NULL: a window
  const int32_t *counts;   // [batch] or NULL
  unsigned *status;
  int n, h_q, G, window, sink;
  float scale_log2;        // softmax scale * log2(e)
};

// Length and number of queries of request b, clamped.
__device__ __forceinline__ void span_sizes(const SpanArgs &a, int b, bool report, int &L, int &c) {
  L = a.kv.seq_lens[b];
  c = a.counts ? a.counts[b] : a.n;
  const bool bad = c < 0 || c > a.n || L < c || L > a.kv.max_seq_len;
  c = min(max(c, 0), a.n);
  L = min(max(L, 0), a.kv.max_seq_len);
  if (bad && report) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
}

// The tokens that the queries [i0, i1] of a request see, in a row: first the sinks, then the window, each from and to a
// multiple of `grain` (a power of two; what a copy takes at once).  Place v of the row holds token(v); a tile is TILE places.
// A token t is seen by one of the queries iff t < hi and (t < sink or t >= lo); places without one of these are
// [sink, lo + off) and those from hi + off on.
struct SpanTiles {
  int base, lo, hi, sink, split, off, n_tiles;  // from place `split` on token v - off is at place v
  __device__ __forceinline__ int token(int v) const { return v < split ? v : v - off; }
  __device__ __forceinline__ bool seen(int t) const { return t < hi && (t < sink || t >= lo); }
};

template <int TILE>
__device__ __forceinline__ SpanTiles span_tiles(const SpanArgs &a, int L, int c, int i0, int i1, int grain) {
  SpanTiles s;
  s.base = L - c;
  i0 = max(i0, -s.base);
  i1 = min(i1, c - 1);
  s.hi = s.lo = s.sink = s.split = s.off = s.n_tiles = 0;
  if (i0 > i1) return s;
  s.hi = s.base + i1 + 1;
  s.lo = max(0, s.base + i0 - a.window + 1);
  s.sink = min(a.sink, s.hi);
  const int first = (s.sink + grain - 1) & -grain, from = s.lo & -grain;
  if (from > first) s.split = first, s.off = first - from;  // (else one stretch from token 0 on)
  s.n_tiles = cdiv(s.hi + s.off, TILE);
  return s;
}

// Bits of the tokens [t0, t0 + 32) in [lo, hi).
__device__ __forceinline__ uint32_t span_bits(int t0, int lo, int hi) {
  const int a = max(lo - t0, 0), e = min(hi - t0, 32);
  if (a >= e) return 0u;
  return (0xffffffffu >> (32 - (e - a))) << a;
}

// What row i of the request (p = base + i >= 0, i < count) sees of the W * 32 places from v0 on.
template <int W>
__device__ __forceinline__ void span_mask(const SpanArgs &a, const int32_t *parents, int base, int off, int i, int v0, unsigned *status,
                                          uint32_t (&m)[W]) {
  const int p = base + i;
  if (!a.parents) {
#pragma unroll
    for (int w = 0; w < W; ++w)
      m[w] = span_bits(v0 + 32 * w, max(0, p - a.window + 1) + off, p + 1 + off) | span_bits(v0 + 32 * w, 0, min(a.sink, p + 1));
    return;
  }
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = span_bits(v0 + 32 * w, 0, base);
  for (int j = i; j >= 0 && base + j >= v0;) {
    const int t = base + j - v0;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if ((t >> 5) == w) m[w] |= 1u << (t & 31);
    const int up = parents[j];
    if (up >= j || up < -1) {
      atomicOr(status, (unsigned)SSD_FAULT_INDEX);
      break;
    }
    j = up;
  }
}

}  // namespace ssd
