// ssd_span.cu -- ssd_tree_attn and ssd_window_attn: argument checks and the choice of a path.
#include "ssd_span.h"

#include <math.h>

namespace ssd {

// Fills `a` but for its pointers; the checks that need no device.
static int span_args(const char *who, const ssd_paged_kv *kv, int h_q, int n, int window, int sink, bool tree, SpanArgs *a) {
  int rc = validate_kv(kv, &a->kv, who);
  if (rc) return rc;
  if (h_q <= 0 || h_q % kv->h_kv) return fail(SSD_ERR_INVALID_ARG, "%s: h_q %d is not a positive multiple of h_kv %d", who, h_q, kv->h_kv);
  if (n < 1) return fail(SSD_ERR_INVALID_ARG, "%s: n %d < 1", who, n);
  a->G = h_q / kv->h_kv;
  if (a->G > kSpanMaxGroup) return fail(SSD_ERR_UNSUPPORTED, "%s: %d query heads per KV head (at most %d)", who, a->G, kSpanMaxGroup);
  if (window < 1 || window > kSpanAll || sink < 0 || sink > kSpanAll)
    return fail(SSD_ERR_INVALID_ARG, "%s: window %d or sink %d out of range", who, window, sink);
  if (tree && (n > kSpanMaxNodes || n * a->G > kSpanMaxTreeRows))
    return fail(SSD_ERR_UNSUPPORTED, "%s: %d nodes (at most %d, and %d rows per KV head)", who, n, kSpanMaxNodes, kSpanMaxTreeRows);
  if ((int64_t)n * a->G >= 1 << 27) return fail(SSD_ERR_UNSUPPORTED, "%s: %d queries", who, n);
  a->n = n;
  a->h_q = h_q;
  a->window = window;
  a->sink = sink;
  return SSD_OK;
}

static size_t span_workspace(const ssd_paged_kv *kv, const SpanArgs &a) {
  return span_tc_takes(kv) ? span_tc_workspace(kv, a) : span_simt_workspace(kv, a);
}

static int span_attn(const char *who, const ssd_paged_kv *kv, const void *q, int h_q, int n, const int32_t *parents,
                     const int32_t *counts, int window, int sink, bool tree, float scale, void *out, float *lse,
                     void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  SpanArgs a = {};
  int rc = span_args(who, kv, h_q, n, window, sink, tree, &a);
  if (rc) return rc;
  if (!(scale > 0.f) || isinf(scale * kLog2e)) return fail(SSD_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
  if (kv->batch == 0) return SSD_OK;
  if (!q || !out || (tree && !parents)) return fail(SSD_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned16(q) || !aligned16(out)) return fail(SSD_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  if (!workspace || workspace_bytes < span_workspace(kv, a)) return fail(SSD_ERR_WORKSPACE, "%s: workspace too small", who);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(SSD_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.parents = tree ? parents : nullptr;
  a.counts = counts;
  a.scale_log2 = scale * kLog2e;
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return span_tc_takes(kv) ? span_tc(kv, a, workspace, st) : span_simt(kv, a, workspace, st);
}

}  // namespace ssd

using namespace ssd;

extern "C" size_t ssd_tree_workspace_bytes(const ssd_paged_kv *kv, int h_q, int n) {
  SpanArgs a = {};
  return span_args("ssd_tree_workspace_bytes", kv, h_q, n, kSpanAll, 0, true, &a) ? 0 : span_workspace(kv, a);
}

extern "C" int ssd_tree_attn(const ssd_paged_kv *kv, const void *q, int h_q, int n, const int32_t *parents, const int32_t *counts,
                             float scale, void *out, float *lse, void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  return span_attn("ssd_tree_attn", kv, q, h_q, n, parents, counts, kSpanAll, 0, true, scale, out, lse, workspace, workspace_bytes, stream);
}

extern "C" size_t ssd_window_workspace_bytes(const ssd_paged_kv *kv, int h_q, int n, int window, int sink) {
  SpanArgs a = {};
  return span_args("ssd_window_workspace_bytes", kv, h_q, n, window, sink, false, &a) ? 0 : span_workspace(kv, a);
}

extern "C" int ssd_window_attn(const ssd_paged_kv *kv, const void *q, int h_q, int n, const int32_t *counts, int window, int sink,
                               float scale, void *out, float *lse, void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  return span_attn("ssd_window_attn", kv, q, h_q, n, nullptr, counts, window, sink, false, scale, out, lse, workspace, workspace_bytes,
                   stream);
}
