// ssd_kv4.cu -- entry points of the attention over a 4-bit cache (kernels: ssd_kv4_attn.cuh).
#include <math.h>

#include <initializer_list>

#include "ssd_cache.h"
#include "ssd_kv4_tc.cuh"

namespace ssd {

int kv4_dense_d64(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st);
int kv4_dense_d128(const Kv4AttnArgs &a, int grid, cudaStream_t st);
int kv4_tc_attn(Kv4AttnArgs a, int rows, int grid, cudaStream_t st);
int kv4_tc_crit(const Kv4AttnArgs &a, int grid, cudaStream_t st);
int kv4_list_d64(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st);
int kv4_list_d128(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st);
int kv4_crit_d64(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st);

// Query rows padded to what a pass takes, and the passes: up to 32 rows go in one.
static int kv4_nt(int R) { return R > 8 * kKv4MaxNT ? kKv4MaxNT : cdiv(R, 8); }
static int kv4_np(int R) { return R <= 16 ? 16 : 32; }
static int kv4_chunks(int R) { return cdiv(R, 32); }

// Blocks of a launch over `units` units of at most `max_tokens` tokens, `tile` of which a block takes at least.
static int64_t kv4_grid_bound(int64_t units, int max_tokens, int tile) {
  const int64_t tiles = units * (max_tokens > 0 ? cdiv(max_tokens, kKv4Tile) : 1);
  const int64_t blocks = cdiv64(tiles * kKv4Tile, tile);
  return blocks > kKv4MaxBlocks ? kKv4MaxBlocks : blocks;
}

struct Kv4Layout {
  size_t o, ml, fin, total;
};
static Kv4Layout kv4_layout(const ssd_paged_kv *kv, int h_q, int n_rows, int max_tokens) {
  const int R = h_q / kv->h_kv * n_rows, rows = kv4_np(R);
  const size_t slots = 2 * (size_t)kv4_grid_bound((int64_t)kv->batch * kv->h_kv * kv4_chunks(R), max_tokens, kKv4Tile);
  Kv4Layout y{};
  y.o = kCounterBytes;
  y.ml = y.o + align256(slots * rows * kv->d * sizeof(float));
  y.fin = y.ml + align256(slots * rows * 2 * sizeof(float));
  y.total = y.fin + align256((size_t)kv->batch * n_rows * h_q * sizeof(float2));
  return y;
}

static bool kv4_shape_ok(const ssd_paged_kv *kv, int h_q, int n) {
  return kv && kv->h_kv > 0 && h_q > 0 && h_q % kv->h_kv == 0 && n > 0 && kv->batch >= 0 && kv->max_seq_len >= 0 &&
         (kv->d == 64 || kv->d == 128) && (int64_t)(h_q / kv->h_kv) * n <= kMaxRows;
}

struct Kv4Call {
  const ssd_paged_kv *kv;
  const void *q;
  int q_dtype, h_q, n_rows;
  float scale, k_scale, v_scale;
  void *out;
  int out_dtype;
  float *lse;
  void *workspace;
  size_t workspace_bytes;
};

// Argument checks and launch arguments common to both calls.
static int kv4_prepare(const Kv4Call &c, int max_tokens, Kv4AttnArgs *a, Kv4Layout *lay, const char *who) {
  int rc = validate_cache(c.kv, &a->kv, who, kCacheNvfp4);
  if (rc) return rc;
  if (!c.q || !c.out) return fail(SSD_ERR_INVALID_ARG, "%s: q and out must be non-NULL", who);
  if (!aligned16(c.q) || !aligned16(c.out)) return fail(SSD_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  for (int t : {c.q_dtype, c.out_dtype})
    if (t != SSD_DTYPE_BF16 && t != SSD_DTYPE_F32)
      return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d (q and out: SSD_DTYPE_BF16 or SSD_DTYPE_F32)", who, t);
  if (c.h_q <= 0 || c.h_q % c.kv->h_kv) return fail(SSD_ERR_INVALID_ARG, "%s: h_q %d not a multiple of h_kv", who, c.h_q);
  if (c.n_rows <= 0) return fail(SSD_ERR_INVALID_ARG, "%s: n_cand %d", who, c.n_rows);
  const int64_t R = (int64_t)(c.h_q / c.kv->h_kv) * c.n_rows;
  if (R > kMaxRows) return fail(SSD_ERR_UNSUPPORTED, "%s: %lld query rows per KV head (at most %d)", who, (long long)R, kMaxRows);
  if (!isfinite(c.scale)) return fail(SSD_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if ((rc = kv4_scales_ok(c.k_scale, c.v_scale, who))) return rc;
  if ((int64_t)c.kv->batch * c.kv->h_kv > 65535) return fail(SSD_ERR_UNSUPPORTED, "%s: batch*h_kv above 65535", who);
  *lay = kv4_layout(c.kv, c.h_q, c.n_rows, max_tokens);
  if (!c.workspace || c.workspace_bytes < lay->total)
    return fail(SSD_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", who, c.workspace_bytes, lay->total);
  if (reinterpret_cast<uintptr_t>(c.workspace) & 255u)
    return fail(SSD_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  char *ws = static_cast<char *>(c.workspace);
  a->q = c.q, a->out = c.out, a->lse = c.lse;
  a->q_f32 = c.q_dtype == SSD_DTYPE_F32, a->out_f32 = c.out_dtype == SSD_DTYPE_F32;
  a->h_q = c.h_q, a->G = c.h_q / c.kv->h_kv, a->n_c = c.n_rows, a->R = (int)R;
  a->n_chunk = kv4_chunks(a->R);
  a->n_units = c.kv->batch * c.kv->h_kv * a->n_chunk;
  a->scale_log2 = c.scale * kLog2e * c.k_scale;
  a->v_scale = c.v_scale;
  a->counters = reinterpret_cast<unsigned *>(ws);
  a->part_o = reinterpret_cast<float *>(ws + lay->o);
  a->part_ml = reinterpret_cast<float *>(ws + lay->ml);
  return SSD_OK;
}

static int kv4_grid(int64_t units, int max_tokens, int tile, int blocks_per_sm) {
  const int64_t bound = kv4_grid_bound(units, cdiv(max_tokens, tile) * tile, tile), dev = (int64_t)sm_count() * blocks_per_sm;
  return (int)(bound < dev ? bound : dev);
}

// Blocks per SM of kv4_attn_kernel: at d = 128 it takes up to 16 rows (drafts), at d = 64 up to 32.
static int kv4_blocks_per_sm(int d, int nt) {
  if (d == 128) return nt == 1 ? Kv4Tune<128, 1>::kBlocks : Kv4Tune<128, 2>::kBlocks;
  return nt == 1 ? Kv4Tune<64, 1>::kBlocks : nt == 2 ? Kv4Tune<64, 2>::kBlocks : nt == 3 ? Kv4Tune<64, 3>::kBlocks : Kv4Tune<64, 4>::kBlocks;
}

}  // namespace ssd

using namespace ssd;

extern "C" size_t ssd_kv4_verify_workspace_bytes(const ssd_paged_kv *kv, int h_q, int n_cand) {
  return kv4_shape_ok(kv, h_q, n_cand) ? kv4_layout(kv, h_q, n_cand, kv->max_seq_len).total : 0;
}

extern "C" int ssd_kv4_verify_attn(const ssd_paged_kv *kv, const void *q, int q_dtype, int h_q, int n_cand, float scale,
                                   float k_scale, float v_scale, void *out, int out_dtype, float *lse, float *scores,
                                   int64_t scores_stride, void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  const char *who = "ssd_kv4_verify_attn";
  const Kv4Call c{kv, q, q_dtype, h_q, n_cand, scale, k_scale, v_scale, out, out_dtype, lse, workspace, workspace_bytes};
  Kv4AttnArgs a{};
  Kv4Layout lay;
  int rc = kv4_prepare(c, kv ? kv->max_seq_len : 0, &a, &lay, who);
  if (rc) return rc;
  if (scores && scores_stride < kv->max_seq_len)
    return fail(SSD_ERR_INVALID_ARG, "%s: scores_stride %lld < max_seq_len %d", who, (long long)scores_stride, kv->max_seq_len);
  if (kv->batch == 0) return SSD_OK;
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  if (scores) a.fin = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + lay.fin);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // d = 128 runs on tcgen05 from 9 rows on.  32 requests of 2048 to 8192 tokens, 8 heads: 4 rows 48 us on mma.sync
  // against 62, 8 rows 49 against 63, 12 rows 70.5 against 68.5 (fp32 outputs: 78 against 70), 16 rows 72
  // against 70.  (Two such requests alone, 4 rows: 11.8 against 13.6; 16 rows: 16 against 22.)  d = 64 has no tcgen05
  // form: V^T would fill half of M = 128, and M = 64 (which kind::f16 has too) has not been built.
  const int nt = kv4_nt(a.R);
  if (kv->d == 128 && a.R <= 8)
    rc = kv4_dense_d128(a, kv4_grid(a.n_units, kv->max_seq_len, kKv4Tile * 4, kv4_blocks_per_sm(kv->d, nt)), st);
  else if (kv->d == 128)
    rc = kv4_tc_attn(a, a.R > 32 ? 32 : a.R, kv4_grid(a.n_units, kv->max_seq_len, kKv4TcTile, 2), st);
  else
    rc = kv4_dense_d64(a, nt, kv4_grid(a.n_units, kv->max_seq_len, kKv4Tile * 4, kv4_blocks_per_sm(kv->d, nt)), st);
  if (rc || !scores) return rc;
  a.scores = scores;
  a.scores_stride = scores_stride;
  a.n_chunk = 1;
  a.n_units = kv->batch * kv->h_kv;
  if (kv->d == 128)
    return kv4_tc_crit(a, kv4_grid(a.n_units, kv->max_seq_len, kKv4TcTile, kKv4CritTcBlocks), st);
  return kv4_crit_d64(a, nt, kv4_grid(a.n_units, kv->max_seq_len, kKv4Tile * 4, kKv4CritBlocks), st);
}

extern "C" size_t ssd_kv4_draft_workspace_bytes(const ssd_paged_kv *kv, int h_q, int k_max) {
  return kv4_shape_ok(kv, h_q, 1) && k_max >= 0 && k_max <= kMaxList ? kv4_layout(kv, h_q, 1, k_max).total : 0;
}

extern "C" int ssd_kv4_draft_attn(const ssd_paged_kv *kv, const void *q, int q_dtype, int h_q, const int32_t *idx, int k_max,
                                  const int32_t *cnt, float scale, float k_scale, float v_scale, void *out, int out_dtype,
                                  float *lse, void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  const char *who = "ssd_kv4_draft_attn";
  const Kv4Call c{kv, q, q_dtype, h_q, 1, scale, k_scale, v_scale, out, out_dtype, lse, workspace, workspace_bytes};
  Kv4AttnArgs a{};
  Kv4Layout lay;
  if (k_max < 0) return fail(SSD_ERR_INVALID_ARG, "%s: k_max < 0", who);
  if (k_max > kMaxList) return fail(SSD_ERR_UNSUPPORTED, "%s: k_max above 2^24", who);
  int rc = kv4_prepare(c, k_max, &a, &lay, who);
  if (rc) return rc;
  if (!cnt || (!idx && k_max > 0)) return fail(SSD_ERR_INVALID_ARG, "%s: idx and cnt must be non-NULL", who);
  if (a.G > 16) return fail(SSD_ERR_UNSUPPORTED, "%s: group size %d > 16", who, a.G);
  if (kv->batch == 0) return SSD_OK;
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  a.idx = idx, a.cnt = cnt, a.k_max = k_max;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int nt = kv4_nt(a.R), grid = kv4_grid(a.n_units, k_max, kKv4Tile * 4, kv4_blocks_per_sm(kv->d, nt));
  return kv->d == 128 ? kv4_list_d128(a, nt, grid, st) : kv4_list_d64(a, nt, grid, st);
}
