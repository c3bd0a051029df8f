// ssd_tree.cu -- which nodes of a drafted tree stay, and moving their K / V rows together.
//
// SparseSpec §2.3: a verify checks the drafted tokens and gives one more; SpecSA, "branch handling": the KV of accepted
// tokens stays for later queries, that of rejected ones is dropped.
#include <math.h>

#include "ssd_host.h"
#include "ssd_span.cuh"

namespace ssd {

constexpr int kTreeThreads = 128;

struct AcceptArgs {
  const int32_t *parents, *tokens, *target, *counts;
  const float *logprob, *entropy;
  float ln_epsilon, ln_delta;
  int n, max_path;
  int32_t *path, *cnt, *next, *advance;
  unsigned *status;
};

// A block per tree.  Each node's link to its parent is kept in shared memory, or broken where the node fails its own
// test; then every node walks its links to node 0, and the deepest that arrives wins.  What bounds it: latency, two loads
// (the parents, then what the test reads) and as many shared loads as the tree is deep: 512 trees of 128 to 255 nodes 3.9 us.
__global__ void __launch_bounds__(kTreeThreads) tree_accept_kernel(AcceptArgs a) {
  __shared__ int16_t s_up[kSpanMaxNodes];
  __shared__ int s_best;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int64_t at = (int64_t)b * a.n;
  if (tid == 0) s_best = -1;
  pdl_trigger();
  pdl_wait();
  int c = a.counts ? a.counts[b] : a.n;
  if (c < 0 || c > a.n) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    c = min(max(c, 0), a.n);
  }
  for (int i = tid; i < c; i += kTreeThreads) {
    const int up = a.parents[at + i];
    bool ok = up >= 0 && up < i;
    if (up < -1 || up >= max(i, 0)) atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
    if (ok && a.logprob) {
      // NaN on either side keeps nothing
      const float h = a.ln_delta - a.entropy[at + up], low = h > a.ln_epsilon ? a.ln_epsilon : h;
      ok = a.logprob[at + i] > low;
    } else if (ok) {
      ok = a.tokens[at + i] == a.target[at + up];
    }
    s_up[i] = ok ? (int16_t)up : (int16_t)-1;
  }
  __syncthreads();
  for (int i = tid; i < c; i += kTreeThreads) {
    int depth = 0, j = i;
    while (j > 0) j = s_up[j], ++depth;
    if (j == 0 && depth < a.max_path) atomicMax(&s_best, depth << 16 | (kSpanMaxNodes - 1 - i));
  }
  __syncthreads();
  const int best = s_best, m = best < 0 ? 0 : (best >> 16) + 1;
  int32_t *path = a.path + (int64_t)b * a.max_path;
  for (int k = m + tid; k < a.max_path; k += kTreeThreads) path[k] = -1;
  if (tid) return;
  int j = best < 0 ? -1 : kSpanMaxNodes - 1 - (best & 0xffff);
  a.next[b] = j < 0 ? -1 : a.target[at + j];
  a.cnt[b] = m;
  a.advance[b] = m - c;
  for (int k = m - 1; k >= 0; --k) path[k] = j, j = s_up[j];
}

struct CommitArgs {
  KVView kv;
  char *pool;
  const int32_t *counts, *path, *cnt;
  int n, max_path, row_bytes;
  unsigned *status;
};

constexpr int kCommitBatch = 8;  // rows of a column that are in flight together

// Blocks (column chunk, request): a thread moves one 16-byte column of a (K|V, head) through all of the path's rows, so
// that no row is written before its column has been read: entries ascend and are not below their index, and a source
// is never a row already written.  What bounds it: latency, the entry, its page and the row: 160 requests of up to 12 rows, 8
// heads of 128 in bf16, 3.5 us (2.4 TB/s of what it reads and writes).
__global__ void __launch_bounds__(kTreeThreads) tree_commit_kernel(CommitArgs a) {
  __shared__ int64_t s_src[kSpanMaxNodes];  // row numbers of head 0's K, -1: the page is bad
  __shared__ int64_t s_dst[kSpanMaxNodes];
  const int b = blockIdx.y, tid = threadIdx.x, ps = a.kv.page_size;
  pdl_trigger();
  pdl_wait();
  const int L = a.kv.seq_lens[b], c = a.counts ? a.counts[b] : a.n, m = a.cnt[b], base = L - c;
  unsigned bad = 0;
  if (c < 0 || c > a.n || L < c || L > a.kv.max_seq_len)
    bad = SSD_FAULT_SEQLEN;
  else if (m < 0 || m > a.max_path || m > c)
    bad = SSD_FAULT_KMAX;
  const int32_t *path = a.path + (int64_t)b * a.max_path, *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
  if (!bad) {
    auto row = [&](int t) -> int64_t {
      const int32_t p = table[t >> a.kv.log2_ps];
      if (p < 0 || (int64_t)p >= a.kv.num_pages) {
        bad |= SSD_FAULT_PAGE;
        return -1;
      }
      return (int64_t)p * 2 * a.kv.h_kv * ps + (t & (ps - 1));
    };
    for (int j = tid; j < m; j += kTreeThreads) {
      const int x = path[j];
      if (x < 0 || x >= c || (j && path[j - 1] >= x))
        bad |= SSD_FAULT_INDEX;
      else
        s_src[j] = row(base + x), s_dst[j] = row(base + j);
    }
  }
  const bool bad_any = __syncthreads_or(bad != 0);
  if (bad) atomicOr(a.status, bad);
  if (bad_any) return;
  const int cpr = a.row_bytes / 16, col = blockIdx.x * kTreeThreads + tid;
  if (col >= 2 * a.kv.h_kv * cpr) return;
  const int64_t block = (int64_t)(col / cpr) * ps;  // (K|V, head) in a page, in rows
  char *mine = a.pool + (col % cpr) * 16;
  for (int j0 = 0; j0 < m; j0 += kCommitBatch) {
    uint4 v[kCommitBatch];
#pragma unroll
    for (int k = 0; k < kCommitBatch; ++k)
      if (j0 + k < m && s_src[j0 + k] != s_dst[j0 + k]) v[k] = *reinterpret_cast<const uint4 *>(mine + (s_src[j0 + k] + block) * a.row_bytes);
#pragma unroll
    for (int k = 0; k < kCommitBatch; ++k)
      if (j0 + k < m && s_src[j0 + k] != s_dst[j0 + k]) *reinterpret_cast<uint4 *>(mine + (s_dst[j0 + k] + block) * a.row_bytes) = v[k];
  }
}

}  // namespace ssd

using namespace ssd;

extern "C" int ssd_tree_accept(const int32_t *parents, const int32_t *tokens, const int32_t *target, const float *logprob,
                               const float *entropy, double epsilon, double delta, const int32_t *counts, int batch, int n,
                               int max_path, int32_t *path, int32_t *cnt, int32_t *next, int32_t *advance, ssd_stream_t stream) {
  const char *who = "ssd_tree_accept";
  if (batch < 0 || n < 1 || max_path < 1) return fail(SSD_ERR_INVALID_ARG, "%s: batch %d < 0, n %d < 1 or max_path %d < 1", who, batch, n, max_path);
  if (n > kSpanMaxNodes) return fail(SSD_ERR_UNSUPPORTED, "%s: %d nodes (at most %d)", who, n, kSpanMaxNodes);
  if (!logprob != !entropy) return fail(SSD_ERR_INVALID_ARG, "%s: logprob and entropy go together", who);
  if (logprob && (!(epsilon > 0) || !(delta > 0) || isinf(epsilon) || isinf(delta)))
    return fail(SSD_ERR_INVALID_ARG, "%s: epsilon and delta must be positive and finite", who);
  if (batch == 0) return SSD_OK;
  if (!parents || (!tokens && !logprob) || !target || !path || !cnt || !next || !advance)
    return fail(SSD_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  unsigned *status = device_status();
  if (!status) return SSD_ERR_CUDA;
  const AcceptArgs a = {parents, tokens, target, counts, logprob, entropy, logprob ? (float)log(epsilon) : 0.f,
                        logprob ? (float)log(delta) : 0.f, n, max_path, path, cnt, next, advance, status};
  return launch(tree_accept_kernel, dim3(batch), dim3(kTreeThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                "tree_accept_kernel", a);
}

extern "C" int ssd_tree_commit(const ssd_paged_kv *kv, int n, const int32_t *counts, const int32_t *path, int max_path,
                               const int32_t *cnt, ssd_stream_t stream) {
  const char *who = "ssd_tree_commit";
  CommitArgs a = {};
  int rc = validate_kv(kv, &a.kv, who);
  if (rc) return rc;
  if (n < 1 || max_path < 1) return fail(SSD_ERR_INVALID_ARG, "%s: n %d < 1 or max_path %d < 1", who, n, max_path);
  if (max_path > kSpanMaxNodes) return fail(SSD_ERR_UNSUPPORTED, "%s: max_path %d (at most %d)", who, max_path, kSpanMaxNodes);
  if (kv->batch > 65535) return fail(SSD_ERR_UNSUPPORTED, "%s: batch %d (at most 65535)", who, kv->batch);
  if (kv->batch == 0) return SSD_OK;
  if (!path || !cnt) return fail(SSD_ERR_INVALID_ARG, "%s: path and cnt must be non-NULL", who);
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  a.pool = static_cast<char *>(const_cast<void *>(kv->pool));
  a.counts = counts, a.path = path, a.cnt = cnt;
  a.n = n, a.max_path = max_path;
  a.row_bytes = kv->d * (kv->dtype == SSD_DTYPE_BF16 ? 2 : 4);
  return launch(tree_commit_kernel, dim3(cdiv(2 * kv->h_kv * (a.row_bytes / 16), kTreeThreads), kv->batch), dim3(kTreeThreads), 0,
                reinterpret_cast<cudaStream_t>(stream), "tree_commit_kernel", a);
}
