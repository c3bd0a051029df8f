// ssd_score.cu -- log probabilities of given tokens under rows of logits, with log-sum-exp, entropy and top alternatives.
//
// One pass over a row.  Every thread keeps m = max x, s = sum e^(x - m), t = sum (x - m) e^(x - m) of its elements; joined over
// the row they give  lse = m + ln s  and  entropy = ln s - t / s  (no term is larger than the entropy itself).  The top k
// need no second pass over the row: the k-th largest of 128 maxima over groups of four threads is a bound that k elements
// reach, and only the threads whose own maximum reaches it read their elements again (about k of 512, from L2).
#include "ssd_host.h"

namespace ssd {

constexpr int kScoreThreads = 512;
constexpr int kScoreGroups = 128;  // maxima that bound the k-th largest from below
constexpr int kScoreMaxK = 64;
constexpr int kScoreCand = 1024;   // candidates for the top k; more: score_ties

struct ScoreArgs {
  const void *logits;
  int64_t stride;
  int n_rows, vocab, k;
  const int32_t *tokens, *rows;
  int n_tokens;
  float *logprob, *lse, *entropy;
  int32_t *top_ids;
  float *top_logprobs;
  unsigned *status;
};

// a, or NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// m (at least the lowest float, so that differences to it are no NaN), s and t as above.
struct ScoreSums {
  float m, s, t;
  // 2^x of a clamped exponent: below -1e4 the term is 0 and (x - m) times it has to be 0 too.
  __device__ __forceinline__ void add(float x) {
    const float z = max_nan(x - m, -1e4f), e = fast_exp2(z * kLog2e);
    s += e;
    t = fmaf(z, e, t);
  }
  __device__ __forceinline__ void move(float to) {  // the reference from m to `to` >= m
    const float z = fmaxf(m - to, -1e4f), f = fast_exp2(z * kLog2e);
    t = (t + s * z) * f;
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(float m2, float s2, float t2) {
    ScoreSums o = {m2, s2, t2};
    const float to = fmaxf(m, m2);
    move(to);
    o.move(to);
    s += o.s;
    t += o.t;
  }
};

template <typename T>
struct ScoreVec;  // 16 bytes of logits
template <>
struct ScoreVec<float> {
  static constexpr int N = 4;
  __device__ static void get(const uint4 &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct ScoreVec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void get(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
};

// (value, index) before (value2, index2) in the order of the top.
__device__ __forceinline__ bool score_before(float v, int i, float v2, int i2) { return v > v2 || (v == v2 && i < i2); }

struct ScoreSmem {
  float gmax[kScoreGroups];
  float val[kScoreCand];
  int idx[kScoreCand];
  float wm[kScoreThreads / 32], ws[kScoreThreads / 32], wt[kScoreThreads / 32];
  int count, hits, hit[kScoreThreads];
  float tau, m, lns;
  float best_v[kScoreThreads / 32];
  int best_i[kScoreThreads / 32];
};

// A row of logits: `head` elements up to the first 16-byte boundary, nv vectors, `tail` elements.
template <typename T>
struct ScoreRow {
  static constexpr int N = ScoreVec<T>::N;
  const T *x;
  int head, nv, tail, vocab;
  __device__ ScoreRow(const ScoreArgs &a, int r) : x(static_cast<const T *>(a.logits) + r * a.stride), vocab(a.vocab) {
    const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15u) / (int)sizeof(T);
    head = min(off ? N - off : 0, vocab);
    nv = (vocab - head) / N;
    tail = vocab - head - nv * N;
  }
  __device__ __forceinline__ uint4 vec(int v) const { return __ldg(reinterpret_cast<const uint4 *>(x + head) + v); }
  // element `e` of the edges: the head's, then the tail's
  __device__ __forceinline__ int edge(int e) const { return e < head ? e : head + nv * N + (e - head); }
};

// The top k where more than kScoreCand elements reach the bound (ties, or fewer than k above -inf): k times the next
// largest.  Reads the row up to k times; rows like these hold mostly equal values.
template <typename T>
__device__ void score_ties(const ScoreArgs &a, const ScoreRow<T> &row, ScoreSmem &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float pv = INFINITY;
  int pi = -1;
  __syncthreads();
  for (int k = 0; k < a.k; ++k) {
    float bv = 0.f;
    int bi = -1;
    for (int i = tid; i < row.vocab; i += kScoreThreads) {
      const float v = to_f32<T>(row.x[i]);
      if (score_before(pv, pi, v, i) && (bi < 0 ? v == v : score_before(v, i, bv, bi))) bv = v, bi = i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, bv, o);
      const int i = __shfl_xor_sync(0xffffffffu, bi, o);
      if (i >= 0 && (bi < 0 || score_before(v, i, bv, bi))) bv = v, bi = i;
    }
    if (lane == 0) sm.best_v[warp] = bv, sm.best_i[warp] = bi;
    __syncthreads();
    bv = sm.best_v[0], bi = sm.best_i[0];
    for (int w = 1; w < kScoreThreads / 32; ++w)
      if (sm.best_i[w] >= 0 && (bi < 0 || score_before(sm.best_v[w], sm.best_i[w], bv, bi))) bv = sm.best_v[w], bi = sm.best_i[w];
    pv = bv, pi = bi;
    __syncthreads();
    if (tid == 0) sm.val[k] = bi < 0 ? -INFINITY : bv, sm.idx[k] = bi;
    if (bi < 0) {  // only NaN is left
      for (int j = k + tid; j < a.k; j += kScoreThreads) sm.val[j] = -INFINITY, sm.idx[j] = -1;
      break;
    }
  }
  __syncthreads();
}

// ln softmax of x in a row with maximum m and ln of the sum lns (or m = the log-sum-exp and lns = 0).
__device__ __forceinline__ float score_logprob(float x, float m, float lns) {
  return x == -INFINITY && m + lns == m + lns ? -INFINITY : (x - m) - lns;
}

template <typename T>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(ScoreArgs a) {
  constexpr int N = ScoreVec<T>::N;
  __shared__ ScoreSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x;
  pdl_wait();
  const ScoreRow<T> row(a, r);
  ScoreSums u = {-3.402823466e38f, 0.f, 0.f};
  float top = -INFINITY;  // largest element
  auto take = [&](const uint4 &v) {
    float x[N];
    ScoreVec<T>::get(v, x);
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mx = fmaxf(mx, x[i]);
    if (mx > top) {
      top = mx;
      if (mx > u.m) u.move(mx);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) u.add(x[i]);
  };
  constexpr int U = 4;
  int v = tid;
  for (; v + (U - 1) * kScoreThreads < row.nv; v += U * kScoreThreads) {
    uint4 w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) w[i] = row.vec(v + i * kScoreThreads);
#pragma unroll
    for (int i = 0; i < U; ++i) take(w[i]);
  }
  for (; v < row.nv; v += kScoreThreads) take(row.vec(v));
  const int n_edge = row.head + row.tail;
  if (tid < n_edge) {
    const float x = to_f32<T>(row.x[row.edge(tid)]);
    top = fmaxf(top, x);
    if (x > u.m) u.move(x);
    u.add(x);
  }
  pdl_trigger();
  // The row's sums.
  {
    ScoreSums w = u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      w.join(__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.s, o), __shfl_xor_sync(0xffffffffu, w.t, o));
    if (lane == 0) sm.wm[warp] = w.m, sm.ws[warp] = w.s, sm.wt[warp] = w.t;
  }
  float g = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((tid & 3) == 0) sm.gmax[tid >> 2] = g;
  if (tid == 0) sm.count = sm.hits = 0, sm.tau = -INFINITY;
  __syncthreads();
  if (tid == 0) {
    ScoreSums w = {sm.wm[0], sm.ws[0], sm.wt[0]};
    for (int i = 1; i < kScoreThreads / 32; ++i) w.join(sm.wm[i], sm.ws[i], sm.wt[i]);
    const float lns = logf(w.s);  // -inf: nothing but -inf
    sm.m = w.m;
    sm.lns = lns;
    a.lse[r] = w.m + lns;
    if (a.entropy) a.entropy[r] = w.s == 0.f ? 0.f : lns - w.t / w.s;
  }
  if (a.k && tid < kScoreGroups) {
    const float mine = sm.gmax[tid];
    int rank = 0;
    for (int j = 0; j < kScoreGroups; ++j) rank += score_before(sm.gmax[j], j, mine, tid);
    if (rank == a.k - 1) sm.tau = mine;
  }
  __syncthreads();
  const float m = sm.m, lns = sm.lns;
  if (!a.rows)  // the row's own tokens
    for (int j = tid; j < a.n_tokens / a.n_rows; j += kScoreThreads) {
      const int64_t at = (int64_t)r * (a.n_tokens / a.n_rows) + j;
      const int tok = a.tokens[at];
      if (tok < 0 || tok >= a.vocab) atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
      a.logprob[at] = tok < 0 || tok >= a.vocab ? NAN : score_logprob(to_f32<T>(row.x[tok]), m, lns);
    }
  if (!a.k) return;
  const float tau = sm.tau;
  auto offer = [&](float x, int i) {
    if (x >= tau) {
      const int at = atomicAdd(&sm.count, 1);
      if (at < kScoreCand) sm.val[at] = x, sm.idx[at] = i;
    }
  };
  // Threads whose maximum reaches the bound: a warp reads each one's vectors again.
  if (top >= tau) sm.hit[atomicAdd(&sm.hits, 1)] = tid;
  if (tid < n_edge) offer(to_f32<T>(row.x[row.edge(tid)]), row.edge(tid));
  __syncthreads();
  const int hits = sm.hits;
  for (int h = warp; h < hits; h += kScoreThreads / 32) {
    if (*(volatile int *)&sm.count > kScoreCand) break;
    for (int w = sm.hit[h] + lane * kScoreThreads; w < row.nv; w += 32 * kScoreThreads) {
      float x[N];
      ScoreVec<T>::get(row.vec(w), x);
#pragma unroll
      for (int i = 0; i < N; ++i) offer(x[i], row.head + w * N + i);
    }
  }
  __syncthreads();
  const int count = sm.count;
  int32_t *ids = a.top_ids + (int64_t)r * a.k;
  float *lps = a.top_logprobs + (int64_t)r * a.k;
  if (count > kScoreCand || count < a.k) {
    score_ties<T>(a, row, sm);
    if (tid < a.k) ids[tid] = sm.idx[tid], lps[tid] = score_logprob(sm.val[tid], m, lns);
    return;
  }
  for (int c = tid; c < count; c += kScoreThreads) {
    const float x = sm.val[c];
    const int i = sm.idx[c];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += score_before(sm.val[j], sm.idx[j], x, i);
    if (rank < a.k) ids[rank] = i, lps[rank] = score_logprob(x, m, lns);
  }
}

// Tokens looked up in rows of their own choice.
template <typename T>
__global__ void __launch_bounds__(128) score_tokens_kernel(ScoreArgs a) {
  const int j = blockIdx.x * 128 + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (j >= a.n_tokens) return;
  const int r = a.rows[j], tok = a.tokens[j];
  float lp = 0.f;
  if (r != -1) {
    if (r < 0 || r >= a.n_rows || tok < 0 || tok >= a.vocab) {
      atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
      lp = NAN;
    } else {
      lp = score_logprob(to_f32<T>(static_cast<const T *>(a.logits)[r * a.stride + tok]), a.lse[r], 0.f);
    }
  }
  a.logprob[j] = lp;
}

template <typename T>
static int score_launch(const ScoreArgs &a, cudaStream_t st) {
  int rc = launch(score_kernel<T>, dim3(a.n_rows), dim3(kScoreThreads), 0, st, "score_kernel", a);
  if (rc || !a.rows || a.n_tokens == 0) return rc;
  return launch(score_tokens_kernel<T>, dim3(cdiv(a.n_tokens, 128)), dim3(128), 0, st, "score_tokens_kernel", a);
}

}  // namespace ssd

using namespace ssd;

extern "C" int ssd_token_logprobs(const void *logits, int dtype, int64_t row_stride, int n_rows, int vocab, const int32_t *tokens,
                                  const int32_t *rows, int n_tokens, float *logprob, float *lse, float *entropy, int32_t *top_ids,
                                  float *top_logprobs, int top_k, ssd_stream_t stream) {
  const char *who = "ssd_token_logprobs";
  if (dtype != SSD_DTYPE_BF16 && dtype != SSD_DTYPE_F32) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d", who, dtype);
  if (n_rows < 0 || vocab < 1 || n_tokens < 0 || row_stride < 0 || vocab > 1 << 30)
    return fail(SSD_ERR_INVALID_ARG, "%s: n_rows %d, vocab %d, n_tokens %d or row_stride out of range", who, n_rows, vocab, n_tokens);
  if (top_k < 0 || top_k > vocab || top_k > kScoreMaxK)
    return fail(SSD_ERR_INVALID_ARG, "%s: top_k %d outside [0, min(vocab, %d)]", who, top_k, kScoreMaxK);
  if (!rows && (n_rows ? n_tokens % n_rows : n_tokens)) return fail(SSD_ERR_INVALID_ARG, "%s: %d tokens for %d rows", who, n_tokens, n_rows);
  if ((n_rows && (!logits || !lse)) || (n_tokens && (!tokens || !logprob)) || (n_rows && top_k && (!top_ids || !top_logprobs)))
    return fail(SSD_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SSD_DTYPE_BF16 ? 2 : 4))
    return fail(SSD_ERR_INVALID_ARG, "%s: logits are not aligned to their type", who);
  if (n_rows == 0 && n_tokens == 0) return SSD_OK;
  if (n_rows == 0) return fail(SSD_ERR_INVALID_ARG, "%s: tokens without rows", who);
  unsigned *status = device_status();
  if (!status) return SSD_ERR_CUDA;
  const ScoreArgs a = {logits, row_stride, n_rows, vocab, top_k, tokens, rows, n_tokens, logprob, lse, entropy, top_ids, top_logprobs, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SSD_DTYPE_BF16 ? score_launch<__nv_bfloat16>(a, st) : score_launch<float>(a, st);
}
