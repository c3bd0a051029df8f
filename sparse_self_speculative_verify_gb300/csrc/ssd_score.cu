// ssd_score.cu -- log probabilities of given tokens under rows of logits, with log-sum-exp, entropy and top alternatives.
//
// One pass over a row.  Every thread keeps m = max x, s = sum e^(x - m), t = sum (x - m) e^(x - m) of its elements; joined over
// the row they give  lse = m + ln s  and  entropy = ln s - t / s  (no term is larger than the entropy itself).  The top k
// need no second pass over the row: the k-th largest of 128 to 256 maxima over groups of threads is a bound that k elements
// reach, and only the threads whose own maximum reaches it read elements again: those of the stage that held it, or all of theirs
// where another stage's maximum reaches it too.
// A cluster of 1 to 8 blocks takes a row, by distributed shared memory: sums and group maxima are read by the others, candidates
// are pushed into the first block's list.
//
// What bounds it: the bytes of the logits where they are many (1000 rows of 151936 bf16: 50 us, 6.0 TB/s), else what comes before
// and behind them: 512 rows 38.0 us (4.1 TB/s), of which the top 20 are 6 and the start, the ends and the cluster's barriers 6
// more; one row 8.6.  A warp of its own brings the logits to shared memory by bulk copies, two stages of 8 KB a block and eight
// blocks an SM (loads into registers, taken and used in turn by the same threads, kept half as much in flight: 44 us where this
// first took 40).  Threads that have met nothing but banned tokens (-inf, or beyond kScoreFar) take element after element: 512 rows in which 99 % are
// banned 53 us without a top, else 32.  Where no more than about k tokens are allowed, the top k is score_ties' work: 512 rows with 5
// allowed 2.9 ms for the top 5, 11.6 for the top 20.
#include <cooperative_groups.h>

#include "ssd_host.h"
#include "ssd_sm100.cuh"
#include "ssd_sm100_pairs.cuh"

namespace ssd {
namespace cg = cooperative_groups;
using namespace sm100;

constexpr int kScoreThreads = 128;  // and a warp that loads
constexpr int kScoreBlocks = 8;     // of an SM
constexpr int kScoreVectors = 4, kScoreStages = 2, kScoreStage = kScoreThreads * 16 * kScoreVectors;  // vectors of a thread; bytes
// A thread's reference follows its maximum only when that has grown by this.
constexpr float kScoreLazy = 4.f;
constexpr int kScoreGroups = 256;  // most maxima that bound the k-th largest from below
// Tokens of chosen rows that the rows' blocks look for themselves; more: score_tokens_kernel.  (512 rows, 512 / 2000 / 4000
// tokens: 41.5 / 44.1 / 45.7 us, by the other kernel 45.2 / 45.8 / 46.6; 8000 tokens 52 and 43.)
constexpr int kScoreFused = 4096;
constexpr int kScoreMaxK = 64;
constexpr int kScoreCand = 512;    // candidates for the top k; more: score_ties

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

// Where m is within kScoreFar, m log2 e rounded lies within 1/4 of itself (2^-24 of less than 2^23), so that exponents relative to it are as
// good as those relative to m; they are finite for every x raised to kScoreLow.  Larger m, and m of banned tokens that hold a large
// negative number: x - m itself.
constexpr float kScoreFar = 4194304.f, kScoreLow = -1e38f;

template <int V>
struct ScoreInt {
  static constexpr int value = V;
};

// 16 bytes of logits.
template <typename T>
struct ScoreVec;
template <>
struct ScoreVec<float> {
  static constexpr int N = 4;
  template <int C = 1>
  __device__ static float max(const uint4 *v) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < C; ++q)
      m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[q].x), __uint_as_float(v[q].y))), fmaxf(__uint_as_float(v[q].z), __uint_as_float(v[q].w)));
    return m;
  }
  __device__ static void get(const uint4 &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  // with -inf (and what is as far off) as a number, NaN kept
  __device__ static void get_finite(const uint4 &v, float (&x)[4]) {
    get(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = max_nan(x[i], kScoreLow);
  }
};
template <>
struct ScoreVec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  template <int C = 1>
  __device__ static float max(const uint4 *v) {
    uint32_t m = max2(max2(v[0].x, v[0].y), max2(v[0].z, v[0].w));
#pragma unroll
    for (int q = 1; q < C; ++q) m = max2(m, max2(max2(v[q].x, v[q].y), max2(v[q].z, v[q].w)));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  __device__ static void get(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
  __device__ static void get_finite(const uint4 &v, float (&x)[8]) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(0xfe96fe96u));  // about kScoreLow
    get(make_uint4(w[0], w[1], w[2], w[3]), x);
  }
};

// Unsigned keys in the order of the floats.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u >> 31 ? ~u : u | 0x80000000u;
}
// (value, index) before (value2, index2) in the order of the top.
__device__ __forceinline__ bool score_before(float v, int i, float v2, int i2) { return v > v2 || (v == v2 && i < i2); }

struct ScoreSmem {
  char stage[kScoreStages][kScoreStage];
  uint64_t full[kScoreStages], empty[kScoreStages];
  int abort;
  float own[kScoreThreads];  // maxima over groups of threads
  float val[kScoreCand];
  int idx[kScoreCand];
  float wm[kScoreThreads / 32], ws[kScoreThreads / 32], wt[kScoreThreads / 32];
  float sums[3];  // of this block's slice
  int count, hits, full_hits, hit[kScoreThreads];
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

// Barrier of the threads that are not the loading warp's.
__device__ __forceinline__ void score_sync() { named_sync(1, kScoreThreads); }

// The top k where more than kScoreCand elements reach the bound (ties, or fewer than k above -inf): k times the next
// largest.  Reads the row up to k times; rows like these hold mostly equal values.
template <typename T>
__device__ void score_ties(const ScoreArgs &a, const ScoreRow<T> &row, ScoreSmem &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float pv = INFINITY;
  int pi = -1;
  score_sync();
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
    score_sync();
    bv = sm.best_v[0], bi = sm.best_i[0];
    for (int w = 1; w < kScoreThreads / 32; ++w)
      if (sm.best_i[w] >= 0 && (bi < 0 || score_before(sm.best_v[w], sm.best_i[w], bv, bi))) bv = sm.best_v[w], bi = sm.best_i[w];
    pv = bv, pi = bi;
    score_sync();
    if (tid == 0) sm.val[k] = bi < 0 ? -INFINITY : bv, sm.idx[k] = bi;
    if (bi < 0) {  // only NaN is left
      for (int j = k + tid; j < a.k; j += kScoreThreads) sm.val[j] = -INFINITY, sm.idx[j] = -1;
      break;
    }
  }
  score_sync();
}

// ln softmax of x in a row with maximum m and ln of the sum lns (or m = the log-sum-exp and lns = 0).
__device__ __forceinline__ float score_logprob(float x, float m, float lns) {
  return x == -INFINITY && m + lns == m + lns ? -INFINITY : (x - m) - lns;
}

// What a token outside the vocabulary or a row outside the logits gets.
__device__ __forceinline__ bool score_bad(const ScoreArgs &a, int tok) {
  if (tok >= 0 && tok < a.vocab) return false;
  atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kScoreThreads + 32, kScoreBlocks) score_kernel(ScoreArgs a) {
  constexpr int N = ScoreVec<T>::N;
  extern __shared__ __align__(16) char smem_raw[];
  ScoreSmem &sm = *reinterpret_cast<ScoreSmem *>(smem_raw);
  auto cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x / ranks;
  if (tid == 0) {
    sm.count = sm.hits = sm.full_hits = sm.abort = 0, sm.tau = -INFINITY;
    for (int i = 0; i < kScoreStages; ++i) mbar_init(smem_u32(sm.full + i), 1), mbar_init(smem_u32(sm.empty + i), kScoreThreads / 32);
    mbar_init_fence();
  }
  __syncthreads();
  pdl_wait();
  const ScoreRow<T> row(a, r);
  const int v0 = (int)((int64_t)row.nv * rank / ranks), v1 = (int)((int64_t)row.nv * (rank + 1) / ranks);
  ScoreSums u = {-3.402823466e38f, 0.f, 0.f};
  // Sums of even and odd elements, in log2 and relative to `ref`, u.m log2 e rounded: one instruction gives (x - m) log2 e.
  uint64_t s2 = 0, t2 = 0;
  float ref = 0.f;
  bool near = false;  // |u.m| is within kScoreFar
  float top = -INFINITY, next = -INFINITY;  // largest element, and the largest of the other stages
  int top_stage = 0;
  const uint64_t log2e2 = pack2(kLog2e, kLog2e);
  auto fold = [&]() {
    if (!near) return;
    const float d = fmaf(-u.m, kLog2e, ref), f = fast_exp2(d);  // what the rounding moved the reference by, 1/4 at most
    float p, q;
    unpack2(s2, p, q);
    const float s = p + q;
    unpack2(t2, p, q);
    u.s = fmaf(s, f, u.s);
    u.t = fmaf((p + q + s * d) * kLn2, f, u.t);
    s2 = t2 = 0;
  };
  float limit = u.m;        // a maximum above it moves the reference
  auto far = [&](uint4 v) {  // (the vector turns, so that its words are taken from one place)
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      if (N == 4) {
        u.add(__uint_as_float(v.x));
      } else {
        u.add(bf16_lo(v.x));
        u.add(bf16_hi(v.x));
      }
      v = make_uint4(v.y, v.z, v.w, v.x);
    }
  };
  auto take = [&](const uint4 *v, auto count) {
    constexpr int C = decltype(count)::value;
    const float mx = ScoreVec<T>::template max<C>(v);
    if (mx > limit) {
      fold();
      u.move(mx);
      limit = mx + kScoreLazy;
      near = fabsf(mx) < kScoreFar;
      ref = mx * kLog2e;
    }
    if (near) {
      const uint64_t ref2 = pack2(-ref, -ref);
#pragma unroll
      for (int q = 0; q < C; ++q) {
        float x[N];
        ScoreVec<T>::get_finite(v[q], x);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint64_t z = fma2(pack2(x[i], x[i + 1]), log2e2, ref2);
          float y0, y1;
          unpack2(z, y0, y1);
          const uint64_t e = pack2(fast_exp2(y0), fast_exp2(y1));
          s2 = add2(s2, e);
          t2 = fma2(z, e, t2);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < C; ++q) far(v[q]);
    }
    return mx;
  };
  // A stage: kScoreStage bytes of the slice's vectors; the loading warp goes to the next barrier at once.
  constexpr int PER = kScoreStage / 16;
  const int stages = cdiv(v1 - v0, PER);
  volatile int *abort = &sm.abort;
  if (warp == kScoreThreads / 32) {
    if (lane == 0) {
      int i = 0;
      for (; i < stages; ++i) {
        const int st = i % kScoreStages, bytes = min(PER, v1 - v0 - i * PER) * 16;
        if (!mbar_wait(smem_u32(sm.empty + st), (i / kScoreStages & 1) ^ 1, abort)) break;
        mbar_arrive_expect_tx(smem_u32(sm.full + st), bytes);
        bulk_load(smem_u32(sm.stage[st]), reinterpret_cast<const char *>(row.x + row.head) + ((int64_t)v0 + (int64_t)i * PER) * 16, bytes,
                  smem_u32(sm.full + st));
      }
      volatile int never = 0;  // (a wait ran out: the copies in flight land before the block ends)
      for (int j = max(0, i - kScoreStages); i < stages && j < i; ++j)
        mbar_wait(smem_u32(sm.full + j % kScoreStages), j / kScoreStages & 1, &never, 200000000ll);
    }
    __syncwarp();
  } else {
    for (int i = 0; i < stages; ++i) {
      const int st = i % kScoreStages, n = min(PER, v1 - v0 - i * PER);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(sm.full + st), i / kScoreStages & 1, abort))) break;
      const uint4 *from = reinterpret_cast<const uint4 *>(sm.stage[st]) + tid;
      uint4 w[kScoreVectors];
      float mx = -INFINITY;
      if (n == PER) {
#pragma unroll
        for (int q = 0; q < kScoreVectors; ++q) w[q] = from[q * kScoreThreads];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(sm.empty + st));
        mx = take(w, ScoreInt<kScoreVectors>{});
      } else {  // (the last stage: nobody waits for its place)
#pragma unroll 1
        for (int q = tid; q < n; q += kScoreThreads) {
          w[0] = reinterpret_cast<const uint4 *>(sm.stage[st])[q];
          mx = fmaxf(mx, take(w, ScoreInt<1>{}));
        }
      }
      next = fmaxf(next, fminf(top, mx));
      if (mx > top) top = mx, top_stage = i;
    }
  }
  fold();
  const int n_edge = rank == 0 ? row.head + row.tail : 0;
  float edge = -INFINITY;
  if (tid < n_edge) {
    edge = to_f32<T>(row.x[row.edge(tid)]);
    if (edge > u.m) u.move(edge);
    u.add(edge);
  }
  pdl_trigger();
  // The slice's sums, and the maxima over groups of `per` threads: 128, 64 or 32 of a block.
  {
    ScoreSums w = u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      w.join(__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.s, o), __shfl_xor_sync(0xffffffffu, w.t, o));
    if (lane == 0 && warp < kScoreThreads / 32) sm.wm[warp] = w.m, sm.ws[warp] = w.s, sm.wt[warp] = w.t;
  }
  const int per = min(ranks, 4), groups = kScoreThreads / per;
  float g = fmaxf(top, edge);
  for (int o = 1; o < per; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  if (tid < kScoreThreads && tid % per == 0) sm.own[tid / per] = g;
  __syncthreads();
  if (warp == 0) {
    ScoreSums w = {-3.402823466e38f, 0.f, 0.f};
    if (lane < kScoreThreads / 32) w = {sm.wm[lane], sm.ws[lane], sm.wt[lane]};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      w.join(__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.s, o), __shfl_xor_sync(0xffffffffu, w.t, o));
    if (lane == 0) sm.sums[0] = w.m, sm.sums[1] = w.s, sm.sums[2] = w.t;
  }
  if (tid == 0 && sm.abort) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
  if (ranks > 1) cluster.sync(); else __syncthreads();
  if (rank == 0 && warp == 0) {
    ScoreSums w = {-3.402823466e38f, 0.f, 0.f};
    if (lane < ranks) {
      const float *o = cluster.map_shared_rank(sm.sums, lane);
      w = {o[0], o[1], o[2]};
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      w.join(__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.s, o), __shfl_xor_sync(0xffffffffu, w.t, o));
    if (lane == 0) {
      const float lns = logf(w.s);  // -inf: nothing but -inf
      sm.m = w.m;
      sm.lns = lns;
      a.lse[r] = w.m + lns;
      if (a.entropy) a.entropy[r] = w.s == 0.f ? 0.f : lns - w.t / w.s;
    }
  }
  if (a.k) {
    // The bound: bit by bit the largest key, of its upper bits, that k maxima reach.  (Comparing them all with one another took
    // a third of the call.)
    if (warp == 0) {
      uint32_t key[kScoreGroups / 32], t = 0;
#pragma unroll
      for (int q = 0; q < kScoreGroups / 32; ++q) {
        const int j = q * 32 + lane;
        key[q] = j < ranks * groups ? score_key(cluster.map_shared_rank(sm.own, j / groups)[j % groups]) : 0u;
      }
#pragma unroll 1
      for (uint32_t bit = 1u << 31; bit >= 1u << 12; bit >>= 1) {
        int n = 0;
#pragma unroll
        for (int q = 0; q < kScoreGroups / 32; ++q) n += key[q] >= (t | bit);
        if (__reduce_add_sync(0xffffffffu, n) >= a.k) t |= bit;
      }
      if (lane == 0) sm.tau = t <= score_key(-INFINITY) ? -INFINITY : __uint_as_float(t >> 31 ? t ^ 0x80000000u : ~t);
    }
    __syncthreads();
    const float tau = sm.tau;
    int *count = cluster.map_shared_rank(&sm.count, 0);
    float *val = cluster.map_shared_rank(sm.val, 0);
    int *idx = cluster.map_shared_rank(sm.idx, 0);
    auto offer = [&](float x, int i) {
      if (x >= tau) {
        const int at = atomicAdd(count, 1);
        if (at < kScoreCand) val[at] = x, idx[at] = i;
      }
    };
    // Vectors of the threads whose maximum reaches the bound, read again by everybody and four at a time: of one stage, or all.
    if (tid < kScoreThreads && top >= tau) {
      if (next < tau)
        sm.hit[atomicAdd(&sm.hits, 1)] = top_stage * kScoreThreads + tid;
      else
        sm.hit[kScoreThreads - 1 - atomicAdd(&sm.full_hits, 1)] = tid;  // (from the list's other end)
    }
    if (tid < n_edge) offer(edge, row.edge(tid));
    __syncthreads();
    auto again = [&](int hits, int from, int each, auto vector_of) {
      const unsigned total = hits * each;
      constexpr int U = 4;
      for (unsigned e0 = tid; e0 < total && *(volatile int *)count <= kScoreCand; e0 += U * (kScoreThreads + 32)) {
        int at[U];
        uint4 w[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const unsigned e = e0 + q * (kScoreThreads + 32), h = e / each;
          at[q] = e < total ? v0 + vector_of(sm.hit[from + h], (int)(e - h * each)) : v1;
          if (at[q] < v1) w[q] = row.vec(at[q]);
        }
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (at[q] < v1 && ScoreVec<T>::max(w + q) >= tau) {
            float x[N];
            ScoreVec<T>::get(w[q], x);
#pragma unroll
            for (int i = 0; i < N; ++i) offer(x[i], row.head + at[q] * N + i);
          }
      }
    };
    again(sm.hits, 0, kScoreVectors, [&](int hit, int q) { return hit / kScoreThreads * PER + hit % kScoreThreads + q * kScoreThreads; });
    again(sm.full_hits, kScoreThreads - sm.full_hits, cdiv(v1 - v0, kScoreThreads), [&](int hit, int q) { return hit + q * kScoreThreads; });
  }
  if (ranks > 1) cluster.sync(); else __syncthreads();
  if (rank || tid >= kScoreThreads) return;
  const float m = sm.m, lns = sm.lns;
  if (!a.rows) {  // the row's own tokens
    const int each = a.n_tokens / a.n_rows;
    for (int j = tid; j < each; j += kScoreThreads) {
      const int64_t at = (int64_t)r * each + j;
      const int tok = a.tokens[at];
      a.logprob[at] = score_bad(a, tok) ? NAN : score_logprob(to_f32<T>(row.x[tok]), m, lns);
    }
  } else if (a.n_tokens <= kScoreFused) {
    for (int j = tid; j < a.n_tokens; j += kScoreThreads) {
      const int of = a.rows[j];
      if (of == r) {
        const int tok = a.tokens[j];
        a.logprob[j] = score_bad(a, tok) ? NAN : score_logprob(to_f32<T>(row.x[tok]), m, lns);
      } else if (r == 0 && (of < 0 || of >= a.n_rows)) {
        if (of != -1) atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
        a.logprob[j] = of == -1 ? 0.f : NAN;
      }
    }
  }
  if (!a.k) return;
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
    int before = 0;
    for (int j = 0; j < count; ++j) before += score_before(sm.val[j], sm.idx[j], x, i);
    if (before < a.k) ids[before] = i, lps[before] = score_logprob(x, m, lns);
  }
}

// Tokens looked up in rows of their own choice, where they are many.
template <typename T>
__global__ void __launch_bounds__(128) score_tokens_kernel(ScoreArgs a) {
  const int j = blockIdx.x * 128 + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (j >= a.n_tokens) return;
  const int r = a.rows[j], tok = a.tokens[j];
  float lp = 0.f;
  if (r != -1) {
    if (r < 0 || r >= a.n_rows || score_bad(a, tok)) {
      atomicOr(a.status, (unsigned)SSD_FAULT_INDEX);
      lp = NAN;
    } else {
      lp = score_logprob(to_f32<T>(static_cast<const T *>(a.logits)[r * a.stride + tok]), a.lse[r], 0.f);
    }
  }
  a.logprob[j] = lp;
}

// Blocks of a row's cluster: so many that six lie on every SM, with a vector a thread at least.  (512 rows of 151936 bf16: 46
// us with three an SM, whose shares differ too much, 40 with six, 48 with twelve, which do not all fit; 300 rows 33.5, 34.2
// and 43.7.)
static int score_ranks(const ScoreArgs &a, int per_vector) {
  int ranks = 1;
  while (ranks < 8 && (int64_t)a.n_rows * ranks < 6 * sm_count() && a.vocab >= 2 * ranks * kScoreThreads * per_vector) ranks *= 2;
  return ranks;
}

template <typename T>
static int score_launch(const ScoreArgs &a, cudaStream_t st) {
  const int ranks = score_ranks(a, ScoreVec<T>::N);
  int rc = ensure_smem<score_kernel<T>>(sizeof(ScoreSmem));
  if (rc) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_rows * ranks);
  cfg.blockDim = dim3(kScoreThreads + 32);
  cfg.dynamicSmemBytes = sizeof(ScoreSmem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, score_kernel<T>, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(SSD_ERR_CUDA, "score_kernel: %s", cudaGetErrorString(e));
  }
  rc = check_launch("score_kernel");
  if (rc || !a.rows || a.n_tokens <= kScoreFused) return rc;
  return launch(score_tokens_kernel<T>, dim3(cdiv(a.n_tokens, 128)), dim3(128), 0, st, "score_tokens_kernel", a);
}

}  // namespace ssd

using namespace ssd;

extern "C" int ssd_token_logprobs(const void *logits, int dtype, int64_t row_stride, int n_rows, int vocab, const int32_t *tokens,
                                  const int32_t *rows, int n_tokens, float *logprob, float *lse, float *entropy, int32_t *top_ids,
                                  float *top_logprobs, int top_k, ssd_stream_t stream) {
  const char *who = "ssd_token_logprobs";
  if (dtype != SSD_DTYPE_BF16 && dtype != SSD_DTYPE_F32) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d", who, dtype);
  if (n_rows < 0 || vocab < 1 || n_tokens < 0 || row_stride < 0 || vocab > 1 << 30 || n_rows > 1 << 27)
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
