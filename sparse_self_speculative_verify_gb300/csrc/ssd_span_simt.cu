// ssd_span_simt.cu -- span attention on CUDA cores: fp32 caches, and bf16 ones whose pages are below 8 tokens.
//
// A block takes up to ROWS query rows of one (request, KV head) and a part of their tiles of 64 tokens.  K and V of a tile
// are brought to shared memory as fp32; the scores, 64 per row, go there too; the softmax keeps a running maximum and sum
// per row and O stays in registers.  An element of K and V in shared memory meets 2 or 4 rows of registers in S and in
// O, so that shared-memory reads and FMAs take about the same time.  Where the (request, head, rows) blocks do not fill
// the SMs, each is cut into equal parts of its tiles, joined by span_join_kernel.
#include "ssd_host.h"
#include "ssd_span.h"

namespace ssd {

constexpr int kSimtTile = 64;
constexpr int kSimtThreads = 256;

struct SimtPlan {
  int chunks, parts;  // row chunks of a (request, head), parts of a chunk's tiles
  float *o, *lse;     // [item][ROWS][D], [item][ROWS] (log2), parts > 1
};

template <int D, int ROWS>
struct SimtSmem {
  float q[ROWS][D + 4], k[kSimtTile][D + 4], v[kSimtTile][D], s[ROWS][kSimtTile + 4];
  float m[ROWS], l[ROWS], alpha[ROWS];
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ void store4(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kSimtThreads) span_simt_kernel(SpanArgs a, SimtPlan pl) {
  extern __shared__ __align__(16) char smem_raw[];
  auto &sm = *reinterpret_cast<SimtSmem<D, ROWS> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h_kv = a.kv.h_kv, rows = a.n * a.G;
  int64_t x = blockIdx.x;
  const int part = (int)(x % pl.parts);
  x /= pl.parts;
  const int chunk = (int)(x % pl.chunks);
  x /= pl.chunks;
  const int g = (int)(x % h_kv), b = (int)(x / h_kv);
  const int r0 = chunk * ROWS, nr = min(ROWS, rows - r0);
  pdl_wait();
  int L, c;
  span_sizes(a, b, g == 0 && chunk == 0 && part == 0 && tid == 0, L, c);
  const SpanTiles st = span_tiles<kSimtTile>(a, L, c, r0 / a.G, (r0 + nr - 1) / a.G);
  const int k0 = (int)((int64_t)st.n_tiles * part / pl.parts), k1 = (int)((int64_t)st.n_tiles * (part + 1) / pl.parts);
  const int32_t *parents = a.parents ? a.parents + (int64_t)b * a.n : nullptr;

  auto row_at = [&](int r) {  // element offset of row r0 + r in q and out
    const int i = (r0 + r) / a.G;
    return (((int64_t)b * a.n + i) * a.h_q + g * a.G + (r0 + r - i * a.G)) * D;
  };
  for (int e = tid; e < ROWS * (D / 4); e += kSimtThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    store4(&sm.q[r][col], r < nr ? load4<T>(static_cast<const T *>(a.q) + row_at(r) + col) : make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (tid < ROWS) sm.m[tid] = -INFINITY, sm.l[tid] = 0.f;

  constexpr int TC = D / 4, TR = kSimtThreads / TC, RT = ROWS / TR;  // O: rows per thread, four columns
  static_assert(RT >= 1 && ROWS % 16 == 0, "tile");
  const int oc = tid % TC * 4, orow = tid / TC * RT;
  constexpr int SR = ROWS / 16;  // S: SR rows and tokens st_ + 16 j per thread
  const int s_t = tid % 16, s_r = tid / 16 * SR;
  float4 o[RT];
#pragma unroll
  for (int k = 0; k < RT; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int k = k0; k < k1; ++k) {
    const int t0 = st.tile(k) * kSimtTile;
    __syncthreads();  // the tile before has been used
    for (int e = tid; e < kSimtTile * TC; e += kSimtThreads) {
      const int t = e / TC, col = e % TC * 4;
      float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
      if (st.seen(t0 + t)) {
        const T *kr = kv_row<D, T>(a.kv, b, 0, g, t0 + t, a.status);
        if (kr) {
          kk = load4<T>(kr + col);
          vv = load4<T>(kr + (int64_t)h_kv * a.kv.page_size * D + col);
        }
      }
      store4(&sm.k[t][col], kk);
      store4(&sm.v[t][col], vv);
    }
    __syncthreads();
    float s[SR][4];
#pragma unroll
    for (int i = 0; i < SR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 qv[SR], kv4[4];
#pragma unroll
      for (int i = 0; i < SR; ++i) qv[i] = *reinterpret_cast<const float4 *>(&sm.q[s_r + i][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv4[j] = *reinterpret_cast<const float4 *>(&sm.k[s_t + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < SR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(qv[i].x, kv4[j].x, fmaf(qv[i].y, kv4[j].y, fmaf(qv[i].z, kv4[j].z, fmaf(qv[i].w, kv4[j].w, s[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < SR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.s[s_r + i][s_t + 16 * j] = s[i][j] * a.scale_log2;
    __syncthreads();
    for (int r = warp; r < ROWS; r += kSimtThreads / 32) {  // a warp per row, two tokens per lane
      const int i = (r0 + r) / a.G;
      uint32_t m2[2] = {0u, 0u};
      if (r < nr && i < c && st.base + i >= 0) span_mask<2>(a, parents, st.base, i, t0, a.status, m2);
      const float x0 = (m2[0] >> lane & 1) ? sm.s[r][lane] : -INFINITY, x1 = (m2[1] >> lane & 1) ? sm.s[r][lane + 32] : -INFINITY;
      const float m_old = sm.m[r], m_new = fmaxf(m_old, warp_max(fmaxf(x0, x1)));
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float p0 = exp2f(x0 - ref), p1 = exp2f(x1 - ref), sum = warp_sum(p0 + p1);
      sm.s[r][lane] = p0;
      sm.s[r][lane + 32] = p1;
      __syncwarp();
      if (lane == 0) {
        const float f = exp2f(m_old - ref);
        sm.alpha[r] = f;
        sm.m[r] = m_new;
        sm.l[r] = sm.l[r] * f + sum;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float f = sm.alpha[orow + i];
      o[i].x *= f, o[i].y *= f, o[i].z *= f, o[i].w *= f;
    }
#pragma unroll 4
    for (int t = 0; t < kSimtTile; t += 4) {
      float4 pv[RT], vv[4];
#pragma unroll
      for (int i = 0; i < RT; ++i) pv[i] = *reinterpret_cast<const float4 *>(&sm.s[orow + i][t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) vv[j] = *reinterpret_cast<const float4 *>(&sm.v[t + j][oc]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float p[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[i].x = fmaf(p[j], vv[j].x, o[i].x), o[i].y = fmaf(p[j], vv[j].y, o[i].y);
          o[i].z = fmaf(p[j], vv[j].z, o[i].z), o[i].w = fmaf(p[j], vv[j].w, o[i].w);
        }
      }
    }
  }
  pdl_trigger();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = orow + i;
    if (r >= nr) continue;
    const float l = sm.l[r], f = l > 0.f || l != l ? 1.f / l : 0.f;
    const float4 v = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
    if (pl.parts > 1)
      store4(pl.o + ((int64_t)blockIdx.x * ROWS + r) * D + oc, v);
    else
      store4(static_cast<T *>(a.out) + row_at(r) + oc, v);
  }
  if (tid < nr) {
    const float l = sm.l[tid];
    const float lse2 = l > 0.f || l != l ? sm.m[tid] + log2f(l) : -INFINITY;
    if (pl.parts > 1)
      pl.lse[(int64_t)blockIdx.x * ROWS + tid] = lse2;
    else if (a.lse)
      a.lse[row_at(tid) / D] = lse2 * kLn2;
  }
}

// Joins the parts of a row: weights 2^(lse2 - max) / their sum.  A warp per row.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(256) span_simt_join_kernel(SpanArgs a, SimtPlan pl) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), rows = (int64_t)a.n * a.G;
  pdl_wait();
  pdl_trigger();
  if (row >= rows * a.kv.h_kv * a.kv.batch) return;
  const int64_t bg = row / rows;
  const int r = (int)(row - bg * rows), b = (int)(bg / a.kv.h_kv), g = (int)(bg % a.kv.h_kv);
  const int64_t item = (bg * pl.chunks + r / ROWS) * pl.parts;
  const float *lse = pl.lse + item * ROWS + r % ROWS;
  float m = -INFINITY;
  for (int k = lane; k < pl.parts; k += 32) m = fmaxf(m, lse[(int64_t)k * ROWS]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float z = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool mine = lane * 4 < D;
  for (int k = 0; k < pl.parts; ++k) {
    const float w = exp2f(lse[(int64_t)k * ROWS] - ref);
    z += w;
    if (mine && w != 0.f) {
      const float4 v = load4<float>(pl.o + ((item + k) * ROWS + r % ROWS) * D + lane * 4);
      o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    }
  }
  const float f = z > 0.f || z != z ? 1.f / z : 0.f;
  const int i = r / a.G;
  const int64_t at = (((int64_t)b * a.n + i) * a.h_q + g * a.G + (r - i * a.G));
  if (mine) store4(static_cast<T *>(a.out) + at * D + lane * 4, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
  if (a.lse && lane == 0) a.lse[at] = z > 0.f || z != z ? (m + log2f(z)) * kLn2 : -INFINITY;
}

// Row chunks of 16 where that many cover a head's rows, else 32.
static int simt_rows(const SpanArgs &a) { return (int64_t)a.n * a.G <= 16 ? 16 : 32; }

static SimtPlan simt_plan(const ssd_paged_kv *kv, const SpanArgs &a) {
  const int rows = simt_rows(a);
  SimtPlan p = {};
  p.chunks = (int)cdiv64((int64_t)a.n * a.G, rows);
  const int64_t units = (int64_t)kv->batch * kv->h_kv * p.chunks;
  // tiles of a chunk, at most: the sinks', the window's and those that its ends cut
  const int64_t all = cdiv(kv->max_seq_len, kSimtTile);
  const int64_t tiles = all < cdiv64(a.sink, kSimtTile) + ((int64_t)a.window + rows / a.G) / kSimtTile + 2
                            ? all
                            : cdiv64(a.sink, kSimtTile) + ((int64_t)a.window + rows / a.G) / kSimtTile + 2;
  // about four blocks per SM, two tiles each at least
  const int64_t want = 4 * (int64_t)sm_count();
  int64_t parts = units >= want ? 1 : cdiv64(want, units > 0 ? units : 1);
  if (parts > tiles / 2) parts = tiles / 2;
  p.parts = parts < 1 ? 1 : (int)parts;
  return p;
}

static size_t simt_carve(const ssd_paged_kv *kv, const SpanArgs &a, SimtPlan &p, void *ws) {
  Carver c(ws);
  c.take<char>(kCounterBytes);
  if (p.parts > 1) {
    const size_t items = (size_t)kv->batch * kv->h_kv * p.chunks * p.parts, rows = simt_rows(a);
    p.o = c.take<float>(items * rows * kv->d);
    p.lse = c.take<float>(items * rows);
  }
  return c.off;
}

size_t span_simt_workspace(const ssd_paged_kv *kv, const SpanArgs &a) {
  SimtPlan p = simt_plan(kv, a);
  return simt_carve(kv, a, p, nullptr);
}

template <typename T, int D, int ROWS>
static int simt_launch(const ssd_paged_kv *kv, const SpanArgs &a, const SimtPlan &p, cudaStream_t st) {
  constexpr auto kernel = span_simt_kernel<T, D, ROWS>;
  constexpr int smem = sizeof(SimtSmem<D, ROWS>);
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  const int64_t items = (int64_t)kv->batch * kv->h_kv * p.chunks * p.parts;
  if (items >= (int64_t)1 << 31) return fail(SSD_ERR_UNSUPPORTED, "span attention: %lld blocks", (long long)items);
  if ((rc = launch(kernel, dim3((unsigned)items), dim3(kSimtThreads), smem, st, "span_simt_kernel", a, p)) || p.parts == 1) return rc;
  const int64_t rows = (int64_t)kv->batch * kv->h_kv * a.n * a.G;
  return launch(span_simt_join_kernel<T, D, ROWS>, dim3((unsigned)cdiv64(rows, 8)), dim3(256), 0, st, "span_simt_join_kernel", a, p);
}

int span_simt(const ssd_paged_kv *kv, const SpanArgs &a, void *workspace, cudaStream_t st) {
  SimtPlan p = simt_plan(kv, a);
  simt_carve(kv, a, p, workspace);
  const bool few = simt_rows(a) == 16, wide = kv->d == 128;
  if (kv->dtype == SSD_DTYPE_F32)
    return wide ? (few ? simt_launch<float, 128, 16>(kv, a, p, st) : simt_launch<float, 128, 32>(kv, a, p, st))
                : (few ? simt_launch<float, 64, 16>(kv, a, p, st) : simt_launch<float, 64, 32>(kv, a, p, st));
  using H = __nv_bfloat16;
  return wide ? (few ? simt_launch<H, 128, 16>(kv, a, p, st) : simt_launch<H, 128, 32>(kv, a, p, st))
              : (few ? simt_launch<H, 64, 16>(kv, a, p, st) : simt_launch<H, 64, 32>(kv, a, p, st));
}

}  // namespace ssd
