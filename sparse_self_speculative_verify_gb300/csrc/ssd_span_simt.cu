// ssd_span_simt.cu -- span attention on CUDA cores: fp32 caches, and bf16 ones whose pages are below 8 tokens.
//
// A block of eight warps takes ROWS = 8 RW query rows of one (request, KV head) and a part of their tiles of 64 tokens; a warp
// has RW rows for itself.  K and V come to shared memory by cp.async, V of a tile while S is computed and K of the next while O
// is, from row addresses that are looked up one tile ahead.  In S a lane has two tokens and all of the warp's rows: the queries
// are read by broadcast, and 12 wavefronts of shared memory feed 32 multiply-adds of each lane; in O a lane has four columns
// (two at d = 64) and all rows.  A row's softmax stays inside its warp.  What bounds it: shared memory (69 % busy) and the
// latencies of a tile's four barriers; 16 requests of 1000 to 4000 tokens, 8 heads of 4 queries, 8 nodes in fp32: 224 us, 23
// TFLOP/s (231 with unpaired multiply-adds; four warps with twice the rows each: 269; about two blocks an SM instead of eight:
// 293); one request of 300 tokens: 10, latency.  A long request of one
// head and a deep tree are far from that: 8 nodes, 4 queries a head, over 16000 / 131072 tokens 57 / 326 us (8 heads 144 / 670, the last
// at 26 TFLOP/s): the join reads up to eight parts an SM one after the other; 512 nodes in a chain over 4000 tokens, 2 heads, 1.56 ms, side
// by side 0.17: the mask walks a row's ancestors in every tile.  Where the (request, head, rows) blocks do not fill the SMs, each is cut into
// equal parts of its tiles, joined by span_simt_join_kernel.
#include <type_traits>

#include "ssd_host.h"
#include "ssd_sm100_pairs.cuh"
#include "ssd_span.h"

namespace ssd {
using namespace sm100;

constexpr int kSimtTile = 64;
constexpr int kSimtWarps = 8;
constexpr int kSimtThreads = 32 * kSimtWarps;

struct SimtPlan {
  int chunks, parts;  // row chunks of a (request, head), parts of a chunk's tiles
  float *o, *lse;     // [item][ROWS][D], [item][ROWS] (log2), parts > 1
};

template <typename T, int D, int ROWS>
struct SimtSmem {
  float q[ROWS][D], p[ROWS][kSimtTile];
  T kv[2][kSimtTile][D + 16 / sizeof(T)];
  int64_t row[2][kSimtTile];  // offsets of the K rows of a tile and the next, -1: zeros
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

__device__ __forceinline__ void load2(const float *p, float &x, float &y) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  x = v.x, y = v.y;
}
__device__ __forceinline__ void load2(const __nv_bfloat16 *p, float &x, float &y) {
  const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
  x = bf16_lo(v), y = bf16_hi(v);
}
__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) { *reinterpret_cast<uint32_t *>(p) = pack_bf16(x, y); }

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kSimtThreads, 2) span_simt_kernel(SpanArgs a, SimtPlan pl) {
  constexpr int RW = ROWS / kSimtWarps, CL = D / 32;  // rows of a warp, columns of a lane
  extern __shared__ __align__(16) char smem_raw[];
  auto &sm = *reinterpret_cast<SimtSmem<T, D, ROWS> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, w0 = (tid >> 5) * RW;  // the warp's first row
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
  const SpanTiles st = span_tiles<kSimtTile>(a, L, c, r0 / a.G, (r0 + nr - 1) / a.G, 1);
  const int k0 = (int)((int64_t)st.n_tiles * part / pl.parts), k1 = (int)((int64_t)st.n_tiles * (part + 1) / pl.parts);
  const int32_t *parents = a.parents ? a.parents + (int64_t)b * a.n : nullptr;

  auto row_at = [&](int r) {  // row r0 + r of q and out
    const int i = (r0 + r) / a.G;
    return ((int64_t)b * a.n + i) * a.h_q + g * a.G + (r0 + r - i * a.G);
  };
  for (int e = tid; e < ROWS * (D / 4); e += kSimtThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    store4(&sm.q[r][col], r < nr ? load4<T>(static_cast<const T *>(a.q) + row_at(r) * D + col) : make_float4(0.f, 0.f, 0.f, 0.f));
  }
  float m[RW], l[RW], o[RW][CL];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < CL; ++j) o[i][j] = 0.f;
  }
  auto look_up = [&](int k) {
    if (k >= k1 || tid >= kSimtTile) return;
    const int t = st.token(k * kSimtTile + tid);
    const T *row = st.seen(t) ? kv_row<D, T>(a.kv, b, 0, g, t, a.status) : nullptr;
    sm.row[k & 1][tid] = row ? row - static_cast<const T *>(a.kv.pool) : -1;
  };
  // K (which = 0) or V of tile k; a group of its own.
  auto load = [&](int which, int k) {
    constexpr int C = D * (int)sizeof(T) / 16;
    if (k < k1) {
      const T *pool = static_cast<const T *>(a.kv.pool) + (which ? (int64_t)h_kv * a.kv.page_size * D : 0);
#pragma unroll
      for (int e0 = 0; e0 < kSimtTile * C; e0 += kSimtThreads) {
        const int t = (e0 + tid) / C, col = (e0 + tid) % C * (16 / (int)sizeof(T));
        const int64_t row = sm.row[k & 1][t];
        cp_async16(smem_u32(&sm.kv[which][t][col]), row < 0 ? a.kv.pool : pool + row + col, row < 0 ? 0 : 16);
      }
    }
    cp_async_commit();
  };
  look_up(k0);
  __syncthreads();
  load(0, k0);
  load(1, k0);
  look_up(k0 + 1);
  for (int k = k0; k < k1; ++k) {
    const int t0 = k * kSimtTile;  // its first place
    const int end = st.hi + st.off - t0;  // nothing is seen from this place of the tile on
    cp_async_wait<1>();
    __syncthreads();
    uint64_t s2[RW][2];  // sums over even and odd columns
#pragma unroll
    for (int i = 0; i < RW; ++i) s2[i][0] = s2[i][1] = 0;
    auto products = [&](auto both) {
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        const float4 ka = load4<T>(&sm.kv[0][lane][d]);
        const uint64_t a0 = pack2(ka.x, ka.y), a1 = pack2(ka.z, ka.w);
        float4 kb = {};
        if (decltype(both)::value) kb = load4<T>(&sm.kv[0][lane + 32][d]);
        const uint64_t b0 = pack2(kb.x, kb.y), b1 = pack2(kb.z, kb.w);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float4 q = *reinterpret_cast<const float4 *>(&sm.q[w0 + i][d]);
          const uint64_t q0 = pack2(q.x, q.y), q1 = pack2(q.z, q.w);
          s2[i][0] = fma2(q0, a0, fma2(q1, a1, s2[i][0]));
          if (decltype(both)::value) s2[i][1] = fma2(q0, b0, fma2(q1, b1, s2[i][1]));
        }
      }
    };
    if (end > 32)
      products(std::true_type());
    else
      products(std::false_type());
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int node = (r0 + w0 + i) / a.G;
      float s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float even, odd;
        unpack2(s2[i][h], even, odd);
        s[h] = even + odd;
      }
      uint32_t seen[2] = {0u, 0u};
      if (w0 + i < nr && node < c && st.base + node >= 0) span_mask<2>(a, parents, st.base, st.off, node, t0, a.status, seen);
      const float x0 = (seen[0] >> lane & 1) ? s[0] * a.scale_log2 : -INFINITY, x1 = (seen[1] >> lane & 1) ? s[1] * a.scale_log2 : -INFINITY;
      const float top = fmaxf(m[i], warp_max(fmaxf(x0, x1))), ref = top == -INFINITY ? 0.f : top;
      const float p0 = exp2f(x0 - ref), p1 = exp2f(x1 - ref), f = exp2f(m[i] - ref);
      m[i] = top;
      l[i] = l[i] * f + warp_sum(p0 + p1);
      sm.p[w0 + i][lane] = p0;
      sm.p[w0 + i][lane + 32] = p1;
#pragma unroll
      for (int j = 0; j < CL; ++j) o[i][j] *= f;
    }
    __syncthreads();
    load(0, k + 1);
    cp_async_wait<1>();
    __syncthreads();
#pragma unroll 2
    for (int t = 0; t < min(end, kSimtTile); t += 4) {
      uint64_t v[4][CL / 2];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < CL; j += 2) {
          float x, y;
          load2(&sm.kv[1][t + u][lane * CL + j], x, y);
          v[u][j / 2] = pack2(x, y);
        }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float4 p = *reinterpret_cast<const float4 *>(&sm.p[w0 + i][t]);
        const uint64_t px = pack2(p.x, p.x), py = pack2(p.y, p.y), pz = pack2(p.z, p.z), pw = pack2(p.w, p.w);
#pragma unroll
        for (int j = 0; j < CL; j += 2) {
          const uint64_t sum = fma2(px, v[0][j / 2], fma2(py, v[1][j / 2], fma2(pz, v[2][j / 2], fma2(pw, v[3][j / 2], pack2(o[i][j], o[i][j + 1])))));
          unpack2(sum, o[i][j], o[i][j + 1]);
        }
      }
    }
    __syncthreads();
    load(1, k + 1);
    look_up(k + 2);
  }
  cp_async_wait<0>();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = w0 + i;
    if (r >= nr) break;
    const bool some = l[i] > 0.f || l[i] != l[i];
    const float f = some ? 1.f / l[i] : 0.f, lse2 = some ? m[i] + log2f(l[i]) : -INFINITY;
    const int64_t at = row_at(r), slot = (int64_t)blockIdx.x * ROWS + r;
    if (pl.parts > 1) {
#pragma unroll
      for (int j = 0; j < CL; ++j) o[i][j] *= f;
#pragma unroll
      for (int j = 0; j < CL; j += 2) *reinterpret_cast<float2 *>(pl.o + slot * D + lane * CL + j) = make_float2(o[i][j], o[i][j + 1]);
      if (lane == 0) pl.lse[slot] = lse2;
    } else {
#pragma unroll
      for (int j = 0; j < CL; j += 2) store2(static_cast<T *>(a.out) + at * D + lane * CL + j, o[i][j] * f, o[i][j + 1] * f);
      if (a.lse && lane == 0) a.lse[at] = lse2 * kLn2;
    }
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

// Tiles of a chunk of `rows` rows, at most: the sinks', the window's and those that its ends cut.
static int64_t simt_tiles(const ssd_paged_kv *kv, const SpanArgs &a, int rows) {
  const int64_t all = cdiv(kv->max_seq_len, kSimtTile);
  const int64_t most = cdiv64(a.sink, kSimtTile) + ((int64_t)a.window + rows / a.G) / kSimtTile + 2;
  return all < most ? all : most;
}

// Rows of a block: 32; 48, which take 1.45 times as long, where that saves one of two or three chunks (36 rows 166 us, by 32 218; 72 rows
// 621 and 664; 256 rows 235 and 217, so not there); or 8 or 16 where these cover a head's or where all tiles of such chunks are on the SMs at once, two an SM or
// four at d = 64.  (One request of 300 tokens, 2 heads of 64, 20 rows: 10 us by 8 rows, 11.2 by 32; of 400 tokens, 8 heads of
// 128, 32 rows: 11.5 and 14.6.  Up to twice as many blocks, d = 64 with 256 rows: 12.5, else 13.7; d = 128, two of 800 tokens:
// 25.3, else 20.8.)
static int simt_rows(const ssd_paged_kv *kv, const SpanArgs &a) {
  const int64_t rows = (int64_t)a.n * a.G;
  for (int r = 8; r < 32; r *= 2)
    if (rows <= r || (int64_t)kv->batch * kv->h_kv * cdiv64(rows, r) * simt_tiles(kv, a, r) <= 256 / kv->d * sm_count()) return r;
  return rows > 32 && rows <= 96 && cdiv64(rows, 48) < cdiv64(rows, 32) ? 48 : 32;
}

static SimtPlan simt_plan(const ssd_paged_kv *kv, const SpanArgs &a) {
  const int rows = simt_rows(kv, a);
  SimtPlan p = {};
  p.chunks = (int)cdiv64((int64_t)a.n * a.G, rows);
  const int64_t units = (int64_t)kv->batch * kv->h_kv * p.chunks, tiles = simt_tiles(kv, a, rows);
  // about eight blocks per SM (one request of 300 tokens, 2 heads, 20 rows in fp32: two tiles a part 22 us, one 12)
  const int64_t want = 8 * (int64_t)sm_count();
  int64_t parts = units >= want ? 1 : cdiv64(want, units > 0 ? units : 1);
  if (parts > tiles) parts = tiles;
  // of two tiles at least where the units fill the SMs (7 requests of 64 tokens, 8 heads, 264 rows: 34 us; of one tile: 42)
  if (units >= 2 * (int64_t)sm_count() && parts > tiles / 2) parts = tiles / 2;
  p.parts = parts < 1 ? 1 : (int)parts;
  return p;
}

static size_t simt_carve(const ssd_paged_kv *kv, const SpanArgs &a, SimtPlan &p, void *ws) {
  Carver c(ws);
  c.take<char>(kCounterBytes);
  if (p.parts > 1) {
    const size_t items = (size_t)kv->batch * kv->h_kv * p.chunks * p.parts, rows = simt_rows(kv, a);
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
  constexpr int smem = sizeof(SimtSmem<T, D, ROWS>);
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  const int64_t items = (int64_t)kv->batch * kv->h_kv * p.chunks * p.parts;
  if (items >= (int64_t)1 << 31) return fail(SSD_ERR_UNSUPPORTED, "span attention: %lld blocks", (long long)items);
  if ((rc = launch(kernel, dim3((unsigned)items), dim3(kSimtThreads), smem, st, "span_simt_kernel", a, p)) || p.parts == 1) return rc;
  const int64_t rows = (int64_t)kv->batch * kv->h_kv * a.n * a.G;
  return launch(span_simt_join_kernel<T, D, ROWS>, dim3((unsigned)cdiv64(rows, 8)), dim3(256), 0, st, "span_simt_join_kernel", a, p);
}

template <typename T, int D>
static int simt_launch_rows(const ssd_paged_kv *kv, const SpanArgs &a, const SimtPlan &p, cudaStream_t st) {
  switch (simt_rows(kv, a)) {
    case 8: return simt_launch<T, D, 8>(kv, a, p, st);
    case 16: return simt_launch<T, D, 16>(kv, a, p, st);
    case 32: return simt_launch<T, D, 32>(kv, a, p, st);
    default: return simt_launch<T, D, 48>(kv, a, p, st);
  }
}

int span_simt(const ssd_paged_kv *kv, const SpanArgs &a, void *workspace, cudaStream_t st) {
  SimtPlan p = simt_plan(kv, a);
  simt_carve(kv, a, p, workspace);
  const bool wide = kv->d == 128;
  if (kv->dtype == SSD_DTYPE_F32) return wide ? simt_launch_rows<float, 128>(kv, a, p, st) : simt_launch_rows<float, 64>(kv, a, p, st);
  return wide ? simt_launch_rows<__nv_bfloat16, 128>(kv, a, p, st) : simt_launch_rows<__nv_bfloat16, 64>(kv, a, p, st);
}

}  // namespace ssd
