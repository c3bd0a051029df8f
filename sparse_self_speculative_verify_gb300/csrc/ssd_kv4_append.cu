// ssd_kv4_append.cu -- quantising new K / V rows into a 4-bit paged cache, and reading rows back.
//
// Per group of 16 elements x (after division by the cache's k_scale or v_scale, a power of two, so
// exact):  s = e4m3(max |x| / 6),  code_i = e2m1(x_i / s), both to nearest with ties to even and
// saturating; s = 0 stores zeros.  SparseSpec §2.3 / SpecSA "branch handling": the candidates of a round
// are appended at the request's end, as ssd_kv_append does for 16- and 32-bit caches.
#include "ssd_cache.h"
#include "ssd_kv4.cuh"

namespace ssd {

constexpr int kKv4Threads = 256;

struct Kv4RowsArgs {
  KVView kv;
  char *pool;
  const void *k_in, *v_in;  // append
  void *k_out, *v_out;      // read
  const int32_t *first;     // read: first token of each request
  const int32_t *counts;    // rows of each request, or NULL: n for all
  int n, d, gpb;            // gpb: groups of 16 per block
  float k_mul, v_mul;       // append: 1 / scale, read: scale
  unsigned *status;
};

// 16 elements from global memory as fp32.
template <typename T>
__device__ __forceinline__ void load_group(const T *p, float (&x)[16]);
template <>
__device__ __forceinline__ void load_group<float>(const float *p, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + k);
    x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
  }
}
template <>
__device__ __forceinline__ void load_group<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + k);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[8 * k + 2 * i] = bf16_lo(w[i]), x[8 * k + 2 * i + 1] = bf16_hi(w[i]);
  }
}

// Division by the group's scale.  fp32 inputs take the IEEE division.  bf16 inputs (8 significant
// bits) take the product with the rounded reciprocal, off by less than 2^-22 relative, rounded to 17
// significant bits: x / s is either one of e2m1's ties (3 significant bits, times s's 4: 7 bits, so the
// rounding restores it exactly) or at least 2^-8 relative away from every tie, so the code is that of
// the exact quotient.
template <typename T>
__device__ __forceinline__ float scaled(float x, float s, float r);
template <>
__device__ __forceinline__ float scaled<float>(float x, float s, float r) { return __fdiv_rn(x, s); }
template <>
__device__ __forceinline__ float scaled<__nv_bfloat16>(float x, float s, float r) {
  return __uint_as_float((__float_as_uint(x * r) + 0x40u) & ~0x7fu);
}

// One group of 16 elements per thread and step; consecutive threads take consecutive groups of a row,
// then the next head, K before V of a token.  blockIdx.y is the request; a request is appended whole or
// not at all, so every block first looks at all the page ids its request needs.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(Kv4RowsArgs a) {
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int L = a.kv.seq_lens[b];
  const int n = a.counts ? a.counts[b] : a.n;
  if (n < 0 || n > a.n || L < 0 || (int64_t)L + n > a.kv.max_seq_len) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    return;
  }
  const int gpr = a.d / kKv4Group;                      // groups per row
  const int64_t total = (int64_t)n * a.kv.h_kv * gpr;   // of K, and of V
  const int64_t e0 = (int64_t)blockIdx.x * a.gpb;
  if (e0 >= total) return;
  const int32_t *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
  bool ok = true;
  for (int j = (L >> a.kv.log2_ps) + tid; j <= (L + n - 1) >> a.kv.log2_ps; j += kKv4Threads) {
    const int32_t p = __ldg(table + j);
    ok &= p >= 0 && (int64_t)p < a.kv.num_pages;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
    return;
  }
  const int64_t e1 = min(total, e0 + a.gpb);
  const int cb = kv4_code_bytes(a.d), sb = kv4_scale_bytes(a.d);
  const int64_t block_bytes = (int64_t)a.kv.page_size * (cb + sb);
  bool bad = false;
  for (int64_t e = e0 + tid; e < e1; e += kKv4Threads) {
    const int c = (int)(e % gpr);
    const int64_t row = e / gpr;
    const int g = (int)(row % a.kv.h_kv);
    const int j = (int)(row / a.kv.h_kv);
    const int t = L + j, slot = t & (a.kv.page_size - 1);
    const int32_t p = __ldg(table + (t >> a.kv.log2_ps));
    const int64_t src = (((int64_t)b * a.n + j) * a.kv.h_kv + g) * a.d + c * kKv4Group;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[16];
      load_group(static_cast<const T *>(which ? a.v_in : a.k_in) + src, x);
      const float mul = which ? a.v_mul : a.k_mul;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        bad |= !isfinite(x[i]);
        x[i] = isnan(x[i]) ? 0.f : x[i] * mul;
        amax = fmaxf(amax, fabsf(x[i]));
      }
      const uint32_t sc = f32_to_e4m3(__fdiv_rn(amax, 6.f));
      const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sc) & 0xffffu)));
      const float r = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = s > 0.f ? scaled<T>(x[i], s, r) : 0.f;
      char *blk = a.pool + (((int64_t)p * 2 + which) * a.kv.h_kv + g) * block_bytes;
      *reinterpret_cast<uint2 *>(blk + slot * cb + c * 8) = make_uint2(f32_to_e2m1(x), f32_to_e2m1(x + 8));
      blk[a.kv.page_size * cb + slot * sb + c] = (char)sc;
    }
  }
  if (bad) atomicOr(a.status, (unsigned)SSD_FAULT_VALUE);
}

__device__ __forceinline__ void store_group(float *p, const float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    reinterpret_cast<float4 *>(p)[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
}
__device__ __forceinline__ void store_group(__nv_bfloat16 *p, const float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    reinterpret_cast<uint4 *>(p)[k] = make_uint4(pack_bf16(x[8 * k], x[8 * k + 1]), pack_bf16(x[8 * k + 2], x[8 * k + 3]),
                                                 pack_bf16(x[8 * k + 4], x[8 * k + 5]), pack_bf16(x[8 * k + 6], x[8 * k + 7]));
}

// The reverse: rows first[b] + j, j < counts[b], as T; rows from counts[b] on are zeros.  The values are
// exact in both types (6 significant bits times a power of two).
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(Kv4RowsArgs a) {
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int n = a.counts ? a.counts[b] : a.n;
  const int f0 = a.first[b];
  if (n < 0 || n > a.n || f0 < 0 || (int64_t)f0 + n > a.kv.max_seq_len) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    n = 0;
  }
  const int gpr = a.d / kKv4Group;
  const int64_t total = (int64_t)a.n * a.kv.h_kv * gpr;
  const int64_t e0 = (int64_t)blockIdx.x * a.gpb, e1 = min(total, e0 + a.gpb);
  const int32_t *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
  const int cb = kv4_code_bytes(a.d), sb = kv4_scale_bytes(a.d);
  const int64_t block_bytes = (int64_t)a.kv.page_size * (cb + sb);
  for (int64_t e = e0 + tid; e < e1; e += kKv4Threads) {
    const int c = (int)(e % gpr);
    const int64_t row = e / gpr;
    const int g = (int)(row % a.kv.h_kv);
    const int j = (int)(row / a.kv.h_kv);
    const int t = f0 + j, slot = t & (a.kv.page_size - 1);
    int32_t p = -1;
    if (j < n) {
      p = __ldg(table + (t >> a.kv.log2_ps));
      if (p < 0 || (int64_t)p >= a.kv.num_pages) {
        atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
        p = -1;
      }
    }
    const int64_t dst = (((int64_t)b * a.n + j) * a.kv.h_kv + g) * a.d + c * kKv4Group;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[16];
      if (p >= 0) {
        const char *blk = a.pool + (((int64_t)p * 2 + which) * a.kv.h_kv + g) * block_bytes;
        const uint2 w = *reinterpret_cast<const uint2 *>(blk + slot * cb + c * 8);
        const uint32_t sc = (unsigned char)blk[a.kv.page_size * cb + slot * sb + c];
        const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sc) & 0xffffu))) *
                        (which ? a.v_mul : a.k_mul);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[4];
          e2m1_to_f16x2(k ? w.y : w.x, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            x[8 * k + 2 * i] = v.x * s;
            x[8 * k + 2 * i + 1] = v.y * s;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
      store_group(static_cast<T *>(which ? a.v_out : a.k_out) + dst, x);
    }
  }
}

// Groups per block: whole multiples of the block's threads, few enough that the grid covers the SMs.
static int groups_per_block(int64_t total, int batch) {
  const int64_t per_sm = total * batch / ((int64_t)sm_count() * 8 * kKv4Threads);
  const int64_t steps = per_sm < 1 ? 1 : (per_sm > 8 ? 8 : per_sm);
  return (int)steps * kKv4Threads;
}

static int rows_checks(const ssd_paged_kv *kv, KVView *v, const void *k, const void *vv, int dtype, int n, float k_scale,
                       float v_scale, const char *who) {
  int rc = validate_cache(kv, v, who, kCacheNvfp4);
  if (rc) return rc;
  if (n < 0) return fail(SSD_ERR_INVALID_ARG, "%s: %d rows", who, n);
  if (dtype != SSD_DTYPE_BF16 && dtype != SSD_DTYPE_F32)
    return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d (expected SSD_DTYPE_BF16 or SSD_DTYPE_F32)", who, dtype);
  if ((rc = kv4_scales_ok(k_scale, v_scale, who))) return rc;
  if (kv->batch == 0 || n == 0) return SSD_OK;
  if (kv->batch > 65535) return fail(SSD_ERR_UNSUPPORTED, "%s: batch above 65535", who);
  if (!k || !vv) return fail(SSD_ERR_INVALID_ARG, "%s: the K and V rows must be non-NULL", who);
  if (!aligned16(k) || !aligned16(vv)) return fail(SSD_ERR_INVALID_ARG, "%s: the K and V rows must be 16-byte aligned", who);
  return SSD_OK;
}

}  // namespace ssd

using namespace ssd;

extern "C" int ssd_kv4_append(const ssd_paged_kv *kv, const void *k_new, const void *v_new, int dtype, int n_new,
                              const int32_t *counts, float k_scale, float v_scale, ssd_stream_t stream) {
  const char *who = "ssd_kv4_append";
  Kv4RowsArgs a{};
  int rc = rows_checks(kv, &a.kv, k_new, v_new, dtype, n_new, k_scale, v_scale, who);
  if (rc || kv->batch == 0 || n_new == 0) return rc;
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  a.pool = static_cast<char *>(const_cast<void *>(kv->pool));
  a.k_in = k_new, a.v_in = v_new, a.counts = counts, a.n = n_new, a.d = kv->d;
  a.k_mul = 1.f / k_scale, a.v_mul = 1.f / v_scale;
  const int64_t total = (int64_t)n_new * kv->h_kv * (kv->d / kKv4Group);
  a.gpb = groups_per_block(total, kv->batch);
  const dim3 grid((unsigned)cdiv64(total, a.gpb), kv->batch), block(kKv4Threads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SSD_DTYPE_BF16) return launch(kv4_append_kernel<__nv_bfloat16>, grid, block, 0, st, "kv4_append_kernel", a);
  return launch(kv4_append_kernel<float>, grid, block, 0, st, "kv4_append_kernel", a);
}

extern "C" int ssd_kv4_read(const ssd_paged_kv *kv, const int32_t *first, const int32_t *counts, int n, float k_scale,
                            float v_scale, int dtype, void *k, void *v, ssd_stream_t stream) {
  const char *who = "ssd_kv4_read";
  Kv4RowsArgs a{};
  int rc = rows_checks(kv, &a.kv, k, v, dtype, n, k_scale, v_scale, who);
  if (rc || kv->batch == 0 || n == 0) return rc;
  if (!first) return fail(SSD_ERR_INVALID_ARG, "%s: first must be non-NULL", who);
  if (!(a.status = device_status())) return SSD_ERR_CUDA;
  a.pool = static_cast<char *>(const_cast<void *>(kv->pool));
  a.k_out = k, a.v_out = v, a.first = first, a.counts = counts, a.n = n, a.d = kv->d;
  a.k_mul = k_scale, a.v_mul = v_scale;
  const int64_t total = (int64_t)n * kv->h_kv * (kv->d / kKv4Group);
  a.gpb = groups_per_block(total, kv->batch);
  const dim3 grid((unsigned)cdiv64(total, a.gpb), kv->batch), block(kKv4Threads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SSD_DTYPE_BF16) return launch(kv4_read_kernel<__nv_bfloat16>, grid, block, 0, st, "kv4_read_kernel", a);
  return launch(kv4_read_kernel<float>, grid, block, 0, st, "kv4_read_kernel", a);
}
