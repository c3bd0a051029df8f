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
  int n, d;
  int tokens;               // tokens per block
  float k_mul, v_mul;       // append: 1 / scale, read: scale
  unsigned *status;
};

// 32 bytes from and to global memory: in one access where the base is 32-byte aligned (torch's allocations are; the
// calls ask for 16).
__device__ __forceinline__ void load32(const void *p, bool wide, uint4 &x, uint4 &y) {
  if (wide) {
    asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                 : "l"(p));
  } else {
    x = static_cast<const uint4 *>(p)[0];
    y = static_cast<const uint4 *>(p)[1];
  }
}
__device__ __forceinline__ void store32(void *p, bool wide, const uint4 &x, const uint4 &y) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y),
                 "r"(y.z), "r"(y.w)
                 : "memory");
  } else {
    static_cast<uint4 *>(p)[0] = x;
    static_cast<uint4 *>(p)[1] = y;
  }
}

// 16 elements as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  uint4 v[4];
  __device__ __forceinline__ void load(const float *p, bool wide) {
    load32(p, wide, v[0], v[1]);
    load32(p + 8, wide, v[2], v[3]);
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[4 * k] = __uint_as_float(v[k].x), x[4 * k + 1] = __uint_as_float(v[k].y);
      x[4 * k + 2] = __uint_as_float(v[k].z), x[4 * k + 3] = __uint_as_float(v[k].w);
    }
  }
  // Largest magnitude; infinity or NaN when an element is.
  __device__ __forceinline__ float amax() const {
    float x[16], m = 0.f;
    get(x);
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) odd |= isnan(x[i]), m = fmaxf(m, fabsf(x[i]));
    return odd ? NAN : m;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool wide) { load32(p, wide, v[0], v[1]); }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[8 * k + 2 * i] = bf16_lo(w[i]), x[8 * k + 2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ __forceinline__ float amax() const {  // pairs; max.NaN keeps a NaN
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    }
    const float lo = bf16_lo(m), hi = bf16_hi(m);
    return isnan(lo) || isnan(hi) ? NAN : fmaxf(lo, hi);
  }
};

// A group's scale byte, e4m3(m mul / 6) of its largest magnitude m, and eight values x mul over the scale s as codes.
// fp32 inputs take IEEE divisions.  For bf16 inputs (8 significant bits) the quotients are approximated and
// rounded to fewer bits first:
//   m mul / 6, off by less than 2^-22 relative, to 12 significant bits: it is either one of e4m3's ties (at most
//   5 significant bits, so the rounding restores it exactly) or at least 2^-8 relative away from every tie;
//   x mul r with r = 1 / s, off by less than 2^-21, to a multiple of 2^-10 by adding and taking away 1.5 * 2^13:
//   it is either one of e2m1's ties (multiples of 1/4) or at least 2^-8 relative, so 2^-10, away from every
//   tie.  (Above 8 the spacing is wider, but everything there is 6.)
// The bytes are those of the exact quotients either way.
template <typename T>
__device__ __forceinline__ uint32_t scale_of(float m, float mul);
template <>
__device__ __forceinline__ uint32_t scale_of<float>(float m, float mul) {
  return f32_to_e4m3(__fdiv_rn(m * mul, 6.f));
}
template <>
__device__ __forceinline__ uint32_t scale_of<__nv_bfloat16>(float m, float mul) {
  return f32_to_e4m3(__uint_as_float((__float_as_uint(m * mul * (1.f / 6.f)) + 0x400u) & 0xfffff800u));
}
template <typename T>
__device__ __forceinline__ uint32_t codes_of(const float *x, float mul, float s);
template <>
__device__ __forceinline__ uint32_t codes_of<float>(const float *x, float mul, float s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i] * mul, s);
  return f32_to_e2m1(y);
}
template <>
__device__ __forceinline__ uint32_t codes_of<__nv_bfloat16>(const float *x, float mul, float s) {
  const float r = __fdividef(mul, s);
  constexpr float C = 12288.f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = copysignf(__fadd_rn(__fmaf_rn(x[i], r, C), -C), x[i]);
  return f32_to_e2m1(y);
}

// Quantises one group of K or V into codes (two words) and its scale byte.
template <typename T>
__device__ __forceinline__ bool quantise(const Raw<T> &raw, float mul, uint2 &codes, uint32_t &sc) {
  float x[16];
  raw.get(x);
  float amax = raw.amax();
  const bool bad = !isfinite(amax);
  if (bad) {  // NaN counts as 0
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (isnan(x[i])) x[i] = 0.f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
  }
  sc = scale_of<T>(amax, mul);
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sc) & 0xffffu)));
  codes = s > 0.f ? make_uint2(codes_of<T>(x, mul, s), codes_of<T>(x + 8, mul, s)) : make_uint2(0, 0);
  return bad;
}

// One group of 16 elements per thread and step, of K and of V; consecutive threads take consecutive groups of a
// row, then the next head, then the next token.  blockIdx.y is the request; a request is appended whole or not
// at all, so every block first looks at all the page ids its request needs.
//
// Bound: 2.56 bytes per bf16 element against about 8 instructions; at the first version's 13 (an element's NaN
// looked at on its own, 64-bit index divisions) issue bound it, 62 us for 168 MB of input; 45 us now, 0.7 of the
// measured HBM rate, at 60 % of the issue rate.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads, sizeof(T) == 2 ? 5 : 4) kv4_append_kernel(Kv4RowsArgs a) {
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int L = a.kv.seq_lens[b];
  const int n = a.counts ? a.counts[b] : a.n;
  if (n < 0 || n > a.n || L < 0 || (int64_t)L + n > a.kv.max_seq_len) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_SEQLEN);
    return;
  }
  const int j0 = blockIdx.x * a.tokens, nt = min(a.tokens, n - j0);
  if (nt <= 0) return;
  const int32_t *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
  bool ok = true;
  for (int j = (L >> a.kv.log2_ps) + tid; j <= (L + n - 1) >> a.kv.log2_ps; j += kKv4Threads) {
    const int32_t p = table[j];
    ok &= p >= 0 && (int64_t)p < a.kv.num_pages;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
    return;
  }
  const int log2_gpr = a.d == 128 ? 3 : 2;
  const unsigned per_token = (unsigned)a.kv.h_kv << log2_gpr, total = nt * per_token;
  const int cb = kv4_code_bytes(a.d), sb = kv4_scale_bytes(a.d);
  const int64_t block_bytes = (int64_t)a.kv.page_size * (cb + sb), v_off = a.kv.h_kv * block_bytes;
  const int64_t src0 = ((int64_t)b * a.n + j0) * a.kv.h_kv * a.d;
  const T *kin = static_cast<const T *>(a.k_in) + src0, *vin = static_cast<const T *>(a.v_in) + src0;
  bool bad = false;
  auto store = [&](unsigned e, const Raw<T> &k, const Raw<T> &v) {
    const unsigned jt = e / per_token, in = e - jt * per_token;
    const int g = in >> log2_gpr, c = in & ((1 << log2_gpr) - 1);
    const int t = L + j0 + (int)jt, slot = t & (a.kv.page_size - 1);
    const int32_t p = table[t >> a.kv.log2_ps];
    char *blk = a.pool + ((int64_t)p * 2 * a.kv.h_kv + g) * block_bytes;
    char *to = blk + slot * cb + c * 8, *ts = blk + a.kv.page_size * cb + slot * sb + c;
    uint2 w;
    uint32_t sc;
    bad |= quantise<T>(k, a.k_mul, w, sc);
    *reinterpret_cast<uint2 *>(to) = w;
    *ts = (char)sc;
    bad |= quantise<T>(v, a.v_mul, w, sc);
    *reinterpret_cast<uint2 *>(to + v_off) = w;
    ts[v_off] = (char)sc;
  };
  const bool wide = ((reinterpret_cast<uintptr_t>(a.k_in) | reinterpret_cast<uintptr_t>(a.v_in)) & 31) == 0;
#pragma unroll 1
  for (unsigned e = tid; e < total; e += kKv4Threads) {
    Raw<T> k, v;
    k.load(kin + (int64_t)e * 16, wide), v.load(vin + (int64_t)e * 16, wide);
    store(e, k, v);
  }
  if (bad) atomicOr(a.status, (unsigned)SSD_FAULT_VALUE);
}

__device__ __forceinline__ uint4 bits4(float a, float b, float c, float d) {
  return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ void store_group(float *p, const float (&x)[16], bool wide) {
#pragma unroll
  for (int k = 0; k < 16; k += 8) store32(p + k, wide, bits4(x[k], x[k + 1], x[k + 2], x[k + 3]), bits4(x[k + 4], x[k + 5], x[k + 6], x[k + 7]));
}
__device__ __forceinline__ void store_group(__nv_bfloat16 *p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
  store32(p, wide, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
}

// The reverse: rows first[b] + j, j < counts[b], as T; rows from counts[b] on are zeros.  The values are
// exact in both types (6 significant bits times a power of two).
// Bound by HBM: 8 requests of up to 8192 rows of 8 heads of 128, 53 MB read and 268 MB written (rows behind the counts
// included) in 49 us, 0.97 of its measured rate.
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
  const int j0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n - j0), live = min(nt, n - j0);
  const int log2_ppr = a.d == 128 ? 2 : 1;
  const unsigned per_token = (unsigned)a.kv.h_kv << log2_ppr, total = nt * per_token;
  const int32_t *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
  const int cb = kv4_code_bytes(a.d), sb = kv4_scale_bytes(a.d);
  const int64_t block_bytes = (int64_t)a.kv.page_size * (cb + sb), v_off = a.kv.h_kv * block_bytes;
  const int64_t dst0 = ((int64_t)b * a.n + j0) * a.kv.h_kv * a.d;
  T *ko = static_cast<T *>(a.k_out) + dst0, *vo = static_cast<T *>(a.v_out) + dst0;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out)) & 31) == 0;
  // Two groups of 16 elements per thread and step (with one, the narrow loads filled the load/store queue).
#pragma unroll 1
  for (unsigned e = tid; e < total; e += kKv4Threads) {
    const unsigned jt = e / per_token, in = e - jt * per_token;
    uint4 w[2] = {};
    uint32_t sc[2] = {};
    if ((int)jt < live) {
      const int g = in >> log2_ppr, c = in & ((1 << log2_ppr) - 1);
      const int t = f0 + j0 + (int)jt, slot = t & (a.kv.page_size - 1);
      const int32_t p = table[t >> a.kv.log2_ps];
      if (p < 0 || (int64_t)p >= a.kv.num_pages) {
        atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
      } else {
        const char *blk = a.pool + ((int64_t)p * 2 * a.kv.h_kv + g) * block_bytes;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          w[which] = *reinterpret_cast<const uint4 *>(blk + which * v_off + slot * cb + c * 16);
          sc[which] = *reinterpret_cast<const uint16_t *>(blk + which * v_off + a.kv.page_size * cb + slot * sb + c * 2);
        }
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint32_t s2 = e4m3x2_to_f16x2(sc[which]);
      const float2 s = __half22float2(*reinterpret_cast<const __half2 *>(&s2));
      const float mul = which ? a.v_mul : a.k_mul;
      const uint32_t words[4] = {w[which].x, w[which].y, w[which].z, w[which].w};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float f = (y ? s.y : s.x) * mul;
        float x[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[4];
          e2m1_to_f16x2(words[2 * y + k], h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            x[8 * k + 2 * i] = v.x * f;
            x[8 * k + 2 * i + 1] = v.y * f;
          }
        }
        store_group((which ? vo : ko) + (int64_t)e * 32 + y * 16, x, wide);
      }
    }
  }
}

// Tokens per block: enough groups for the threads, more (up to four steps each) while the grid still covers the
// SMs eight times.  (8 prompts of up to 8192 tokens, 1 / 2 / 4 / 8 / 16 steps: 104 / 96 / 95 / 97 / 109 us with the read.)
static int tokens_per_block(const ssd_paged_kv *kv, int n) {
  const int64_t per_token = (int64_t)kv->h_kv * (kv->d / kKv4Group);
  int64_t steps = per_token * n * kv->batch / ((int64_t)sm_count() * 8 * kKv4Threads);
  steps = steps < 1 ? 1 : (steps > 4 ? 4 : steps);
  int64_t t = steps * kKv4Threads / per_token;
  const int64_t least = cdiv64(n, 65535 * 16);  // grid.x stays far below its limit
  t = t < least ? least : t;
  return (int)(t < 1 ? 1 : t);
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
  a.tokens = tokens_per_block(kv, n_new);
  const dim3 grid(cdiv(n_new, a.tokens), kv->batch), block(kKv4Threads);
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
  a.tokens = tokens_per_block(kv, n);
  const dim3 grid(cdiv(n, a.tokens), kv->batch), block(kKv4Threads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SSD_DTYPE_BF16) return launch(kv4_read_kernel<__nv_bfloat16>, grid, block, 0, st, "kv4_read_kernel", a);
  return launch(kv4_read_kernel<float>, grid, block, 0, st, "kv4_read_kernel", a);
}
