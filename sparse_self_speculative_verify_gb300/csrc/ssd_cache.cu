// ssd_cache.cu -- host-side checks of caches of any element type.
#include "ssd_cache.h"

#include <math.h>

#include "ssd_kv4.cuh"

namespace ssd {

int validate_cache(const ssd_paged_kv *kv, KVView *v, const char *who, unsigned kinds) {
  if (!kv) return fail(SSD_ERR_INVALID_ARG, "%s: kv is NULL", who);
  if (kv->dtype != SSD_DTYPE_NVFP4) {
    if (!(kinds & kCache16Or32)) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype %d (expected SSD_DTYPE_NVFP4)", who, kv->dtype);
    return validate_kv(kv, v, who);
  }
  if (!(kinds & kCacheNvfp4)) return fail(SSD_ERR_UNSUPPORTED, "%s: dtype SSD_DTYPE_NVFP4", who);
  ssd_paged_kv c = *kv;  // everything but the element type is checked alike
  c.dtype = SSD_DTYPE_BF16;
  const int rc = validate_kv(&c, v, who);
  if (rc) return rc;
  if (kv->page_size < kKv4MinPage)
    return fail(SSD_ERR_UNSUPPORTED, "%s: page_size %d of a 4-bit cache is below %d", who, kv->page_size, kKv4MinPage);
  if ((int64_t)kv->page_size * kv->h_kv * kv4_row_bytes(kv->d) >= (int64_t)1 << 30)  // offsets inside a page: 32 bits
    return fail(SSD_ERR_UNSUPPORTED, "%s: a page of 2 GB or more", who);
  return SSD_OK;
}

int kv4_scales_ok(float k_scale, float v_scale, const char *who) {
  for (int i = 0; i < 2; ++i) {
    const float s = i ? v_scale : k_scale;
    int e = 0;
    if (!(s > 0.f) || frexpf(s, &e) != 0.5f || e < -31 || e > 33)
      return fail(SSD_ERR_INVALID_ARG, "%s: k_scale and v_scale must be powers of two between 2^-32 and 2^32", who);
  }
  return SSD_OK;
}

}  // namespace ssd
