// ssd_cache.h -- host-side checks of caches of any element type.
#pragma once

#include "ssd_host.h"

namespace ssd {

// As validate_kv, for the element types listed as bits in `kinds`.
constexpr unsigned kCache16Or32 = 1u, kCacheNvfp4 = 2u;
int validate_cache(const ssd_paged_kv *kv, KVView *v, const char *who, unsigned kinds);
// Longest token list of a call, as max_seq_len: positions, and tiles past their end, stay in 32 bits.
constexpr int kMaxList = 1 << 24;
// A 4-bit cache's k_scale and v_scale: powers of two, so that applying them never rounds.
int kv4_scales_ok(float k_scale, float v_scale, const char *who);

}  // namespace ssd
