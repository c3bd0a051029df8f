// ssd_span.h -- host side of span attention: its two paths.
#pragma once

#include "ssd_host.h"
#include "ssd_span.cuh"

namespace ssd {

// CUDA cores: fp32 caches, pages below 8 tokens.
size_t span_simt_workspace(const ssd_paged_kv *kv, const SpanArgs &a);
int span_simt(const ssd_paged_kv *kv, const SpanArgs &a, void *workspace, cudaStream_t st);

}  // namespace ssd
