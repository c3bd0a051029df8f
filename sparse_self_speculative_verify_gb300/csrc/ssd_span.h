// ssd_span.h -- host side of span attention: its two paths.
#pragma once

#include "ssd_host.h"
#include "ssd_span.cuh"

namespace ssd {

// CUDA cores: fp32 caches, pages below 8 tokens.
size_t span_simt_workspace(const ssd_paged_kv *kv, const SpanArgs &a);
int span_simt(const ssd_paged_kv *kv, const SpanArgs &a, void *workspace, cudaStream_t st);

// Tensor cores: the others.
bool span_tc_takes(const ssd_paged_kv *kv);
size_t span_tc_workspace(const ssd_paged_kv *kv, const SpanArgs &a);
int span_tc(const ssd_paged_kv *kv, const SpanArgs &a, void *workspace, cudaStream_t st);

}  // namespace ssd
