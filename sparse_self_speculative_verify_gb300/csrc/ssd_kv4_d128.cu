// ssd_kv4_d128.cu -- the mma.sync 4-bit attention kernels at d = 128: drafts, and the dense pass of up to 8 rows.
#include "ssd_kv4_attn.cuh"

namespace ssd {
int kv4_dense_d128(const Kv4AttnArgs &a, int grid, cudaStream_t st) { return kv4_attn_types<128, 1, false>(a, grid, st); }
int kv4_list_d128(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st) {
  return nt == 1 ? kv4_attn_types<128, 1, true>(a, grid, st) : kv4_attn_types<128, 2, true>(a, grid, st);
}
}  // namespace ssd
