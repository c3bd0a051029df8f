// ssd_kv4_list_d128.cu -- the 4-bit draft kernels at d = 128.
#include "ssd_kv4_attn.cuh"

namespace ssd {
int kv4_list_d128(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st) {
  return nt == 1 ? kv4_attn_types<128, 1, true>(a, grid, st) : kv4_attn_types<128, 2, true>(a, grid, st);
}
}  // namespace ssd
