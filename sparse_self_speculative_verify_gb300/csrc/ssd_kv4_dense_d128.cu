// ssd_kv4_dense_d128.cu -- the dense 4-bit attention kernels at d = 128.
#include "ssd_kv4_attn.cuh"

namespace ssd {
int kv4_dense_d128(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st) {
  switch (nt) {
    case 1: return kv4_attn_types<128, 1, false>(a, grid, st);
    case 2: return kv4_attn_types<128, 2, false>(a, grid, st);
    case 3: return kv4_attn_types<128, 3, false>(a, grid, st);
    default: return kv4_attn_types<128, 4, false>(a, grid, st);
  }
}
}  // namespace ssd
