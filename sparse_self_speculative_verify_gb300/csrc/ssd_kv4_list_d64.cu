// ssd_kv4_list_d64.cu -- the 4-bit draft and criticality kernels at d = 64.
#include "ssd_kv4_attn.cuh"

namespace ssd {
int kv4_list_d64(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st) {
  return nt == 1 ? kv4_attn_types<64, 1, true>(a, grid, st) : kv4_attn_types<64, 2, true>(a, grid, st);
}
int kv4_crit_d64(const Kv4AttnArgs &a, int nt, int grid, cudaStream_t st) {
  switch (nt) {
    case 1: return a.q_f32 ? kv4_launch_crit<1, 2>(a, grid, st) : kv4_launch_crit<1, 1>(a, grid, st);
    case 2: return a.q_f32 ? kv4_launch_crit<2, 2>(a, grid, st) : kv4_launch_crit<2, 1>(a, grid, st);
    case 3: return a.q_f32 ? kv4_launch_crit<3, 2>(a, grid, st) : kv4_launch_crit<3, 1>(a, grid, st);
    default: return a.q_f32 ? kv4_launch_crit<4, 2>(a, grid, st) : kv4_launch_crit<4, 1>(a, grid, st);
  }
}
}  // namespace ssd
