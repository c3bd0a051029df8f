// ssd_kv4_tc.cu -- launches of the tcgen05 kernels over a 4-bit cache (d = 128).
#include "ssd_host.h"
#include "ssd_kv4_tc.cuh"

namespace ssd {

template <int NP, int CW, int QS, int PS>
static int launch_tc(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr auto kernel = kv4_tc_kernel<NP, CW, QS, PS>;
  constexpr int smem = Kv4TcCfg<NP, QS, PS>::kSmem;
  int rc = ensure_smem<kernel>(smem);
  static_assert(smem * 2 <= 225 * 1024, "the blocks of an SM fit");
  if (rc) return rc;
  if ((rc = launch(kernel, dim3(grid), dim3(kKv4TcWarps * 32), smem, st, "kv4_tc_kernel", a)) || !a.join_blocks) return rc;
  return launch(kv4_join_kernel<NP>, dim3(cdiv(2 * CW, kKv4JoinRows), a.n_units), dim3(kKv4JoinRows * 32), 0, st,
                "kv4_join_kernel", a);
}

template <int NP, int CW>
static int launch_types(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  return a.q_f32 ? launch_tc<NP, CW, 2, 2>(a, grid, st) : a.out_f32 ? launch_tc<NP, CW, 1, 2>(a, grid, st) : launch_tc<NP, CW, 1, 1>(a, grid, st);
}

template <int NP, int CR, int QS>
static int launch_crit(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  constexpr int BPS = QS == 2 && NP == 64 ? 2 : NP == 64 ? 3 : kKv4CritTcBlocks;
  constexpr auto kernel = kv4_crit_tc_kernel<NP, CR, QS, BPS>;
  constexpr int smem = Kv4CritCfg<NP, QS>::kSmem;
  static_assert(smem * BPS <= 227 * 1024, "the blocks of an SM fit");
  int rc = ensure_smem<kernel>(smem);
  if (rc) return rc;
  const int most = sm_count() * BPS;
  return launch(kernel, dim3(grid < most ? grid : most), dim3(kKv4CritTcWarps * 32), smem, st, "kv4_crit_tc_kernel", a);
}

template <int NP, int CR>
static int launch_crit_types(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  return a.q_f32 ? launch_crit<NP, CR, 2>(a, grid, st) : launch_crit<NP, CR, 1>(a, grid, st);
}

// rows: of a pass (more than 8, at most 32).
int kv4_tc_attn(Kv4AttnArgs a, int rows, int grid, cudaStream_t st) {
  // Units of six parts and more: a launch of its own joins them.  8 heads, 20 rows, in place against apart: 4096
  // tokens 22.5 us, 15.7; 131072 tokens 74, 61; 4 requests of 2048 to 8192 tokens 28, 24; 6 of them 30, 27; 8 of
  // them (64 units) 32.5, 31, with the criticality 43, 46.
  a.join_blocks = grid >= 6 * a.n_units && a.n_units <= kKv4JoinMost ? grid : 0;
  return rows <= 16   ? launch_types<16, 8>(a, grid, st)
         : rows <= 24 ? launch_types<32, 12>(a, grid, st)
                      : launch_types<32, 16>(a, grid, st);
}

// All rows (up to 64) at once.
int kv4_tc_crit(const Kv4AttnArgs &a, int grid, cudaStream_t st) {
  return a.R <= 8    ? launch_crit_types<16, 8>(a, grid, st)
         : a.R <= 16 ? launch_crit_types<16, 16>(a, grid, st)
         : a.R <= 24 ? launch_crit_types<32, 24>(a, grid, st)
         : a.R <= 32 ? launch_crit_types<32, 32>(a, grid, st)
         : a.R <= 48 ? launch_crit_types<64, 48>(a, grid, st)
                     : launch_crit_types<64, 64>(a, grid, st);
}

}  // namespace ssd
