// ssd_kv4_tc.cuh -- the dense 4-bit attention at d = 128 on the 5th-generation tensor cores (tcgen05), and the
// criticality pass.
//
// Per tile of 128 tokens of a (request, KV head):
//   S^T [128 tokens x N rows] = K [128 x 128] Q^T,   O^T [128 d x N rows] += V^T [128 x 128 tokens] P^T,
// both M = 128, the narrow N side the padded query rows.  K and V^T are the A operands and live in tensor
// memory: warps convert 4-bit codes to f16 in registers (code times scale is exact in f16) and store
// them there, so that the 512 bytes a dequantised token takes never pass through shared memory, whose
// 128 bytes a clock they would exhaust (1.2 KB a token against 0.5 KB here; HBM delivers a token's 144
// bytes every 6.1 clocks an SM).  The fragments of mma.sync (ssd_kv4_attn.cuh) took 930 instructions per 32 tokens
// and head at 20 rows and 800 for the K half alone of the criticality; converting 144 bytes to 512 takes
// about 350 whatever the rows.
//
// What bounds it: instructions.  A tile takes about 1000 per warp's 32 tokens (V's conversion 260, K's 200, the
// softmax and its probabilities 160, loads 75), at two thirds of the issue rate; the MMAs fill 40 % of their pipe.
// 8 heads, 20 rows: 32 requests of 2048 to 8192 tokens 81 us with bf16 outputs (35 % of the measured HBM rate; mma.sync
// took 120), 92 with fp32 ones, 8 requests of 131072 tokens 335 us (53 %) and 387.
//
// Roles of a block (two blocks share an SM, each filling the other's gaps):
//   warps 0-7  two groups of four (a group covers the 128 lanes), each with half of every step:
//              K: a thread converts 64 d of a token's row into its TMEM lane;
//              V, 64 tokens: ldmatrix transposes pairs of bytes so that a thread holds the codes of two
//              tokens of one d; conversion, tcgen05.st.16x128b into V^T's lanes;
//              softmax, half of the rows: a thread reads its token's lane of S^T and stores the probabilities
//              to shared memory as the B operand, N-major with 128-byte rows; each half has its own references
//              (warps 4-7 also write the output at a segment's end)
//   warp 8     issues the MMAs
//   warp 9     loads the raw tiles (cp.async, four stages for bf16 outputs, three for fp32)
#pragma once

#include "ssd_kv4_attn.cuh"
#include "ssd_sm100.cuh"
#include "ssd_sm100_pairs.cuh"

namespace ssd {

constexpr int kKv4TcTile = 128;
constexpr int kKv4TcWarps = 10;

// For fp32 outputs O^T leaves tensor memory every so many tiles, to be added up in shared memory: the tensor cores add
// with truncation, and over a block's whole part of a context that grew to 3.0e-6 of the output (relative 2-norm; a
// plain fp32 computation is off by 1.2e-6).  Every 8 tiles 2.0e-6, 4 tiles 1.0e-6, 2 tiles 0.6e-6; the round 116.5 us
// without, 119, 119.7, 121.
constexpr int kKv4TcFlush = 4;

template <int NP, int QS, int PS>
struct Kv4TcCfg {
  static constexpr int kStages = PS == 1 ? 4 : 3;  // raw tiles: two blocks' shared memory fits an SM
  // raw stage: K codes, V codes (64 bytes a token, 16-byte pieces permuted), K scales, V scales
  static constexpr int kCodes = kKv4TcTile * 64, kScales = kKv4TcTile * 8;
  static constexpr int kVCodes = kCodes, kKScales = 2 * kCodes, kVScales = 2 * kCodes + kScales;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;
  static constexpr int kP = kStages * kStage;  // offsets
  static constexpr int kQ = kP + kKv4TcTile * 128;
  static constexpr int kQBytes = NP * 256;          // one part of Q: two panels of 64 d
  static constexpr int kSv = kQ + QS * kQBytes;     // V scales as f16 [2][8 groups][128 tokens]
  static constexpr int kO = kSv + 2 * 8 * kKv4TcTile * 2;  // O^T so far [NP][128]
  static constexpr int kMisc = kO + (PS == 2 ? NP * 128 * 4 : 0);
  // per row: factor, reference, change of it, final reference, join's three; per warp and row: two
  static constexpr int kSmem = kMisc + (7 * NP + 8 * NP) * 4 + 32 * 8 + 64 + 1024;
  static constexpr int kTmem = 256;
  // tensor memory columns: K, V^T of two tiles, S^T, O^T
  static constexpr int kColV = 64, kColS = 192, kColO = 224;
};

// D[tmem] (+)= A[tmem] * B[smem], f16 operands.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem), "r"(a_tmem),
      "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 16 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 8 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 4 columns.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float *v) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// N = 8, 12 or 16 columns.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float *v) {
  if (N == 16) tmem_ld16(taddr, v);
  if (N == 8 || N == 12) tmem_ld8(taddr, v);
  if (N == 12) tmem_ld4(taddr + 8, v + 8);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const float *v) {
  const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
  if (N == 16) tmem_st16(taddr, r);
  if (N == 8 || N == 12) tmem_st8(taddr, r);
  if (N == 12) tmem_st4(taddr + 8, r + 8);
}
// 16 lanes x 16 columns: register 2 j + e of lane 4 r + c is row r + 8 e, column 4 j + c.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Arrives once on `bar` when every cp.async issued so far by this thread has landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool group_any(int id, int count, bool v) {
  int r;
  asm volatile(
      "{ .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.s32 %0, 1, 0, q; }\n"
      : "=r"(r)
      : "r"((int)v), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// Byte of 16-byte piece c (of 4) of token t in a raw tile's codes: rows of 64 bytes, two to a line, the pieces
// of four consecutive lines permuted differently.  A thread per token reading one piece each, and ldmatrix
// reading one piece of eight tokens, both touch every bank once.
__device__ __forceinline__ int kv4_raw_piece(int t, int c) { return (t >> 1) * 128 + (((t & 1) * 4 + (c ^ ((t >> 1) & 3))) << 4); }

// Page `lane` of the tile of tokens [t0, t0 + nv) (0 where it has none).
__device__ __forceinline__ int32_t kv4_raw_peek(const Kv4AttnArgs &a, const int32_t *table, int t0, int nv, int lane) {
  const int log2_cs = min(a.kv.log2_ps, 7), at = lane << log2_cs;
  return lane < (kKv4TcTile >> log2_cs) && at < nv ? table[(t0 + at) >> a.kv.log2_ps] : 0;
}
// That raw tile of head `head` (its K block of page 0).
template <bool WITH_V>
__device__ __forceinline__ void kv4_raw_load(const Kv4AttnArgs &a, const char *head, int32_t pid, int t0, int nv, uint32_t dst, int lane) {
  constexpr int kCodes = kKv4TcTile * 64, kScaleAt = (WITH_V ? 2 : 1) * kCodes, kScales = kKv4TcTile * 8;
  const int log2_cs = min(a.kv.log2_ps, 7), mask = a.kv.page_size - 1;
  const uint32_t v_off = (uint32_t)a.kv.h_kv * a.kv.page_size * 72, page_bytes = 2 * v_off;
  const bool ok = pid >= 0 && (int64_t)pid < a.kv.num_pages;
  const unsigned bad = __ballot_sync(0xffffffffu, !ok);
  if (!ok) pid = 0;
  const uint32_t swz = dst + kv4_raw_piece(lane >> 2, lane & 3);
  const char *mine = head + lane * 16;
  auto codes = [&](int i) {  // eight tokens: 512 consecutive bytes of a page
    const int32_t p = __shfl_sync(0xffffffffu, pid, (8 * i) >> log2_cs);
    const char *src = mine + (uint64_t)(uint32_t)p * page_bytes + ((t0 + 8 * i) & mask) * 64;
    cp_async16(swz + i * 512, src, 16);
    if (WITH_V) cp_async16(swz + kCodes + i * 512, src + v_off, 16);
  };
  if (nv >= kKv4TcTile) {
#pragma unroll
    for (int i = 0; i < 16; ++i) codes(i);
  } else {
#pragma unroll 1
    for (int i = 0; 8 * i < nv; ++i) codes(i);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // two tokens' scales to a piece
    const int e = i * 32 + lane, t = 2 * e;
    const int32_t p = __shfl_sync(0xffffffffu, pid, t >> log2_cs);
    if (t < nv) {
      const char *src = head + (uint64_t)(uint32_t)p * page_bytes + a.kv.page_size * 64 + ((t0 + t) & mask) * 8;
      cp_async16(dst + kScaleAt + e * 16, src, 16);
      if (WITH_V) cp_async16(dst + kScaleAt + kScales + e * 16, src + v_off, 16);
    }
  }
  if (bad) {  // rows of pages outside the pool read as zeros: scales of 0
    if (!ok) atomicOr(a.status, (unsigned)SSD_FAULT_PAGE);
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    for (int t = lane; t < kKv4TcTile; t += 32)
      if (bad >> (t >> log2_cs) & 1)
        for (int w = 0; w < (WITH_V ? 2 : 1); ++w)
          asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst + kScaleAt + w * kScales + t * 8), "r"(0) : "memory");
    __threadfence_block();
    __syncwarp();
  }
}

// Pieces [c0, c0 + NC) of 32 d of the K row of token `tw` of a raw tile -> its TMEM lane, 16 columns of two f16 each.
template <int NC>
__device__ __forceinline__ void kv4_convert_k(const char *codes, const char *scales, int tw, int c0, uint32_t taddr) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = c0 + k;
    const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(scales + tw * 8 + 2 * c));
    const uint4 v = *reinterpret_cast<const uint4 *>(codes + kv4_raw_piece(tw, c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t lo = __byte_perm(s2, 0, 0x1010), hi = __byte_perm(s2, 0, 0x3232);
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t f[4];
      e2m1_to_f16x2(w[i], f);
#pragma unroll
      for (int y = 0; y < 4; ++y) r[4 * i + y] = mul_f16x2(f[y], i < 2 ? lo : hi);
    }
    tmem_st16(taddr + 16 * c, r);
  }
}

// Query rows [r0, r0 + rows) as the K-major B operand (128-byte swizzle, panels of 64 d), by four warps; scaling
// as in Kv4Queries.  Rows go CW at a time to the starts of H operand rows; the others hold zeros.
template <int NP, int QS, int H, int CW>
__device__ __forceinline__ void kv4_tc_stage_q(const Kv4AttnArgs &a, int b, int g, int r0, int rows, char *qs, float *s_sl) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  constexpr int U = 4;
#pragma unroll 1
  for (int n0 = warp; n0 < NP; n0 += 4 * U) {
    float x[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int n = n0 + 4 * k, row = n / H * CW + n % H;
#pragma unroll
      for (int y = 0; y < 4; ++y) x[k][y] = 0.f;
      if (n < NP && n % H < CW && row < rows) {
        const int rr = r0 + row;
        const int64_t off = (((int64_t)b * a.n_c + rr / a.G) * a.h_q + g * a.G + rr % a.G) * 128 + lane * 4;
        if (QS == 2) {
          const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + off);
          x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + off);
          x[k][0] = bf16_lo(v.x), x[k][1] = bf16_hi(v.x), x[k][2] = bf16_lo(v.y), x[k][3] = bf16_hi(v.y);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int n = n0 + 4 * k;
      if (n >= NP) break;
      float mx = fmaxf(fmaxf(fabsf(x[k][0]), fabsf(x[k][1])), fmaxf(fabsf(x[k][2]), fabsf(x[k][3])));
      mx = warp_max(mx);
      const int e = (int)(__float_as_uint(mx) >> 23) - 127;
      const int up = (mx == 0.f || e == 128) ? 0 : min(13 - e, 126);
      const float f = __uint_as_float((uint32_t)(127 + up) << 23);
      if (lane == 0) s_sl[n] = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
      const int d = lane * 4;
      char *dst = qs + (d >> 6) * (NP * 128) + sm100::sw128_offset(n, d & 63);
      float lo[4];
      __half hh[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) hh[y] = __float2half_rn(x[k][y] * f), lo[y] = x[k][y] * f - __half2float(hh[y]);
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(pack_half(__half2float(hh[0]), __half2float(hh[1])), pack_half(__half2float(hh[2]), __half2float(hh[3])));
      if (QS == 2) *reinterpret_cast<uint2 *>(dst + NP * 256) = make_uint2(pack_half(lo[0], lo[1]), pack_half(lo[2], lo[3]));
    }
  }
}

// PS = 2: probabilities as the sum of two f16, in 2 NP columns (see kv4_attn_kernel).
// A group of warps has CW rows (of the pass's up to 2 CW) in H = NP / 2 columns: NP is a multiple of 16, but the
// softmax of padding is not worth its instructions.
template <int NP, int CW, int QS, int PS>
__global__ void __launch_bounds__(kKv4TcWarps * 32, 2) kv4_tc_kernel(Kv4AttnArgs a) {
  using C = Kv4TcCfg<NP, QS, PS>;
  constexpr int H = NP / 2;
  constexpr float kLift = kv4_lift(PS), kSlack = kv4_slack(PS);
  using namespace sm100;
  extern __shared__ __align__(16) char smem_raw[];
  char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(sm);
  float *s_sl = reinterpret_cast<float *>(sm + C::kMisc), *s_ms = s_sl + NP, *s_f = s_ms + NP, *s_mfin = s_f + NP, *s_jm = s_mfin + NP,
        *s_jf = s_jm + NP, *s_jl = s_jf + NP, *s_lw = s_jl + NP, *s_red = s_lw + 4 * NP;
  const uint32_t bars = smem_u32(s_red + 4 * NP);
  const uint32_t b_raw = bars, b_free = bars + 8 * C::kStages, b_k = b_free + 8 * C::kStages, b_s = b_k + 8, b_v = b_s + 8, b_p = b_v + 16,
                 b_pv = b_p + 8, b_l = b_pv + 8, b_lfree = b_l + 8, b_drain = b_lfree + 8;
  __shared__ int64_t s_scan[kKv4TcWarps + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < C::kStages; ++i) mbar_init(b_raw + 8 * i, 32), mbar_init(b_free + 8 * i, 8);
    mbar_init(b_k, 8), mbar_init(b_s, 1), mbar_init(b_v, 8), mbar_init(b_v + 8, 8), mbar_init(b_p, 8), mbar_init(b_pv, 1);
    mbar_init(b_l, 4), mbar_init(b_lfree, 4), mbar_init(b_drain, 1);
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&s_tmem), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  pdl_wait();
  Kv4Range rg;
  const bool mine = kv4_range<false, kKv4TcWarps, kKv4TcTile, 1>(a, rg, s_scan);
  if (blockIdx.x == 0)
    for (int b = tid; b < a.kv.batch; b += kKv4TcWarps * 32) effective_len(a.kv, b, a.n_c, a.status);

  // Every role walks the same segments and tiles.  A wait that runs out raises the fault and the abort flag,
  // after which no wait blocks: the roles run to their ends, their results invalid.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!mbar_wait(bar, parity & 1, &s_abort)) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
  };
  struct Seg {
    int b, g, r0, rows, n_tiles, t0, t1, L;
  };
  auto segment = [&]() {
    Seg s;
    s.b = rg.u / (a.kv.h_kv * a.n_chunk), s.g = (rg.u / a.n_chunk) % a.kv.h_kv, s.r0 = (rg.u % a.n_chunk) * 2 * CW;
    s.rows = min(2 * CW, a.R - s.r0);
    s.n_tiles = kv4_tiles<false, kKv4TcTile>(a, rg.u);
    s.t0 = rg.off, s.t1 = kv4_range_end<kKv4TcTile>(rg, s.n_tiles);
    s.L = min(max(a.kv.seq_lens[s.b], 0), a.kv.max_seq_len);
    return s;
  };
  auto advance = [&](const Seg &s) { kv4_range_next<kKv4TcTile>(rg, s.n_tiles); };
  uint32_t n = 0;  // tiles so far
  if (!mine) rg.x = rg.x1 = 0;

  if (warp == 9) {
    // ---------------------------------------------------------------- raw tiles
    for (; rg.x < rg.x1;) {
      const Seg s = segment();
      const char *head = static_cast<const char *>(a.kv.pool) + (uint32_t)s.g * a.kv.page_size * 72;
      const int32_t *table = a.kv.page_table + (int64_t)s.b * a.kv.max_pages;
      int32_t pid = kv4_raw_peek(a, table, s.t0 * kKv4TcTile, s.L - s.t0 * kKv4TcTile, lane);
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int st = n % C::kStages, t0 = t * kKv4TcTile;
        const int32_t now = pid;
        if (t + 1 < s.t1) pid = kv4_raw_peek(a, table, t0 + kKv4TcTile, s.L - t0 - kKv4TcTile, lane);
        wait(b_free + 8 * st, (n / C::kStages + 1) & 1);
        kv4_raw_load<true>(a, head, now, t0, s.L - t0, sbase + st * C::kStage, lane);
        cp_async_arrive(b_raw + 8 * st);
      }
      advance(s);
    }
    pdl_trigger();
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    // The whole warp walks the tiles and one lane issues: operands stay warp-uniform (a single thread's loop
    // took 70 to 95 clocks for each instruction).
    const uint32_t id_qk = idesc_f16_f32(128, NP, 0), id_pv = idesc_f16_f32(128, NP, 1);
    const uint64_t qd = smem_desc(sbase + C::kQ, 16, 1024), pd = smem_desc(sbase + C::kP, kKv4TcTile * 128, 1024);
    const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
    auto qk = [&](uint32_t tile) {
      wait(b_k, tile);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int q = 0; q < QS; ++q)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tmu + C::kColS, tmu + 8 * kk, qd + (uint64_t)((q * C::kQBytes + (kk >> 2) * (NP * 128) + (kk & 3) * 32) >> 4), id_qk,
                       q + kk > 0 ? 1u : 0u);
        mma_commit(b_s);
      }
      __syncwarp();
    };
    for (; rg.x < rg.x1;) {
      const Seg s = segment();
      qk(n);
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        if (t + 1 < s.t1) qk(n + 1);
        wait(b_v + 8 * (n & 1), n >> 1);
        wait(b_p, n);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t vt = tmu + C::kColV + (n & 1) * 64, acc = (PS == 2 ? (t - s.t0) % kKv4TcFlush != 0 : t > s.t0) ? 1u : 0u;
          // The parts of P are panels' columns [0, NP) and [NP, 2 NP).
#pragma unroll
          for (int q = 0; q < PS; ++q)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_f16_ts(tmu + C::kColO, vt + 8 * kk, pd + (uint64_t)((kk * 2048 + q * NP * 2) >> 4), id_pv, q + kk > 0 ? 1u : acc);
          mma_commit(b_pv);
        }
        __syncwarp();
      }
      advance(s);
    }
    // Drain every MMA this warp issued before the tensor memory is released.
    if (elect_one()) mma_commit(b_drain);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(b_drain, 0, &never);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- conversion, softmax, output
    const int grp = warp >> 2, w = warp & 3, tw = tid & 127, c0 = grp * H, bar = 1 + grp;
    const int r = lane >> 2, col = lane & 3;
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    uint32_t seg = 0;
    auto arrive = [&](uint32_t b) {  // for the warp, whose lanes have done what is announced
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    // The group's half of K: 64 d of every token; and V's scales of its 64 tokens as f16 by group of 16 d, so that
    // a thread of convert_v (after a barrier of the group) reads two tokens' at once; 0 behind the request's
    // end, where a slot may hold anything.  left: tokens of the request from the tile's first on.
    auto convert_k = [&](uint32_t tile, int left) {
      const int st = tile % C::kStages;
      const char *raw = sm + st * C::kStage;
      wait(b_raw + 8 * st, tile / C::kStages);
      kv4_convert_k<2>(raw, raw + C::kKScales, tw, 2 * grp, tm + lanes);
      __half *sv = reinterpret_cast<__half *>(sm + C::kSv) + (tile & 1) * 8 * kKv4TcTile + 64 * grp;
      const int tok = 64 * grp + (tw & 63), g4 = (tw >> 6) * 4;
      uint32_t v = *reinterpret_cast<const uint32_t *>(raw + C::kVScales + tok * 8 + g4);
      if (tok >= left) v = 0;
      const uint32_t f[2] = {e4m3x2_to_f16x2(v & 0xffffu), e4m3x2_to_f16x2(v >> 16)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __half2 h2 = *reinterpret_cast<const __half2 *>(&f[k]);
        sv[(g4 + 2 * k) * kKv4TcTile + (tw & 63)] = __low2half(h2);
        sv[(g4 + 2 * k + 1) * kKv4TcTile + (tw & 63)] = __high2half(h2);
      }
    };
    // The group's half of V: 64 tokens.  The stores to tensor memory are waited for with the next K's.
    auto convert_v = [&](uint32_t tile) {
      const int st = tile % C::kStages;
      const __half *sv = reinterpret_cast<const __half *>(sm + C::kSv) + (tile & 1) * 8 * kKv4TcTile + 64 * grp;
      const uint32_t codes = sbase + st * C::kStage + C::kVCodes + grp * 4096 + kv4_raw_piece(lane, w);
      const uint32_t to = tm + C::kColV + (tile & 1) * 64 + 32 * grp + lanes;
      const uint32_t *sg = reinterpret_cast<const uint32_t *>(sv + (2 * w + (r >> 2)) * kKv4TcTile) + col;
      uint32_t m[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) ldsm_x4_t(codes + k * 2048, m[k][0], m[k][1], m[k][2], m[k][3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // 32 tokens: 16 columns
        uint32_t v[2][8];  // [half of the 32 lanes][register of the store]
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // 16 tokens: groups of eight 2 y and 2 y + 1
          const uint32_t ta = __byte_perm(m[k][2 * y], m[k][2 * y + 1], 0x5410), tb = __byte_perm(m[k][2 * y], m[k][2 * y + 1], 0x7632);
          uint32_t ev[4], od[4];
          e2m1_to_f16x2((ta & 0x0f0f0f0fu) | ((tb << 4) & 0xf0f0f0f0u), ev);
          e2m1_to_f16x2(((ta >> 4) & 0x0f0f0f0fu) | (tb & 0xf0f0f0f0u), od);
          const uint32_t s0 = sg[(32 * k + 16 * y) / 2], s1 = sg[(32 * k + 16 * y + 8) / 2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[h][4 * y] = mul_f16x2(ev[h], s0), v[h][4 * y + 1] = mul_f16x2(od[h], s0);
            v[h][4 * y + 2] = mul_f16x2(ev[2 + h], s1), v[h][4 * y + 3] = mul_f16x2(od[2 + h], s1);
          }
        }
        tmem_st_16x128b_x4(to + 16 * k, v[0]);
        tmem_st_16x128b_x4(to + (16u << 16) + 16 * k, v[1]);
      }
      arrive(b_free + 8 * st);
    };

    for (; rg.x < rg.x1; ++seg) {
      const Seg s = segment();
      if (grp == 0) {
        kv4_tc_stage_q<NP, QS, H, CW>(a, s.b, s.g, s.r0, s.rows, sm + C::kQ, s_sl);
        fence_proxy_async_smem();
      }
      convert_k(n, s.L - s.t0 * kKv4TcTile);
      tmem_st_wait();
      tc_fence_before();
      arrive(b_k);
      named_sync(3, 256);  // s_sl and the V scales are staged
      convert_v(n);
      float l[CW];
#pragma unroll
      for (int q = 0; q < CW; ++q) l[q] = 0.f;
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int t0 = t * kKv4TcTile;
        const bool edge = t0 + kKv4TcTile > s.L - a.n_c + 1, more = t + 1 < s.t1;
        wait(b_s, n);
        tc_fence_after();
        float x[CW];
        tmem_ld_n<CW>(tm + lanes + C::kColS + c0, x);
        if (more) convert_k(n + 1, s.L - t0 - kKv4TcTile);
        tmem_ld_wait();
        tmem_st_wait();
        tc_fence_before();
        if (more) arrive(b_k);  // the next tile's K is in place, and S^T has been read
        arrive(b_v + 8 * (n & 1));
        // The group's row i sees the token when it is the request's and its candidate may look at it.
        int first = 0;
        if (edge) first = t0 + tw < s.L ? (t0 + tw - (s.L - a.n_c)) * a.G - s.r0 - grp * CW : CW;
        if (t == s.t0) {  // first references: the tile's largest logits
#pragma unroll
          for (int q = 0; q < CW; ++q) {
            const float v = q < first ? -INFINITY : x[q] * s_sl[c0 + q];
            const float mx = warp_max(v);
            if (lane == 0) s_red[w * NP + c0 + q] = mx;
          }
          named_sync(bar, 128);
          if (tw < CW) {
            const int q = c0 + tw;
            s_ms[q] = fmaxf(fmaxf(fmaxf(s_red[q], s_red[NP + q]), fmaxf(s_red[2 * NP + q], s_red[3 * NP + q])), -1e30f) - kLift;
          }
          named_sync(bar, 128);
        }
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < CW; q += 4) {
          const float4 sl = *reinterpret_cast<const float4 *>(s_sl + c0 + q), ms = *reinterpret_cast<const float4 *>(s_ms + c0 + q);
          x[q] = fmaf(x[q], sl.x, -ms.x), x[q + 1] = fmaf(x[q + 1], sl.y, -ms.y);
          x[q + 2] = fmaf(x[q + 2], sl.z, -ms.z), x[q + 3] = fmaf(x[q + 3], sl.w, -ms.w);
        }
        if (edge) {
#pragma unroll
          for (int q = 0; q < CW; ++q)
            if (q < first) x[q] = -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < CW; ++q) top = fmaxf(top, x[q]);
        const bool moved = group_any(bar, 128, top > kSlack);  // (and the next V scales are staged)
        if (n > 0) wait(b_pv, n - 1);  // P, O and the other V^T are free
        const bool flush = PS == 2 && t > s.t0 && (t - s.t0) % kKv4TcFlush == 0;
        float *so = reinterpret_cast<float *>(sm + C::kO) + c0 * 128 + tw;  // this lane's [CW]
        if (flush) {
          tc_fence_after();
          float o[CW];
          tmem_ld_n<CW>(tm + lanes + C::kColO + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < CW; ++k) so[k * 128] = t == s.t0 + kKv4TcFlush ? o[k] : so[k * 128] + o[k];
        }
        if (moved) {
          // The references move up to the tile's largest logits; O and the sums follow.
#pragma unroll
          for (int q = 0; q < CW; ++q) {
            const float mx = warp_max(x[q]);
            if (lane == 0) s_red[w * NP + c0 + q] = mx;
          }
          named_sync(bar, 128);
          if (tw < CW) {
            const int q = c0 + tw;
            const float up =
                fmaxf(fmaxf(fmaxf(s_red[q], s_red[NP + q]), fmaxf(s_red[2 * NP + q], s_red[3 * NP + q])) - kLift, 0.f);
            s_f[q] = up;
            s_ms[q] += up;
          }
          named_sync(bar, 128);
#pragma unroll
          for (int q = 0; q < CW; ++q) x[q] -= s_f[c0 + q], l[q] *= fast_exp2(-s_f[c0 + q]);
          if (PS == 2 && t - s.t0 >= kKv4TcFlush) {
#pragma unroll
            for (int k = 0; k < CW; ++k) so[k * 128] *= fast_exp2(-s_f[c0 + k]);
          }
          if (t > s.t0 && !flush) {
            tc_fence_after();
            float o[CW];
            tmem_ld_n<CW>(tm + lanes + C::kColO + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < CW; ++k) o[k] *= fast_exp2(-s_f[c0 + k]);
            tmem_st_n<CW>(tm + lanes + C::kColO + c0, o);
            tmem_st_wait();
          }
        }
        char *prow = sm + C::kP + tw * 128;
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          float e[4];
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = fast_exp2(x[c + k]), l[c + k] += e[k];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 h2 = __floats2half2_rn(e[2 * k], e[2 * k + 1]);
            hi[k] = *reinterpret_cast<const uint32_t *>(&h2);
            if (PS == 2) {
              const float2 back = __half22float2(h2);
              lo[k] = pack_half(e[2 * k] - back.x, e[2 * k + 1] - back.y);
            }
          }
          const int piece = (c0 + c) >> 3, in = (c & 4) * 2;
          *reinterpret_cast<uint2 *>(prow + ((piece ^ (tw & 7)) << 4) + in) = make_uint2(hi[0], hi[1]);
          if (PS == 2) *reinterpret_cast<uint2 *>(prow + (((NP / 8 + piece) ^ (tw & 7)) << 4) + in) = make_uint2(lo[0], lo[1]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(b_p);
        if (more) convert_v(n + 1);
      }
      // The segment's sums and references, for the warps that write the output.
#pragma unroll
      for (int q = 0; q < CW; ++q) l[q] = warp_sum(l[q]);
      if (grp == 0) wait(b_lfree, seg + 1);
#pragma unroll
      for (int q = 0; q < CW; ++q)
        if (lane == q) s_lw[w * NP + c0 + q] = l[q];
      if (tw < CW) s_mfin[c0 + tw] = s_ms[c0 + tw];
      if (grp == 0) arrive(b_l);
      // Both groups have read s_sl for the last time: Q is staged again after this.
      named_sync(3, 256);
      if (grp == 0) {
        advance(s);
        continue;
      }
      // Output: lane 16 h + 8 e + rr of the warp's 32 holds d = 32 w + 4 rr + 2 h + e.
      wait(b_pv, n - 1);
      wait(b_l, seg);
      tc_fence_after();
      const int d = 32 * w + 4 * (lane & 7) + 2 * (lane >> 4) + ((lane >> 3) & 1);
      const Kv4Parts<kKv4TcTile> parts(rg, rg.x, s.n_tiles);
      const bool whole = parts.more == 0;
      const int64_t slot = parts.slot((int)blockIdx.x - parts.first);
      auto column = [&](int q) { return q / CW * H + q % CW; };  // of the pass's row q
      auto row_of = [&](int q) {
        const int rr = s.r0 + q;
        return ((int64_t)s.b * a.n_c + rr / a.G) * a.h_q + s.g * a.G + rr % a.G;
      };
      auto sum_of = [&](int c) { return s_lw[c] + s_lw[NP + c] + s_lw[2 * NP + c] + s_lw[3 * NP + c]; };
      auto write = [&](int64_t elem, float v) {
        if (a.out_f32)
          static_cast<float *>(a.out)[elem] = v;
        else
          static_cast<__nv_bfloat16 *>(a.out)[elem] = __float2bfloat16(v);
      };
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float o[CW];
        tmem_ld_n<CW>(tm + lanes + C::kColO + h * H, o);
        tmem_ld_wait();
        if (PS == 2 && s.t1 - s.t0 > kKv4TcFlush) {
          const float *so = reinterpret_cast<const float *>(sm + C::kO) + h * H * 128 + tw;
#pragma unroll
          for (int k = 0; k < CW; ++k) o[k] += so[k * 128];
        }
#pragma unroll
        for (int k = 0; k < CW; ++k) {
          const int q = h * CW + k;
          if (q >= s.rows) break;
          const float Z = sum_of(h * H + k);
          if (whole)
            write(row_of(q) * 128 + d, Z == 0.f ? 0.f : o[k] * (a.v_scale / Z));
          else
            __stcg(a.part_o + (slot * NP + q) * 128 + d, o[k]);
        }
      }
      if (tw < s.rows) {
        const float Z = sum_of(column(tw)), M = s_mfin[column(tw)];
        if (!whole)
          __stcg(reinterpret_cast<float2 *>(a.part_ml) + slot * NP + tw, make_float2(M, Z));
        else
          kv4_row_done(a, row_of(tw), M, Z);
      }
      tc_fence_before();
      arrive(b_lfree);
      if (!whole && !a.join_blocks) {
        // The last block of the unit to arrive joins the partial results.
        named_sync(2, 128);
        if (tw == 0) {
          s_last = kv4_arrive(a.counters + parts.first) == (unsigned)parts.more;
          if (s_last) a.counters[parts.first] = 0;
        }
        named_sync(2, 128);
        if (s_last)
          kv4_join<128, 128>(
              a, parts.more + 1, s.rows, tw, s_jm, s_jf, s_jl, [&](int k) { return parts.slot(k) * NP; }, row_of,
              [] { named_sync(2, 128); });
        named_sync(2, 128);
      }
      advance(s);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tm, C::kTmem);
}

// Joins the units' parts where a unit has many: a warp per row of a unit, 16 parts' loads on their way at once.  The
// last block's 128 threads took 12 us for 17 parts of 20 rows and would take 19 for the 38 of a single long request.
constexpr int kKv4JoinRows = 4;          // per block
constexpr int kKv4JoinMost = 64;         // units
template <int NP>
__global__ void __launch_bounds__(kKv4JoinRows * 32) kv4_join_kernel(Kv4AttnArgs a) {
  constexpr int LEAD = kKv4Lead<kKv4TcTile>;
  const int lane = threadIdx.x & 31, u = blockIdx.y, q = blockIdx.x * kKv4JoinRows + (threadIdx.x >> 5);
  pdl_wait();
  // The unit's place in the line, as kv4_range has it.
  int64_t at = 0, total = 0;
#pragma unroll
  for (int k = 0; k < kKv4JoinMost; k += 32) {
    const int64_t own = k + lane < a.n_units ? kv4_tiles<false, kKv4TcTile>(a, k + lane) + LEAD : 0;
    int64_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int64_t before = __shfl_sync(0xffffffffu, total + inc - own, u & 31);
    if (u >> 5 == k >> 5) at = before;
    total += __shfl_sync(0xffffffffu, inc, 31);
  }
  Kv4Range r;
  r.per = kv4_per(total, a.join_blocks, 1);
  const Kv4Parts<kKv4TcTile> parts(r, at, kv4_tiles<false, kKv4TcTile>(a, u));
  const int r0 = u % a.n_chunk * 32;
  if (parts.more == 0 || q >= min(32, a.R - r0)) return;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.part_o);
  float M = -1e30f, Z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 16;
  for (int k0 = 0; k0 <= parts.more; k0 += U) {
    float2 v[U];
    float4 y[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      v[k] = make_float2(-1e30f, 0.f), y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k <= parts.more) {
        const int64_t row = parts.slot(k0 + k) * NP + q;
        v[k] = __ldcg(ml + row), y[k] = __ldcg(po + row * 32 + lane);
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < U; ++k) top = fmaxf(top, v[k].x);
    const float f0 = fast_exp2(M - top);
    Z *= f0, acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
    M = top;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float f = fast_exp2(v[k].x - M);
      Z = fmaf(v[k].y, f, Z);
      acc.x = fmaf(y[k].x, f, acc.x), acc.y = fmaf(y[k].y, f, acc.y), acc.z = fmaf(y[k].z, f, acc.z), acc.w = fmaf(y[k].w, f, acc.w);
    }
  }
  const int rr = r0 + q, unit = u / a.n_chunk, b = unit / a.kv.h_kv, g = unit % a.kv.h_kv;
  const int64_t row = ((int64_t)b * a.n_c + rr / a.G) * a.h_q + g * a.G + rr % a.G;
  const float f = Z == 0.f ? 0.f : a.v_scale / Z;
  kv4_write4(a, row * 128 + lane * 4, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
  if (lane == 0) kv4_row_done(a, row, M, Z);
}

// ---- criticality ------------------------------------------------------------------------------
constexpr int kKv4CritTcWarps = 6;  // 0-3: K and the sums, 4: MMA issue, 5: raw tiles
constexpr int kKv4CritTcStages = 4;
constexpr int kKv4CritTcBlocks = 4;  // per SM

template <int NP, int QS>
struct Kv4CritCfg {
  static constexpr int kStage = kKv4TcTile * 72;
  static constexpr int kQ = (kKv4CritTcStages * kStage + 1023) / 1024 * 1024;
  static constexpr int kQBytes = NP * 256;
  static constexpr int kMisc = kQ + QS * kQBytes;
  static constexpr int kSmem = kMisc + 3 * NP * 4 + 16 * 8 + 64 + 1024;
  // tensor memory: K, S^T of two tiles (of one, where the rows are many)
  static constexpr int kBufs = NP <= 32 ? 2 : 1;
  static constexpr int kTmem = 128, kColS = 64;
  static_assert(kColS + kBufs * NP <= kTmem, "tensor memory");
};

// A second pass over K alone recomputes the logits of all rows and sums exp2(x - m) / l per token, from each row's
// reference m and 1 / l.  (Keeping them from the first pass would cost 2 R bytes per token each way, more than K's 72
// for R > 18, and a rounding to f16.)
//
// CR: columns that hold rows (the MMA takes NP).  Four blocks share an SM (two, and one S^T: attention and
// criticality of 32 requests of 2048 to 8192 tokens, 8 heads, 20 rows, took 134 us instead of 128).
template <int NP, int CR, int QS, int BPS>
__global__ void __launch_bounds__(kKv4CritTcWarps * 32, BPS) kv4_crit_tc_kernel(Kv4AttnArgs a) {
  using C = Kv4CritCfg<NP, QS>;
  using namespace sm100;
  extern __shared__ __align__(16) char smem_raw[];
  char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(sm);
  float *s_sl = reinterpret_cast<float *>(sm + C::kMisc), *s_ref = s_sl + NP, *s_inv = s_ref + NP;
  const uint32_t bars = smem_u32(s_inv + NP);
  const uint32_t b_raw = bars, b_free = bars + 8 * kKv4CritTcStages, b_k = b_free + 8 * kKv4CritTcStages, b_s = b_k + 8, b_drain = b_s + 16;
  __shared__ int64_t s_scan[kKv4CritTcWarps + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kKv4CritTcStages; ++i) mbar_init(b_raw + 8 * i, 32), mbar_init(b_free + 8 * i, 4);
    mbar_init(b_k, 4), mbar_init(b_s, 1), mbar_init(b_s + 8, 1), mbar_init(b_drain, 1);
    mbar_init_fence();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(&s_tmem), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  // Everything but a.fin was written before the attention kernel ran, which waited for it and only then let
  // this one start; a.fin is waited for below.
  Kv4Range rg;
  const bool mine = kv4_range<false, kKv4CritTcWarps, kKv4TcTile, 1>(a, rg, s_scan);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!mbar_wait(bar, parity & 1, &s_abort)) atomicOr(a.status, (unsigned)SSD_FAULT_TIMEOUT);
  };
  uint32_t n = 0;
  if (!mine) rg.x = rg.x1 = 0;
  if (warp == 5) {
    for (; rg.x < rg.x1;) {
      const int b = rg.u / a.kv.h_kv, g = rg.u % a.kv.h_kv, n_tiles = kv4_tiles<false, kKv4TcTile>(a, rg.u);
      const int t1 = kv4_range_end<kKv4TcTile>(rg, n_tiles);
      const int L = min(max(a.kv.seq_lens[b], 0), a.kv.max_seq_len);
      const char *head = static_cast<const char *>(a.kv.pool) + (uint32_t)g * a.kv.page_size * 72;
      const int32_t *table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
      int32_t pid = kv4_raw_peek(a, table, rg.off * kKv4TcTile, L - rg.off * kKv4TcTile, lane);
      for (int t = rg.off; t < t1; ++t, ++n) {
        const int st = n % kKv4CritTcStages, t0 = t * kKv4TcTile;
        const int32_t now = pid;
        if (t + 1 < t1) pid = kv4_raw_peek(a, table, t0 + kKv4TcTile, L - t0 - kKv4TcTile, lane);
        wait(b_free + 8 * st, (n / kKv4CritTcStages + 1) & 1);
        kv4_raw_load<false>(a, head, now, t0, L - t0, sbase + st * C::kStage, lane);
        cp_async_arrive(b_raw + 8 * st);
      }
      kv4_range_next<kKv4TcTile>(rg, n_tiles);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 4) {
    const uint32_t id_qk = idesc_f16_f32(128, NP, 0), tmu = __shfl_sync(0xffffffffu, tm, 0);
    const uint64_t qd = smem_desc(sbase + C::kQ, 16, 1024);
    uint32_t total = 0;
    while (rg.x < rg.x1) {
      const int n_tiles = kv4_tiles<false, kKv4TcTile>(a, rg.u);
      total += kv4_range_end<kKv4TcTile>(rg, n_tiles) - rg.off;
      kv4_range_next<kKv4TcTile>(rg, n_tiles);
    }
    for (; n < total; ++n) {
      wait(b_k, n);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int q = 0; q < QS; ++q)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tmu + C::kColS + n % C::kBufs * NP, tmu + 8 * kk, qd + (uint64_t)((q * C::kQBytes + (kk >> 2) * (NP * 128) + (kk & 3) * 32) >> 4), id_qk,
                       q + kk > 0 ? 1u : 0u);
        mma_commit(b_s + 8 * (n % C::kBufs));
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(b_drain);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(b_drain, 0, &never);
    __syncwarp();
  } else {
    const int tw = tid;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    auto convert = [&](uint32_t tile) {
      const int st = tile % kKv4CritTcStages;
      wait(b_raw + 8 * st, tile / kKv4CritTcStages);
      kv4_convert_k<4>(sm + st * C::kStage, sm + st * C::kStage + kKv4TcTile * 64, tw, 0, tm + lanes);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_k), mbar_arrive(b_free + 8 * st);
    };
    for (; rg.x < rg.x1;) {
      const int b = rg.u / a.kv.h_kv, g = rg.u % a.kv.h_kv, n_tiles = kv4_tiles<false, kKv4TcTile>(a, rg.u);
      const int t1 = kv4_range_end<kKv4TcTile>(rg, n_tiles);
      const int L = min(max(a.kv.seq_lens[b], 0), a.kv.max_seq_len);
      kv4_tc_stage_q<NP, QS, NP, NP>(a, b, g, 0, min(NP, a.R), sm + C::kQ, s_sl);
      fence_proxy_async_smem();
      named_sync(1, 128);
      convert(n);
      pdl_wait();
      for (int q = tw; q < NP; q += 128) {
        float2 v = make_float2(INFINITY, 0.f);  // the padding, as rows that see nothing: exp2(x - inf) = 0
        if (q < a.R) v = __ldcg(a.fin + ((int64_t)b * a.n_c + q / a.G) * a.h_q + g * a.G + q % a.G);
        s_ref[q] = v.x, s_inv[q] = v.y;
      }
      named_sync(1, 128);
      for (int t = rg.off; t < t1; ++t, ++n) {
        const int tok = t * kKv4TcTile + tw;
        const bool edge = (t + 1) * kKv4TcTile > L - a.n_c + 1;
        wait(b_s + 8 * (n % C::kBufs), n / C::kBufs);
        tc_fence_after();
        const uint32_t s_at = tm + lanes + C::kColS + n % C::kBufs * NP;
        float x[C::kBufs == 1 ? CR : 4];
        if (C::kBufs == 1) {  // the one buffer is read before the next tile's K is announced
#pragma unroll
          for (int c = 0; c < CR; c += 4) tmem_ld4(s_at + c, x + (C::kBufs == 1 ? c : 0));
          tmem_ld_wait();
          tc_fence_before();
        }
        if (t + 1 < t1) convert(n + 1);
        int first = 0;
        if (edge) first = tok < L ? (tok - (L - a.n_c)) * a.G : NP;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CR; c += 8) {
          constexpr int W = 8;
          float v[W];
          if (C::kBufs == 1) {
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] = x[C::kBufs == 1 ? c + k : 0];
          } else {
            tmem_ld8(s_at + c, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int q = 0; q < W; q += 4) {
            const float4 sl = *reinterpret_cast<const float4 *>(s_sl + c + q), ls = *reinterpret_cast<const float4 *>(s_ref + c + q);
            v[q] = fmaf(v[q], sl.x, -ls.x), v[q + 1] = fmaf(v[q + 1], sl.y, -ls.y);
            v[q + 2] = fmaf(v[q + 2], sl.z, -ls.z), v[q + 3] = fmaf(v[q + 3], sl.w, -ls.w);
          }
          if (edge) {
#pragma unroll
            for (int q = 0; q < W; ++q)
              if (c + q < first) v[q] = -INFINITY;
          }
#pragma unroll
          for (int q = 0; q < W; q += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(s_inv + c + q);
            sum[0] = fmaf(fast_exp2(v[q]), f.x, sum[0]), sum[1] = fmaf(fast_exp2(v[q + 1]), f.y, sum[1]);
            sum[2] = fmaf(fast_exp2(v[q + 2]), f.z, sum[2]), sum[3] = fmaf(fast_exp2(v[q + 3]), f.w, sum[3]);
          }
        }
        if (tok < L) a.scores[(int64_t)rg.u * a.scores_stride + tok] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc_fence_before();
      }
      named_sync(1, 128);
      kv4_range_next<kKv4TcTile>(rg, n_tiles);
    }
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tm, C::kTmem);
}

}  // namespace ssd
