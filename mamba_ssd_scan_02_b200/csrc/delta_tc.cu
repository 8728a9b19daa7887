// delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor cores (tcgen05 + TMEM).
//
// Within a chunk, with cs the prefix sums of log2(alpha), S the state (P x N) that enters it and the
// rows of K, Q, V its tokens, the token recurrence is
//   (I + L) U = R,   R = beta (V - 2^cs K S^T),   L_ij = beta_i 2^{cs_i - cs_j} k_i.k_j  (j < i)
//   S' = 2^{cs_C} S + U^T diag(2^{cs_C - cs}) K,   y = 2^cs Q S^T + A U,  A_ij = 2^{cs_i - cs_j} q_i.k_j (j <= i)
// (U: what each token really writes, once the tokens before it are erased).  With T = (I + L)^-1,
// everything that does not depend on the state is taken out of the chain from chunk to chunk:
//   M = K^T diag(2^{cs_C - cs}) T  (N x 64),   AT = A T  (64 x 64)
//   chain:  R from K S^T,  then  S'^T = 2^{cs_C} S^T + M R  and  y = 2^cs Q S^T + AT R:
// two dependent products per chunk, K S^T and M R.  One CTA carries 64 state rows of one head through
// the sequence (the rows are independent given K, so a head of 128 rows is two CTAs).
//
// Precision.  The state is fp32, in registers.  Its products run on fp16 operands in two parts,
// hi = fp16(x), lo = fp16(x - hi), which keep 22 bits; the products hi.hi + hi.lo + lo.hi leave an error
// of about 2^-22, so the state stays as near to the fp64 rule as the fp32 recurrence does
// (4e-7 to 7e-7 of its norm at 8192 tokens for both).  K and Q need one part: a row of bf16 numbers times
// a power of two is exact in fp16, and the power and the norm's factor come back in the fp32
// factors rho.  S and R are scaled by powers of two from running bounds of |S| and |V| (state_scale), so
// that fp16's range holds any size of input.  Only what goes into y alone (A, AT, one part of R in
// AT R) is rounded to 11 bits: y is then rounded to bf16's 8.
// T is inverted in fp32: 16 x 16 diagonal blocks by substitution, the rest by block products with
// tf32 in two parts (22 bits).
//
// Roles (16 warps, so that a thread may have 128 registers): warps 0-7 the chain; warps 8-15 the
// chunk's own part (decay masks, inverse, M, AT), one chunk ahead of the chain; the last of them also
// loads (bulk copies of the tiles that the front end prepared and of the rows of V).  The leader thread of each group issues the group's MMAs right after the
// group's barrier and all its threads wait for the commit, so a hand-over is one barrier and one
// mbarrier.  Every wait is bounded: a timeout makes every role leave and latches SSD_ERR_TIMEOUT.
#include "common.cuh"
#include "delta_plan.h"
#include "plan.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int C = kDeltaChunk;
constexpr int kThreads = 16 * 32;
constexpr int kStages = 3;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes
// stage
constexpr uint32_t OFF_RHOK = 2 * kHalf;          // the tile's row factors follow its operands
constexpr uint32_t OFF_RHOQ = OFF_RHOK + 256;
constexpr uint32_t OFF_HI = OFF_RHOQ + 256;       // the head's gates record
constexpr uint32_t OFF_LO = OFF_HI + 256;
constexpr uint32_t OFF_BETA = OFF_LO + 256;
constexpr uint32_t OFF_V = OFF_BETA + 256;        // 64 rows of 128 bytes, 144 apart (no bank conflicts)
constexpr uint32_t kVPitch = 144;
constexpr uint32_t kStage = (OFF_V + C * kVPitch + 1023) / 1024 * 1024;
static_assert(OFF_HI == kDeltaTileBytes && OFF_V == kDeltaTileBytes + kDeltaGateBytes, "records as loaded");
// CTA
constexpr uint32_t OFF_SB = kStages * kStage;     // S operand: [n][p] hi, then lo (128 rows x 128 bytes each)
constexpr uint32_t OFF_RB = OFF_SB + 2 * kHalf;   // R operand: [token][p] hi, lo (64 rows x 128 bytes each)
constexpr uint32_t OFF_T = OFF_RB + 16384;        // [j][i]: T_ij 2^{cs_C - cs_i} rho_i hi, lo; T_ij
constexpr uint32_t OFF_W = OFF_T + 3 * 8192;      // fp32 64 x 72: L below the diagonal, T^T above
constexpr int kWPitch = 72;                       // = 8 mod 32: conflict-free fragment reads
constexpr uint32_t OFF_X = OFF_W + 64 * kWPitch * 4;  // fp32 products of the inverse, 1 KB per warp
constexpr uint32_t OFF_SRHO = OFF_X + 4096;       // 2^{cs_C - cs_i} rho_i
constexpr uint32_t OFF_MAXS = OFF_SRHO + 256;     // largest |S| per chain warp
constexpr uint32_t OFF_MAXV = OFF_MAXS + 32;      // largest |V| per warp, two chunks
constexpr uint32_t OFF_BAR = OFF_MAXV + 64;
enum {
  BAR_FULL,                        // [kStages] stage loaded
  BAR_G = BAR_FULL + kStages,      // K K^T, Q K^T done
  BAR_MM,                          // M and AT done
  BAR_MREADY,                      // M and AT operands in tensor memory (8 warps)
  BAR_MAXV,                        // [2] largest |V| known
  BAR_D1 = BAR_MAXV + 2,           // K S^T, Q S^T done
  BAR_S,                           // M R done
  BAR_O,                           // AT R done
  BAR_END,                         // [2] nothing of a leader's left in flight
  kNumBars = BAR_END + 2
};
constexpr uint32_t OFF_MISC = OFF_BAR + 8 * 32;   // [0] TMEM base, [1] abort flag
constexpr uint32_t kSmem = OFF_MISC + 16 + 1024;  // room to align the base to 1024 bytes
static_assert(kNumBars <= 32 && kSmem <= 232448, "shared memory");
static_assert(OFF_SB % 1024 == 0 && OFF_RB % 1024 == 0 && OFF_T % 1024 == 0, "swizzle alignment");

// TMEM columns.  K rows are lanes 0-63 of G and D1, Q rows lanes 64-127; A (fp16) replaces the Q rows
// of G, the AT operand those of AT (lanes 0-63 of both are never used).
constexpr uint32_t TM_G = 0, TM_M = 64, TM_AT = 128, TM_D1 = 192, TM_S = 320, TM_O = 384, TM_MHI = 448, TM_MLO = 480,
                   TM_COLS = 512;

constexpr uint32_t IDESC_KK = idesc_f16(128, 64, false, false, kFmtF16);   // G: both K-major; AT: A from TMEM
constexpr uint32_t IDESC_D1 = idesc_f16(128, 128, false, true, kFmtF16);   // [K; Q] . [S hi | S lo]
constexpr uint32_t IDESC_M = idesc_f16(128, 64, true, false, kFmtF16);     // K^T . T
constexpr uint32_t IDESC_R = idesc_f16(128, 64, false, true, kFmtF16);     // M or AT (TMEM) . R

__device__ __forceinline__ uint64_t adv(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(d) + (bytes >> 4));
}
__device__ __forceinline__ constexpr uint32_t kstep(int j) { return (j >> 2) * kHalf + (j & 3) * 32; }

__device__ __forceinline__ void issue_G(uint32_t kq, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, 16, 1024);
#pragma unroll
  for (int j = 0; j < 8; ++j) mma_f16_ss(d, adv(a, kstep(j)), adv(a, kstep(j)), IDESC_KK, j > 0);
}
__device__ __forceinline__ void issue_D1(uint32_t kq, uint32_t sbuf, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, 16, 1024), b = smem_desc_sw128(sbuf, kHalf, 1024);
#pragma unroll
  for (int j = 0; j < 8; ++j) mma_f16_ss(d, adv(a, kstep(j)), adv(b, j * 2048), IDESC_D1, j > 0);
}
__device__ __forceinline__ void issue_M(uint32_t kq, uint32_t t, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, kHalf, 1024), b = smem_desc_sw128(t, 16, 1024);
#pragma unroll
  for (int j = 0; j < 8; ++j)  // hi, then lo
    mma_f16_ss(d, adv(a, (j & 3) * 2048), adv(b, (j >> 2) * 8192 + (j & 3) * 32), IDESC_M, j > 0);
}
__device__ __forceinline__ void issue_AT(uint32_t a_tmem, uint32_t t, uint32_t d) {
  const uint64_t b = smem_desc_sw128(t, 16, 1024);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_f16_ts(d, a_tmem + 8 * j, adv(b, 32 * j), IDESC_KK, j > 0);
}
// (a_tmem: 64 columns of K, fp16) . R part, adding to d if acc
__device__ __forceinline__ void issue_R(uint32_t a_tmem, uint32_t r, uint32_t d, bool acc) {
  const uint64_t b = smem_desc_sw128(r, 8192, 1024);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_f16_ts(d, a_tmem + 8 * j, adv(b, 2048 * j), IDESC_R, (acc || j > 0) ? 1u : 0u);
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return (uint32_t)row * 128u + ((uint32_t)(chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
// fp16 pairs of (a, b): hi, and lo = what hi leaves
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = h2(h);
  lo = h2(__floats2half2_rn(a - f.x, b - f.y));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Powers of two that bring a quantity bounded by m to [64, 128) and back.  Headroom: with alpha <= 1
// and beta |k|^2 <= 2 the transition does not expand a state row s, so over a chunk
// |s'| <= gamma |s| + 64 * 2 max|V|, and |R| <= 2 (max|V| + |s|).  With m = gamma max|S_old| + max|V| that
// is |S| <= (sqrt(128) + 128) m < 140 m and |R| < 282 max(m, max|V|): both below 65504 / 128 = 511.
__device__ __forceinline__ float2 state_scale(float m) {
  const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u), 8), 254);
  return make_float2(__uint_as_float((uint32_t)(260 - e) << 23), __uint_as_float((uint32_t)(e - 6) << 23));
}

// ---- tf32 block products of the inverse -----------------------------------------------------------
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// c += A . B with A[r][k] = a[r * ar + k * ak] (16 x 8) and B[k][n] = b[k * bk + n] (8 x 8)
__device__ __forceinline__ void block_mma(float (&c)[4], const float *a, int ar, int ak, const float *b, int bk, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t ah[4], al[4], bh[2], bl[2];
  split_tf32(a[g * ar + t * ak], ah[0], al[0]);
  split_tf32(a[(g + 8) * ar + t * ak], ah[1], al[1]);
  split_tf32(a[g * ar + (t + 4) * ak], ah[2], al[2]);
  split_tf32(a[(g + 8) * ar + (t + 4) * ak], ah[3], al[3]);
  split_tf32(b[t * bk + g], bh[0], bl[0]);
  split_tf32(b[(t + 4) * bk + g], bh[1], bl[1]);
  mma_tf32(c, al, bh);
  mma_tf32(c, ah, bl);
  mma_tf32(c, ah, bh);
}

// W = T^T of the 32 x 32 diagonal block at p0 of L (both in w, see OFF_W), by one warp.
__device__ __forceinline__ void invert32(float *w, float *x, int p0, int lane) {
  {  // the two 16 x 16 blocks, a column of T per lane: t_i = [i == j] - sum_{m < i} L_im t_m
    const int b0 = p0 + (lane & 16), j = lane & 15;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int m4 = 0; m4 < (i + 3) / 4; ++m4) {
        const float4 l = *reinterpret_cast<const float4 *>(w + (b0 + i) * kWPitch + b0 + 4 * m4);
        s0 = fmaf(-l.x, t[4 * m4], s0);
        if (4 * m4 + 1 < i) s1 = fmaf(-l.y, t[4 * m4 + 1], s1);
        if (4 * m4 + 2 < i) s0 = fmaf(-l.z, t[4 * m4 + 2], s0);
        if (4 * m4 + 3 < i) s1 = fmaf(-l.w, t[4 * m4 + 3], s1);
      }
      t[i] = s0 + s1;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4 *>(w + (b0 + j) * kWPitch + b0 + i) = make_float4(t[i], t[i + 1], t[i + 2], t[i + 3]);
  }
  __syncwarp();
  // W12 = -W11 Z12 W22 with Z12[j][i] = L_ij of the block below
  const int g = lane >> 2, t = lane & 3;
  const float *w22 = w + (p0 + 16) * kWPitch + p0 + 16;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kt = 0; kt <= nt; ++kt)  // W22 is upper triangular
      block_mma(c, w + (p0 + 16 + 8 * kt) * kWPitch + p0, 1, kWPitch, w22 + 8 * kt * kWPitch + 8 * nt, kWPitch, lane);
    *reinterpret_cast<float2 *>(x + nt * 128 + g * 8 + 2 * t) = make_float2(c[0], c[1]);
    *reinterpret_cast<float2 *>(x + nt * 128 + (g + 8) * 8 + 2 * t) = make_float2(c[2], c[3]);
  }
  __syncwarp();
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
      block_mma(c, w + p0 * kWPitch + p0 + 8 * kt, kWPitch, 1, x + nt * 128 + kt * 64, 8, lane);
    float *o = w + p0 * kWPitch + p0 + 16 + 8 * nt + 2 * t;
    *reinterpret_cast<float2 *>(o + g * kWPitch) = make_float2(-c[0], -c[1]);
    *reinterpret_cast<float2 *>(o + (g + 8) * kWPitch) = make_float2(-c[2], -c[3]);
  }
}

__global__ void __launch_bounds__(kThreads, 1) ssd_delta_chunk_kernel(const DeltaPlan p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int halves = p.P >> 6;
  const int h = blockIdx.x / halves, ph = blockIdx.x % halves;
  const int seq = p.order ? p.order[blockIdx.y] : (int)blockIdx.y;
  const int len = seq_len(p.cu, seq, p.L);
  const long long base = seq_base(p.cu, seq, p.L);
  const int nck = (len + C - 1) / C;
  const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
  const uint32_t bar0 = sb + OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
  const auto wait = [&](int bar, uint32_t parity) { return mbar_wait(BAR(bar), parity, abort_flag, p.err); };

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(BAR(i), i == BAR_MREADY ? 8 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // the part of T above the diagonal blocks stays zero
  for (int i = tid; i < 3 * 8192 / 16; i += kThreads) reinterpret_cast<uint4 *>(smem + OFF_T)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == 14) {
    tmem_alloc(sb + OFF_MISC, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int q4 = warp & 3;                           // TMEM lanes 32 q4 ..
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
  const int hf = (warp >> 2) & 1;                    // columns 32 hf ..

  if (warp >= 8) {
    // ------------------------------------------------------------------ the chunk's own part
    const int ow = warp - 8;
    const bool leader = ow == 0 && lane == 0;
    float *w = reinterpret_cast<float *>(smem + OFF_W);
    float *srho = reinterpret_cast<float *>(smem + OFF_SRHO);
    const int row = 32 * (q4 & 1) + lane;  // K or Q row of this thread's lane of G
    const bool is_q = q4 >= 2;
    int loaded = 0;
    const auto load = [&](int c) {  // chunk c into its stage, by the last warp
      const int rows = min(C, len - c * C);
      const uint32_t dst = sb + c % kStages * kStage, full = BAR(BAR_FULL + c % kStages);
      if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(kDeltaTileBytes + kDeltaGateBytes) + rows * 128);
      __syncwarp();
      const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + (base + c * C) * p.vs + h * p.P + 64 * ph;
      for (int r = lane; r < rows; r += 32) bulk_load(dst + OFF_V + r * kVPitch, v + r * p.vs, 128, full);
      if (lane == 0) {
        // V is the caller's; the tiles and gates are the front end's, which may still be running
        // (programmatic dependent launch)
        if (c == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        bulk_load(dst, p.tiles + ((ck0 + c) * p.G + h / p.hpg) * kDeltaTileBytes, (uint32_t)kDeltaTileBytes, full);
        bulk_load(dst + OFF_HI, p.gates + ((ck0 + c) * p.H + h) * (kDeltaGateBytes / 4), (uint32_t)kDeltaGateBytes, full);
      }
      __syncwarp();
      ++loaded;
    };
    if (ow == 7)
      for (int c = 0; c < min(nck, kStages); ++c) load(c);
    for (int c = 0; c < nck; ++c) {
      const int st = c % kStages;
      unsigned char *stage = smem + st * kStage;
      const float *hi = reinterpret_cast<const float *>(stage + OFF_HI), *lo = reinterpret_cast<const float *>(stage + OFF_LO);
      const float *rk = reinterpret_cast<const float *>(stage + OFF_RHOK);
      wait(BAR_FULL + st, (c / kStages) & 1);
      if (c == 0) {
        if (leader) {
          issue_G(sb + st * kStage, tmem + TM_G);
          mma_commit(BAR(BAR_G));
        }
        __syncwarp();
      }
      {  // largest |V| of the chunk
        const int rows = min(C, len - c * C), t = tid - 256;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = t + 256 * i;
          if ((at >> 3) < rows) {
            const uint4 u = *reinterpret_cast<const uint4 *>(stage + OFF_V + (at >> 3) * kVPitch + (at & 7) * 16);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(x[k] & 0x7fffu, (x[k] >> 16) & 0x7fffu));
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) reinterpret_cast<uint32_t *>(smem + OFF_MAXV)[8 * (c & 1) + ow] = top << 16;
      }
      const float hi_end = hi[C - 1], lo_end = lo[C - 1];
      if (tid - 256 < C) srho[tid - 256] = ex2((hi_end - hi[tid - 256]) + (lo_end - lo[tid - 256])) * rk[tid - 256];
      wait(BAR_G, c & 1);
      __syncwarp();
      tc_fence_after();
      uint32_t pk[16];
      {
        // rows of L = beta_i 2^{cs_i - cs_j} k_i.k_j for j < i, or of A = 2^{cs_i - cs_j} q_i.k_j for j <= i
        // (Q's row factor is applied to y)
        float v[32];
        const bool none = hf == 1 && (q4 & 1) == 0;  // columns 32.. of rows 0-31
        if (!none) {
          tmem_ld32(tmem + TM_G + 32 * hf + lane_off, v);
          tmem_ld_wait();
          const float hr = hi[row], lr = lo[row];
          const float f = is_q ? 1.f : reinterpret_cast<const float *>(stage + OFF_BETA)[row] * rk[row];
          const int last = row - 32 * hf - (is_q ? 0 : 1);  // last column kept
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 hj = *reinterpret_cast<const float4 *>(hi + 32 * hf + j);
            const float4 lj = *reinterpret_cast<const float4 *>(lo + 32 * hf + j);
            const float4 rj = *reinterpret_cast<const float4 *>(rk + 32 * hf + j);
            v[j] = j <= last ? v[j] * (f * rj.x) * ex2((hr - hj.x) + (lr - lj.x)) : 0.f;
            v[j + 1] = j + 1 <= last ? v[j + 1] * (f * rj.y) * ex2((hr - hj.y) + (lr - lj.y)) : 0.f;
            v[j + 2] = j + 2 <= last ? v[j + 2] * (f * rj.z) * ex2((hr - hj.z) + (lr - lj.z)) : 0.f;
            v[j + 3] = j + 3 <= last ? v[j + 3] * (f * rj.w) * ex2((hr - hj.w) + (lr - lj.w)) : 0.f;
          }
        }
        if (is_q) {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = none ? 0u : h2(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
        } else if (!none) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(w + row * kWPitch + 32 * hf + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
      tc_fence_before();
      if (named_bar_or(2, 256, *abort_flag != 0)) break;
      if (leader) mbar_arrive(BAR(BAR_MAXV + (c & 1)));
      if (is_q) {  // every warp has read G: A over its Q rows
        tc_fence_after();
        tmem_st16(tmem + TM_G + 16 * hf + lane_off, pk);
        tmem_st_wait();
      } else if (ow < 2) {
        invert32(w, reinterpret_cast<float *>(smem + OFF_X) + 256 * ow, 32 * ow, lane);
      }
      named_bar(2, 256);
      if (ow < 4) {
        // W12 = -W11 Z12 W22 of the 32 x 32 blocks, 8 columns per warp; out as T operands
        float *x = reinterpret_cast<float *>(smem + OFF_X) + 256 * ow;
        const int g = lane >> 2, t = lane & 3;
        float cc[2][4] = {};
        for (int kt = 0; kt <= ow; ++kt) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
            block_mma(cc[mt], w + (32 + 8 * kt) * kWPitch + 16 * mt, 1, kWPitch,
                      w + (32 + 8 * kt) * kWPitch + 32 + 8 * ow, kWPitch, lane);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          *reinterpret_cast<float2 *>(x + (16 * mt + g) * 8 + 2 * t) = make_float2(cc[mt][0], cc[mt][1]);
          *reinterpret_cast<float2 *>(x + (16 * mt + g + 8) * 8 + 2 * t) = make_float2(cc[mt][2], cc[mt][3]);
        }
        __syncwarp();
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kt = 2 * mt; kt < 4; ++kt)  // W11 is upper triangular
            block_mma(d, w + 16 * mt * kWPitch + 8 * kt, kWPitch, 1, x + kt * 64, 8, lane);
          const float2 f = *reinterpret_cast<const float2 *>(srho + 32 + 8 * ow + 2 * t);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int j = 16 * mt + g + 8 * u;
            const float a = -d[2 * u], b = -d[2 * u + 1];
            unsigned char *o = smem + OFF_T + swz(j, 4 + ow) + 4 * t;
            uint32_t hv, lv;
            split2(a * f.x, b * f.y, hv, lv);
            *reinterpret_cast<uint32_t *>(o) = hv;
            *reinterpret_cast<uint32_t *>(o + 8192) = lv;
            *reinterpret_cast<uint32_t *>(o + 16384) = h2(__floats2half2_rn(a, b));
          }
        }
      } else {
        // the diagonal 32 x 32 blocks of T, 16 elements of a row of T^T per thread
        const int t = 32 * (ow - 4) + lane, j = t >> 1, i0 = (j & 32) + 16 * (t & 1);
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(w + j * kWPitch + i0 + i);
          v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
        }
        uint32_t hv[8], lv[8], tv[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float a = i0 + i >= j ? v[i] : 0.f, b = i0 + i + 1 >= j ? v[i + 1] : 0.f;
          const float2 f = *reinterpret_cast<const float2 *>(srho + i0 + i);
          split2(a * f.x, b * f.y, hv[i / 2], lv[i / 2]);
          tv[i / 2] = h2(__floats2half2_rn(a, b));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          unsigned char *o = smem + OFF_T + swz(j, i0 / 8 + u);
          *reinterpret_cast<uint4 *>(o) = make_uint4(hv[4 * u], hv[4 * u + 1], hv[4 * u + 2], hv[4 * u + 3]);
          *reinterpret_cast<uint4 *>(o + 8192) = make_uint4(lv[4 * u], lv[4 * u + 1], lv[4 * u + 2], lv[4 * u + 3]);
          *reinterpret_cast<uint4 *>(o + 16384) = make_uint4(tv[4 * u], tv[4 * u + 1], tv[4 * u + 2], tv[4 * u + 3]);
        }
      }
      fence_proxy_async();
      tc_fence_before();
      if (named_bar_or(2, 256, *abort_flag != 0)) break;
      if (leader) {
        tc_fence_after();
        issue_M(sb + st * kStage, sb + OFF_T, tmem + TM_M);
        issue_AT(tmem + TM_G, sb + OFF_T + 16384, tmem + TM_AT);
        mma_commit(BAR(BAR_MM));
      }
      __syncwarp();
      wait(BAR_MM, c & 1);
      __syncwarp();
      tc_fence_after();
      if (leader) {
        if (c + 1 < nck && wait(BAR_FULL + (c + 1) % kStages, ((c + 1) / kStages) & 1)) {
          issue_G(sb + (c + 1) % kStages * kStage, tmem + TM_G);
          mma_commit(BAR(BAR_G));
        }
      }
      __syncwarp();
      // M and AT become operands in tensor memory once the chain's products of the chunk before have
      // read the previous ones
      {
        float m[32];
        tmem_ld32(tmem + TM_M + 32 * hf + lane_off, m);
        tmem_ld_wait();
        uint32_t mh[16], ml[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) split2(m[2 * j], m[2 * j + 1], mh[j], ml[j]);
        if (is_q) {
          tmem_ld32(tmem + TM_AT + 32 * hf + lane_off, m);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = h2(__floats2half2_rn(m[2 * j], m[2 * j + 1]));
          tc_fence_before();
          named_bar(3, 128);  // both halves of the row are read: the operand goes over them
          tc_fence_after();
        }
        if (c > 0) {
          const bool ok = wait(BAR_O, (c - 1) & 1);
          // that was the last use of chunk c - 1's stage, by the chain and here
          if (ow == 7 && c - 1 + kStages < nck && __all_sync(0xffffffffu, ok)) load(c - 1 + kStages);
        }
        __syncwarp();
        tc_fence_after();
        tmem_st16(tmem + TM_MHI + 16 * hf + lane_off, mh);
        tmem_st16(tmem + TM_MLO + 16 * hf + lane_off, ml);
        if (is_q) tmem_st16(tmem + TM_AT + 16 * hf + lane_off, pk);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_MREADY));
    }
    if (leader) {  // no MMA may still be running when TMEM is released
      mma_commit(BAR(BAR_END));
      int never_abort = 0;
      mbar_wait(BAR(BAR_END), 0, &never_abort, p.err);
    }
    if (ow == 7 && lane == 0) {  // and every load must have landed before the CTA may exit
      int never_abort = 0;
      for (int j = max(0, loaded - kStages); j < loaded; ++j)
        mbar_wait(BAR(BAR_FULL + j % kStages), (j / kStages) & 1, &never_abort, p.err);
    }
  } else {
    // ------------------------------------------------------------------ the chain
    const bool leader = tid == 0;
    const int n = 32 * q4 + lane;           // state column of this thread; it holds rows 32 hf ..
    const int row = 32 * (q4 & 1) + lane;   // token of this thread's lane of D1 and O
    const bool is_q = q4 >= 2;
    const long long soff = (((long long)seq * p.H + h) * p.P + 64 * ph + 32 * hf) * kDState + n;
    uint32_t *max_s = reinterpret_cast<uint32_t *>(smem + OFF_MAXS);
    const uint32_t *max_v = reinterpret_cast<const uint32_t *>(smem + OFF_MAXV);
    float S[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) S[i] = p.h0 ? p.h0[soff + (long long)i * kDState] : 0.f;
    const auto publish_max = [&] {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(S[i]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) max_s[warp] = top;
    };
    const auto read_max = [](const uint32_t *m) {
      const uint4 a = *reinterpret_cast<const uint4 *>(m), b = *reinterpret_cast<const uint4 *>(m + 4);
      return __uint_as_float(max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w))));
    };
    publish_max();
    named_bar(1, 256);
    float m = read_max(max_s);  // bounds |S| as described at state_scale
    float qs[32];               // 2^cs Q S^T of the chunk whose y is still to come
    float back_o = 0.f, rho_q = 0.f;
    const auto put_y = [&](int c) {  // Q rows: y of chunk c
      wait(BAR_O, c & 1);
      __syncwarp();
      tc_fence_after();
      const int t = c * C + row;
      const long long yo = (base + t) * p.ys + (long long)h * p.P + 64 * ph + 32 * hf;
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + yo);
      const bool store = t < len && in_bounds(yo + 31, p.y_extent, p.err);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float o[16];
        tmem_ld16(tmem + TM_O + 32 * hf + 16 * x + lane_off, o);
        tmem_ld_wait();
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(rho_q * fmaf(back_o, o[2 * i], qs[16 * x + 2 * i]),
                                                         rho_q * fmaf(back_o, o[2 * i + 1], qs[16 * x + 2 * i + 1]));
          u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if (store) {
          dst[2 * x] = make_uint4(u[0], u[1], u[2], u[3]);
          dst[2 * x + 1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
      tc_fence_before();
    };
    bool done = true;
    for (int c = 0; c < nck; ++c) {
      const int st = c % kStages;
      const unsigned char *stage = smem + st * kStage;
      const float2 sc = state_scale(m);
      // S into its operand
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hv[4], lv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(S[8 * k + 2 * i] * sc.x, S[8 * k + 2 * i + 1] * sc.x, hv[i], lv[i]);
        unsigned char *o = smem + OFF_SB + swz(n, 4 * hf + k);
        *reinterpret_cast<uint4 *>(o) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        *reinterpret_cast<uint4 *>(o + kHalf) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
      }
      fence_proxy_async();
      tc_fence_before();
      if (named_bar_or(1, 256, *abort_flag != 0)) { done = false; break; }
      if (leader && wait(BAR_FULL + st, (c / kStages) & 1)) {
        tc_fence_after();
        issue_D1(sb + st * kStage, sb + OFF_SB, tmem + TM_D1);
        mma_commit(BAR(BAR_D1));
      }
      __syncwarp();
      // meanwhile: y of the chunk before, the bound of |S|, this chunk's rows
      if (is_q && c > 0) put_y(c - 1);
      publish_max();
      wait(BAR_FULL + st, (c / kStages) & 1);
      const float *hi = reinterpret_cast<const float *>(stage + OFF_HI), *lo = reinterpret_cast<const float *>(stage + OFF_LO);
      const float gamma = ex2(hi[row] + lo[row]) * sc.y, gamma_end = ex2(hi[C - 1] + lo[C - 1]);
      uint4 vv[4];
      float beta = 0.f, back_k = 0.f;
      const bool live = c * C + row < len;
      if (!is_q) {
        beta = reinterpret_cast<const float *>(stage + OFF_BETA)[row];
        back_k = gamma * reinterpret_cast<const float *>(stage + OFF_RHOK)[row];
        const uint4 *src = reinterpret_cast<const uint4 *>(stage + OFF_V + row * kVPitch + 64 * hf);
#pragma unroll
        for (int i = 0; i < 4; ++i) vv[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
      } else {
        rho_q = reinterpret_cast<const float *>(stage + OFF_RHOQ)[row];
      }
      wait(BAR_MAXV + (c & 1), (c >> 1) & 1);
      const float vmax = read_max(max_v + 8 * (c & 1));
      const float2 rsc = state_scale(fmaxf(m, vmax));
      back_o = rsc.y;
      wait(BAR_D1, c & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16], e[16];
        tmem_ld16(tmem + TM_D1 + 32 * hf + 16 * x + lane_off, d);
        tmem_ld16(tmem + TM_D1 + 64 + 32 * hf + 16 * x + lane_off, e);
        tmem_ld_wait();
        if (is_q) {
#pragma unroll
          for (int i = 0; i < 16; ++i) qs[16 * x + i] = gamma * (d[i] + e[i]);
        } else {
          uint32_t hv[8], lv[8];
          const float b = live ? beta * rsc.x : 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 u4 = vv[2 * x + (i >> 2)];
            const uint32_t u = (i & 3) == 0 ? u4.x : (i & 3) == 1 ? u4.y : (i & 3) == 2 ? u4.z : u4.w;
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
            split2(b * fmaf(-back_k, d[2 * i] + e[2 * i], v.x), b * fmaf(-back_k, d[2 * i + 1] + e[2 * i + 1], v.y), hv[i], lv[i]);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            unsigned char *o = smem + OFF_RB + swz(row, 4 * hf + 2 * x + u);
            *reinterpret_cast<uint4 *>(o) = make_uint4(hv[4 * u], hv[4 * u + 1], hv[4 * u + 2], hv[4 * u + 3]);
            *reinterpret_cast<uint4 *>(o + 8192) = make_uint4(lv[4 * u], lv[4 * u + 1], lv[4 * u + 2], lv[4 * u + 3]);
          }
        }
      }
      fence_proxy_async();
      tc_fence_before();
      if (named_bar_or(1, 256, *abort_flag != 0)) { done = false; break; }
      if (leader && wait(BAR_MREADY, c & 1)) {
        tc_fence_after();
        issue_R(tmem + TM_MHI, sb + OFF_RB, tmem + TM_S, false);
        issue_R(tmem + TM_MHI, sb + OFF_RB + 8192, tmem + TM_S, true);
        issue_R(tmem + TM_MLO, sb + OFF_RB, tmem + TM_S, true);
        mma_commit(BAR(BAR_S));
        issue_R(tmem + TM_AT, sb + OFF_RB, tmem + TM_O, false);
        mma_commit(BAR(BAR_O));
      }
      __syncwarp();
      m = fmaf(gamma_end, read_max(max_s), vmax);
      wait(BAR_S, c & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16];
        tmem_ld16(tmem + TM_S + 32 * hf + 16 * x + lane_off, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[16 * x + i] = fmaf(rsc.y, d[i], gamma_end * S[16 * x + i]);
      }
    }
    if (done && *abort_flag == 0) {
      if (is_q && nck > 0) put_y(nck - 1);
      if (p.h_final) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (in_bounds(soff + (long long)i * kDState, p.state_extent, p.err)) p.h_final[soff + (long long)i * kDState] = S[i];
      }
    }
    if (leader) {
      mma_commit(BAR(BAR_END + 1));
      int never_abort = 0;
      mbar_wait(BAR(BAR_END + 1), 0, &never_abort, p.err);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 14) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
#undef BAR
}

// ---- front end: the operand tiles and gates of every chunk -----------------------------------------
// One CTA per (chunk, group).  A warp takes 16 of the 128 rows (64 of K, 64 of Q): a row is scaled
// by the power of two that brings its largest element to [1, 2), which is exact in fp16 down to
// 2^-17 of it, and stored where the swizzled operand tile wants it; rho is that power and the norm's
// factor.  Then each warp scans the gates of its heads: the prefix sums of log2(alpha) in fp64,
// left as two floats, so that differences keep fp32's relative precision however large the sums.
// Bound by HBM: per token and group 512 bytes read and 520 written, per token and head 4 and 12.
__global__ void __launch_bounds__(256) ssd_delta_front_kernel(const DeltaPlan p) {
  const long long ck = blockIdx.x;
  const int g = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int seq;
  long long first;
  if (p.chunk0) {  // the last sequence that starts at or before this chunk and has one
    int a = 0, b = p.B - 1;
    while (a < b) {
      const int mid = (a + b + 1) / 2;
      if (p.chunk0[mid] <= ck) a = mid;
      else b = mid - 1;
    }
    seq = a;
    first = p.chunk0[a];
  } else {
    const int nc = (p.L + C - 1) / C;
    seq = (int)(ck / nc);
    first = (long long)seq * nc;
  }
  const int t0 = (int)(ck - first) * C, rows = min(C, seq_len(p.cu, seq, p.L) - t0);
  const long long base = seq_base(p.cu, seq, p.L) + t0;
  unsigned char *tile = p.tiles + (ck * p.G + g) * kDeltaTileBytes;
  uint2 raw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 16 * warp + i, t = r & 63;
    const __nv_bfloat16 *src = r < 64 ? static_cast<const __nv_bfloat16 *>(p.k) + (base + t) * p.ks
                                      : static_cast<const __nv_bfloat16 *>(p.q) + (base + t) * p.qs;
    raw[i] = t < rows ? *reinterpret_cast<const uint2 *>(src + g * kDState + 4 * lane) : make_uint2(0, 0);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 16 * warp + i;
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw[i].x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw[i].y));
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(__float_as_uint(a.x) & 0x7fffffffu, __float_as_uint(a.y) & 0x7fffffffu),
                                                            max(__float_as_uint(b.x) & 0x7fffffffu, __float_as_uint(b.y) & 0x7fffffffu)));
    const uint32_t e = min(max(top >> 23, 1u), 253u);
    const float f = __uint_as_float((254u - e) << 23);
    const int chunk = (lane & 15) >> 1;
    *reinterpret_cast<uint2 *>(tile + (lane >> 4) * kHalf + swz(r, chunk) + 8 * (lane & 1)) =
        make_uint2(h2(__floats2half2_rn(a.x * f, a.y * f)), h2(__floats2half2_rn(b.x * f, b.y * f)));
    float rho = __uint_as_float(e << 23);
    if (p.qk_norm) rho *= 1.f / sqrtf(warp_sum(a.x * a.x + a.y * a.y + b.x * b.x + b.y * b.y) + p.qk_eps);
    if (r >= 64) rho *= p.q_scale;
    if (lane == 0) reinterpret_cast<float *>(tile + OFF_RHOK)[r] = rho;
  }
  for (int hh = warp; hh < p.hpg; hh += 8) {
    const int h = g * p.hpg + hh;
    const float A = p.A[h], bias = p.dt_bias[h];
    double s[2];
    float beta[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 2 * lane + u;
      s[u] = 0.0;
      beta[u] = 0.f;
      if (t < rows) {
        float d = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.dt)[(base + t) * p.ds + h]) + bias;
        const float b = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.b)[(base + t) * p.bs + h]);
        if (p.softplus) d = d > 20.f ? d : log1pf(expf(d));
        d = fminf(fmaxf(d, p.dt_min), p.dt_max);
        s[u] = (double)A * d * 1.4426950408889634;
        beta[u] = p.beta_scale * (p.beta_sigmoid ? 1.f / (1.f + expf(-b)) : b);
      }
    }
    s[1] += s[0];
    double sum = s[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const double before = sum - s[1];
    const float h0 = (float)(before + s[0]), h1 = (float)sum;
    float *out = p.gates + (ck * p.H + h) * (kDeltaGateBytes / 4) + 2 * lane;
    *reinterpret_cast<float2 *>(out) = make_float2(h0, h1);
    *reinterpret_cast<float2 *>(out + C) = make_float2((float)(before + s[0] - h0), (float)(sum - h1));
    *reinterpret_cast<float2 *>(out + 2 * C) = make_float2(beta[0], beta[1]);
  }
}

}  // namespace

cudaError_t launch_delta_front(const DeltaPlan &p, cudaStream_t s) {
  ssd_delta_front_kernel<<<dim3((unsigned)p.n_chunks, p.G), 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_delta_chunks(const DeltaPlan &p, cudaStream_t s) {
  cudaError_t e = set_smem_attr(ssd_delta_chunk_kernel, kSmem, s);
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the front end: its set-up and first loads of V overlap the front
  // end's tail
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(p.H * (p.P / 64)), (unsigned)p.B);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kSmem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, ssd_delta_chunk_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ssd
