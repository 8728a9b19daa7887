// delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor cores (tcgen05 + TMEM).
//
// Within a chunk, with cs the prefix sums of log2(alpha), S the state (P x N) that enters it and the
// rows of K, Q, V its tokens, the token recurrence is
//   (I + L) U = R,   R_j = beta_j (v_j - 2^{cs_j} S k_j),   L_ij = beta_i 2^{cs_i - cs_j} k_i.k_j  (j < i)
//   S' = 2^{cs_C} S + sum_i 2^{cs_C - cs_i} U_i k_i^T,   y_t = 2^{cs_t} S q_t + sum_{i <= t} 2^{cs_t - cs_i} (q_t.k_i) U_i
// (U_i: what token i really writes, once the tokens before it are erased).  Keys are k_i = rho_i K_i with
// K_i exact in fp16.  The decays and the rho are a similarity of L: with
//   L~_ij = beta_i rho_i^2 K_i.K_j  (j < i),   T~ = (I + L~)^-1,
// (I + L)^-1_ij = T~_ij 2^{cs_i - cs_j} rho_j / rho_i, so that
//   S' = 2^{cs_C} S + sum_j (rho_j 2^{cs_C - cs_j} R_j) M_j^T,          M = K^T T~          (N x 64)
//   y_t = 2^{cs_t} S q_t + sum_j 2^{cs_t - cs_j} rho_j (A~ T~)_tj R_j,   A~_ti = q_t.K_i     (i <= t)
// The inverse, M and A~ T~ know no decay, and nothing of them depends on the state: the chain from chunk
// to chunk is two dependent products, K S^T (which gives R) and M R~.  One CTA carries 64 state rows
// of one head through the sequence (the rows are independent given K, so a head of 128 rows is two
// CTAs).
//
// Precision.  The state is fp32, in registers.  Its products run on fp16 operands in two parts,
// hi = fp16(x), lo = fp16(x - hi), which keep 22 bits; the products hi.hi + hi.lo + lo.hi leave an error
// of about 2^-22, so the state stays as near to the fp64 rule as an fp32 recurrence does.  K and Q need
// one part: a row of bf16 numbers times a power of two is exact in fp16, and the power and the norm's
// factor come back in the fp32 factors rho.  |T~| and |M| are bounded (beta |k|^2 <= 2 and
// 1 <= |K_i| < 23); S and R are scaled by powers of two from running bounds of |S| and |V|
// (state_scale), so that fp16's range holds any size of input.  Only what goes into y alone (A~, A~ T~,
// the R beside it) is rounded to 11 bits: y is then rounded to bf16's 8.
// T~ is inverted in fp32: 16 x 16 diagonal blocks by substitution, joined by block products with tf32
// in two parts (22 bits).
//
// Roles (20 warps).  Warps 0-7, the chain: S into its operand, R from K S^T, the new S, y.  Warps
// 8-15, the chunk's own part, one chunk ahead of the chain: the decay masks of K K^T and Q K^T, the
// inverse, M and AT into operands.  Warps 16 and 17 issue the MMAs of the one and of the other (an
// issuing thread is held up for about as long as its MMAs run), warp 18 loads (bulk copies of the
// tiles that the front end prepared and of the rows of V), warp 19 finds the largest |V| of each
// chunk.  Hand-overs are mbarriers; every wait is bounded: a timeout makes every role leave and latches
// SSD_ERR_TIMEOUT.
#include "common.cuh"
#include "delta_plan.h"
#include "plan.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int C = kDeltaChunk;
constexpr int kThreads = 20 * 32;
constexpr int kStages = 3;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes
// stage
constexpr uint32_t OFF_RHOK = 2 * kHalf;          // the tile's row factors follow its operands
constexpr uint32_t OFF_RHOQ = OFF_RHOK + 256;
constexpr uint32_t OFF_HI = OFF_RHOQ + 256;       // the head's gates record, six arrays of 64 floats
constexpr uint32_t OFF_LO = OFF_HI + 256;
constexpr uint32_t OFF_BETA = OFF_LO + 256;
constexpr uint32_t OFF_GAMMA = OFF_BETA + 256;
constexpr uint32_t OFF_COL = OFF_GAMMA + 256;
constexpr uint32_t OFF_END = OFF_COL + 256;
constexpr uint32_t OFF_V = OFF_END + 256;         // 64 rows of 128 bytes, 144 apart (no bank conflicts)
constexpr uint32_t kVPitch = 144;
constexpr uint32_t kStage = (OFF_V + C * kVPitch + 1023) / 1024 * 1024;
static_assert(OFF_HI == kDeltaTileBytes && OFF_V == kDeltaTileBytes + kDeltaGateBytes, "records as loaded");
// CTA
constexpr uint32_t OFF_SB = kStages * kStage;     // S operand: [n][p] hi, then lo (128 rows x 128 bytes each)
constexpr uint32_t OFF_RB = OFF_SB + 2 * kHalf;   // R operands: [token][p] R~ hi, lo; R (64 rows x 128 bytes each)
constexpr uint32_t OFF_T = OFF_RB + 3 * 8192;     // T operand: [j][i] T~_ij hi, lo
constexpr uint32_t OFF_W = OFF_T + 2 * 8192;      // fp32 64 x 72: (-L~)^T, its diagonal 32 x 32 blocks then T~^T's
constexpr int kWPitch = 72;                       // = 8 mod 32: conflict-free fragment reads
constexpr uint32_t OFF_MAXS = OFF_W + 64 * kWPitch * 4;  // largest |S| per chain warp, two chunks
constexpr uint32_t OFF_MAXV = OFF_MAXS + 64;      // bound of what the chunk adds, per stage
constexpr uint32_t OFF_BAR = OFF_MAXV + 64;
// A barrier that can complete again before every waiter has seen the phase before has one copy per
// buffer, so that a parity test never sees two phases at once.
enum {
  BAR_FULL,                        // [kStages] stage loaded
  BAR_EMPTY = BAR_FULL + kStages,  // [kStages] its last product is done (and every read before it)
  BAR_MAXV = BAR_EMPTY + kStages,  // [kStages] bound of what the chunk adds known
  BAR_G = BAR_MAXV + kStages,      // [2] K K^T, Q K^T done
  BAR_Z = BAR_G + 2,               // L21 and the inverted diagonal blocks in w (3 warps)
  BAR_WFREE,                       // w read (4 warps)
  BAR_T,                           // T and A operands written (6 warps)
  BAR_MM,                          // M and AT done
  BAR_MREADY,                      // M and AT operands in tensor memory (6 warps)
  BAR_SREADY,                      // S operand written (8 warps)
  BAR_D1,                          // K S^T, Q S^T done
  BAR_RREADY,                      // R operand written, D1 read (8 warps)
  BAR_S,                           // M R done
  BAR_O,                           // AT R done
  BAR_DONE,                        // [2] nothing of an issuer's left in flight
  kNumBars = BAR_DONE + 2
};
constexpr uint32_t OFF_MISC = OFF_BAR + 8 * 32;   // [0] TMEM base, [1] abort flag
constexpr uint32_t kSmem = OFF_MISC + 16 + 1024;  // room to align the base to 1024 bytes
static_assert(kNumBars <= 32 && kSmem <= 232448, "shared memory");
static_assert(OFF_SB % 1024 == 0 && OFF_RB % 1024 == 0 && OFF_T % 1024 == 0, "swizzle alignment");

// TMEM columns.  K rows are lanes 0-63 of G and D1, Q rows lanes 64-127.  fp16 operands replace the
// products they come from: A the Q rows of G, the AT operand those of AT (lanes 0-63 of both are never
// used), the M operand's two parts M.  Tokens 32 b .. 32 b + 31 of an operand lie in the columns
// 32 b .. of their own 32 fp32 columns: hi (or the only part) first, lo 16 columns on.  So a warp writes only
// over columns that it alone has read.
constexpr uint32_t TM_G = 0, TM_M = 128, TM_AT = 192, TM_D1 = 256, TM_S = 384, TM_O = 448, TM_COLS = 512;

constexpr uint32_t IDESC_KK = idesc_f16(128, 64, false, false, kFmtF16);   // G: both K-major; AT: A from TMEM
constexpr uint32_t IDESC_D1 = idesc_f16(128, 128, false, true, kFmtF16);   // [K; Q] . [S hi | S lo]
constexpr uint32_t IDESC_M = idesc_f16(128, 64, true, false, kFmtF16);     // K^T . T
constexpr uint32_t IDESC_R = idesc_f16(128, 64, false, true, kFmtF16);     // M or AT (TMEM) . R

// A bounded wait like tc::mbar_wait, but with the hardware's own suspension instead of a time hint: with
// the hint a failed try sleeps in software, and each hand-over waits for the end of a sleep.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_retry(uint32_t bar, uint32_t parity, volatile int *abort, int *err) {
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        *abort = 1;
        latch_error(err, (int)SSD_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ uint64_t adv(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(d) + (bytes >> 4));
}
__device__ __forceinline__ constexpr uint32_t kstep(int j) { return (j >> 2) * kHalf + (j & 3) * 32; }

__device__ __forceinline__ constexpr uint32_t tstep(int j) { return (j >> 1) * 32 + (j & 1) * 8; }

// The issuing loops stay rolled: an MMA runs for 32 to 64 clocks, and what the instruction cache holds
// decides this kernel's speed (unrolled everywhere, 100 KB of code, it took twice as long).
__device__ __forceinline__ void issue_G(uint32_t kq, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, 16, 1024);
#pragma unroll 1
  for (int j = 0; j < 8; ++j) mma_f16_ss(d, adv(a, kstep(j)), adv(a, kstep(j)), IDESC_KK, j > 0);
}
__device__ __forceinline__ void issue_D1(uint32_t kq, uint32_t sbuf, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, 16, 1024), b = smem_desc_sw128(sbuf, kHalf, 1024);
#pragma unroll 1
  for (int j = 0; j < 8; ++j) mma_f16_ss(d, adv(a, kstep(j)), adv(b, j * 2048), IDESC_D1, j > 0);
}
__device__ __forceinline__ void issue_M(uint32_t kq, uint32_t t, uint32_t d) {
  const uint64_t a = smem_desc_sw128(kq, kHalf, 1024), b = smem_desc_sw128(t, 16, 1024);
#pragma unroll 1
  for (int j = 0; j < 8; ++j)  // hi, then lo
    mma_f16_ss(d, adv(a, (j & 3) * 2048), adv(b, (j >> 2) * 8192 + (j & 3) * 32), IDESC_M, j > 0);
}
__device__ __forceinline__ void issue_AT(uint32_t a_tmem, uint32_t t, uint32_t d) {
  const uint64_t b = smem_desc_sw128(t, 16, 1024);
#pragma unroll 1
  for (int j = 0; j < 4; ++j) mma_f16_ts(d, a_tmem + tstep(j), adv(b, 32 * j), IDESC_KK, j > 0);
}
// d = M_hi R~_hi + M_hi R~_lo + M_lo R~_hi  (64 tokens each)
__device__ __forceinline__ void issue_S(uint32_t m, uint32_t r, uint32_t d) {
  const uint64_t b = smem_desc_sw128(r, 8192, 1024);
#pragma unroll 1
  for (int j = 0; j < 12; ++j)
    mma_f16_ts(d, m + tstep(j & 3) + (j >> 3) * 16, adv(b, 2048 * (j & 3) + (j >> 2 & 1) * 8192), IDESC_R, j > 0);
}
__device__ __forceinline__ void issue_O(uint32_t at, uint32_t r, uint32_t d) {
  const uint64_t b = smem_desc_sw128(r, 8192, 1024);
#pragma unroll 1
  for (int j = 0; j < 4; ++j) mma_f16_ts(d, at + tstep(j), adv(b, 2048 * j), IDESC_R, j > 0);
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return (uint32_t)row * 128u + ((uint32_t)(chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
// fp16 pairs: hi, and lo = what hi leaves
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __float22half2_rn(v);
  hi = h2(h);
  lo = h2(__float22half2_rn(__ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), v)));
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, float (&v)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  v[0] = __uint_as_float(r[0]);
  v[1] = __uint_as_float(r[1]);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Powers of two that bring a quantity bounded by m to [64, 128) and back.  Headroom: with alpha <= 1
// and beta |k|^2 <= 2 the transition does not expand a state row s, so over a chunk
// |s'| <= gamma |s| + 64 * 2 max|V|, and |R|, |R~| <= 2 (max|V| + |s|).  With m = gamma max|S_old| + max|V| that
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
struct FragA {
  uint32_t h[4], l[4];
};
struct FragB {
  uint32_t h[2], l[2];
};
// 16 x 8 of A, row-major at a
__device__ __forceinline__ FragA load_a(const float *a, int lane) {
  const float *x = a + (lane >> 2) * kWPitch + (lane & 3);
  FragA f;
  split_tf32(x[0], f.h[0], f.l[0]);
  split_tf32(x[8 * kWPitch], f.h[1], f.l[1]);
  split_tf32(x[4], f.h[2], f.l[2]);
  split_tf32(x[8 * kWPitch + 4], f.h[3], f.l[3]);
  return f;
}
// 8 x 8 of B, row-major at b: its rows r0 and r1 per lane are t and t + 4, or, where A comes from an
// accumulator (from_acc), 2t and 2t + 1
__device__ __forceinline__ FragB load_b(const float *b, bool from_acc, int lane) {
  const int t = lane & 3;
  const float *x = b + (from_acc ? 2 * t : t) * kWPitch + (lane >> 2);
  FragB f;
  split_tf32(x[0], f.h[0], f.l[0]);
  split_tf32(x[from_acc ? kWPitch : 4 * kWPitch], f.h[1], f.l[1]);
  return f;
}
// An accumulator tile as an A fragment: a lane's elements of a row are columns 2t and 2t + 1, which the
// product takes as k = t and t + 4 (B's rows permuted alike).
__device__ __forceinline__ FragA acc_as_a(const float (&c)[4]) {
  FragA f;
  split_tf32(c[0], f.h[0], f.l[0]);
  split_tf32(c[2], f.h[1], f.l[1]);
  split_tf32(c[1], f.h[2], f.l[2]);
  split_tf32(c[3], f.h[3], f.l[3]);
  return f;
}

// 16 rows and two 8-column tiles of W12 = W11 Z W22, the block that joins two inverted diagonal blocks
// (transposed, so upper triangular; their zeros are stored) of 8 K rows each: w11 at its row and
// first column, z at its corner, w22 at its first row and the tiles' column.  No branches: the
// products of one tile would otherwise wait for those of the one before.
template <int K>
__device__ __forceinline__ void join(const float *w11, const float *z, const float *w22, float (&d)[2][4], int lane) {
  FragA a[K];
#pragma unroll
  for (int kk = 0; kk < K; ++kk) a[kk] = load_a(w11 + 8 * kk, lane);
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[nt][e] = 0.f;
#pragma unroll
  for (int kt = 0; kt < K; ++kt) {
    float hh[4] = {}, hl[4] = {}, lh[4] = {};
#pragma unroll
    for (int kk = 0; kk < K; ++kk) {
      const FragB b = load_b(z + 8 * kk * kWPitch + 8 * kt, false, lane);
      mma_tf32(hh, a[kk].h, b.h);
      mma_tf32(hl, a[kk].h, b.l);
      mma_tf32(lh, a[kk].l, b.h);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) hh[e] += hl[e] + lh[e];
    const FragA x = acc_as_a(hh);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const FragB b = load_b(w22 + 8 * kt * kWPitch + 8 * nt, true, lane);
      mma_tf32(d[nt], x.l, b.h);
      mma_tf32(d[nt], x.h, b.l);
      mma_tf32(d[nt], x.h, b.h);
    }
  }
}

// The 16 x 16 diagonal blocks at p0 and p0 + 16, by one warp: t = column `lane & 15` of T~'s block lane / 16,
//   t_i = [i == j] - sum_{m < i} L~_im t_m,
// the column of m taken off every later element as soon as t_m is known (so the chain is one
// multiply-add per row).  z = (-L~)^T at w; a row is read while the one before is used.
__device__ __forceinline__ void invert16(const float *w, int p0, int lane, float2 (&t)[8]) {
  const int b0 = p0 + (lane & 16), j = lane & 15;
  const float *zr = w + b0 * kWPitch + b0;
  float4 z[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    z[q] = *reinterpret_cast<const float4 *>(zr + 4 * q);
    t[2 * q] = make_float2(4 * q == j ? 1.f : 0.f, 4 * q + 1 == j ? 1.f : 0.f);
    t[2 * q + 1] = make_float2(4 * q + 2 == j ? 1.f : 0.f, 4 * q + 3 == j ? 1.f : 0.f);
  }
#pragma unroll
  for (int m = 0; m < 15; ++m) {
    const float tm = m & 1 ? t[m / 2].y : t[m / 2].x;
    const float2 t2 = make_float2(tm, tm);
#pragma unroll
    for (int q = m / 4; q < 4; ++q) {
      if (2 * q >= (m + 1) / 2) t[2 * q] = __ffma2_rn(make_float2(z[q].x, z[q].y), t2, t[2 * q]);
      if (2 * q + 1 >= (m + 1) / 2) t[2 * q + 1] = __ffma2_rn(make_float2(z[q].z, z[q].w), t2, t[2 * q + 1]);
      if (m < 14 && q >= (m + 1) / 4) z[q] = *reinterpret_cast<const float4 *>(zr + (m + 1) * kWPitch + 4 * q);
    }
  }
}

// Two neighbouring elements (i, i + 1) of row j of the T operand, from an accumulator tile's lane
__device__ __forceinline__ void put_t(unsigned char *t, int j, int chunk, int lane, float a, float b) {
  uint32_t hv, lv;
  split2(make_float2(a, b), hv, lv);
  unsigned char *o = t + swz(j, chunk) + 4 * (lane & 3);
  *reinterpret_cast<uint32_t *>(o) = hv;
  *reinterpret_cast<uint32_t *>(o + 8192) = lv;
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
  const uint32_t bar0 = sb + OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
  const auto wait = [&](int bar, uint32_t parity) {
    return try_wait(BAR(bar), parity) || wait_retry(BAR(bar), parity, abort_flag, p.err);
  };
  const auto wait_stage = [&](int bar, int c) { return wait(bar + c % kStages, (c / kStages) & 1); };

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(BAR(i), i == BAR_SREADY || i == BAR_RREADY ? 8 : i == BAR_T || i == BAR_MREADY ? 6 : i == BAR_Z ? 3 : i == BAR_WFREE ? 4 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // the part of T above the diagonal blocks stays zero
  for (int i = tid; i < 2 * 8192 / 16; i += kThreads) reinterpret_cast<uint4 *>(smem + OFF_T)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == 19) {
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
  const bool is_q = q4 >= 2;
  const int row = 32 * (q4 & 1) + lane;              // token of this thread's lane of G, D1 and O

  // Registers: 640 threads have 96 each; the chain's eight warps take 24 more from the last four
  // (256 x 24 = 128 x 48).
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 16) {
      // ---------------------------------------------------------------- MMAs of the chain
      if (lane == 0) {
        for (int c = 0; c < nck; ++c) {
          if (!wait_stage(BAR_FULL, c) || !wait(BAR_SREADY, c & 1)) break;
          tc_fence_after();
          issue_D1(sb + c % kStages * kStage, sb + OFF_SB, tmem + TM_D1);
          mma_commit(BAR(BAR_D1));
          if (!wait(BAR_MREADY, c & 1) || !wait(BAR_RREADY, c & 1)) break;
          tc_fence_after();
          issue_S(tmem + TM_M, sb + OFF_RB, tmem + TM_S);
          mma_commit(BAR(BAR_S));
          issue_O(tmem + TM_AT, sb + OFF_RB + 16384, tmem + TM_O);
          mma_commit(BAR(BAR_O));
          mma_commit(BAR(BAR_EMPTY + c % kStages));
        }
        mma_commit(BAR(BAR_DONE));  // no MMA may still be running when TMEM is released
        int never_abort = 0;
        mbar_wait(BAR(BAR_DONE), 0, &never_abort, p.err);
      }
    } else if (warp == 17) {
      // ---------------------------------------------------------------- MMAs of the chunk's own part
      if (lane == 0) {
        for (int c = -1; c < nck; ++c) {
          if (c + 1 < nck) {  // G of the next chunk, over that of the one before, which AT has read
            if (!wait_stage(BAR_FULL, c + 1) || (c > 0 && !wait(BAR_MM, (c - 1) & 1))) break;
            tc_fence_after();
            issue_G(sb + (c + 1) % kStages * kStage, tmem + TM_G + 64 * ((c + 1) & 1));
            mma_commit(BAR(BAR_G + ((c + 1) & 1)));
          }
          if (c < 0) continue;
          // M and AT over those of the chunk before, which the chain's products have read
          if (!wait(BAR_T, c & 1) || (c > 0 && !wait(BAR_O, (c - 1) & 1))) break;
          tc_fence_after();
          issue_AT(tmem + TM_G + 64 * (c & 1), sb + OFF_T, tmem + TM_AT);
          issue_M(sb + c % kStages * kStage, sb + OFF_T, tmem + TM_M);
          mma_commit(BAR(BAR_MM));
        }
        mma_commit(BAR(BAR_DONE + 1));
        int never_abort = 0;
        mbar_wait(BAR(BAR_DONE + 1), 0, &never_abort, p.err);
      }
    } else if (warp == 18) {
      // ---------------------------------------------------------------- loads
      const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
      const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + base * p.vs + h * p.P + 64 * ph;
      int c = 0;
      for (; c < nck; ++c) {
        const int rows = min(C, len - c * C);
        const uint32_t dst = sb + c % kStages * kStage, full = BAR(BAR_FULL + c % kStages);
        bool ok = true;
        if (lane == 0) {
          ok = c < kStages || wait_stage(BAR_EMPTY, c - kStages);
          if (ok) mbar_arrive_expect_tx(full, (uint32_t)(kDeltaTileBytes + kDeltaGateBytes) + rows * 128);
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        for (int r = lane; r < rows; r += 32) bulk_load(dst + OFF_V + r * kVPitch, v + (c * C + r) * p.vs, 128, full);
        if (lane == 0) {
          // V is the caller's; the tiles and gates are the front end's, which may still be running
          // (programmatic dependent launch)
          if (c == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
          bulk_load(dst, p.tiles + ((ck0 + c) * p.G + h / p.hpg) * kDeltaTileBytes, (uint32_t)kDeltaTileBytes, full);
          bulk_load(dst + OFF_HI, p.gates + ((ck0 + c) * p.H + h) * (kDeltaGateBytes / 4), (uint32_t)kDeltaGateBytes, full);
        }
        __syncwarp();
      }
      if (lane == 0) {  // every load must land before the CTA may exit
        int never_abort = 0;
        for (int j = max(0, c - kStages); j < c; ++j)
          mbar_wait(BAR(BAR_FULL + j % kStages), (j / kStages) & 1, &never_abort, p.err);
      }
    } else {
      // ---------------------------------------------------------------- largest |V| of each chunk,
      // times the largest |beta| / 2 where that is above one
      for (int c = 0; c < nck; ++c) {
        const bool ok = wait_stage(BAR_FULL, c);
        if (!__all_sync(0xffffffffu, ok)) break;
        const unsigned char *v = smem + c % kStages * kStage + OFF_V;
        const int rows = min(C, len - c * C);
        uint32_t top = 0;
#pragma unroll 4
        for (int r = lane >> 3; r < rows; r += 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(v + r * kVPitch + (lane & 7) * 16);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                       __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const float2 b = reinterpret_cast<const float2 *>(smem + c % kStages * kStage + OFF_BETA)[lane];
        const uint32_t bt = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(b.x), fabsf(b.y))));
        if (lane == 0) {
          reinterpret_cast<float *>(smem + OFF_MAXV)[c % kStages] = __uint_as_float(top << 16) * fmaxf(1.f, 0.5f * __uint_as_float(bt));
          mbar_arrive(BAR(BAR_MAXV + c % kStages));
        }
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ the chunk's own part
    const int ow = warp - 8;
    // By 32 x 32 blocks of L~ (rows, columns): warp 0 masks and inverts block (0, 0) and writes its part of
    // the T operand, warp 5 block (1, 1), warp 1 masks block (1, 0); the four Q warps mask A~ and join
    // the blocks of the inverse.  M's operand is made by warp 4 (lanes 0-31), warp 1 (lanes 32-63)
    // and the Q warps (lanes 64-127, with A~ T~).
    float *w = reinterpret_cast<float *>(smem + OFF_W);
    // columns 32 b .. of M into operands
    const auto convert_m = [&](int b) {
      float m[32];
      uint32_t hv[16], lv[16];
      tmem_ld32(tmem + TM_M + 32 * b + lane_off, m);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) split2(make_float2(m[2 * j], m[2 * j + 1]), hv[j], lv[j]);
      tmem_st16(tmem + TM_M + 32 * b + lane_off, hv);
      tmem_st16(tmem + TM_M + 32 * b + 16 + lane_off, lv);
    };
    // Columns 32 hf .. of A~ T~, times 2^{cs_t - cs_j} rho_j.  2^{cs_t - cs_j} = 2^{cs_t - r} 2^{r - cs_j} with
    // r the prefix sum at the end of the columns' block of 32: a factor per row and one per column.
    // In the blocks on the diagonal the row's is above one: where it could overflow the power is
    // taken directly.
    const auto convert_at = [&](const unsigned char *stage) {
      const auto arr = [&](uint32_t off) { return reinterpret_cast<const float *>(stage + off) + 32 * hf; };
      float v[32];
      uint32_t pk[16];
      const float *hi = arr(OFF_HI), *lo = arr(OFF_LO);
      const int at = row - 32 * hf;  // this row's column
      const float hr = hi[at], lr = lo[at], hb = hi[31], lb = lo[31];
      if (hf == (q4 & 1) && hi[0] - hb > 64.f) {
#pragma unroll 1
        for (int j = 0; j < 32; j += 2) {
          float x[2];
          tmem_ld2(tmem + TM_AT + 32 * hf + j + lane_off, x);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 2; ++u)
            x[u] *= arr(OFF_RHOK)[j + u] * ex2(j + u <= at ? (hr - hi[j + u]) + (lr - lo[j + u]) : -INFINITY);
          tmem_st1(tmem + TM_AT + 32 * hf + j / 2 + lane_off, h2(__floats2half2_rn(x[0], x[1])));
          tmem_st_wait();
        }
        return;
      }
      tmem_ld32(tmem + TM_AT + 32 * hf + lane_off, v);
      tmem_ld_wait();
      const float fr = ex2((hr - hb) + (lr - lb));
      const float2 f2 = make_float2(fr, fr);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 cf = *reinterpret_cast<const float4 *>(arr(OFF_COL) + 4 * j);
        pk[2 * j] = h2(__float22half2_rn(__fmul2_rn(__fmul2_rn(make_float2(v[4 * j], v[4 * j + 1]), f2), make_float2(cf.x, cf.y))));
        pk[2 * j + 1] = h2(__float22half2_rn(__fmul2_rn(__fmul2_rn(make_float2(v[4 * j + 2], v[4 * j + 3]), f2), make_float2(cf.z, cf.w))));
      }
      tmem_st16(tmem + TM_AT + 32 * hf + lane_off, pk);
    };
    const bool none = hf == 1 && (q4 & 1) == 0;  // columns 32.. of rows 0-31: zeros
    const auto convert_chunk = [&](int c) {
      const bool ok = wait(BAR_MM, c & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int b = is_q ? hf : 0; b < (is_q ? hf + 1 : 2); ++b) convert_m(b);
      if (is_q) {
        if (!none) {
          convert_at(smem + c % kStages * kStage);
        } else {  // (zero already, but in fp32: the operand takes half the columns)
          uint32_t zero[16] = {};
          tmem_st16(tmem + TM_AT + 32 * hf + lane_off, zero);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_MREADY));
      return ok;
    };
    const bool inverts = ow == 0 || ow == 5;
    for (int c = 0; c <= nck; ++c) {  // (the last turn only converts)
      const unsigned char *stage = smem + c % kStages * kStage;
      const auto arr = [&](uint32_t off) { return reinterpret_cast<const float *>(stage + off); };
      bool ok = true;
      const bool live = c < nck;
      if (ow != 4 && live) {
        // rows of -L~ (j < i), or of A~ (j <= i)
        ok = wait_stage(BAR_FULL, c);
        ok = wait(BAR_G + (c & 1), (c >> 1) & 1) && ok;
        __syncwarp();
        tc_fence_after();
        float v[32];
        const uint32_t tg = tmem + TM_G + 64 * (c & 1) + lane_off;
        if (!none) {
          tmem_ld32(tg + 32 * hf, v);
          tmem_ld_wait();
          if (hf == (q4 & 1)) {
            const int last = lane - (is_q ? 0 : 1);  // last column kept
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = j <= last ? v[j] : 0.f;
          }
        }
        if (is_q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = none ? 0u : h2(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
          tmem_st16(tg + 32 * hf, pk);
          tmem_st_wait();
        } else {
          const float rho = arr(OFF_RHOK)[row], f = -arr(OFF_BETA)[row] * rho * rho;
          if (c > 0) ok = wait(BAR_WFREE, (c - 1) & 1) && ok;
#pragma unroll
          for (int j = 0; j < 32; ++j) w[(32 * hf + j) * kWPitch + row] = f * v[j];
          __syncwarp();
        }
      }
      if (inverts) {
        if (!live) break;
        const int p0 = 32 * hf, j = p0 + lane, g = lane >> 2;
        float2 t[8];
        invert16(w, p0, lane, t);
        __syncwarp();
        float *o = w + j * kWPitch + p0 + (lane & 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4 *>(o + 4 * i) = make_float4(t[2 * i].x, t[2 * i].y, t[2 * i + 1].x, t[2 * i + 1].y);
        __syncwarp();
        float d[2][4];
        const float *wp = w + p0 * kWPitch + p0;
        join<2>(wp, wp + 16, wp + 16 * kWPitch + 16, d, lane);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float *x = w + (p0 + g) * kWPitch + p0 + 16 + 8 * nt + 2 * (lane & 3);
          *reinterpret_cast<float2 *>(x) = make_float2(d[nt][0], d[nt][1]);
          *reinterpret_cast<float2 *>(x + 8 * kWPitch) = make_float2(d[nt][2], d[nt][3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_Z));
        if (c > 0) ok = wait(BAR_MM, (c - 1) & 1) && ok;  // the T of the chunk before is read
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t hv[4], lv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split2(t[4 * u + k], hv[k], lv[k]);
          unsigned char *x = smem + OFF_T + swz(j, (p0 + (lane & 16)) / 8 + u);
          *reinterpret_cast<uint4 *>(x) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
          *reinterpret_cast<uint4 *>(x + 8192) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          put_t(smem + OFF_T, p0 + g, p0 / 8 + 2 + nt, lane, d[nt][0], d[nt][1]);
          put_t(smem + OFF_T, p0 + g + 8, p0 / 8 + 2 + nt, lane, d[nt][2], d[nt][3]);
        }
      } else {
        if (ow == 1 && live && lane == 0) mbar_arrive(BAR(BAR_Z));
        if (c > 0) ok = convert_chunk(c - 1) && ok;
        if (is_q && live) {
          // T~^T's block (0, 1): 16 rows and 16 columns per warp
          ok = wait(BAR_Z, c & 1) && ok;
          __syncwarp();
          const int mt = hf, nh = q4 & 1, g = lane >> 2;
          float d[2][4];
          join<4>(w + 16 * mt * kWPitch, w + 32, w + 32 * kWPitch + 32 + 16 * nh, d, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(BAR_WFREE));
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            put_t(smem + OFF_T, 16 * mt + g, 4 + 2 * nh + nt, lane, d[nt][0], d[nt][1]);
            put_t(smem + OFF_T, 16 * mt + g + 8, 4 + 2 * nh + nt, lane, d[nt][2], d[nt][3]);
          }
        }
      }
      if ((inverts || is_q) && live) {
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_T));
      }
      if (!__all_sync(0xffffffffu, ok)) break;
    }
  } else {
    // ------------------------------------------------------------------ the chain
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    const int n = 32 * q4 + lane;  // state column of this thread; it holds rows 32 hf ..
    const long long soff = (((long long)seq * p.H + h) * p.P + 64 * ph + 32 * hf) * kDState + n;
    uint32_t *max_s = reinterpret_cast<uint32_t *>(smem + OFF_MAXS);
    float2 S[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      S[i].x = p.h0 ? p.h0[soff + (2 * i) * kDState] : 0.f;
      S[i].y = p.h0 ? p.h0[soff + (2 * i + 1) * kDState] : 0.f;
    }
    const auto publish_max = [&](int buf) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fmaxf(fabsf(S[i].x), fabsf(S[i].y)));
      const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      if (lane == 0) max_s[8 * buf + warp] = bits;
    };
    const auto read_max = [&](int buf) {
      const uint4 a = *reinterpret_cast<const uint4 *>(max_s + 8 * buf), b = *reinterpret_cast<const uint4 *>(max_s + 8 * buf + 4);
      return __uint_as_float(max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w))));
    };
    publish_max(1);
    named_bar(1, 256);
    float m = read_max(1);  // bounds |S| as described at state_scale
    float2 qs[16];          // 2^cs Q S^T of the chunk whose y is still to come
    float back_o = 0.f, rho_q = 0.f;
    const auto put_y = [&](int c) {  // Q rows: y of chunk c
      wait(BAR_O, c & 1);
      __syncwarp();
      tc_fence_after();
      const int t = c * C + row;
      const long long yo = (base + t) * p.ys + (long long)h * p.P + 64 * ph + 32 * hf;
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + yo);
      const bool store = t < len && in_bounds(yo + 31, p.y_extent, p.err);
      const float2 b2 = make_float2(back_o, back_o), r2 = make_float2(rho_q, rho_q);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float o[16];
        tmem_ld16(tmem + TM_O + 32 * hf + 16 * x + lane_off, o);
        tmem_ld_wait();
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = __fmul2_rn(r2, __ffma2_rn(b2, make_float2(o[2 * i], o[2 * i + 1]), qs[8 * x + i]));
          const __nv_bfloat162 v = __float22bfloat162_rn(f);
          u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if (store) {
          dst[2 * x] = make_uint4(u[0], u[1], u[2], u[3]);
          dst[2 * x + 1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
    };
    bool ok = true;
    for (int c = 0;; ++c) {
      const unsigned char *stage = smem + c % kStages * kStage;
      const auto arr = [&](uint32_t off) { return reinterpret_cast<const float *>(stage + off); };
      const float2 sc = state_scale(m), sc2 = make_float2(sc.x, sc.x);
      // S into its operand (after the last chunk too, where no product takes it)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hv[4], lv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(__fmul2_rn(S[4 * k + i], sc2), hv[i], lv[i]);
        unsigned char *o = smem + OFF_SB + swz(n, 4 * hf + k);
        *reinterpret_cast<uint4 *>(o) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        *reinterpret_cast<uint4 *>(o + kHalf) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
      }
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_SREADY));
      // while K S^T runs: y of the chunk before, the bound of |S|, this chunk's rows
      if (is_q && c > 0) put_y(c - 1);
      if (c == nck) break;
      publish_max(c & 1);
      ok = wait_stage(BAR_FULL, c);
      ok = wait_stage(BAR_MAXV, c) && ok;
      const float gamma = arr(OFF_GAMMA)[row] * sc.y, gamma_end = arr(OFF_GAMMA)[C - 1];
      const float vmax = reinterpret_cast<const float *>(smem + OFF_MAXV)[c % kStages];
      const float2 rsc = state_scale(fmaxf(m, vmax));
      uint4 vv[4];
      float b = 0.f, back_k = 0.f, to_end = 0.f;
      if (!is_q) {
        const bool live = c * C + row < len;
        to_end = arr(OFF_END)[row];
        if (live) b = arr(OFF_BETA)[row] * rsc.x;
        back_k = -gamma * arr(OFF_RHOK)[row];
        const uint4 *src = reinterpret_cast<const uint4 *>(stage + OFF_V + row * kVPitch + 64 * hf);
#pragma unroll
        for (int i = 0; i < 4; ++i) vv[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
      } else {
        rho_q = arr(OFF_RHOQ)[row];
        back_o = rsc.y;
      }
      ok = wait(BAR_D1, c & 1) && ok;
      __syncwarp();
      tc_fence_after();
      const float2 g2 = make_float2(gamma, gamma), k2 = make_float2(back_k, back_k), b2 = make_float2(b, b);
      const float2 e2 = make_float2(to_end, to_end);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16], e[16];
        tmem_ld16(tmem + TM_D1 + 32 * hf + 16 * x + lane_off, d);
        tmem_ld16(tmem + TM_D1 + 64 + 32 * hf + 16 * x + lane_off, e);
        tmem_ld_wait();
        if (is_q) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            qs[8 * x + i] = __fmul2_rn(g2, __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(e[2 * i], e[2 * i + 1])));
        } else {
          uint32_t hv[8], lv[8], rv[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 u4 = vv[2 * x + (i >> 2)];
            const uint32_t u = (i & 3) == 0 ? u4.x : (i & 3) == 1 ? u4.y : (i & 3) == 2 ? u4.z : u4.w;
            const float2 v = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
            const float2 ks = __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(e[2 * i], e[2 * i + 1]));
            const float2 r = __fmul2_rn(b2, __ffma2_rn(k2, ks, v));
            rv[i] = h2(__float22half2_rn(r));
            split2(__fmul2_rn(e2, r), hv[i], lv[i]);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            unsigned char *o = smem + OFF_RB + swz(row, 4 * hf + 2 * x + u);
            *reinterpret_cast<uint4 *>(o) = make_uint4(hv[4 * u], hv[4 * u + 1], hv[4 * u + 2], hv[4 * u + 3]);
            *reinterpret_cast<uint4 *>(o + 8192) = make_uint4(lv[4 * u], lv[4 * u + 1], lv[4 * u + 2], lv[4 * u + 3]);
            *reinterpret_cast<uint4 *>(o + 16384) = make_uint4(rv[4 * u], rv[4 * u + 1], rv[4 * u + 2], rv[4 * u + 3]);
          }
        }
      }
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_RREADY));
      // S = gamma_end S + M R
      const float2 ge = make_float2(gamma_end, gamma_end), y2 = make_float2(rsc.y, rsc.y);
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = __fmul2_rn(S[i], ge);
      ok = wait(BAR_S, c & 1) && ok;
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      m = fmaf(gamma_end, read_max(c & 1), vmax);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16];
        tmem_ld16(tmem + TM_S + 32 * hf + 16 * x + lane_off, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) S[8 * x + i] = __ffma2_rn(y2, make_float2(d[2 * i], d[2 * i + 1]), S[8 * x + i]);
      }
    }
    if (ok) {
      if (p.h_final) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (in_bounds(soff + (long long)i * kDState, p.state_extent, p.err))
            p.h_final[soff + (long long)i * kDState] = i & 1 ? S[i / 2].y : S[i / 2].x;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 19) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
#undef BAR
}

// ---- front end: the operand tiles and gates of every chunk -----------------------------------------
// One CTA per (chunk, group).  A warp takes 16 of the 128 rows (64 of K, 64 of Q): a row is scaled
// by the power of two that brings its largest element to [1, 2), which is exact in fp16 down to
// 2^-17 of it, and stored where the swizzled operand tile wants it; rho is that power and the norm's
// factor.  Then each warp scans the gates of its heads, in fp64, so that differences of the prefix
// sums keep fp32's relative precision however large the sums, and leaves per token cs (as two floats),
// beta, 2^cs, and rho 2^{r - cs} for r the prefix sum at the end of its block of 32 and of the chunk.
// Bound by HBM: per token and group 512 bytes read and 520 written, per token and head 4 and 24.

// 2^x for x <= 0, to fp32's precision: the whole part of x as an exponent, the rest by exp2f
__device__ __forceinline__ float exp2_split(double x) {
  const double w = rint(x);
  return ldexpf(exp2f((float)(x - w)), (int)fmax(w, -200.0));
}

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
  __shared__ float s_rho[C];
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
    if (lane == 0) {
      reinterpret_cast<float *>(tile + OFF_RHOK)[r] = rho;
      if (r < 64) s_rho[r] = rho;
    }
  }
  __syncthreads();  // rho of the keys
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
    const double cs[2] = {sum - s[1] + s[0], sum};
    const double mid = __shfl_sync(0xffffffffu, sum, 15), end = __shfl_sync(0xffffffffu, sum, 31);
    const double ref = lane < 16 ? mid : end;  // cs at the end of this token's block of 32
    float out[6][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float rho = s_rho[2 * lane + u];
      out[0][u] = (float)cs[u];
      out[1][u] = (float)(cs[u] - out[0][u]);
      out[2][u] = beta[u];
      out[3][u] = exp2_split(cs[u]);
      out[4][u] = rho * exp2_split(ref - cs[u]);
      out[5][u] = rho * exp2_split(end - cs[u]);
    }
    float *dst = p.gates + (ck * p.H + h) * (kDeltaGateBytes / 4) + 2 * lane;
#pragma unroll
    for (int i = 0; i < 6; ++i) *reinterpret_cast<float2 *>(dst + i * C) = make_float2(out[i][0], out[i][1]);
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
