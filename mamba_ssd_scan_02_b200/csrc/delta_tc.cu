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
// The front end (delta_prep.cu) computes T~ and A T = 2^{cs_t - cs_j} rho_j (A~ T~)_tj.
//
// Precision.  The state is fp32, in registers.  Its products run on fp16 operands in two parts,
// hi = fp16(x), lo = fp16(x - hi), which keep 22 bits; the products hi.hi + hi.lo + lo.hi leave an error
// of about 2^-22, so the state stays as near to the fp64 rule as an fp32 recurrence does.  K and Q need
// one part: a row of bf16 numbers times a power of two is exact in fp16, and the power and the norm's
// factor come back in the fp32 factors rho.  |T~| and |M| are bounded (beta |k|^2 <= 2 and
// 1 <= |K_i| < 23); S and R are scaled by powers of two from running bounds of |S| and |V|
// (state_scale), so that fp16's range holds any size of input.  Only what goes into y alone (A~, A T, the R
// beside it) is rounded to 11 bits: y is then rounded to bf16's 8.
//
// Roles (16 warps, so that a thread may have 128 registers).  Warps 0-7, the chain: S into its operand, R
// from K S^T, the new S, y.  Warps 8-11 bring M (of the chunk after) into its operand.  Warps 12 and 13
// issue the MMAs of the chain and of M (an issuing thread is held up for about as long as its MMAs
// run), warp 14 loads (bulk copies of the front end's tiles and records and of the rows of V), warp 15
// finds the largest |V| of each chunk.  Hand-overs are mbarriers; every wait is bounded: a timeout makes
// every role leave and latches SSD_ERR_TIMEOUT.
#include "common.cuh"
#include "delta_mma.cuh"
#include "delta_plan.h"
#include "plan.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;
using namespace delta;

constexpr int C = kDeltaChunk;
constexpr int kThreads = 16 * 32;
constexpr int kStages = 2;
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes
// stage
constexpr uint32_t OFF_RHOK = 2 * kHalf;          // the tile's row factors follow its operands
constexpr uint32_t OFF_RHOQ = OFF_RHOK + 256;
constexpr uint32_t OFF_T = 33 * 1024;             // the record: T~^T hi, lo, A T; three arrays of 64 floats
constexpr uint32_t OFF_AT = OFF_T + 2 * 8192;
constexpr uint32_t OFF_BETA = OFF_T + 3 * 8192;
constexpr uint32_t OFF_GAMMA = OFF_BETA + 256;
constexpr uint32_t OFF_END = OFF_GAMMA + 256;
constexpr uint32_t OFF_V = OFF_END + 256;         // 64 rows of 128 bytes, 144 apart (no bank conflicts)
constexpr uint32_t kVPitch = 144;
constexpr uint32_t kStage = (OFF_V + C * kVPitch + 1023) / 1024 * 1024;
static_assert(OFF_RHOQ + 256 == kDeltaTileBytes && kDeltaTileBytes <= OFF_T && OFF_V - OFF_T == kDeltaRecordBytes, "as loaded");
// CTA
constexpr uint32_t OFF_SB = kStages * kStage;     // S operand: [n][p] hi, then lo (128 rows x 128 bytes each)
constexpr uint32_t OFF_RB = OFF_SB + 2 * kHalf;   // R operands: [token][p] R~ hi, lo; R (64 rows x 128 bytes each)
constexpr uint32_t OFF_MAXS = OFF_RB + 3 * 8192;  // largest |S| per chain warp, two chunks
constexpr uint32_t OFF_MAXV = OFF_MAXS + 64;      // bound of what the chunk adds, per stage
constexpr uint32_t OFF_BAR = OFF_MAXV + 64;
// A barrier that can complete again before every waiter has seen the phase before has one copy per
// buffer, so that a parity test never sees two phases at once.
enum {
  BAR_FULL,                        // [2] stage loaded
  BAR_EMPTY = BAR_FULL + kStages,  // [2] its last product is done (and every read before it)
  BAR_MAXV = BAR_EMPTY + kStages,  // [2] bound of what the chunk adds known
  BAR_M = BAR_MAXV + kStages,      // [2] M done
  BAR_MREADY = BAR_M + 2,          // [2] M operand in tensor memory (4 warps)
  BAR_SREADY = BAR_MREADY + 2,     // S operand written (8 warps)
  BAR_D1,                          // K S^T, Q S^T done
  BAR_RREADY,                      // R operands written, D1 read (8 warps)
  BAR_S,                           // M R~ done
  BAR_O,                           // A T R done
  BAR_DONE,                        // [2] nothing of an issuer's left in flight
  kNumBars = BAR_DONE + 2
};
constexpr uint32_t OFF_MISC = OFF_BAR + 8 * 32;   // [0] TMEM base, [1] abort flag
constexpr uint32_t kSmem = OFF_MISC + 16 + 1024;  // room to align the base to 1024 bytes
static_assert(kNumBars <= 32 && kSmem <= 232448, "shared memory");
static_assert(OFF_SB % 1024 == 0 && OFF_RB % 1024 == 0 && OFF_T % 1024 == 0, "swizzle alignment");

// TMEM columns.  K rows are lanes 0-63 of D1, Q rows lanes 64-127, as are the rows of A T R (lanes 0-63
// of it are never used).  The M operand replaces M: tokens 32 b .. 32 b + 31 lie in the columns 32 b .. of
// their own 32 fp32 columns, hi first, lo 16 columns on.
constexpr uint32_t TM_M = 0, TM_D1 = 128, TM_S = 256, TM_O = 320, TM_COLS = 512;

constexpr uint32_t IDESC_D1 = idesc_f16(128, 128, false, true, kFmtF16);   // [K; Q] . [S hi | S lo]
constexpr uint32_t IDESC_M = idesc_f16(128, 64, true, false, kFmtF16);     // K^T . T
constexpr uint32_t IDESC_R = idesc_f16(128, 64, false, true, kFmtF16);     // M (TMEM) or A T . R

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

// The issuing loops stay rolled: an MMA runs for 32 to 64 clocks, and the chain's code should stay in
// the instruction cache.
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
// d = M_hi R~_hi + M_hi R~_lo + M_lo R~_hi  (64 tokens each)
__device__ __forceinline__ void issue_S(uint32_t m, uint32_t r, uint32_t d) {
  const uint64_t b = smem_desc_sw128(r, 8192, 1024);
#pragma unroll 1
  for (int j = 0; j < 12; ++j)
    mma_f16_ts(d, m + tstep(j & 3) + (j >> 3) * 16, adv(b, 2048 * (j & 3) + (j >> 2 & 1) * 8192), IDESC_R, j > 0);
}
// A T . R: rows 64-127 of the A operand are A T's; rows 0-63 are what lies 8 KB before it, and their
// results are not used
__device__ __forceinline__ void issue_O(uint32_t at, uint32_t r, uint32_t d) {
  const uint64_t a = smem_desc_sw128(at - 8192, 16, 1024), b = smem_desc_sw128(r, 8192, 1024);
#pragma unroll 1
  for (int j = 0; j < 4; ++j) mma_f16_ss(d, adv(a, 32 * j), adv(b, 2048 * j), IDESC_R, j > 0);
}

// Powers of two that bring a quantity bounded by m to [64, 128) and back.  Headroom: with alpha <= 1
// and beta |k|^2 <= 2 the transition does not expand a state row s, so over a chunk
// |s'| <= gamma |s| + 64 * 2 max|V|, and |R|, |R~| <= 2 (max|V| + |s|).  With m = gamma max|S_old| + max|V| that
// is |S| <= (sqrt(128) + 128) m < 140 m and |R| < 282 max(m, max|V|): both below 65504 / 128 = 511.
__device__ __forceinline__ float2 state_scale(float m) {
  const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u), 8), 254);
  return make_float2(__uint_as_float((uint32_t)(260 - e) << 23), __uint_as_float((uint32_t)(e - 6) << 23));
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
  const auto wait_buf = [&](int bar, int c) { return wait(bar + (c & 1), (c >> 1) & 1); };  // one of two copies

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(BAR(i), i == BAR_SREADY || i == BAR_RREADY ? 8 : i == BAR_MREADY || i == BAR_MREADY + 1 ? 4 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 15) {
    tmem_alloc(sb + OFF_MISC, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int q4 = warp & 3;                           // TMEM lanes 32 q4 ..
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16;

  if (warp == 12) {
    // ------------------------------------------------------------------ MMAs of the chain
    if (lane == 0) {
      for (int c = 0; c < nck; ++c) {
        const uint32_t stage = sb + (c & 1) * kStage;
        if (!wait_buf(BAR_FULL, c) || !wait(BAR_SREADY, c & 1)) break;
        tc_fence_after();
        issue_D1(stage, sb + OFF_SB, tmem + TM_D1);
        mma_commit(BAR(BAR_D1));
        if (!wait_buf(BAR_MREADY, c) || !wait(BAR_RREADY, c & 1)) break;
        tc_fence_after();
        issue_S(tmem + TM_M + 64 * (c & 1), sb + OFF_RB, tmem + TM_S);
        mma_commit(BAR(BAR_S));
        issue_O(stage + OFF_AT, sb + OFF_RB + 16384, tmem + TM_O);
        mma_commit(BAR(BAR_O));
        mma_commit(BAR(BAR_EMPTY + (c & 1)));
      }
      mma_commit(BAR(BAR_DONE));  // no MMA may still be running when TMEM is released
      int never_abort = 0;
      mbar_wait(BAR(BAR_DONE), 0, &never_abort, p.err);
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMAs of M
    if (lane == 0) {
      for (int c = 0; c < nck; ++c) {
        // a loaded stage also says that the chain is through with the M of two chunks before
        if (!wait_buf(BAR_FULL, c)) break;
        tc_fence_after();
        issue_M(sb + (c & 1) * kStage, sb + (c & 1) * kStage + OFF_T, tmem + TM_M + 64 * (c & 1));
        mma_commit(BAR(BAR_M + (c & 1)));
      }
      mma_commit(BAR(BAR_DONE + 1));
      int never_abort = 0;
      mbar_wait(BAR(BAR_DONE + 1), 0, &never_abort, p.err);
    }
  } else if (warp == 14) {
    // ------------------------------------------------------------------ loads
    const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + base * p.vs + h * p.P + 64 * ph;
    int c = 0;
    for (; c < nck; ++c) {
      const int rows = min(C, len - c * C);
      const uint32_t dst = sb + (c & 1) * kStage, full = BAR(BAR_FULL + (c & 1));
      bool ok = true;
      if (lane == 0) {
        ok = c < kStages || wait_buf(BAR_EMPTY, c - kStages);
        if (ok) mbar_arrive_expect_tx(full, (uint32_t)(kDeltaTileBytes + kDeltaRecordBytes) + rows * 128);
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      for (int r = lane; r < rows; r += 32) bulk_load(dst + OFF_V + r * kVPitch, v + (c * C + r) * p.vs, 128, full);
      if (lane == 0) {
        // V is the caller's; tiles and records are the front end's, which may still be running
        // (programmatic dependent launch)
        if (c == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        bulk_load(dst, p.tiles + ((ck0 + c) * p.G + h / p.hpg) * kDeltaTileBytes, (uint32_t)kDeltaTileBytes, full);
        bulk_load(dst + OFF_T, p.records + ((ck0 + c) * p.H + h) * kDeltaRecordBytes, (uint32_t)kDeltaRecordBytes, full);
      }
      __syncwarp();
    }
    if (lane == 0) {  // every load must land before the CTA may exit
      int never_abort = 0;
      for (int j = max(0, c - kStages); j < c; ++j) mbar_wait(BAR(BAR_FULL + (j & 1)), (j >> 1) & 1, &never_abort, p.err);
    }
  } else if (warp == 15) {
    // ------------------------------------------------------------------ largest |V| of each chunk, times the
    // largest |beta| / 2 where that is above one
    for (int c = 0; c < nck; ++c) {
      const bool ok = wait_buf(BAR_FULL, c);
      if (!__all_sync(0xffffffffu, ok)) break;
      const unsigned char *stage = smem + (c & 1) * kStage;
      const int rows = min(C, len - c * C);
      uint32_t top = 0;
#pragma unroll 4
      for (int r = lane >> 3; r < rows; r += 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(stage + OFF_V + r * kVPitch + (lane & 7) * 16);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                     __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
      }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
      const float2 b = reinterpret_cast<const float2 *>(stage + OFF_BETA)[lane];
      const uint32_t bt = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(b.x), fabsf(b.y))));
      if (lane == 0) {
        reinterpret_cast<float *>(smem + OFF_MAXV)[c & 1] = __uint_as_float(top << 16) * fmaxf(1.f, 0.5f * __uint_as_float(bt));
        mbar_arrive(BAR(BAR_MAXV + (c & 1)));
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ M into its operand
    for (int c = 0; c < nck; ++c) {
      const bool ok = wait_buf(BAR_M, c);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const uint32_t at = tmem + TM_M + 64 * (c & 1) + 32 * b + lane_off;
        float m[32];
        uint32_t hv[16], lv[16];
        tmem_ld32(at, m);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) split2(make_float2(m[2 * j], m[2 * j + 1]), hv[j], lv[j]);
        tmem_st16(at, hv);
        tmem_st16(at + 16, lv);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_MREADY + (c & 1)));
    }
  } else {
    // ------------------------------------------------------------------ the chain
    const int hf = warp >> 2;                // state rows (columns of D1, S and O) 32 hf ..
    const bool is_q = q4 >= 2;
    const int row = 32 * (q4 & 1) + lane;    // token of this thread's lane of D1 and O
    const int n = 32 * q4 + lane;            // state column of this thread
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
      const unsigned char *stage = smem + (c & 1) * kStage;
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
      ok = wait_buf(BAR_FULL, c);
      ok = wait_buf(BAR_MAXV, c) && ok;
      const float gamma = arr(OFF_GAMMA)[row] * sc.y, gamma_end = arr(OFF_GAMMA)[C - 1];
      const float vmax = reinterpret_cast<const float *>(smem + OFF_MAXV)[c & 1];
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
      // S = gamma_end S + M R~
      const float2 ge = make_float2(gamma_end, gamma_end), y2 = make_float2(rsc.y, rsc.y);
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = __fmul2_rn(S[i], ge);
      ok = wait(BAR_S, c & 1) && ok;
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
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
    if (ok && p.h_final) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (in_bounds(soff + (long long)i * kDState, p.state_extent, p.err))
          p.h_final[soff + (long long)i * kDState] = i & 1 ? S[i / 2].y : S[i / 2].x;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
#undef BAR
}

}  // namespace

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
