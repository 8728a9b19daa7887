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
//   S' = 2^{cs_C} S + sum_j R_j (rho_j 2^{cs_C - cs_j} M_j)^T,          M = K^T T~          (N x 64)
//   y_t = 2^{cs_t} S q_t + sum_j 2^{cs_t - cs_j} rho_j (A~ T~)_tj R_j,   A~_ti = q_t.K_i     (i <= t)
// The inverse, M and A~ T~ know no decay, and nothing of them depends on the state: the chain from chunk
// to chunk is two dependent products, K S^T (which gives R) and M R.  One CTA carries 64 state rows
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
// from K S^T, the new S, y.  Their two halves, 32 state rows each, are chains of their own, one
// product apart, so that the conversions of the one run beside the products of the other.  Warps 8-11 bring M
// (of the chunk after) into its operand.  Warp 12 issues the MMAs of the chains, warp 13 those of M, warp
// 14 loads, warp 15 loads T and finds the largest |V| of each chunk.  Hand-overs are mbarriers; every
// wait is bounded: a timeout makes every role leave and latches SSD_ERR_TIMEOUT.
#include <cudaTypedefs.h>

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
constexpr uint32_t kHalf = 16384;  // 128 rows x 128 bytes
// Rings of what is loaded, as deep as it is needed early: the group's tile (K and Q; M takes K a chunk ahead of
// the chain, and a load takes more than half a chunk) three, T two (M alone takes it), A T two, V
// with the head's gates three.
constexpr int kDeep = 3;
constexpr uint32_t OFF_RHOK = 2 * kHalf;          // the tile's row factors follow its operands
constexpr uint32_t OFF_RHOQ = OFF_RHOK + 256;
constexpr uint32_t kTile = 33 * 1024;
static_assert(OFF_RHOQ + 256 == kDeltaTileBytes && kDeltaTileBytes <= kTile, "as loaded");
constexpr uint32_t kT = 16384, kAT = 8192;        // T~^T hi, lo; A T
constexpr uint32_t OFF_BETA = 8192;               // after V (64 rows of 128 bytes, swizzled): three arrays of 64 floats
constexpr uint32_t OFF_GAMMA = OFF_BETA + 256;
constexpr uint32_t OFF_END = OFF_GAMMA + 256;
constexpr uint32_t kVG = 9 * 1024;
static_assert(kT + kAT + 3 * 256 == kDeltaRecordBytes && OFF_END + 256 <= kVG, "as loaded");
// CTA
constexpr uint32_t OFF_T = kDeep * kTile;
constexpr uint32_t OFF_AT = OFF_T + 2 * kT;
constexpr uint32_t OFF_VG = OFF_AT + 2 * kAT;
constexpr uint32_t OFF_SB = OFF_VG + kDeep * kVG;  // S operands of the halves: [n][32 p hi, 32 p lo], 128 rows each
constexpr uint32_t OFF_R = OFF_SB + 2 * kHalf;    // R operands of the halves: [token][32 p hi, 32 p lo], 64 rows each
constexpr uint32_t OFF_MAXS = OFF_R + 2 * 8192;      // largest |S| per chain warp, two chunks
constexpr uint32_t OFF_MAXV = OFF_MAXS + 64;      // bound of what the chunk adds, per place in the ring
constexpr uint32_t OFF_BAR = OFF_MAXV + 64;
// A barrier that can complete again before every waiter has seen the phase before has one copy per
// buffer, so that a parity test never sees two phases at once.
enum {
  BAR_TILE,                        // [3] tile loaded
  BAR_VG = BAR_TILE + kDeep,       // [3] V and gates loaded
  BAR_READY = BAR_VG + kDeep,      // [3] both, and the bound of what the chunk adds known
  BAR_EMPTY = BAR_READY + kDeep,   // [3] the chunk's last product (and every read before it) is done
  BAR_T = BAR_EMPTY + kDeep,       // [2] T loaded
  BAR_AT = BAR_T + 2,              // [2] A T loaded
  BAR_M = BAR_AT + 2,              // [2] M done
  BAR_MREADY = BAR_M + 2,          // [2] M operand in tensor memory (4 warps)
  BAR_SREADY = BAR_MREADY + 2,     // [2 halves] S operand written (4 warps)
  BAR_RREADY = BAR_SREADY + 2,     // [2 halves] R operand written, D1 read (4 warps)
  BAR_D1 = BAR_RREADY + 2,         // [2 halves] K S^T, Q S^T done
  BAR_S = BAR_D1 + 2,              // [2 halves] M R done
  BAR_O = BAR_S + 2,               // [2 halves] A T R done
  BAR_DONE = BAR_O + 2,            // [2] nothing of an issuer's left in flight
  kNumBars = BAR_DONE + 2
};
constexpr uint32_t OFF_MISC = OFF_BAR + 8 * 32;   // [0] TMEM base, [1] abort flag, [2] the same for the last waits
constexpr uint32_t kSmem = OFF_MISC + 16 + 1024;  // room to align the base to 1024 bytes
static_assert(kNumBars <= 32 && kSmem <= 232448, "shared memory");
static_assert(OFF_SB % 1024 == 0 && OFF_R % 1024 == 0 && OFF_T % 1024 == 0 && OFF_VG % 1024 == 0, "swizzle alignment");

// TMEM columns.  K rows are lanes 0-63 of D1, Q rows lanes 64-127, as are the rows of A T R (lanes 0-63
// of it are never used).  D1 and S have per half 32 columns of the products with hi, 32 of those with
// lo, O 32 columns.  The M operand replaces M: tokens 32 b .. 32 b + 31 lie in the columns 32 b .. of their own 32 fp32
// columns, hi first, lo 16 columns on.
constexpr uint32_t TM_M = 0, TM_D1 = 128, TM_S = 256, TM_O = 384, TM_COLS = 512;

constexpr uint32_t IDESC_N64 = idesc_f16(128, 64, false, true, kFmtF16);   // [K; Q] . S, M (TMEM) . R
constexpr uint32_t IDESC_N32 = idesc_f16(128, 32, false, true, kFmtF16);   // M_lo (TMEM) . R_hi, A T . R_hi
constexpr uint32_t IDESC_M = idesc_f16(128, 64, true, false, kFmtF16);     // K^T . T

// A bounded wait.  A try suspends the warp for a while in hardware; after every 256 the abort flag is
// looked at, and after 2^17 times that (about a second) the flag is set to 2.  In one piece of
// assembly, because a warp that waits should issue little (about half of them wait at any time), and
// because every wait of every role sits in the instruction cache.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint32_t abort) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n, m, f;\n\t"
      "mov.u32 m, 131072;\n"
      "OUTER_%=:\n\t"
      "mov.u32 n, 256;\n"
      "TRY_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra TRY_%=;\n\t"
      "ld.volatile.shared.u32 f, [%3];\n\t"
      "setp.ne.u32 q, f, 0;\n\t"
      "@q bra DONE_%=;\n\t"
      "sub.u32 m, m, 1;\n\t"
      "setp.ne.u32 q, m, 0;\n\t"
      "@q bra OUTER_%=;\n\t"
      "st.volatile.shared.u32 [%3], 2;\n"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(abort)
      : "memory");
  return ok != 0;
}

// Position in a ring of D places: the place, and the parity of its current use
template <int D>
struct Ring {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == D) {
      at = 0;
      parity ^= 1;
    }
  }
};

// Start address field of an operand's descriptor, advanced by adding to it (16-byte units; every operand lies
// below 256 KB); the other word holds the strides, the version bits and the 128-byte swizzle.
__device__ __forceinline__ uint32_t op_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t kOpHi = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ constexpr uint32_t kstep(int j) { return ((j >> 2) * kHalf + (j & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint32_t tstep(int j) { return (j >> 1) * 32 + (j & 1) * 8; }

// The issuing warps run converged and elect a lane per instruction, and what the descriptors come from is
// broadcast with shuffles: the compiler then knows it to be uniform and keeps the descriptors in uniform
// registers.  Moved there from a divergent branch for every MMA, they cost 50 to 80 clocks each, more
// than the MMA (SS N = 64: 49 clocks, its operands' shared-memory reads; TS N = 64: 32, N = 32: 16).
template <uint32_t kIdesc>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "n"(kIdesc), "r"((uint32_t)acc), "n"(kOpHi)
      : "memory");
}
template <uint32_t kIdesc>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "n"(kIdesc), "r"((uint32_t)acc), "n"(kOpHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void issue_D1(uint32_t kq, uint32_t sbuf, uint32_t d) {
  const uint32_t a = op_lo(kq, 16), b = op_lo(sbuf, 8192);
#pragma unroll
  for (int j = 0; j < 8; ++j) mma_ss<IDESC_N64>(d, a + kstep(j), b + j * 128, j > 0);
}
__device__ __forceinline__ void issue_M(uint32_t kq, uint32_t t, uint32_t d) {
  const uint32_t a = op_lo(kq, kHalf), b = op_lo(t, 16);
#pragma unroll
  for (int j = 0; j < 8; ++j)  // hi, then lo
    mma_ss<IDESC_M>(d, a + (j & 3) * 128, b + (j >> 2) * 512 + (j & 3) * 2, j > 0);
}
// d = M_hi R_hi + M_lo R_hi | M_hi R_lo  (64 tokens)
__device__ __forceinline__ void issue_S(uint32_t m, uint32_t r, uint32_t d) {
  const uint32_t b = op_lo(r, 8192);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ts<IDESC_N64>(d, m + tstep(j), b + 128 * j, j > 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ts<IDESC_N32>(d, m + tstep(j) + 16, b + 128 * j, true);
}
// A T . R_hi: rows 64-127 of the A operand are A T's; rows 0-63 are what lies 8 KB before it, and their
// results are not used
__device__ __forceinline__ void issue_O(uint32_t at, uint32_t r, uint32_t d) {
  const uint32_t a = op_lo(at - 8192, 16), b = op_lo(r, 8192);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ss<IDESC_N32>(d, a + 2 * j, b + 128 * j, j > 0);
}

// Powers of two that bring a quantity bounded by m to [64, 128) and back.  Headroom: with alpha <= 1
// and beta |k|^2 <= 2 the transition does not expand a state row s, so over a chunk
// |s'| <= gamma |s| + 64 * 2 max|V|, and |R| <= 2 (max|V| + |s|).  With m = gamma max|S_old| + max|V| that
// is |S| <= (sqrt(128) + 128) m < 140 m and |R| < 282 max(m, max|V|): both below 65504 / 128 = 511.
__device__ __forceinline__ float2 state_scale(float m) {
  const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u), 8), 254);
  return make_float2(__uint_as_float((uint32_t)(260 - e) << 23), __uint_as_float((uint32_t)(e - 6) << 23));
}

__global__ void __launch_bounds__(kThreads, 1)
    ssd_delta_chunk_kernel(const __grid_constant__ CUtensorMap tm_v, const DeltaPlan p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int halves = p.P >> 6;
  const int h = blockIdx.x / halves, ph = blockIdx.x % halves;
  const int seq = p.order ? p.order[blockIdx.y] : (int)blockIdx.y;
  const int len = seq_len(p.cu, seq, p.L);
  const long long base = seq_base(p.cu, seq, p.L);
  const int nck = (len + C - 1) / C;
  const uint32_t bar0 = sb + OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
  const uint32_t abort_at = sb + OFF_MISC + 4;
  const auto wait = [&](int bar, uint32_t parity) { return wait_bounded(BAR(bar), parity, abort_at); };
  // before leaving, whatever the abort flag says
  const auto settle = [&](int bar, uint32_t parity) { wait_bounded(BAR(bar), parity, abort_at + 4); };
  const auto wait2 = [&](int bar, int c) { return wait(bar + (c & 1), (c >> 1) & 1); };  // one of two copies

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(BAR(i), i >= BAR_MREADY && i < BAR_D1 ? 4 : 1);
    misc[1] = misc[2] = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(sb + OFF_MISC, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const int q4 = warp & 3;                           // TMEM lanes 32 q4 ..
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16;

  const bool lead = lane == 0;
  if (warp == 12) {
    // ------------------------------------------------------------------ MMAs of the chains, one half's after the
    // other's: while those of one run, the other converts
    Ring<kDeep> r;
    bool ok = true;
    for (int c = 0; c < nck && ok; ++c, r.next()) {
      ok = wait(BAR_READY + r.at, r.parity);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        ok = wait(BAR_SREADY + half, c & 1) && ok;
        tc_fence_after();
        issue_D1(sb + r.at * kTile, sb + OFF_SB + half * kHalf, tmem + TM_D1 + 64 * half);
        commit(BAR(BAR_D1 + half));
      }
      ok = wait2(BAR_MREADY, c) && ok;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        ok = wait(BAR_RREADY + half, c & 1) && ok;
        tc_fence_after();
        issue_S(tmem + TM_M + 64 * (c & 1), sb + OFF_R + half * 8192, tmem + TM_S + 64 * half);
        commit(BAR(BAR_S + half));
      }
      ok = wait2(BAR_AT, c) && ok;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        issue_O(sb + OFF_AT + (c & 1) * kAT, sb + OFF_R + half * 8192, tmem + TM_O + 32 * half);
        commit(BAR(BAR_O + half));
      }
      commit(BAR(BAR_EMPTY + r.at));
      ok = __all_sync(0xffffffffu, ok);
    }
    commit(BAR(BAR_DONE));  // no MMA may still be running when TMEM is released
    settle(BAR_DONE, 0);
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMAs of M
    Ring<kDeep> r, e;
    bool ok = true;
    for (int c = 0; c < nck && ok; ++c, r.next()) {
      ok = wait(BAR_TILE + r.at, r.parity);
      ok = wait2(BAR_T, c) && ok;
      if (c >= 2) {  // the M of two chunks before is read
        ok = wait(BAR_EMPTY + e.at, e.parity) && ok;
        e.next();
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      issue_M(sb + r.at * kTile, sb + OFF_T + (c & 1) * kT, tmem + TM_M + 64 * (c & 1));
      commit(BAR(BAR_M + (c & 1)));
    }
    commit(BAR(BAR_DONE + 1));
    settle(BAR_DONE + 1, 0);
  } else if (warp == 14) {
    // ------------------------------------------------------------------ loads of tiles, V, gates, A T
    if (lead) {
      prefetch_tmap(&tm_v);
      const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
      const unsigned char *rec = p.records + (ck0 * p.H + h) * kDeltaRecordBytes + kT;
      const unsigned char *tile = p.tiles + (ck0 * p.G + h / p.hpg) * kDeltaTileBytes;
      const long long rec_step = p.H * kDeltaRecordBytes, tile_step = p.G * kDeltaTileBytes;
      Ring<kDeep> r, e;  // to load; to become free
      int n = 0, n_at = 0;
      // Turn c: tile, V and gates of chunk c, into the place of chunk c - 3; A T of chunk c - 1 (and in
      // turn 0 of chunk 0), whose two places are free then too.  The last turn loads A T alone.
      for (int c = 0; c <= nck; ++c) {
        if (c >= kDeep) {
          if (!wait(BAR_EMPTY + e.at, e.parity)) break;
          e.next();
        }
        if (c < nck) {
          const uint32_t vg = BAR(BAR_VG + r.at), tb = BAR(BAR_TILE + r.at), dst = sb + OFF_VG + r.at * kVG;
          mbar_arrive_expect_tx(vg, 8192 + 768);
          // 64 token rows, the ones after the sequence's end among them (they are not used)
          tma_load_2d(dst, &tm_v, h * p.P + 64 * ph, (int)(base + c * C), vg);
          // V is the caller's; tiles and records are the front end's, which may still be running
          // (programmatic dependent launch)
          if (c == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
          mbar_arrive_expect_tx(tb, (uint32_t)kDeltaTileBytes);
          bulk_load(sb + r.at * kTile, tile + c * tile_step, (uint32_t)kDeltaTileBytes, tb);
          bulk_load(dst + OFF_BETA, rec + c * rec_step + kAT, 768, vg);
          r.next();
          ++n;
        }
        if (c != 1 && n_at < nck) {
          const uint32_t at = BAR(BAR_AT + (n_at & 1));
          mbar_arrive_expect_tx(at, kAT);
          bulk_load(sb + OFF_AT + (n_at & 1) * kAT, rec + n_at * rec_step, kAT, at);
          ++n_at;
        }
      }
      // every load must land before the CTA may exit
      for (int k = 0; k < kDeep; ++k)
        if (k < n) {
          const uint32_t last = k < r.at ? r.parity : r.parity ^ 1;
          settle(BAR_VG + k, last);
          settle(BAR_TILE + k, last);
        }
      for (int k = max(0, n_at - 2); k < n_at; ++k) settle(BAR_AT + (k & 1), (k >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 15) {
    // ------------------------------------------------------------------ loads of T; the largest |V| of each chunk,
    // times the largest |beta| / 2 where that is above one
    const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
    const unsigned char *rec = p.records + (ck0 * p.H + h) * kDeltaRecordBytes;
    if (lead && nck > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    Ring<kDeep> r;
    int n = 0;
    // Turn c: the bound of chunk c, then T of chunk c + 2 over that of chunk c, once M has taken it
    for (int c = -2; c < nck; ++c) {
      if (c >= 0) {
        bool ok = wait(BAR_VG + r.at, r.parity);
        ok = wait(BAR_TILE + r.at, r.parity) && ok;
        const unsigned char *stage = smem + OFF_VG + r.at * kVG;
        const int rows = min(C, len - c * C);
        uint32_t top = 0;
#pragma unroll 4
        for (int i = lane >> 3; i < rows; i += 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(stage + i * 128 + (lane & 7) * 16);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                       __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const float2 b = reinterpret_cast<const float2 *>(stage + OFF_BETA)[lane];
        const uint32_t bt = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(b.x), fabsf(b.y))));
        if (lead) {
          reinterpret_cast<float *>(smem + OFF_MAXV)[r.at] = __uint_as_float(top << 16) * fmaxf(1.f, 0.5f * __uint_as_float(bt));
          mbar_arrive(BAR(BAR_READY + r.at));
        }
        __syncwarp();
        r.next();
        if (c + 2 < nck) ok = wait2(BAR_M, c) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      if (lead && c + 2 < nck) {
        const uint32_t t = BAR(BAR_T + (c & 1));
        mbar_arrive_expect_tx(t, kT);
        bulk_load(sb + OFF_T + (c & 1) * kT, rec + (long long)(c + 2) * p.H * kDeltaRecordBytes, kT, t);
        ++n;
      }
      __syncwarp();
    }
    if (lead)
      for (int k = max(0, n - 2); k < n; ++k) settle(BAR_T + (k & 1), (k >> 1) & 1);
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ M, its columns times
    // rho_j 2^{cs_C - cs_j}, into its operand
    Ring<kDeep> r;
    for (int c = 0; c < nck; ++c, r.next()) {
      bool ok = wait(BAR_VG + r.at, r.parity);  // the factors
      ok = wait2(BAR_M, c) && ok;
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const float4 *f = reinterpret_cast<const float4 *>(smem + OFF_VG + r.at * kVG + OFF_END);
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const uint32_t at = tmem + TM_M + 64 * (c & 1) + 32 * b + lane_off;
        float m[32];
        uint32_t hv[16], lv[16];
        tmem_ld32(at, m);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 x = f[8 * b + j];
          split2(__fmul2_rn(make_float2(m[4 * j], m[4 * j + 1]), make_float2(x.x, x.y)), hv[2 * j], lv[2 * j]);
          split2(__fmul2_rn(make_float2(m[4 * j + 2], m[4 * j + 3]), make_float2(x.z, x.w)), hv[2 * j + 1], lv[2 * j + 1]);
        }
        tmem_st16(at, hv);
        tmem_st16(at + 16, lv);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_MREADY + (c & 1)));
    }
  } else {
    // ------------------------------------------------------------------ the chains
    const int hf = warp >> 2;                // half: state rows (columns of S and O) 32 hf ..
    const bool is_q = q4 >= 2;
    const int row = 32 * (q4 & 1) + lane;    // token of this thread's lane of D1 and O
    const int n = 32 * q4 + lane;            // state column of this thread
    const long long soff = (((long long)seq * p.H + h) * p.P + 64 * ph + 32 * hf) * kDState + n;
    uint32_t *max_s = reinterpret_cast<uint32_t *>(smem + OFF_MAXS) + 8 * hf;
    const uint32_t t_d1 = tmem + TM_D1 + 64 * hf, t_s = tmem + TM_S + 64 * hf, t_o = tmem + TM_O + 32 * hf;
    float2 S[16];  // the state, times sc.x
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
      if (lane == 0) max_s[4 * buf + q4] = bits;
    };
    const auto read_max = [&](int buf) {
      const uint4 a = *reinterpret_cast<const uint4 *>(max_s + 4 * buf);
      return __uint_as_float(max(max(a.x, a.y), max(a.z, a.w)));
    };
    publish_max(1);
    named_bar(1 + hf, 128);
    float m = read_max(1);  // bounds the state as described at state_scale
    float2 sc = state_scale(m);
#pragma unroll
    for (int i = 0; i < 16; ++i) S[i] = __fmul2_rn(S[i], make_float2(sc.x, sc.x));
    // K rows: the chunk's V; Q rows: 2^cs Q S^T of the chunk whose y is still to come
    float2 hold[16];
    float gamma = 0.f, gamma_end = 0.f, beta = 0.f, rho = 0.f, vmax = 0.f;  // of the chunk
    float back_o = 0.f, rho_y = 0.f;                                         // of the y to come
    Ring<kDeep> ring;  // of the rows to load next
    const auto load_rows = [&](int c) {
      const unsigned char *stage = smem + OFF_VG + ring.at * kVG;
      const auto arr = [&](uint32_t off) { return reinterpret_cast<const float *>(stage + off); };
      const bool ok = wait(BAR_READY + ring.at, ring.parity);
      vmax = reinterpret_cast<const float *>(smem + OFF_MAXV)[ring.at];
      gamma = arr(OFF_GAMMA)[row];
      gamma_end = arr(OFF_GAMMA)[C - 1];
      rho = reinterpret_cast<const float *>(smem + ring.at * kTile + (is_q ? OFF_RHOQ : OFF_RHOK))[row];
      if (!is_q) {
        const bool live = c * C + row < len;  // (the rows after may hold anything)
        beta = live ? arr(OFF_BETA)[row] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 u = live ? *reinterpret_cast<const uint4 *>(stage + swz(row, 4 * hf + i)) : make_uint4(0, 0, 0, 0);
          hold[2 * i] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
          hold[2 * i + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
      }
      ring.next();
      return ok;
    };
    const auto put_y = [&](int c) {  // Q rows: y of chunk c
      wait(BAR_O + hf, c & 1);
      __syncwarp();
      tc_fence_after();
      const int t = c * C + row;
      const long long yo = (base + t) * p.ys + (long long)h * p.P + 64 * ph + 32 * hf;
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + yo);
      const bool store = t < len && in_bounds(yo + 31, p.y_extent, p.err);
      const float2 b2 = make_float2(back_o, back_o), r2 = make_float2(rho_y, rho_y);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float o[16];
        tmem_ld16(t_o + 16 * x + lane_off, o);
        tmem_ld_wait();
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = __fmul2_rn(r2, __ffma2_rn(b2, make_float2(o[2 * i], o[2 * i + 1]), hold[8 * x + i]));
          const __nv_bfloat162 v = __float22bfloat162_rn(f);
          u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if (store) {
          dst[2 * x] = make_uint4(u[0], u[1], u[2], u[3]);
          dst[2 * x + 1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
    };
    bool ok = nck == 0 || load_rows(0);
    for (int c = 0; c < nck; ++c) {
      // S into its operand
      unsigned char *so = smem + OFF_SB + hf * kHalf;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hv[4], lv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(S[4 * k + i], hv[i], lv[i]);
        *reinterpret_cast<uint4 *>(so + swz(n, k)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        *reinterpret_cast<uint4 *>(so + swz(n, 4 + k)) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
      }
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lead) mbar_arrive(BAR(BAR_SREADY + hf));
      // while K S^T runs: y of the chunk before, the bound of |S|
      if (is_q && c > 0) put_y(c - 1);
      publish_max(c & 1);
      const float2 rsc = state_scale(fmaxf(m, vmax));
      rho_y = rho;
      back_o = rsc.y;
      const float g = gamma * sc.y, gk = -g * rho, b = beta * rsc.x;
      const float2 g2 = make_float2(g, g), k2 = make_float2(gk, gk), b2 = make_float2(b, b);
      ok = wait(BAR_D1 + hf, c & 1) && ok;
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16], e[16];
        tmem_ld16(t_d1 + 16 * x + lane_off, d);
        tmem_ld16(t_d1 + 32 + 16 * x + lane_off, e);
        tmem_ld_wait();
        if (is_q) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            hold[8 * x + i] = __fmul2_rn(g2, __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(e[2 * i], e[2 * i + 1])));
        } else {
          uint32_t hv[8], lv[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 vp = hold[4 * x + i / 2];  // two bf16 pairs
            const uint32_t u = __float_as_uint(i & 1 ? vp.y : vp.x);
            const float2 v = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
            const float2 ks = __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(e[2 * i], e[2 * i + 1]));
            split2(__fmul2_rn(b2, __ffma2_rn(k2, ks, v)), hv[i], lv[i]);
          }
          unsigned char *o = smem + OFF_R + hf * 8192;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            *reinterpret_cast<uint4 *>(o + swz(row, 2 * x + u)) = make_uint4(hv[4 * u], hv[4 * u + 1], hv[4 * u + 2], hv[4 * u + 3]);
            *reinterpret_cast<uint4 *>(o + swz(row, 4 + 2 * x + u)) = make_uint4(lv[4 * u], lv[4 * u + 1], lv[4 * u + 2], lv[4 * u + 3]);
          }
        }
      }
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lead) mbar_arrive(BAR(BAR_RREADY + hf));
      // S = gamma_end S + M R, in the next chunk's scale; while the product runs: the next chunk's rows
      const float decay = gamma_end * sc.y, bound = vmax;
      if (c + 1 < nck) ok = load_rows(c + 1) && ok;
      ok = wait(BAR_S + hf, c & 1) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      m = fmaf(decay, read_max(c & 1), bound);
      sc = state_scale(m);
      const float ge = decay * sc.x, yn = rsc.y * sc.x;
      const float2 ge2 = make_float2(ge, ge), y2 = make_float2(yn, yn);
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = __fmul2_rn(S[i], ge2);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float d[16], e[16];
        tmem_ld16(t_s + 16 * x + lane_off, d);
        tmem_ld16(t_s + 32 + 16 * x + lane_off, e);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          S[8 * x + i] = __ffma2_rn(y2, __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(e[2 * i], e[2 * i + 1])), S[8 * x + i]);
      }
    }
    if (ok) {
      if (is_q && nck > 0) put_y(nck - 1);
      if (p.h_final) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (in_bounds(soff + (long long)i * kDState, p.state_extent, p.err))
            p.h_final[soff + (long long)i * kDState] = sc.y * (i & 1 ? S[i / 2].y : S[i / 2].x);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && misc[1] != 0) latch_error(p.err, (int)SSD_ERR_TIMEOUT);
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
#undef BAR
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

cudaError_t launch_delta_chunks(const DeltaPlan &p, cudaStream_t s) {
  // V as one matrix of all token rows; a box is 64 rows of 64 state rows
  const auto encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap tm;
  const cuuint64_t dims[2] = {(cuuint64_t)p.H * p.P, (cuuint64_t)p.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)p.vs * 2};
  const cuuint32_t box[2] = {64, C}, ones[2] = {1, 1};
  if (encode(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p.v), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
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
  e = cudaLaunchKernelEx(&lc, ssd_delta_chunk_kernel, tm, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ssd
