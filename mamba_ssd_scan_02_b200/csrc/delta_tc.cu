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
//   X_j = v_j - 2^{cs_j} S k_j,   u_j = beta_j rho_j,   w_j = 2^{cs_C - cs_j} u_j,
//   S' = 2^{cs_C} S + sum_j (w_j X_j) M_j^T,                         M = K^T T~            (N x 64)
//   y_t = 2^{cs_t} S q_t + sum_j 2^{cs_t - cs_j} (A~ T~)_tj (u_j X_j),   A~_ti = q_t.K_i     (i <= t)
// The inverse, M and A~ T~ know no decay, and nothing of them depends on the state: the chain from chunk
// to chunk is two dependent products, K S^T (which gives R = w X) and M R.  A CTA carries 64 state rows of one head
// through a sequence (the rows are independent given K, so a head of 128 rows is two such items), then the next
// item's: the grid is one CTA per SM, and an item's first loads and M run while the one before ends (64
// sequences of up to 700 tokens x 128 heads, when the chunks were slower than now: 715 us with a CTA per item, 606 so;
// now 572).
//
// The front end (delta_prep.cu) computes T~, A T = 2^{cs_t - cs_j} (A~ T~)_tj, u and w.
//
// Precision.  The state is fp32, in registers.  Its products run on fp16 operands in two parts,
// hi = fp16(x), lo = fp16(x - hi), which keep 22 bits; the products hi.hi + hi.lo + lo.hi leave an error
// of about 2^-22, so the state stays as near to the fp64 rule as an fp32 recurrence does (2.3e-7 of its root mean
// square after 8192 tokens, the worst of 128 heads 3.1e-7).  K and Q need
// one part: a row of bf16 numbers times a power of two is exact in fp16, and the power and the norm's
// factor come back in the fp32 factors rho.  What differs in size between tokens and heads - beta, the decays, the
// rho - stands in R, in fp32 before it is split: |T~|, |M| and |A T| are bounded without it (beta |k|^2 <= 2, 1 <=
// |K_i| < 23, alpha <= 1), and R and the next S have one scale, the power of two of a bound of the next S that
// counts each token's value as what is left of it at the chunk's end (state_scale).  So a term loses bits only
// beside larger terms of the same state.  (With the factors in M, which had no scale, and R's scale from |S| and |V|
// alone, a chunk that ended in tokens of small beta or without values lost up to all of the state's bits.)  Only
// what goes into y alone (A~, A T, the R beside it: u X, scaled by the largest |u V| and what the first token leaves
// of the largest |S|) is rounded to 11 bits, and to 2^-24 of the chunk's largest term where that is more: y is then
// rounded to bf16's 8.
//
// Roles (16 warps, so that a thread may have 128 registers).  Warps 0-7, the chain: S into its operand, R
// from K S^T, the new S.  Their two halves, 32 state rows each, share the product with K, whose operand is
// read once for both, and have M R each, so that one converts while the other's runs.  Warps 8-11 bring M (of
// the chunk after) into its operand and make y from Q S^T and A T R, neither in the chain's way.  Warp 12
// issues the MMAs of the chains, warp 13 those of M, warp 14 loads, warp 15 loads T and finds the largest |w V| and
// |u V| of each chunk.  Hand-overs are mbarriers; every wait is bounded: a timeout makes every role leave and
// latches SSD_ERR_TIMEOUT.
//
// What bounds it: the chain.  A chunk takes 1.8 us (8192 tokens x 128 heads: 228 us on 128 SMs, and 220 with one R for
// the state and y, whose scales then left bits out).  Of those 220: S into fp16 0.25 (the halves one after the other
// 0.5), K S^T 0.4, R 0.25, M R 0.35 (the next rows load meanwhile), the new S 0.2.  Now the tensor pipe is 50 % busy,
// the issue slots 59 %, DRAM 27 %.  Measured against it, at the stage each was tried: y by the chain's warps 246 us where this took 226;
// M R waiting for the readers of Q S^T 226 : 213; one M R for both halves 246 : 226; a product per half for
// K S^T (the halves half a chunk apart, one issuer each or one for both) 255 to 260 : 232, since the K and Q
// operand is then read twice.  The code is kept small (loops rolled, one place per inlined part): sixteen
// warps in six roles share an instruction cache, and 10 KB more of it cost 5 to 10 %.
#include <cudaTypedefs.h>
#include <algorithm>

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
// T~^T: four times (16 columns) 64 rows of hi, 64 of lo, 32 bytes each; A T: four times (16 columns) 128 rows,
// 16 of each of two chunks in turn.  In 8 x 8 core matrices; what the triangles leave out stays zero.
constexpr uint32_t kT = 16384, kAT = 8192;
constexpr uint32_t OFF_U = 8192;                  // after V (64 rows of 128 bytes, swizzled): three arrays of 64 floats
constexpr uint32_t OFF_GAMMA = OFF_U + 256;
constexpr uint32_t OFF_W = OFF_GAMMA + 256;
constexpr uint32_t kVG = 9 * 1024;
static_assert(OFF_W + 256 <= kVG, "as loaded");
// CTA
constexpr uint32_t OFF_T = kDeep * kTile;
constexpr uint32_t OFF_AT = OFF_T + 2 * kT;
constexpr uint32_t OFF_VG = OFF_AT + 2 * kAT;
// Per half, S operand: [n][32 p hi, 32 p lo], 128 rows.  Once K S^T is done, R operand: [token][32 p hi, 32 p lo],
// 64 rows.
constexpr uint32_t OFF_SB = OFF_VG + kDeep * kVG;
constexpr uint32_t OFF_R = OFF_SB + 2 * kHalf;    // R operand of y: [token][32 p of each half], 64 rows
constexpr uint32_t OFF_MAXS = OFF_R + 8192;       // largest |S| per chain warp: two chunks, an item's first
constexpr uint32_t OFF_SCALE = OFF_MAXS + 128;    // per half and chunk parity: the scales of S and of y's R, backwards
constexpr uint32_t OFF_BOUND = OFF_SCALE + 32;    // per place in the ring: max |w V|, max |u V|, the first 2^cs, the last
constexpr uint32_t OFF_BAR = OFF_BOUND + 64;
// A barrier that can complete again before every waiter has seen the phase before has one copy per
// buffer, so that a parity test never sees two phases at once.
enum {
  BAR_TILE,                        // [3] tile loaded
  BAR_VG = BAR_TILE + kDeep,       // [3] V and gates loaded
  BAR_READY = BAR_VG + kDeep,      // [3] both, and the bounds of what the chunk adds known
  BAR_EMPTY = BAR_READY + kDeep,   // [3] the chunk's last product (and every read before it) is done
  BAR_T = BAR_EMPTY + kDeep,       // [2] T loaded
  BAR_AT = BAR_T + 2,              // [2] A T loaded
  BAR_M = BAR_AT + 2,              // [2] M done
  BAR_MREADY = BAR_M + 2,          // [2] M operand in tensor memory (4 warps)
  BAR_SREADY = BAR_MREADY + 2,     // S operand written (8 warps)
  BAR_RREADY = BAR_SREADY + 1,     // [2 halves] R operands written, K S^T read (4 warps)
  BAR_D1 = BAR_RREADY + 2,         // K S^T, Q S^T done
  BAR_S = BAR_D1 + 1,              // [2 halves] M R done
  BAR_O = BAR_S + 2,               // A T R done
  BAR_DONE = BAR_O + 1,            // [2] nothing of an issuer's left in flight
  BAR_MAX = BAR_DONE + 2,          // [2 halves] the largest |S| of each warp written (4 warps)
  BAR_QREAD = BAR_MAX + 2,         // Q S^T read, and the y before it done (4 warps)
  kNumBars = BAR_QREAD + 1
};
constexpr uint32_t OFF_MISC = OFF_BAR + 8 * 32;   // [0] TMEM base, [1] abort flag, [2] the same for the last waits
constexpr uint32_t kSmem = OFF_MISC + 16 + 1024;  // room to align the base to 1024 bytes
static_assert(kNumBars <= 32 && kSmem <= 232448, "shared memory");
static_assert(OFF_SB % 1024 == 0 && OFF_R % 1024 == 0 && OFF_T % 1024 == 0 && OFF_VG % 1024 == 0, "swizzle alignment");

// TMEM columns.  M: twice 64 columns of the product with T's hi and 64 of that with its lo; the M operand
// replaces the former (tokens 16 j .. in the columns 16 j .. , hi first, lo 8 columns on).  Of every 32 lanes of
// D1 the first 16 are K rows, the others the Q rows of the same tokens, as are the rows of A T R (the other
// lanes of it are never used): each of the four warps that can read a quarter of the lanes then has as
// much to convert (with the K rows in lanes 0-63, two of them had all of R to convert, on two of the four
// schedulers: 240 us where this took 232, 8192 tokens x 128 heads).  D1 has per half 32 columns of the products
// with hi, 32 of those with lo, S and O 32 columns.
constexpr uint32_t TM_M = 0, TM_D1 = 256, TM_S = 384, TM_O = 448, TM_COLS = 512;

constexpr uint32_t IDESC_D1 = idesc_f16(128, 128, false, true, kFmtF16);  // [K; Q] . S of both halves
constexpr uint32_t IDESC_M = idesc_f16(128, 128, true, false, kFmtF16);   // K^T . [T_hi, T_lo]
constexpr uint32_t IDESC_S = idesc_f16(128, 32, false, true, kFmtF16);    // M (TMEM) . R of a half
constexpr uint32_t IDESC_O = idesc_f16(128, 64, false, true, kFmtF16);    // A T . R of both halves

// A bounded wait.  A try suspends the warp for up to 7800 clocks (4 us); after every 256 the abort flag is
// looked at, and after 2^11 times that (two seconds) the flag is set to 2.  In one piece of
// assembly, because a warp that waits should issue little (about half of them wait at any time), and
// because every wait of every role sits in the instruction cache.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint32_t abort) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n, m, f;\n\t"
      "mov.u32 m, 2048;\n"
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
constexpr uint32_t kCoreHi = 256 >> 4 | 1u << 14;  // the same for rows of 8 x 8 core matrices, two of them 16 columns
__device__ __forceinline__ constexpr uint32_t kstep(int j) { return ((j >> 2) * kHalf + (j & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint32_t tstep(int j) { return 16 * j; }

// The issuing warps run converged and elect a lane per instruction, and what the descriptors come from is
// broadcast with shuffles: the compiler then knows it to be uniform and keeps the descriptors in uniform
// registers.  Moved there from a divergent branch for every MMA, they cost 50 to 80 clocks each, more
// than the MMA (SS N = 64: 49 clocks, its operands' shared-memory reads; TS N = 64: 32, N = 32: 16).
template <uint32_t kIdesc, uint32_t kAHi = kOpHi, uint32_t kBHi = kOpHi>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "n"(kIdesc), "r"((uint32_t)acc), "n"(kAHi), "n"(kBHi)
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
// The operands that the halves share are read once for both: an SS product takes its operands' bytes / 128
// clocks (N = 64: 49, N = 128: 65), a TS product its multiply-adds.
__device__ __forceinline__ void issue_D1(uint32_t kq, uint32_t sbuf, uint32_t d) {
  const uint32_t a = op_lo(kq, 16), b = op_lo(sbuf, kHalf);
#pragma unroll
  for (int j = 0; j < 8; ++j) mma_ss<IDESC_D1>(d, a + kstep(j), b + j * 128, j > 0);
}
__device__ __forceinline__ void issue_M(uint32_t kq, uint32_t t, uint32_t d) {
  const uint32_t a = op_lo(kq, kHalf), b = op_lo(t, 128);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ss<IDESC_M, kOpHi, kCoreHi>(d, a + j * 256, b + j * 256, j > 0);  // 16 K rows of every 32
}
// d = M_lo R_hi + M_hi R_lo + M_hi R_hi  (64 tokens; the small ones first).  The lo columns of R begin 64 bytes into
// its rows.
__device__ __forceinline__ void issue_S(uint32_t m, uint32_t r, uint32_t d) {
  const uint32_t hi = op_lo(r, 8192), lo = hi + 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    mma_ts<IDESC_S>(d, m + tstep(j) + 8, hi + 128 * j, j > 0);
    mma_ts<IDESC_S>(d, m + tstep(j), lo + 128 * j, true);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ts<IDESC_S>(d, m + tstep(j), hi + 128 * j, true);
}
// A T . R.  The rows of A T are the second 16 of every 32 rows of the A operand; the first 16 are the other
// chunk's (or what lies before the first place), and their results are not used.
__device__ __forceinline__ void issue_O(uint32_t at, uint32_t r, uint32_t d) {
  const uint32_t a = op_lo(at - 512, 128), b = op_lo(r, 8192);
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_ss<IDESC_O, kCoreHi, kOpHi>(d, a + 256 * j, b + 128 * j, j > 0);
}

// 16 TMEM lanes (from taddr's on) x 32 columns: thread l has of rows l / 4 and l / 4 + 8 the columns 8 b + 2 (l % 4) and
// the next, at 4 b and 4 b + 2.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Powers of two that bring m to [2^(6 - kUp), 2^(7 - kUp)) and back.  Headroom: with alpha <= 1
// and beta |k|^2 <= 2 the transition does not expand a state row s, so over a chunk
// |s'| <= gamma |s| + 64 max |w V| max |K|, with |K| < 23 and, of 128 elements, |s| <= 12 max |S|; and
// |w X| <= max |w V| + 2 gamma |s|, since w_j 2^{cs_j} rho_j |K_j| = gamma beta_j |k_j|^2 / |K_j| <= 2 gamma.  With
// m = gamma max |S| / 4 + max |w V| and kUp = 2 the next state and R are below 1500 m.  The R of y is below 25 times
// the larger of max |u V| and 2^{cs_0} max |S|, what the first token leaves of the state (kUp = 0).  Scaled, all are
// under 65504.
// Where m is infinite or NaN both are NaN, and so is then every state row: scaled by what is left of such a
// bound, the rows without one in them would silently lose their bits.
template <int kUp>
__device__ __forceinline__ float2 state_scale(float m) {
  const int raw = (int)((__float_as_uint(m) >> 23) & 255u), e = min(max(raw, 8), 254);
  const uint32_t to = (uint32_t)(260 - kUp - e) << 23, from = (uint32_t)(e - 6 + kUp) << 23;
  return make_float2(__uint_as_float(raw == 255 ? 0x7fffffffu : to), __uint_as_float(raw == 255 ? 0x7fffffffu : from));
}
// (fmaxf would drop a NaN)
__device__ __forceinline__ float max_bound(float a, float b) { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); }

__global__ void __launch_bounds__(kThreads, 1)
    ssd_delta_chunk_kernel(const __grid_constant__ CUtensorMap tm_v, const DeltaPlan p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // Items: 64 state rows of a head of a sequence, the longest sequences' first.  CTA b takes items b, b + gridDim.x,
  // ..; every role runs through the chunks of all of them (k counts those, c the item's), so that the loads and M
  // of the next item's first chunks overlap the end of this one's.
  const uint32_t per_seq = p.H * (p.P >> 6), n_items = p.B * per_seq, step = gridDim.x;
  const auto seq_at = [&](uint32_t rank) { return p.order ? p.order[rank] : (int)rank; };
  const auto chunks_of = [&](uint32_t i) { return i < n_items ? (seq_len(p.cu, seq_at(i / per_seq), p.L) + C - 1) / C : 0; };
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
      mbar_init(BAR(i), i == BAR_SREADY ? 8 : i >= BAR_MREADY && i < BAR_D1 || i >= BAR_MAX ? 4 : 1);
    misc[1] = misc[2] = 0;
    fence_mbar_init();
  }
  for (uint32_t i = tid * 16; i < 2 * kT + 2 * kAT; i += kThreads * 16)  // T and A T: what is never loaded
    *reinterpret_cast<uint4 *>(smem + OFF_T + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
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
  if (warp < 8) {
    // ------------------------------------------------------------------ the chains
    const int hf = warp >> 2;                // half: state rows (columns of S and O) 32 hf ..
    const int row = 16 * q4 + (lane >> 2);   // this thread's tokens of D1 and O: row, row + 8
    const int col = 2 * (lane & 3);          // its columns of them: 8 b + col, 8 b + col + 1, b = 0 .. 3
    const int n = 32 * q4 + lane;            // state column of this thread
    // swizzled places: unit k of the thread's row of the S operand at s_at ^ 16 k, columns 8 b of its rows of V and
    // of y's R at r_at ^ 16 b, of R at w_at ^ 16 b (hi), w_at ^ 16 (4 + b) (lo)
    const uint32_t s_at = OFF_SB + hf * kHalf + swz(n, 0), r_at = swz(row, 4 * hf) + 2 * col;
    const uint32_t w_at = OFF_SB + hf * kHalf + swz(row, 0) + 2 * col;
    uint32_t *max_s = reinterpret_cast<uint32_t *>(smem + OFF_MAXS) + 12 * hf;
    const uint32_t t_d1 = tmem + TM_D1 + 64 * hf, t_s = tmem + TM_S + 32 * hf;
    float2 S[16];  // the state, times sc.x
    int len = 0;   // the item's tokens
    const auto publish_max = [&](int buf) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fmaxf(fabsf(S[i].x), fabsf(S[i].y)));
      const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      if (lead) {
        max_s[4 * buf + q4] = bits;
        mbar_arrive(BAR(BAR_MAX + hf));
      }
      __syncwarp();
    };
    const auto read_max = [&](int buf) {
      const uint4 a = *reinterpret_cast<const uint4 *>(max_s + 4 * buf);
      return __uint_as_float(max(max(a.x, a.y), max(a.z, a.w)));
    };
    float2 sc;
    uint32_t v[2][4];                  // the chunk's V, pairs
    float gr[2], u[2], w[2];           // of the chunk: 2^cs rho_k, u, w
    float4 bound = make_float4(0.f, 0.f, 0.f, 0.f);  // max |w V|, max |u V|, the first 2^cs, the last
    Ring<kDeep> ring;  // of the rows to load next
    const auto load_rows = [&](int c) {
      const unsigned char *stage = smem + OFF_VG + ring.at * kVG;
      const auto arr = [&](uint32_t off) { return reinterpret_cast<const float *>(stage + off); };
      const bool ok = wait(BAR_READY + ring.at, ring.parity);
      bound = reinterpret_cast<const float4 *>(smem + OFF_BOUND)[ring.at];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = row + 8 * i;
        const bool live = c * C + t < len;  // (the rows after may hold anything)
        gr[i] = arr(OFF_GAMMA)[t] * reinterpret_cast<const float *>(smem + ring.at * kTile + OFF_RHOK)[t];
        u[i] = arr(OFF_U)[t];
        w[i] = arr(OFF_W)[t];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t x = *reinterpret_cast<const uint32_t *>(stage + (r_at ^ 16 * b) + 1024 * i);
          v[i][b] = live ? x : 0u;
        }
      }
      ring.next();
      return ok;
    };
    bool ok = true;
    int k = 0, maxes = 0;  // chunks; largest |S| exchanged
    int seq = 0, hp_next = 0;  // of the next item
    for (uint32_t i = blockIdx.x; i < n_items + step && ok; i += step) {
      const int seq_now = seq, hp = hp_next;
      if (i < n_items) {  // on its way while the item before runs
        const uint32_t rank = i / per_seq;
        seq = seq_at(rank);
        hp_next = 64 * (i - rank * per_seq);
      }
      if (i < step) continue;
      len = seq_len(p.cu, seq_now, p.L);
      const int nck = (len + C - 1) / C;
      const long long soff = ((long long)seq_now * p.H * p.P + hp + 32 * hf) * kDState + n;
#pragma unroll
      for (int j = 0; j < 16; ++j) S[j] = make_float2(0.f, 0.f);
      if (p.h0) {
        const float *src = p.h0 + soff;
#pragma unroll
        for (int j = 0; j < 16; ++j) S[j] = make_float2(src[(2 * j) * kDState], src[(2 * j + 1) * kDState]);
      }
      if (nck == 0) {  // no tokens: the state goes on as it came, of any size
        if (p.h_final && in_bounds(soff + 31 * kDState, p.state_extent, p.err))
#pragma unroll
          for (int j = 0; j < 32; ++j) p.h_final[soff + j * kDState] = j & 1 ? S[j / 2].y : S[j / 2].x;
        continue;
      }
      float m = 0.f;
      if (p.h0) {
        publish_max(2);
        ok = wait(BAR_MAX + hf, maxes++ & 1);
        m = read_max(2);
      }
      sc = state_scale<0>(m);
#pragma unroll
      for (int j = 0; j < 16; ++j) S[j] = __fmul2_rn(S[j], make_float2(sc.x, sc.x));
      ok = load_rows(0) && ok;
      for (int c = 0;; ++c, ++k) {
        if (c < nck) {
          // S into its operand
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t hv[4], lv[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) split2(S[4 * j + x], hv[x], lv[x]);
            *reinterpret_cast<uint4 *>(smem + (s_at ^ 16 * j)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            *reinterpret_cast<uint4 *>(smem + (s_at ^ 16 * (4 + j))) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (lead) mbar_arrive(BAR(BAR_SREADY));
        } else if (p.h_final && in_bounds(soff + 31 * kDState, p.state_extent, p.err)) {
          float *dst = p.h_final + soff;
#pragma unroll
          for (int j = 0; j < 32; ++j) dst[j * kDState] = sc.y * (j & 1 ? S[j / 2].y : S[j / 2].x);
        }
        if (c == nck) break;
        // while K S^T runs: the largest |S|, and from it the scales of the next S (and R) and of y's R
        publish_max(k & 1);
        ok = wait(BAR_MAX + hf, maxes++ & 1) && ok;
        // (A decay below 2^-126 is zero in 2^{cs_C}, but not yet in w_j 2^{cs_j}: it counts as that in the bound.  And S
        // grows by at most 2^64 in its new scale, where zeros could otherwise meet an infinity.)
        const float top = read_max(k & 1), decay = bound.w * sc.y, least = fmaxf(bound.w, 0x1p-126f) * sc.y;
        const float2 nsc = state_scale<2>(max_bound(fmaf(0.25f * least, top, bound.x), 0x1p-60f * least));
        const float2 ysc = state_scale<0>(max_bound(bound.z * sc.y * top, bound.y));
        ok = wait(BAR_D1, k & 1) && ok;
        __syncwarp();
        tc_fence_after();
        // (for y; the place is free: the product was issued after the y of two chunks before)
        if (q4 == 0 && lead) reinterpret_cast<float2 *>(smem + OFF_SCALE)[2 * hf + (k & 1)] = make_float2(sc.y, ysc.y);
        {
          float d[16], e[16];
          tmem_ld_rows(t_d1 + lane_off, d);
          tmem_ld_rows(t_d1 + 32 + lane_off, e);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float g = -gr[i] * sc.y, wn = w[i] * nsc.x, un = u[i] * ysc.x;
            const float2 k2 = make_float2(g, g), w2 = make_float2(wn, wn), u2 = make_float2(un, un);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int x = 4 * b + 2 * i;
              const float2 vp = make_float2(__uint_as_float(v[i][b] << 16), __uint_as_float(v[i][b] & 0xffff0000u));
              const float2 ks = __fadd2_rn(make_float2(d[x], d[x + 1]), make_float2(e[x], e[x + 1]));
              const float2 xv = __ffma2_rn(k2, ks, vp);
              uint32_t hv, lv;
              split2(__fmul2_rn(w2, xv), hv, lv);
              *reinterpret_cast<uint32_t *>(smem + (w_at ^ 16 * b) + 1024 * i) = hv;
              *reinterpret_cast<uint32_t *>(smem + (w_at ^ 16 * (4 + b)) + 1024 * i) = lv;
              *reinterpret_cast<uint32_t *>(smem + OFF_R + (r_at ^ 16 * b) + 1024 * i) = h2(__float22half2_rn(__fmul2_rn(u2, xv)));
            }
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lead) mbar_arrive(BAR(BAR_RREADY + hf));
        // S = gamma_end S + M R, in the new scale; while the product runs: the next chunk's rows
        const float ge = decay * nsc.x;
        const float2 ge2 = make_float2(ge, ge);
        sc = nsc;
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = __fmul2_rn(S[i], ge2);
        if (c + 1 < nck) ok = load_rows(c + 1) && ok;
        ok = wait(BAR_S + hf, k & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float d[16];
          tmem_ld16(t_s + 16 * x + lane_off, d);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) S[8 * x + i] = __fadd2_rn(make_float2(d[2 * i], d[2 * i + 1]), S[8 * x + i]);
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ M into its operand, a chunk ahead; y
    const int row = 16 * q4 + (lane >> 2), col = 2 * (lane & 3);  // tokens and columns as the chains'
    uint32_t total = 0;  // chunks of all items
    for (uint32_t i = blockIdx.x + lane * step; i < n_items; i += 32 * step) total += chunks_of(i);
    total = __reduce_add_sync(0xffffffffu, total);
    Ring<kDeep> ry;
    bool ok = true;
    const auto convert = [&](uint32_t k) {
      ok = wait2(BAR_M, k) && ok;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {  // 16 tokens
        const uint32_t at = tmem + TM_M + 128 * (k & 1) + lane_off;
        float m[16], e[16];
        uint32_t hv[8], lv[8];
        tmem_ld16(at + 16 * b, m);
        tmem_ld16(at + 64 + 16 * b, e);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          split2(__fadd2_rn(make_float2(m[2 * j], m[2 * j + 1]), make_float2(e[2 * j], e[2 * j + 1])), hv[j], lv[j]);
        tmem_st8(at + 16 * b, hv);
        tmem_st8(at + 16 * b + 8, lv);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lead) mbar_arrive(BAR(BAR_MREADY + (k & 1)));
    };
    uint32_t k = 0;
    if (total > 0) convert(0);
    int seq = 0, hp_next = 0;  // of the next item
    for (uint32_t i = blockIdx.x; i < n_items + step && ok; i += step) {
      const int seq_now = seq, hp = hp_next;
      if (i < n_items) {  // on its way while the item before runs
        const uint32_t rank = i / per_seq;
        seq = seq_at(rank);
        hp_next = 64 * (i - rank * per_seq);
      }
      if (i < step) continue;
      const int len = seq_len(p.cu, seq_now, p.L), nck = (len + C - 1) / C;
      const long long base = seq_base(p.cu, seq_now, p.L);
      for (int c = 0; c < nck; ++c, ++k) {
        // Q S^T, out of the next chunk's way
        ok = wait(BAR_D1, k & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float2 hold[2][2][4];  // [half][token]
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float d[16], e[16];
          tmem_ld_rows(tmem + TM_D1 + 64 * hf + lane_off + (16u << 16), d);
          tmem_ld_rows(tmem + TM_D1 + 64 * hf + 32 + lane_off + (16u << 16), e);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int x = 4 * b + 2 * t;
              hold[hf][t][b] = __fadd2_rn(make_float2(d[x], d[x + 1]), make_float2(e[x], e[x + 1]));
            }
        }
        ok = wait(BAR_TILE + ry.at, ry.parity) && ok;  // (done: what they loaded is read here)
        ok = wait(BAR_VG + ry.at, ry.parity) && ok;
        float gamma[2], rho[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          gamma[t] = reinterpret_cast<const float *>(smem + OFF_VG + ry.at * kVG + OFF_GAMMA)[row + 8 * t];
          rho[t] = reinterpret_cast<const float *>(smem + ry.at * kTile + OFF_RHOQ)[row + 8 * t];
        }
        ry.next();
        tc_fence_before();
        __syncwarp();
        if (lead) mbar_arrive(BAR(BAR_QREAD));
        if (k + 1 < total) convert(k + 1);
        ok = wait(BAR_O, k & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float2 sc = reinterpret_cast<const float2 *>(smem + OFF_SCALE)[2 * hf + (k & 1)];
          float o[16];
          tmem_ld_rows(tmem + TM_O + 32 * hf + lane_off + (16u << 16), o);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int token = c * C + row + 8 * t;
            // (rho first: without it the sums of the largest values would overflow)
            const float g = gamma[t] * (sc.x * rho[t]), yb = sc.y * rho[t];
            const float2 b2 = make_float2(yb, yb), g2 = make_float2(g, g);
            uint32_t u[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float2 w = __ffma2_rn(b2, make_float2(o[4 * b + 2 * t], o[4 * b + 2 * t + 1]), __fmul2_rn(g2, hold[hf][t][b]));
              const __nv_bfloat162 x = __float22bfloat162_rn(w);
              u[b] = *reinterpret_cast<const uint32_t *>(&x);
            }
            // a row's four lanes exchange, so that lane l % 4 has the columns 8 (l % 4) ..: 16 bytes to store
            const bool odd = lane & 1, up = lane & 2;
            uint32_t e0 = __shfl_xor_sync(0xffffffffu, odd ? u[0] : u[1], 1), e1 = __shfl_xor_sync(0xffffffffu, odd ? u[2] : u[3], 1);
            const uint32_t a0 = odd ? e0 : u[0], a1 = odd ? u[1] : e0, c0 = odd ? e1 : u[2], c1 = odd ? u[3] : e1;
            e0 = __shfl_xor_sync(0xffffffffu, up ? a0 : c0, 2);
            e1 = __shfl_xor_sync(0xffffffffu, up ? a1 : c1, 2);
            const long long yo = (base + token) * p.ys + hp + 32 * hf + 4 * col;
            if (token < len && in_bounds(yo + 7, p.y_extent, p.err))
              *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + yo) =
                  up ? make_uint4(e0, e1, c0, c1) : make_uint4(a0, a1, e0, e1);
          }
        }
        tc_fence_before();
      }
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------------ MMAs of the chains
    Ring<kDeep> r;
    bool ok = true;
    int k = 0;
    for (uint32_t i = blockIdx.x, nck = 0, next; i < n_items + step && ok; i += step, nck = next) {
      next = chunks_of(i);  // on its way while the item before runs
      for (uint32_t c = 0; c < nck && ok; ++c, ++k, r.next()) {
        ok = wait(BAR_READY + r.at, r.parity);
        ok = wait(BAR_SREADY, k & 1) && ok;
        tc_fence_after();
        issue_D1(sb + r.at * kTile, sb + OFF_SB, tmem + TM_D1);
        commit(BAR(BAR_D1));
        ok = wait2(BAR_MREADY, k) && ok;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          ok = wait(BAR_RREADY + half, k & 1) && ok;
          tc_fence_after();
          issue_S(tmem + TM_M + 128 * (k & 1), sb + OFF_SB + half * kHalf, tmem + TM_S + 32 * half);
          commit(BAR(BAR_S + half));
        }
        ok = wait2(BAR_AT, k) && ok;
        ok = wait(BAR_QREAD, k & 1) && ok;
        tc_fence_after();
        issue_O(sb + OFF_AT + (k & 1) * 512, sb + OFF_R, tmem + TM_O);
        commit(BAR(BAR_O));
        commit(BAR(BAR_EMPTY + r.at));
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    commit(BAR(BAR_DONE));  // no MMA may still be running when TMEM is released
    settle(BAR_DONE, 0);
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMAs of M
    Ring<kDeep> r, e;
    bool ok = true;
    int k = 0;
    for (uint32_t i = blockIdx.x, nck = 0, next; i < n_items + step && ok; i += step, nck = next) {
      next = chunks_of(i);
      for (uint32_t c = 0; c < nck && ok; ++c, ++k, r.next()) {
        ok = wait(BAR_TILE + r.at, r.parity);
        ok = wait2(BAR_T, k) && ok;
        if (k >= 2) {  // the M of two chunks before is read
          ok = wait(BAR_EMPTY + e.at, e.parity) && ok;
          e.next();
        }
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        issue_M(sb + r.at * kTile, sb + OFF_T + (k & 1) * kT, tmem + TM_M + 128 * (k & 1));
        commit(BAR(BAR_M + (k & 1)));
      }
    }
    commit(BAR(BAR_DONE + 1));
    settle(BAR_DONE + 1, 0);
  } else if (warp == 14) {
    // ------------------------------------------------------------------ loads of tiles, V, gates, A T
    if (lead) {
      prefetch_tmap(&tm_v);
      int n = 0, n_at = 0;
      const long long rec_step = p.H * kDeltaRecordBytes, tile_step = p.G * kDeltaTileBytes;
      Ring<kDeep> r, e;  // to load; to become free
      const unsigned char *before = nullptr;  // A T of the chunk before
      const auto load_at = [&](const unsigned char *src) {
        const uint32_t at = BAR(BAR_AT + (n_at & 1));
        mbar_arrive_expect_tx(at, kDeltaATBytes);
#pragma unroll 1
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll 1
          for (int g = kb; g < 4; ++g, src += 512)  // the two places alternate by 16 rows
            bulk_load(sb + OFF_AT + kb * 4096 + g * 1024 + (n_at & 1) * 512, src, 512, at);
        ++n_at;
      };
      // Chunk k's turn: its tile, V and gates, into the place of chunk k - 3; A T of chunk k - 1 (and in turn 0 of
      // chunk 0), whose two places are free then too.  A last turn loads A T alone.
      bool ok = true;
      for (uint32_t i = blockIdx.x; i < n_items && ok; i += step) {
        const uint32_t rank = i / per_seq, hp = i - rank * per_seq;  // 64 rows of a head: h P / 64 + ..
        const int seq = seq_at(rank), h = hp >> (p.P > 64), nck = (seq_len(p.cu, seq, p.L) + C - 1) / C;
        const long long base = seq_base(p.cu, seq, p.L);
        const long long ck0 = p.chunk0 ? p.chunk0[seq] : (long long)seq * nck;
        const unsigned char *rec = p.records + (ck0 * p.H + h) * kDeltaRecordBytes + kDeltaTBytes;
        const unsigned char *tile = p.tiles + (ck0 * p.G + h / p.hpg) * kDeltaTileBytes;
        for (int c = 0; c < nck; ++c, rec += rec_step, tile += tile_step) {
          if (n >= kDeep) {
            ok = wait(BAR_EMPTY + e.at, e.parity);
            if (!ok) break;
            e.next();
          }
          const uint32_t vg = BAR(BAR_VG + r.at), tb = BAR(BAR_TILE + r.at), dst = sb + OFF_VG + r.at * kVG;
          mbar_arrive_expect_tx(vg, 8192 + 768);
          // 64 token rows, the ones after the sequence's end among them (they are not used)
          tma_load_2d(dst, &tm_v, (int)(64 * hp), (int)(base + c * C), vg);
          // V is the caller's; tiles and records are the front end's, which may still be running
          // (programmatic dependent launch)
          if (n == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
          mbar_arrive_expect_tx(tb, (uint32_t)kDeltaTileBytes);
          bulk_load(sb + r.at * kTile, tile, (uint32_t)kDeltaTileBytes, tb);
          bulk_load(dst + OFF_U, rec + kDeltaATBytes, 768, vg);
          r.next();
          if (n != 1) load_at(n == 0 ? rec : before);
          before = rec;
          ++n;
        }
      }
      if (ok && n >= 2 && (n < kDeep || wait(BAR_EMPTY + e.at, e.parity))) load_at(before);
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
  } else {
    // ------------------------------------------------------------------ loads of T; the bounds of what each chunk
    // adds to the state and to y
    uint32_t i = blockIdx.x - step;  // the item of the T to load, its chunks, the chunk
    int len = 0, nck = 0, c = 0;
    const unsigned char *rec = nullptr;
    int rows = 0, rows_next = 0;     // tokens of chunk k, of chunk k + 1
    Ring<kDeep> r;
    int n = 0;
    // Turn k: the bound of chunk k, then T of chunk k + 2 over that of chunk k, once M has taken it
    for (int k = -2; k < 0 || rows > 0; ++k) {
      while (c == nck && i + step < n_items) {  // the next item that has chunks
        i += step;
        const uint32_t rank = i / per_seq;
        const int seq = seq_at(rank), h = (i - rank * per_seq) >> (p.P > 64);
        len = seq_len(p.cu, seq, p.L);
        nck = (len + C - 1) / C;
        c = 0;
        rec = p.records + ((p.chunk0 ? p.chunk0[seq] : (long long)seq * nck) * p.H + h) * kDeltaRecordBytes;
      }
      if (k >= 0) {
        bool ok = wait(BAR_VG + r.at, r.parity);
        ok = wait(BAR_TILE + r.at, r.parity) && ok;
        const unsigned char *stage = smem + OFF_VG + r.at * kVG;
        const float *u = reinterpret_cast<const float *>(stage + OFF_U), *w = reinterpret_cast<const float *>(stage + OFF_W);
        uint32_t top_w = 0, top_u = 0;
#pragma unroll 4
        for (int t = lane >> 3; t < rows; t += 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(stage + t * 128 + (lane & 7) * 16);
          const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          // at least 2^-100, so that u and w times a scale are finite (as integers, where a NaN ranks highest)
          const float v = __uint_as_float(max(max(m << 16, m & 0x7fff0000u), 0x0d800000u));
          top_w = max(top_w, __float_as_uint(fabsf(w[t] * v)));
          top_u = max(top_u, __float_as_uint(fabsf(u[t] * v)));
        }
        top_w = __reduce_max_sync(0xffffffffu, top_w);
        top_u = __reduce_max_sync(0xffffffffu, top_u);
        if (lead) {
          const float *gamma = reinterpret_cast<const float *>(stage + OFF_GAMMA);
          reinterpret_cast<float4 *>(smem + OFF_BOUND)[r.at] =
              make_float4(__uint_as_float(top_w), __uint_as_float(top_u), gamma[0], gamma[C - 1]);
          mbar_arrive(BAR(BAR_READY + r.at));
        }
        __syncwarp();
        r.next();
        if (c < nck) ok = wait2(BAR_M, k) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      rows = rows_next;
      rows_next = 0;
      if (c < nck) {
        if (k == -2 && lead) asm volatile("griddepcontrol.wait;" ::: "memory");
        if (lead) {
          const uint32_t t = BAR(BAR_T + (k & 1));
          mbar_arrive_expect_tx(t, kDeltaTBytes);
          const unsigned char *src = rec;
          uint32_t dst = sb + OFF_T + (k & 1) * kT, bytes = 512;
#pragma unroll 1
          for (int kb = 0; kb < 4; ++kb, dst += 4096, bytes += 512) {
            bulk_load(dst, src, bytes, t);
            bulk_load(dst + 2048, src + bytes, bytes, t);
            src += 2 * bytes;
          }
        }
        rows_next = min(C, len - c * C);
        rec += p.H * kDeltaRecordBytes;
        ++c;
        ++n;
      }
      __syncwarp();
    }
    if (lead)
      for (int k = max(0, n - 2); k < n; ++k) settle(BAR_T + (k & 1), (k >> 1) & 1);
    __syncwarp();
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
  // (also while the stream is captured: it may be the process's first call)
  cudaError_t e = cudaFuncSetAttribute(ssd_delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  // a programmatic dependent of the front end: its set-up and first loads of V overlap the front
  // end's tail
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)std::min<long long>((long long)p.B * p.H * (p.P / 64), 148));
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
