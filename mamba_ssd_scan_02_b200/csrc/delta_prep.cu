// delta_prep.cu -- the front end of the chunked delta rule: everything of a 64-token chunk that does
// not depend on the state, for all chunks at once.
//
// One CTA per (chunk, group, set of heads).  Shared by the group's heads: K and Q as fp16 operand tiles (a
// row scaled by the power of two that brings its largest element to [1, 2), exact in fp16 down to
// 2^-17 of it; rho is that power and the norm's factor), K K^T (fp32) and A~ = tril(Q K^T) (fp16).  Then
// each warp takes heads of its own:
//   gates  cs = prefix sums of log2(alpha), in fixed point (32 fractional bits), so that their differences are
//          exact however large the sums
//   T~     = (I + L~)^-1, L~_ij = beta_i rho_i^2 K_i.K_j (j < i), in fp32: 16 x 16 diagonal blocks by
//          substitution, joined by block products with tf32 in two parts (22 bits)
//   A T    2^{cs_t - cs_j} (A~ T~)_tj, at most 529 in size, rounded once to fp16
// and leaves the triangles of T~ in two fp16 parts and of A T as the operand images that the chunk kernel loads.
//
// Why apart from the chunk kernel: inside it this part ran in the same SM as the tcgen05 products, which
// slow mma.sync down threefold and shared-memory loads twofold, and its latency (about 5 us a chunk)
// bounded every CTA: 650 us for 8192 tokens x 128 heads, where the two kernels now take 121 and 228.  Here it
// is spread over all chunks, twelve independent warps per SM (three CTAs; two of them with rows of one
// pitch: 154 us).  The price is 16 KB of workspace per chunk and head, written once and read once.
//
// What bounds it (8192 tokens x 128 heads, 16384 heads' chunks: 121 us): the shared-memory and store pipe, two
// thirds busy; 40 % of the issue slots are used, 31 % of the DRAM rate.  Its 264 MB of records alone would
// take 40 us.  As many heads per CTA as share K K^T (16; 8: 166 us where 16 took 154): the K and Q part costs
// as much as one head.
#include "common.cuh"
#include "delta_mma.cuh"
#include "delta_plan.h"
#include "plan.h"

namespace ssd {
namespace {

using namespace delta;

constexpr int C = kDeltaChunk;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHeads = 16;                      // heads of a CTA, at most
constexpr uint32_t kHalf = 16384;
constexpr int kKPitch = 136;                       // halves of a K or Q row
constexpr int kWarpF = 64 + 64 + 96;               // floats per warp: -beta rho^2, rel, column factors
// Upper triangular 64 x 64s of floats, by blocks of 16 rows, each from its diagonal block on: 12 KB instead of
// 18 (three CTAs per SM instead of two).  Row j's column i (i >= 16 (j / 16)) is at row_at(j) + i of T~^T, at
// g_at(j) + i of K K^T.  The pitches of K K^T are 8 or 24 mod 32 (conflict-free reads of 4 rows x 8), those of
// T~^T 12 or 20 (of 8 rows x 4, of 4 rows in steps of 2 x 8, and of 8 rows x 16 bytes).
__host__ __device__ constexpr int pitch(int j) { return j < 32 ? (j < 16 ? 76 : 52) : (j < 48 ? 44 : 20); }
__host__ __device__ constexpr int row_start(int j) {
  return (j < 32 ? (j < 16 ? 0 : 1216) : (j < 48 ? 2048 : 2752)) + (j & 15) * pitch(j);
}
__host__ __device__ constexpr int row_at(int j) { return row_start(j) - 16 * (j >> 4); }
__host__ __device__ constexpr int g_pitch(int j) { return 72 - 16 * (j >> 4); }
__host__ __device__ constexpr int g_start(int j) {
  return 1152 * (j >> 4) - 128 * (j >> 4) * ((j >> 4) - 1) + (j & 15) * g_pitch(j);
}
__host__ __device__ constexpr int g_at(int j) { return g_start(j) - 16 * (j >> 4); }
constexpr int kTri = row_start(63) + 20;
static_assert(g_start(63) + 24 == kTri, "the two layouts have one size");
// A lower triangular one of halves (A~): rows of block b hold columns 0 .. 16 b + 15
__host__ __device__ constexpr int a_pitch(int t) { return 24 + 16 * (t >> 4); }
__host__ __device__ constexpr int a_row(int t) {
  return 384 * (t >> 4) + 128 * (t >> 4) * ((t >> 4) - 1) + (t & 15) * a_pitch(t);
}
constexpr uint32_t OFF_W = 0;                      // per warp: T~^T
constexpr uint32_t OFF_K = OFF_W;                  // before the heads: [128][136] halves: K rows, Q rows
constexpr uint32_t OFF_G = OFF_W + kWarps * kTri * 4;   // K K^T, columns >= row
constexpr uint32_t OFF_A = OFF_G + kTri * 4;            // A~
constexpr uint32_t OFF_RHO = OFF_A + (a_row(63) + 72) * 2;  // rho_k[64]
constexpr uint32_t OFF_F = OFF_RHO + 256;               // per warp: kWarpF floats
constexpr uint32_t OFF_DT = OFF_F + kWarps * kWarpF * 4;   // [16][66] (dt, b) of the CTA's heads
constexpr uint32_t OFF_AB = OFF_DT + kMaxHeads * 66 * 4;   // [16] (A, dt_bias)
constexpr uint32_t kSmem = OFF_AB + kMaxHeads * 8;
static_assert(128 * kKPitch * 2 <= kWarps * kTri * 4, "K and Q lie where the heads' blocks will");
static_assert(3 * (kSmem + 1024) <= 233472, "three CTAs per SM");

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
// rows r .. r + 15 and columns c .. c + 7 of w
__device__ __forceinline__ FragA load_a(const float *w, int r, int c, int lane) {
  const float *x = w + row_at(r) + c + (lane >> 2) * pitch(r) + (lane & 3);
  FragA f;
  split_tf32(x[0], f.h[0], f.l[0]);
  split_tf32(x[8 * pitch(r)], f.h[1], f.l[1]);
  split_tf32(x[4], f.h[2], f.l[2]);
  split_tf32(x[8 * pitch(r) + 4], f.h[3], f.l[3]);
  return f;
}
// rows r .. r + 7 and columns c .. c + 7 of w, for an A from an accumulator: a lane's two rows are 2t, 2t + 1
__device__ __forceinline__ FragB load_b(const float *w, int r, int c, int lane) {
  const float *x = w + row_at(r) + c + 2 * (lane & 3) * pitch(r) + (lane >> 2);
  FragB f;
  split_tf32(x[0], f.h[0], f.l[0]);
  split_tf32(x[pitch(r)], f.h[1], f.l[1]);
  return f;
}
// rows r .. r + 7 and columns c .. c + 7 of -L~^T, which is K K^T times f = -beta rho^2 of the column
__device__ __forceinline__ FragB load_z(const float *gm, int r, int c, float f, int lane) {
  const float *x = gm + g_at(r) + c + (lane & 3) * g_pitch(r) + (lane >> 2);
  FragB b;
  split_tf32(f * x[0], b.h[0], b.l[0]);
  split_tf32(f * x[4 * g_pitch(r)], b.h[1], b.l[1]);
  return b;
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

// W12 = W11 Z W22 (Z of -L~^T), the block that joins two inverted diagonal blocks of 8 K rows at P0 and P0 + 8 K (transposed,
// so upper triangular): its rows 16 MT .. into d.  Straight-line: with a branch per tile the products of one
// would wait for those of the one before.
template <int P0, int K, int MT>
__device__ __forceinline__ void join(const float *w, const float *gm, const float *s_f, float (&d)[K][4], int lane) {
  constexpr int P1 = P0 + 8 * K;
  FragA a[K];
#pragma unroll
  for (int kk = 2 * MT; kk < K; ++kk) a[kk] = load_a(w, P0 + 16 * MT, P0 + 8 * kk, lane);
#pragma unroll
  for (int nt = 0; nt < K; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[nt][e] = 0.f;
#pragma unroll
  for (int kt = 0; kt < K; ++kt) {
    float hh[4] = {}, hl[4] = {}, lh[4] = {};
    const float f = s_f[P1 + 8 * kt + (lane >> 2)];
#pragma unroll
    for (int kk = 2 * MT; kk < K; ++kk) {
      const FragB b = load_z(gm, P0 + 8 * kk, P1 + 8 * kt, f, lane);
      mma_tf32(hh, a[kk].h, b.h);
      mma_tf32(hl, a[kk].h, b.l);
      mma_tf32(lh, a[kk].l, b.h);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) hh[e] += hl[e] + lh[e];
    const FragA x = acc_as_a(hh);
#pragma unroll
    for (int nt = kt; nt < K; ++nt) {
      const FragB b = load_b(w, P1 + 8 * kt, P1 + 8 * nt, lane);
      mma_tf32(d[nt], x.l, b.h);
      mma_tf32(d[nt], x.h, b.l);
      mma_tf32(d[nt], x.h, b.h);
    }
  }
}
template <int P0, int K, int MT>
__device__ __forceinline__ void put_block(float *w, const float (&d)[K][4], int lane) {
  constexpr int r = P0 + 16 * MT;
#pragma unroll
  for (int nt = 0; nt < K; ++nt) {
    float *x = w + row_at(r) + P0 + 8 * K + 8 * nt + (lane >> 2) * pitch(r) + 2 * (lane & 3);
    *reinterpret_cast<float2 *>(x) = make_float2(d[nt][0], d[nt][1]);
    *reinterpret_cast<float2 *>(x + 8 * pitch(r)) = make_float2(d[nt][2], d[nt][3]);
  }
}

// The 16 x 16 diagonal blocks at p0 and p0 + 16, by one warp: t = column `lane & 15` of T~'s block lane / 16,
//   t_i = [i == j] + f_i sum_{m < i} K_m.K_i t_m,   f = -beta rho^2,
// the column of m added to every later sum as soon as t_m is known (so the chain is two multiply-adds per
// row).  A row of K K^T is read while the one before is used.
__device__ __forceinline__ void invert16(const float *gm, const float *s_f, int p0, int lane, float2 (&t)[8]) {
  const int b0 = p0 + (lane & 16), j = lane & 15, step = g_pitch(b0);
  const float *zr = gm + g_start(b0);
  float4 z[4], f[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    z[q] = *reinterpret_cast<const float4 *>(zr + 4 * q);
    f[q] = *reinterpret_cast<const float4 *>(s_f + b0 + 4 * q);
    t[2 * q] = t[2 * q + 1] = make_float2(0.f, 0.f);
  }
#pragma unroll
  for (int m = 0; m < 16; ++m) {
    const float fm = m & 2 ? (m & 1 ? f[m / 4].w : f[m / 4].z) : (m & 1 ? f[m / 4].y : f[m / 4].x);
    float &own = m & 1 ? t[m / 2].y : t[m / 2].x;
    own = fmaf(fm, own, m == j ? 1.f : 0.f);
    const float2 t2 = make_float2(own, own);
    if (!(m & 1)) t[m / 2].y = fmaf(m & 2 ? z[m / 4].w : z[m / 4].y, own, t[m / 2].y);
#pragma unroll
    for (int q = (m + 1) / 4; q < 4; ++q) {
      if (4 * q > m) t[2 * q] = __ffma2_rn(make_float2(z[q].x, z[q].y), t2, t[2 * q]);
      if (4 * q + 2 > m) t[2 * q + 1] = __ffma2_rn(make_float2(z[q].z, z[q].w), t2, t[2 * q + 1]);
      if (m < 14) z[q] = *reinterpret_cast<const float4 *>(zr + (m + 1) * step + 4 * q);
    }
  }
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// four 8 x 8 matrices from fragments like those of an accumulator; lane i gives the address of row i % 8 of number i / 8
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Exponents of decays are sums of up to 64 steps, whose differences should keep an absolute precision (a
// relative one of the decay) however large the sums: fixed point with 32 fractional bits.  A step beyond
// +-2^12 is taken as that: 2^-4096 is zero.
__device__ __forceinline__ long long decay_step(float A, float d) {  // A d log2(e)
  constexpr float kHi = 1.44269504f, kLo = 1.92596299e-8f;           // log2(e) in two parts
  const float x = A * d, xl = fmaf(A, d, -x);
  const float s = x * kHi;
  if (!(fabsf(s) < 4096.f)) return s > 0.f ? 4096ll << 32 : -(4096ll << 32);
  const float w = rintf(s);
  const float f = (s - w) + (fmaf(x, kHi, -s) + fmaf(x, kLo, xl * kHi));
  return ((long long)(int)w << 32) + __float2int_rn(f * 4294967296.f);
}
__device__ __forceinline__ float exp2_fixed(long long x) {
  const int w = min(max((int)(x >> 32), -127), 127);
  return ex2((float)(uint32_t)x * 0x1p-32f) * __uint_as_float((uint32_t)(w + 127) << 23);
}
__device__ __forceinline__ float to_float(long long x) { return fmaf((float)(uint32_t)x, 0x1p-32f, (float)(int)(x >> 32)); }

__global__ void __launch_bounds__(kThreads, 3) ssd_delta_front_kernel(const DeltaPlan p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const long long ck = blockIdx.x;
  const int g = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int seq;
  long long first;
  if (p.chunk0) {  // the last sequence that starts at or before this chunk
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
  float *s_rho = reinterpret_cast<float *>(smem + OFF_RHO);

  const int h0 = g * p.hpg + blockIdx.z * p.heads_per_cta;  // the first of the CTA's heads
  const int n_heads = min(p.heads_per_cta, p.hpg - (int)blockIdx.z * p.heads_per_cta);
  uint32_t *s_dt = reinterpret_cast<uint32_t *>(smem + OFF_DT);
  float2 *s_ab = reinterpret_cast<float2 *>(smem + OFF_AB);

  // Rows after the chunk's last are loaded as that one and then taken as zero: a load under a condition
  // becomes a branch, and the loads would wait for each other.
  // ---- loads, all in flight: dt and b of the heads; K and Q: a warp takes 16 rows of each, a half warp a row,
  // a lane 8 elements
  uint4 kq[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const long long stride = m == 0 ? p.ks : p.qs;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(m == 0 ? p.k : p.q) + base * stride + g * kDState + 8 * (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      kq[m][i] = *reinterpret_cast<const uint4 *>(src + min(16 * warp + 2 * i + (lane >> 4), rows - 1) * stride);
  }
  {
    const int hl = tid & (kMaxHeads - 1), h = h0 + min(hl, n_heads - 1);
    const unsigned short *dt = static_cast<const unsigned short *>(p.dt) + base * p.ds + h;
    const unsigned short *b = static_cast<const unsigned short *>(p.b) + base * p.bs + h;
    uint32_t x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = min((tid >> 4) + 8 * i, rows - 1);
      x[i] = dt[t * p.ds];
      y[i] = b[t * p.bs];
    }
    if (tid < kMaxHeads) s_ab[hl] = make_float2(p.A[h], p.dt_bias[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) s_dt[hl * 66 + (tid >> 4) + 8 * i] = x[i] | y[i] << 16;
  }
  // ---- K and Q
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int r0 = 64 * kind + 16 * warp;
    uint4(&x)[8] = kq[kind];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((r0 & 63) + 2 * i + (lane >> 4) >= rows) x[i] = make_uint4(0, 0, 0, 0);
    uint32_t m[4];  // the largest magnitudes of two rows each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      constexpr uint32_t kAbs = 0x7fff7fffu;
      const uint32_t u = __vmaxu2(__vmaxu2(x[i].x & kAbs, x[i].y & kAbs), __vmaxu2(x[i].z & kAbs, x[i].w & kAbs));
      const uint32_t top = max(u & 0xffffu, u >> 16);
      m[i / 2] = i & 1 ? m[i / 2] | top << 16 : top;
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = __vmaxu2(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
    float sq[8], e2[8];  // a row's sum of squares (of this lane's elements); the power of two below its largest
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = min(max((i & 1 ? m[i / 2] >> 16 : m[i / 2] & 0xffffu) >> 7, 1u), 253u);
      const float f = __uint_as_float((254u - e) << 23);
      e2[i] = __uint_as_float(e << 23);
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t v[4];
      sq[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __uint_as_float(u[k] << 16), b = __uint_as_float(u[k] & 0xffff0000u);
        sq[i] = fmaf(a, a, fmaf(b, b, sq[i]));
        v[k] = h2(__floats2half2_rn(a * f, b * f));
      }
      const int r = r0 + 2 * i + (lane >> 4), c = lane & 15;
      const uint4 o = make_uint4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<uint4 *>(smem + OFF_K + r * kKPitch * 2 + 16 * c) = o;
      const int at = 32 * ((r & 63) >> 4) + 16 * kind + (r & 15);  // 16 K rows, the Q rows of the same tokens, ..
      if (blockIdx.z == 0) *reinterpret_cast<uint4 *>(tile + (c >> 3) * kHalf + swz(at, c & 7)) = o;
    }
    // sums over 16 lanes; lane c of a half warp ends with row c / 2's
#pragma unroll
    for (int o = 8, n = 4; o > 1; o >>= 1, n >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? sq[i] : sq[i + n];
        sq[i] = (up ? sq[i + n] : sq[i]) + __shfl_xor_sync(0xffffffffu, give, o);
        e2[i] = up ? e2[i + n] : e2[i];
      }
    }
    sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], 1);
    float rho = e2[0];
    if (p.qk_norm) rho *= 1.f / sqrtf(sq[0] + p.qk_eps);
    if (kind == 1) rho *= p.q_scale;
    if ((lane & 1) == 0) {
      const int r = r0 + (lane & 14) + (lane >> 4);
      if (blockIdx.z == 0) reinterpret_cast<float *>(tile + 2 * kHalf)[r] = rho;
      if (kind == 0) s_rho[r] = rho;
    }
  }
  __syncthreads();
  // ---- K K^T (its columns from the diagonal on) and A~ (up to it), 16 rows per turn of a warp
#pragma unroll 1
  for (int rb = warp; rb < 8; rb += kWarps) {
    const int rt = rb & 3, lo = rb < 4 ? 2 * rt : 0, hi = rb < 4 ? 8 : 2 * rt + 2;
    const uint32_t kq = tc::smem_u32(smem + OFF_K);
    const uint32_t arow = kq + (16 * rb + (lane & 15)) * kKPitch * 2 + (lane >> 4) * 16;
    const uint32_t brow = kq + (lane & 7) * kKPitch * 2 + (lane >> 3) * 16;
    uint32_t a[8][4];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) ldmatrix4(a[ks], arow + 32 * ks);
#pragma unroll 2
    for (int nt = lo; nt < hi; ++nt) {
      float c0[4] = {}, c1[4] = {};
#pragma unroll
      for (int ks = 0; ks < 8; ks += 2) {
        uint32_t b[4];
        ldmatrix4(b, brow + 8 * nt * kKPitch * 2 + 32 * ks);
        const uint32_t b0[2] = {b[0], b[1]}, b1[2] = {b[2], b[3]};
        mma_f16(c0, a[ks], b0);
        mma_f16(c1, a[ks + 1], b1);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c0[e] += c1[e];
      const int r = 16 * rt + (lane >> 2), j = 8 * nt + 2 * (lane & 3);
      if (rb < 4) {
        float *o = reinterpret_cast<float *>(smem + OFF_G) + g_at(r) + j;
        *reinterpret_cast<float2 *>(o) = make_float2(c0[0], c0[1]);
        *reinterpret_cast<float2 *>(o + 8 * g_pitch(r)) = make_float2(c0[2], c0[3]);
      } else {
        __half *o = reinterpret_cast<__half *>(smem + OFF_A) + a_row(r) + j;
        *reinterpret_cast<__half2 *>(o) = __floats2half2_rn(j <= r ? c0[0] : 0.f, j + 1 <= r ? c0[1] : 0.f);
        *reinterpret_cast<__half2 *>(o + 8 * a_pitch(r)) = __floats2half2_rn(j <= r + 8 ? c0[2] : 0.f, j + 1 <= r + 8 ? c0[3] : 0.f);
      }
    }
  }
  __syncthreads();

  // ---- heads
  float *w = reinterpret_cast<float *>(smem + OFF_W) + warp * kTri;
  float *s_f = reinterpret_cast<float *>(smem + OFF_F) + warp * kWarpF, *s_rel = s_f + 64, *s_col = s_f + 128;
  const float *gm = reinterpret_cast<const float *>(smem + OFF_G);
  for (int hh = warp; hh < n_heads; hh += kWarps) {
    unsigned char *rec = p.records + (ck * p.H + h0 + hh) * kDeltaRecordBytes;
    {  // gates of tokens 2 lane, 2 lane + 1
      const float2 ab = s_ab[hh];
      const uint2 raw = *reinterpret_cast<const uint2 *>(s_dt + 66 * hh + 2 * lane);
      const float2 rho = *reinterpret_cast<const float2 *>(s_rho + 2 * lane);
      long long s[2];
      float beta[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t x = u ? raw.y : raw.x;
        float d = __uint_as_float(x << 16) + ab.y;
        const float b = __uint_as_float(x & 0xffff0000u);
        if (p.softplus) d = d > 20.f ? d : log1pf(expf(d));
        d = d < p.dt_min ? p.dt_min : d > p.dt_max ? p.dt_max : d;
        const bool on = 2 * lane + u < rows;
        s[u] = on ? decay_step(ab.x, d) : 0;
        beta[u] = on ? p.beta_scale * (p.beta_sigmoid ? 1.f / (1.f + expf(-b)) : b) : 0.f;
        if (on && isnan(ab.x * d)) beta[u] = __int_as_float(0x7fffffff);  // not lost in the fixed point
      }
      s[1] += s[0];
      long long sum = s[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const long long cs0 = sum - s[1] + s[0], cs1 = sum;
      const long long end = __shfl_sync(0xffffffffu, sum, 31);
      float2 *o = reinterpret_cast<float2 *>(rec + kDeltaTBytes + kDeltaATBytes) + lane;
      const float2 u = make_float2(beta[0] * rho.x, beta[1] * rho.y);
      o[0] = u;
      o[32] = make_float2(exp2_fixed(cs0), exp2_fixed(cs1));
      o[64] = make_float2(u.x * exp2_fixed(end - cs0), u.y * exp2_fixed(end - cs1));
      *reinterpret_cast<float2 *>(s_f + 2 * lane) = make_float2(-beta[0] * rho.x * rho.x, -beta[1] * rho.y * rho.y);
      // for A T: cs relative to the first token of its 16; 2^(that - cs) for the tokens before
      long long ref[4];
#pragma unroll
      for (int tb = 1; tb < 4; ++tb) {
        ref[tb] = __shfl_sync(0xffffffffu, cs0, 8 * tb);
        if (lane < 8 * tb)
          *reinterpret_cast<float2 *>(s_col + 8 * tb * (tb - 1) + 2 * lane) =
              make_float2(exp2_fixed(ref[tb] - cs0), exp2_fixed(ref[tb] - cs1));
      }
      ref[0] = __shfl_sync(0xffffffffu, cs0, 0);
      const long long mine = lane < 16 ? (lane < 8 ? ref[0] : ref[1]) : (lane < 24 ? ref[2] : ref[3]);
      *reinterpret_cast<float2 *>(s_rel + 2 * lane) = make_float2(to_float(cs0 - mine), to_float(cs1 - mine));
    }
    __syncwarp();
#pragma unroll 1
    for (int p0 = 0; p0 < 64; p0 += 32) {
      float2 t[8];
      invert16(gm, s_f, p0, lane, t);
      float *o = w + row_start(p0 + lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(o + 4 * i) = make_float4(t[2 * i].x, t[2 * i].y, t[2 * i + 1].x, t[2 * i + 1].y);
    }
    __syncwarp();
    {
      float d0[2][4], d1[2][4];
      join<0, 2, 0>(w, gm, s_f, d0, lane);
      join<32, 2, 0>(w, gm, s_f, d1, lane);
      __syncwarp();
      put_block<0, 2, 0>(w, d0, lane);
      put_block<32, 2, 0>(w, d1, lane);
    }
    __syncwarp();
    {
      float d0[4][4], d1[4][4];
      join<0, 4, 0>(w, gm, s_f, d0, lane);
      join<0, 4, 1>(w, gm, s_f, d1, lane);
      __syncwarp();
      put_block<0, 4, 0>(w, d0, lane);
      put_block<0, 4, 1>(w, d1, lane);
    }
    __syncwarp();
    // T operands: 8 elements of a row per lane, of the blocks on and above the diagonal; hi also over the row in w,
    // for A T.  A warp's 16 rows x 16 columns are one block of the image: 512 bytes in a row.
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // two blocks of 16 rows at a time: all reads first
      constexpr int kBlocks[2] = {4 + 3, 2 + 1};
      const int j = lane & 15;
      float4 a[7], b[7];
#pragma unroll
      for (int k = 0; k < kBlocks[half]; ++k) {
        const int rb = 2 * half + (k >= 4 - 2 * half), cb = k >= 4 - 2 * half ? k - 4 + 2 * half : k;  // columns 16 (rb + cb) ..
        const float *src = w + row_start(16 * rb) + j * pitch(16 * rb) + 16 * cb + 8 * (lane >> 4);
        a[k] = *reinterpret_cast<const float4 *>(src);
        b[k] = *reinterpret_cast<const float4 *>(src + 4);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kBlocks[half]; ++k) {
        const int rb = 2 * half + (k >= 4 - 2 * half), cb = k >= 4 - 2 * half ? k - 4 + 2 * half : k, kb = rb + cb;
        uint4 hv, lv;
        split2(make_float2(a[k].x, a[k].y), hv.x, lv.x);
        split2(make_float2(a[k].z, a[k].w), hv.y, lv.y);
        split2(make_float2(b[k].x, b[k].y), hv.z, lv.z);
        split2(make_float2(b[k].z, b[k].w), hv.w, lv.w);
        *reinterpret_cast<uint4 *>(w + row_start(16 * rb) + j * pitch(16 * rb) + 8 * cb + 4 * (lane >> 4)) = hv;
        unsigned char *dst = rec + 512 * (kb * (kb + 1) + rb) + (j >> 3) * 256 + (lane >> 4) * 128 + (j & 7) * 16;
        *reinterpret_cast<uint4 *>(dst) = hv;
        *reinterpret_cast<uint4 *>(dst + 512 * (kb + 1)) = lv;
      }
    }
    __syncwarp();
    // A T: tiles on and below the diagonal.  Decays to a token of an earlier 16 in two factors, both at most
    // one: from the first token of t's 16 on, and up to it.
    const uint32_t aa = tc::smem_u32(smem + OFF_A) + (lane >> 4) * 16, tt = tc::smem_u32(w) + (lane >> 3 & 1) * 16;
    uint32_t b[4][4][4];  // [16 rows of T~^T][16 columns]: the fragments of two tiles of 8 rows
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
#pragma unroll
      for (int kk = rb; kk < 4; ++kk)
        ldmatrix4(b[rb][kk], tt + 4 * row_start(16 * rb) + ((lane & 7) + (lane >> 4) * 8) * 4 * pitch(16 * rb) + 32 * (kk - rb));
    __syncwarp();  // w is free for the image of A T
    unsigned char *image = reinterpret_cast<unsigned char *>(w);
    const uint32_t im = tc::smem_u32(w);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      uint32_t a[4][4];
#pragma unroll
      for (int kk = 0; kk <= mt; ++kk) ldmatrix4(a[kk], aa + 2 * a_row(16 * mt) + (lane & 15) * 2 * a_pitch(16 * mt) + 32 * kk);
      const int t = 16 * mt + (lane >> 2);
      const float d0 = s_rel[t], d1 = s_rel[t + 8], rt0 = ex2(d0), rt1 = ex2(d1);
#pragma unroll
      for (int np = 0; np <= mt; ++np) {  // two tiles of 8 columns
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int nt = 2 * np + k, j = 8 * nt + 2 * (lane & 3);
          float c[4] = {};
#pragma unroll
          for (int kk = np; kk <= mt; ++kk) {
            const uint32_t y[2] = {b[np][kk][2 * k], b[np][kk][2 * k + 1]};
            mma_f16(c, a[kk], y);
          }
          if (np < mt) {
            const float2 f = *reinterpret_cast<const float2 *>(s_col + 8 * mt * (mt - 1) + j);
            c[0] *= rt0 * f.x;
            c[1] *= rt0 * f.y;
            c[2] *= rt1 * f.x;
            c[3] *= rt1 * f.y;
          } else {
            const float2 d = *reinterpret_cast<const float2 *>(s_rel + j);
            // (above the diagonal the products are zero, and the decays could overflow)
            c[0] *= ex2(j <= t ? d0 - d.x : 0.f);
            c[1] *= ex2(j + 1 <= t ? d0 - d.y : 0.f);
            c[2] *= ex2(j <= t + 8 ? d1 - d.x : 0.f);
            c[3] *= ex2(j + 1 <= t + 8 ? d1 - d.y : 0.f);
          }
          o[2 * k] = h2(__floats2half2_rn(c[0], c[1]));
          o[2 * k + 1] = h2(__floats2half2_rn(c[2], c[3]));
        }
        // block (np, mt) is the (4 np - np (np - 1) / 2 + mt - np)-th
        stmatrix4(im + 512 * (3 * np - np * (np - 1) / 2 + mt) + (lane >> 3 & 1) * 256 + (lane >> 4) * 128 + (lane & 7) * 16, o);
      }
    }
    __syncwarp();
    // out by whole lines: written from the fragments, 16 bytes of 8 rows at a time, it would be four times the
    // requests
#pragma unroll
    for (int it = 0; it < 10; ++it)
      *reinterpret_cast<uint4 *>(rec + kDeltaTBytes + 512 * it + 16 * lane) = *reinterpret_cast<const uint4 *>(image + 512 * it + 16 * lane);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_delta_front(const DeltaPlan &p_in, cudaStream_t s) {
  // (also while the stream is captured: it may be the process's first call)
  cudaError_t e = cudaFuncSetAttribute(ssd_delta_front_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  // As many heads per CTA as share its K K^T, but CTAs for every SM: one head per warp where the chunks and
  // groups alone are few.
  DeltaPlan p = p_in;
  p.heads_per_cta = p.n_chunks * p.G >= 2 * 148 ? kMaxHeads : kWarps;
  const dim3 grid((unsigned)p.n_chunks, p.G, (p.hpg + p.heads_per_cta - 1) / p.heads_per_cta);
  ssd_delta_front_kernel<<<grid, kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd
