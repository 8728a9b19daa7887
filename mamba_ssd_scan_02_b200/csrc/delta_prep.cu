// delta_prep.cu -- the front end of the chunked delta rule: everything of a 64-token chunk that does
// not depend on the state, for all chunks at once.
//
// One CTA per (chunk, group, set of heads).  Shared by the group's heads: K and Q as fp16 operand tiles (a
// row scaled by the power of two that brings its largest element to [1, 2), exact in fp16 down to
// 2^-17 of it; rho is that power and the norm's factor), K K^T (fp32) and A~ = tril(Q K^T) (fp16).  Then
// each warp takes heads of its own:
//   gates  cs = prefix sums of log2(alpha), in fp64 so that differences keep fp32's relative precision
//          however large the sums
//   T~     = (I + L~)^-1, L~_ij = beta_i rho_i^2 K_i.K_j (j < i), in fp32: 16 x 16 diagonal blocks by
//          substitution, joined by block products with tf32 in two parts (22 bits)
//   A T    2^{cs_t - cs_j} rho_j (A~ T~)_tj, rounded once to fp16
// and leaves T~ in two fp16 parts and A T as the swizzled operand images that the chunk kernel loads.
//
// Why apart from the chunk kernel: inside it this part ran in the same SM as the tcgen05 products, which
// slow mma.sync down threefold and shared-memory loads twofold, and its latency (about 5 us a chunk)
// bounded every CTA: 650 us for 8192 tokens x 128 heads.  Here it is spread over all chunks, eight
// independent warps per SM.  The price is 25 KB of workspace per chunk and head, written once and read
// once.
#include "common.cuh"
#include "delta_mma.cuh"
#include "delta_plan.h"
#include "plan.h"

namespace ssd {
namespace {

using namespace delta;

constexpr int C = kDeltaChunk;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kHalf = 16384;
constexpr int kWPitch = 72;                        // floats; = 8 mod 32: conflict-free fragment reads
constexpr int kKPitch = 136;                       // halves of a K or Q row
constexpr int kAPitch = 72;                        // halves of a row of A~
constexpr uint32_t OFF_K = 0;                      // [128][136] halves: K rows, Q rows
constexpr uint32_t OFF_G = OFF_K + 128 * kKPitch * 2;   // [64][72] floats: K K^T, columns >= row
constexpr uint32_t OFF_A = OFF_G + 64 * kWPitch * 4;    // [64][72] halves: A~
constexpr uint32_t OFF_RHO = OFF_A + 64 * kAPitch * 2;  // rho_k[64]
constexpr uint32_t OFF_GATE = OFF_RHO + 256;            // per warp: cs hi[64], lo[64], -beta rho^2 [64]
constexpr uint32_t OFF_W = OFF_GATE + kWarps * 768;     // per warp: [64][72] floats
constexpr uint32_t kSmem = OFF_W + kWarps * 64 * kWPitch * 4;
static_assert(kSmem <= 232448, "shared memory");

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

// W12 = W11 Z W22, the block that joins two inverted diagonal blocks of 8 K rows (transposed, so upper
// triangular): rows 16 mt .. of it into d.  w11, z and w22 at their corners.  Straight-line: with a branch
// per tile the products of one would wait for those of the one before.
template <int K, int MT>
__device__ __forceinline__ void join(const float *w11, const float *z, const float *w22, float (&d)[K][4], int lane) {
  FragA a[K];
#pragma unroll
  for (int kk = 2 * MT; kk < K; ++kk) a[kk] = load_a(w11 + 16 * MT * kWPitch + 8 * kk, lane);
#pragma unroll
  for (int nt = 0; nt < K; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[nt][e] = 0.f;
#pragma unroll
  for (int kt = 0; kt < K; ++kt) {
    float hh[4] = {}, hl[4] = {}, lh[4] = {};
#pragma unroll
    for (int kk = 2 * MT; kk < K; ++kk) {
      const FragB b = load_b(z + 8 * kk * kWPitch + 8 * kt, false, lane);
      mma_tf32(hh, a[kk].h, b.h);
      mma_tf32(hl, a[kk].h, b.l);
      mma_tf32(lh, a[kk].l, b.h);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) hh[e] += hl[e] + lh[e];
    const FragA x = acc_as_a(hh);
#pragma unroll
    for (int nt = kt; nt < K; ++nt) {
      const FragB b = load_b(w22 + 8 * kt * kWPitch + 8 * nt, true, lane);
      mma_tf32(d[nt], x.l, b.h);
      mma_tf32(d[nt], x.h, b.l);
      mma_tf32(d[nt], x.h, b.h);
    }
  }
}
template <int K>
__device__ __forceinline__ void put_block(float *o, const float (&d)[K][4], int lane) {
#pragma unroll
  for (int nt = 0; nt < K; ++nt) {
    float *x = o + (lane >> 2) * kWPitch + 8 * nt + 2 * (lane & 3);
    *reinterpret_cast<float2 *>(x) = make_float2(d[nt][0], d[nt][1]);
    *reinterpret_cast<float2 *>(x + 8 * kWPitch) = make_float2(d[nt][2], d[nt][3]);
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


__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// 2^x for x <= 0, to fp32's precision: the whole part of x as an exponent, the rest by exp2f
__device__ __forceinline__ float exp2_split(double x) {
  const double w = rint(x);
  return ldexpf(exp2f((float)(x - w)), (int)fmax(w, -200.0));
}

__global__ void __launch_bounds__(kThreads, 1) ssd_delta_front_kernel(const DeltaPlan p) {
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

  // ---- K and Q: a warp takes 16 of the 128 rows
  {
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
      const uint32_t top = __reduce_max_sync(
          0xffffffffu, max(max(__float_as_uint(a.x) & 0x7fffffffu, __float_as_uint(a.y) & 0x7fffffffu),
                           max(__float_as_uint(b.x) & 0x7fffffffu, __float_as_uint(b.y) & 0x7fffffffu)));
      const uint32_t e = min(max(top >> 23, 1u), 253u);
      const float f = __uint_as_float((254u - e) << 23);
      const uint2 v = make_uint2(h2(__floats2half2_rn(a.x * f, a.y * f)), h2(__floats2half2_rn(b.x * f, b.y * f)));
      *reinterpret_cast<uint2 *>(smem + OFF_K + r * kKPitch * 2 + 8 * lane) = v;
      if (blockIdx.z == 0)
        *reinterpret_cast<uint2 *>(tile + (lane >> 4) * kHalf + swz(r, (lane & 15) >> 1) + 8 * (lane & 1)) = v;
      float rho = __uint_as_float(e << 23);
      if (p.qk_norm) rho *= 1.f / sqrtf(warp_sum(a.x * a.x + a.y * a.y + b.x * b.x + b.y * b.y) + p.qk_eps);
      if (r >= 64) rho *= p.q_scale;
      if (lane == 0) {
        if (blockIdx.z == 0) reinterpret_cast<float *>(tile + 2 * kHalf)[r] = rho;
        if (r < 64) s_rho[r] = rho;
      }
    }
  }
  __syncthreads();
  // ---- K K^T (warps 0-3, 16 rows each, columns from the diagonal on) and A~ (warps 4-7, up to it)
  {
    const int rt = warp & 3, lo = warp < 4 ? 2 * rt : 0, hi = warp < 4 ? 8 : 2 * rt + 2;
    const uint32_t kq = tc::smem_u32(smem + OFF_K);
    const uint32_t arow = kq + (16 * warp + (lane & 15)) * kKPitch * 2 + (lane >> 4) * 16;
    const uint32_t brow = kq + (lane & 7) * kKPitch * 2 + (lane >> 3 & 1) * 16;
    uint32_t a[8][4];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) ldmatrix4(a[ks], arow + 32 * ks);
    for (int nt = lo; nt < hi; ++nt) {
      float c0[4] = {}, c1[4] = {};
#pragma unroll
      for (int ks = 0; ks < 8; ks += 2) {
        uint32_t b[2], d[2];
        ldmatrix2(b, brow + 8 * nt * kKPitch * 2 + 32 * ks);
        ldmatrix2(d, brow + 8 * nt * kKPitch * 2 + 32 * ks + 32);
        mma_f16(c0, a[ks], b);
        mma_f16(c1, a[ks + 1], d);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c0[e] += c1[e];
      const int r = 16 * rt + (lane >> 2), j = 8 * nt + 2 * (lane & 3);
      if (warp < 4) {
        float *o = reinterpret_cast<float *>(smem + OFF_G) + r * kWPitch + j;
        *reinterpret_cast<float2 *>(o) = make_float2(c0[0], c0[1]);
        *reinterpret_cast<float2 *>(o + 8 * kWPitch) = make_float2(c0[2], c0[3]);
      } else {
        __half *o = reinterpret_cast<__half *>(smem + OFF_A) + r * kAPitch + j;
        *reinterpret_cast<__half2 *>(o) = __floats2half2_rn(j <= r ? c0[0] : 0.f, j + 1 <= r ? c0[1] : 0.f);
        *reinterpret_cast<__half2 *>(o + 8 * kAPitch) = __floats2half2_rn(j <= r + 8 ? c0[2] : 0.f, j + 1 <= r + 8 ? c0[3] : 0.f);
      }
    }
  }
  __syncthreads();

  // ---- heads
  float *w = reinterpret_cast<float *>(smem + OFF_W) + warp * 64 * kWPitch;
  float *s_hi = reinterpret_cast<float *>(smem + OFF_GATE) + warp * 192, *s_lo = s_hi + 64, *s_f = s_hi + 128;
  const float *gm = reinterpret_cast<const float *>(smem + OFF_G);
  const int h_end = min((blockIdx.z + 1) * p.heads_per_cta, p.hpg);
  for (int hh = blockIdx.z * p.heads_per_cta + warp; hh < h_end; hh += kWarps) {
    const int h = g * p.hpg + hh;
    unsigned char *rec = p.records + (ck * p.H + h) * kDeltaRecordBytes;
    {  // gates of tokens 2 lane, 2 lane + 1
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
      const double end = __shfl_sync(0xffffffffu, sum, 31);
      float gamma[2], to_end[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float rho = s_rho[2 * lane + u];
        gamma[u] = exp2_split(cs[u]);
        to_end[u] = rho * exp2_split(end - cs[u]);
        const float hi = (float)cs[u];
        s_hi[2 * lane + u] = hi;
        s_lo[2 * lane + u] = (float)(cs[u] - hi);
        s_f[2 * lane + u] = -beta[u] * rho * rho;
      }
      float2 *o = reinterpret_cast<float2 *>(rec + 3 * 8192) + lane;
      o[0] = make_float2(beta[0], beta[1]);
      o[32] = make_float2(gamma[0], gamma[1]);
      o[64] = make_float2(to_end[0], to_end[1]);
    }
    __syncwarp();
    // w = (-L~)^T by 16 x 16 blocks on and above the diagonal
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
#pragma unroll
      for (int cb = rb; cb < 4; ++cb)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = 16 * rb + 8 * u + (lane >> 2), i = 16 * cb + 4 * (lane & 3);
          const float4 x = *reinterpret_cast<const float4 *>(gm + j * kWPitch + i);
          const float4 f = *reinterpret_cast<const float4 *>(s_f + i);
          float4 y = make_float4(f.x * x.x, f.y * x.y, f.z * x.z, f.w * x.w);
          if (rb == cb) y = make_float4(i > j ? y.x : 0.f, i + 1 > j ? y.y : 0.f, i + 2 > j ? y.z : 0.f, i + 3 > j ? y.w : 0.f);
          *reinterpret_cast<float4 *>(w + j * kWPitch + i) = y;
        }
    __syncwarp();
#pragma unroll 1
    for (int p0 = 0; p0 < 64; p0 += 32) {
      float2 t[8];
      invert16(w, p0, lane, t);
      __syncwarp();
      float *o = w + (p0 + lane) * kWPitch + p0 + (lane & 16);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(o + 4 * i) = make_float4(t[2 * i].x, t[2 * i].y, t[2 * i + 1].x, t[2 * i + 1].y);
      __syncwarp();
      float d[2][4];
      float *wp = w + p0 * kWPitch + p0;
      join<2, 0>(wp, wp + 16, wp + 16 * kWPitch + 16, d, lane);
      __syncwarp();
      put_block<2>(wp + 16, d, lane);
    }
    __syncwarp();
    {
      float d0[4][4], d1[4][4];
      join<4, 0>(w, w + 32, w + 32 * kWPitch + 32, d0, lane);
      join<4, 1>(w, w + 32, w + 32 * kWPitch + 32, d1, lane);
      __syncwarp();
      put_block<4>(w + 32, d0, lane);
      put_block<4>(w + 16 * kWPitch + 32, d1, lane);
    }
    __syncwarp();
    // T operands: 8 elements of a row per lane; hi also over the row in w, for A T
    __half *th = reinterpret_cast<__half *>(w);
#pragma unroll 4
    for (int it = 0; it < 16; ++it) {
      const int j = 4 * it + (lane >> 3), u = lane & 7;
      const float *src = w + j * kWPitch + 8 * u;
      const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
      uint4 hv, lv;
      split2(make_float2(a.x, a.y), hv.x, lv.x);
      split2(make_float2(a.z, a.w), hv.y, lv.y);
      split2(make_float2(b.x, b.y), hv.z, lv.z);
      split2(make_float2(b.z, b.w), hv.w, lv.w);
      if ((u >> 1) < (j >> 4)) hv = lv = make_uint4(0, 0, 0, 0);  // below the diagonal blocks: not computed
      __syncwarp();
      *reinterpret_cast<uint4 *>(th + j * 2 * kWPitch + 8 * u) = hv;
      *reinterpret_cast<uint4 *>(rec + swz(j, u)) = hv;
      *reinterpret_cast<uint4 *>(rec + 8192 + swz(j, u)) = lv;
    }
    __syncwarp();
    // A T: tiles on and below the diagonal
    const uint32_t aa = tc::smem_u32(smem + OFF_A) + (lane & 15) * kAPitch * 2 + (lane >> 4) * 16;
    const uint32_t tt = tc::smem_u32(th) + (lane & 7) * 4 * kWPitch + (lane >> 3 & 1) * 16;
    unsigned char *out = rec + 2 * 8192 + 4 * (lane & 3);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      uint32_t a[4][4];
#pragma unroll
      for (int kk = 0; kk <= mt; ++kk) ldmatrix4(a[kk], aa + 16 * mt * kAPitch * 2 + 32 * kk);
      const int t = 16 * mt + (lane >> 2);
      const float hi0 = s_hi[t], lo0 = s_lo[t], hi1 = s_hi[t + 8], lo1 = s_lo[t + 8];
#pragma unroll
      for (int nt = 0; nt < 2 * mt + 2; ++nt) {
        float c[4] = {};
#pragma unroll
        for (int kk = nt / 2; kk <= mt; ++kk) {
          uint32_t b[2];
          ldmatrix2(b, tt + 8 * nt * 4 * kWPitch + 32 * kk);
          mma_f16(c, a[kk], b);
        }
        const int j = 8 * nt + 2 * (lane & 3);
        const float2 hj = *reinterpret_cast<const float2 *>(s_hi + j), lj = *reinterpret_cast<const float2 *>(s_lo + j);
        const float2 rj = *reinterpret_cast<const float2 *>(s_rho + j);
        // (above the diagonal the products are zero; the exponent is kept from overflowing there)
        c[0] *= rj.x * ex2(fminf((hi0 - hj.x) + (lo0 - lj.x), 0.f));
        c[1] *= rj.y * ex2(fminf((hi0 - hj.y) + (lo0 - lj.y), 0.f));
        c[2] *= rj.x * ex2(fminf((hi1 - hj.x) + (lo1 - lj.x), 0.f));
        c[3] *= rj.y * ex2(fminf((hi1 - hj.y) + (lo1 - lj.y), 0.f));
        *reinterpret_cast<uint32_t *>(out + swz(t, nt)) = h2(__floats2half2_rn(c[0], c[1]));
        *reinterpret_cast<uint32_t *>(out + swz(t + 8, nt)) = h2(__floats2half2_rn(c[2], c[3]));
      }
#pragma unroll
      for (int nt = 2 * mt + 2; nt < 8; ++nt) {
        *reinterpret_cast<uint32_t *>(out + swz(t, nt)) = 0u;
        *reinterpret_cast<uint32_t *>(out + swz(t + 8, nt)) = 0u;
      }
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_delta_front(const DeltaPlan &p_in, cudaStream_t s) {
  cudaError_t e = set_smem_attr(ssd_delta_front_kernel, kSmem, s);
  if (e != cudaSuccess) return e;
  // As many heads per CTA as share its K K^T, but CTAs for every SM: one head per warp where the chunks
  // and groups alone are few.
  DeltaPlan p = p_in;
  p.heads_per_cta = p.n_chunks * p.G >= 2 * 148 ? 2 * kWarps : kWarps;
  const dim3 grid((unsigned)p.n_chunks, p.G, (p.hpg + p.heads_per_cta - 1) / p.heads_per_cta);
  ssd_delta_front_kernel<<<grid, kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd
