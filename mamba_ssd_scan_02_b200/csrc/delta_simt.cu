// delta_simt.cu -- the gated delta rule in fp32: the decode step, short prefills and fp32 inputs.
//
// Per head and token, with S the P x N state and k^, q^ the normalised key and scaled query:
//   u = beta (v - alpha S k^),  y = alpha S q^ + u (k^.q^),  S <- alpha S + u k^^T.
// y is S_t q^ written with the old state, so both products with S come from one pass over it and
// one reduction, and k^.q^ is a scalar per token.
//
// The rows of S are independent given k^, so a few lanes hold a row (in registers for the whole call), a warp
// several rows.
//
// A sequence is taken four tokens at a time.  With g_j = alpha_0 .. alpha_j and D_ij = alpha_{i+1} .. alpha_j,
//   u_j = beta_j (v_j - g_j S k_j - sum_{i<j} D_ij (k_i.k_j) u_i)
//   y_j = g_j S q_j + sum_{i<=j} D_ij (k_i.q_j) u_i
//   S  <- g_3 S + sum_j D_j3 u_j k_j^T,
// so eight products with the old S share one reduction over the lanes of a row, and the chain from token to
// token is a quarter of a dot product, a reduction and an update, plus a triangular solve in scalars (about
// 250 clocks a token; token by token it was 630).  The scalars (D, k_i.k_j, k_i.q_j) are the same for all rows:
// four warps of the CTA work them out for a tile of 16 tokens, normalise q and k and put it all into shared
// memory, while the others run the tile before; their loads run two tiles ahead.  What bounds it then is
// shared memory: a warp reads 8 vectors for 4 rows.  256 tokens x 8 heads in fp32: 31 us.
#include "common.cuh"
#include "delta_plan.h"
#include "plan.h"

namespace ssd {
namespace {

__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

__device__ __forceinline__ float step_of(float raw, float bias, const DeltaPlan &p) {
  float d = raw + bias;
  if (p.softplus) d = d > 20.f ? d : log1pf(expf(d));
  return d < p.dt_min ? p.dt_min : d > p.dt_max ? p.dt_max : d;  // (a NaN stays)
}
__device__ __forceinline__ float beta_of(float raw, const DeltaPlan &p) {
  return p.beta_scale * (p.beta_sigmoid ? 1.f / (1.f + expf(-raw)) : raw);
}

// What four tokens share, whatever the row; j the later token, i the earlier
struct Four {
  float g[4], beta[4], end[4];  // g_j, beta_j, D_j3
  float kk[4][4];               // [j][i]: beta_j D_ij k_i.k_j, i < j
  float kq[4][4];               // [j][i]: D_ij k_i.q_j, i <= j
};
__device__ __forceinline__ constexpr int pair_at(int i, int j) { return j * (j + 1) / 2 + i; }  // i <= j

// Warps 0-3 stage a tile, four tokens each, while warps 4 .. 3 + CW run the tokens of the tile before.
constexpr int kStageWarps = 4;

template <typename T, int CW>
__global__ void __launch_bounds__((kStageWarps + CW) * 32, 1) delta_recurrent_kernel(const DeltaPlan p) {
  constexpr int LPR = 8;                // lanes of a row: as many as there are products per reduction
  constexpr int TT = 4 * kStageWarps;   // tokens of a tile
  constexpr int R = CW * 32 / LPR;      // state rows of this CTA
  constexpr int E4 = kDState / LPR / 4; // float4s of a row per lane
  constexpr int NT = kStageWarps * 32;
  constexpr int VPT = (TT * R + NT - 1) / NT;  // v elements of a tile per staging thread
  constexpr int VP = TT + 4;
  __shared__ __align__(16) float sq[2][TT][kDState], sk[2][TT][kDState];
  __shared__ __align__(16) float sv[2][R][VP];
  __shared__ __align__(16) Four s_four[2][TT / 4];
  __shared__ float s_dot[TT / 4][24];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int blocks_per_head = p.P / R;
  const int h = blockIdx.x / blocks_per_head, row0 = (blockIdx.x % blocks_per_head) * R;
  const int seq = p.order ? p.order[blockIdx.y] : (int)blockIdx.y;
  const int g = h / p.hpg;
  const int len = seq_len(p.cu, seq, p.L);
  const long long base = seq_base(p.cu, seq, p.L);
  const float A = len > 0 ? p.A[h] : 0.f, bias = len > 0 ? p.dt_bias[h] : 0.f;  // (null where no tokens are)
  const T *q = static_cast<const T *>(p.q) + base * p.qs + g * kDState + 4 * lane;
  const T *k = static_cast<const T *>(p.k) + base * p.ks + g * kDState + 4 * lane;
  const T *v = static_cast<const T *>(p.v) + base * p.vs + h * p.P + row0;
  const T *dt = static_cast<const T *>(p.dt) + base * p.ds + h;
  const T *bb = static_cast<const T *>(p.b) + base * p.bs + h;
  struct Tile {
    float rq[4][4], rk[4][4], rv[VPT], rdt, rb;
  } even, odd;  // two tiles on the way from memory

  // This thread's part of the tile at t0, into registers.  Tokens after the last are loaded as the last.
  auto fetch = [&](Tile &x, int t0) {
    const int last = len - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = min(t0 + 4 * warp + i, last);
      load4(q + t * p.qs, x.rq[i]);
      load4(k + t * p.ks, x.rk[i]);
    }
    const long long td = min(t0 + 4 * warp + (lane & 3), last);
    x.rdt = io<T>::ld(dt + td * p.ds);
    x.rb = io<T>::ld(bb + td * p.bs);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = min(tid + i * NT, TT * R - 1);
      x.rv[i] = io<T>::ld(v + (long long)min(t0 + at / R, last) * p.vs + at % R);
    }
  };
  // The fetched tile into shared memory.  Tokens after the last: zeros, no decay.
  auto stage = [&](Tile &tile, int t0, int buf) {
    float(&rq)[4][4] = tile.rq, (&rk)[4][4] = tile.rk;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = tid + i * NT;
      if (at < TT * R) sv[buf][at % R][at / R] = t0 + at / R < len ? tile.rv[i] : 0.f;
    }
    const int first = t0 + 4 * warp;
    float x[24];  // k_i.k_j (i <= j), k_i.q_j (i <= j), q_j.q_j
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (first + j >= len)
#pragma unroll
        for (int e = 0; e < 4; ++e) rk[j][e] = rq[j][e] = 0.f;
#pragma unroll
      for (int i = 0; i <= j; ++i) {
        float kk = 0.f, kq = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk = fmaf(rk[i][e], rk[j][e], kk);
          kq = fmaf(rk[i][e], rq[j][e], kq);
        }
        x[pair_at(i, j)] = kk;
        x[10 + pair_at(i, j)] = kq;
      }
      float qq = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) qq = fmaf(rq[j][e], rq[j][e], qq);
      x[20 + j] = qq;
    }
    // all 24 sums over the warp at once: at each of three levels a lane hands half of them over
#pragma unroll
    for (int o = 16, n = 12; o >= 4; o >>= 1, n >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? x[i] : x[i + n];
        x[i] = (up ? x[i + n] : x[i]) + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
#pragma unroll
    for (int o = 2; o >= 1; o >>= 1)
#pragma unroll
      for (int i = 0; i < 3; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if ((lane & 3) < 3) s_dot[warp][3 * (lane >> 2) + (lane & 3)] = (lane & 3) == 0 ? x[0] : (lane & 3) == 1 ? x[1] : x[2];
    __syncwarp();
    const float *dot = s_dot[warp];
    const int i = lane & 3, j = lane >> 2 & 3;  // (lanes 16-31 as lanes 0-15)
    float fk_j = 1.f, fq_j = p.q_scale;
    if (p.qk_norm) {
      fk_j = 1.f / sqrtf(dot[pair_at(j, j)] + p.qk_eps);
      fq_j *= 1.f / sqrtf(dot[20 + j] + p.qk_eps);
    }
    const float fk_i = __shfl_sync(0xffffffffu, fk_j, 4 * i);
    const bool live = first + i < len;  // (rdt and rb are token i's)
    const float alpha = live ? expf(A * step_of(tile.rdt, bias, p)) : 1.f;
    const float beta = live ? beta_of(tile.rb, p) : 0.f;
    const float beta_j = __shfl_sync(0xffffffffu, beta, j);
    float a[4], gj = 1.f, d = 1.f;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      a[l] = __shfl_sync(0xffffffffu, alpha, l);
      if (l <= j) gj *= a[l];
      if (l > i && l <= j) d *= a[l];
    }
    Four &f = s_four[buf][warp];
    if (lane < 16) {
      const int at = i <= j ? pair_at(i, j) : 0;
      f.kk[j][i] = i < j ? beta_j * d * fk_i * fk_j * dot[at] : 0.f;
      f.kq[j][i] = i <= j ? d * fk_i * fq_j * dot[10 + at] : 0.f;
      if (i == 0) f.g[j] = gj;
      if (i == 0) f.beta[j] = beta_j;
      if (j == 3) f.end[i] = d;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float fk = __shfl_sync(0xffffffffu, fk_j, 4 * t), fq = __shfl_sync(0xffffffffu, fq_j, 4 * t);
      *reinterpret_cast<float4 *>(&sk[buf][4 * warp + t][4 * lane]) = make_float4(rk[t][0] * fk, rk[t][1] * fk, rk[t][2] * fk, rk[t][3] * fk);
      *reinterpret_cast<float4 *>(&sq[buf][4 * warp + t][4 * lane]) = make_float4(rq[t][0] * fq, rq[t][1] * fq, rq[t][2] * fq, rq[t][3] * fq);
    }
  };

  if (len == 0 && (warp < kStageWarps || !p.h_final)) return;
  if (warp < kStageWarps) {
    fetch(even, 0);
    if (TT < len) fetch(odd, TT);
    for (int t0 = 0; t0 < len; t0 += 2 * TT) {
      stage(even, t0, 0);
      __syncthreads();
      if (t0 + 2 * TT < len) fetch(even, t0 + 2 * TT);
      if (t0 + TT >= len) break;
      stage(odd, t0 + TT, 1);
      __syncthreads();
      if (t0 + 3 * TT < len) fetch(odd, t0 + 3 * TT);
    }
    return;
  }

  const int r = (warp - kStageWarps) * (32 / LPR) + lane / LPR, s = lane % LPR;
  const long long soff = (((long long)seq * p.H + h) * p.P + row0 + r) * kDState + 4 * s;
  float2 S[E4][2];
#pragma unroll
  for (int j = 0; j < E4; ++j) {
    const float4 x = p.h0 ? *reinterpret_cast<const float4 *>(p.h0 + soff + 4 * LPR * j) : make_float4(0.f, 0.f, 0.f, 0.f);
    S[j][0] = make_float2(x.x, x.y);
    S[j][1] = make_float2(x.z, x.w);
  }
  const int yj = s & 3;  // lane s ends with S k_s (s < 4) or S q_{s - 4}, and the latter stores that token's y
  T *y = static_cast<T *>(p.y);
  long long yo = (base + yj) * p.ys + (long long)h * p.P + row0 + r;
  for (int t0 = 0, buf = 0; t0 < len; t0 += TT, buf ^= 1) {
    __syncthreads();
    const int blocks = (min(TT, len - t0) + 3) / 4;
#pragma unroll 2
    for (int b = 0; b < blocks; ++b) {
      const Four &f = s_four[buf][b];
      const float *kp = &sk[buf][4 * b][4 * s], *qp = &sq[buf][4 * b][4 * s];
      const float4 g4 = *reinterpret_cast<const float4 *>(f.g), b4 = *reinterpret_cast<const float4 *>(f.beta);
      const float4 v4 = *reinterpret_cast<const float4 *>(&sv[buf][r][4 * b]);
      const float4 kk2 = *reinterpret_cast<const float4 *>(f.kk[2]), kk3 = *reinterpret_cast<const float4 *>(f.kk[3]);
      const float4 end = *reinterpret_cast<const float4 *>(f.end);
      const float kk1 = f.kk[1][0];
      float2 kv[4][E4][2], acc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < E4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 x = *reinterpret_cast<const float4 *>(kp + j * kDState + 4 * LPR * e);
          const float4 z = *reinterpret_cast<const float4 *>(qp + j * kDState + 4 * LPR * e);
          const float2 x0 = make_float2(x.x, x.y), x1 = make_float2(x.z, x.w);
          acc[j] = __ffma2_rn(S[e][0], x0, acc[j]);
          acc[j] = __ffma2_rn(S[e][1], x1, acc[j]);
          acc[4 + j] = __ffma2_rn(S[e][0], make_float2(z.x, z.y), acc[4 + j]);
          acc[4 + j] = __ffma2_rn(S[e][1], make_float2(z.z, z.w), acc[4 + j]);
          kv[j][e][0] = x0;
          kv[j][e][1] = x1;
        }
      float x[8];  // S k_j, S q_j: their sums over the row's lanes, handed over like those of stage()
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = acc[j].x + acc[j].y;
#pragma unroll
      for (int o = LPR / 2, n = 4; o > 0; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const float give = up ? x[j] : x[j + n];
          x[j] = (up ? x[j + n] : x[j]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      float dk[4], u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) dk[j] = __shfl_sync(0xffffffffu, x[0], (lane & ~(LPR - 1)) | j);
      u[0] = b4.x * fmaf(-g4.x, dk[0], v4.x);
      u[1] = fmaf(-kk1, u[0], b4.y * fmaf(-g4.y, dk[1], v4.y));
      u[2] = b4.z * fmaf(-g4.z, dk[2], v4.z);
      u[3] = b4.w * fmaf(-g4.w, dk[3], v4.w);
      u[2] = fmaf(-kk2.y, u[1], fmaf(-kk2.x, u[0], u[2]));
      u[3] = fmaf(-kk3.z, u[2], fmaf(-kk3.y, u[1], fmaf(-kk3.x, u[0], u[3])));
      const float2 ge = make_float2(g4.w, g4.w);
      const float w[4] = {u[0] * end.x, u[1] * end.y, u[2] * end.z, u[3] * end.w};
#pragma unroll
      for (int e = 0; e < E4; ++e) {
        S[e][0] = __fmul2_rn(S[e][0], ge);
        S[e][1] = __fmul2_rn(S[e][1], ge);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 w2 = make_float2(w[j], w[j]);
          S[e][0] = __ffma2_rn(w2, kv[j][e][0], S[e][0]);
          S[e][1] = __ffma2_rn(w2, kv[j][e][1], S[e][1]);
        }
      }
      const float4 kq = *reinterpret_cast<const float4 *>(f.kq[yj]);
      // (what comes after token yj is left out, not multiplied by zero: it may be NaN)
      const float o = fmaf(kq.w, yj >= 3 ? u[3] : 0.f, fmaf(kq.z, yj >= 2 ? u[2] : 0.f,
                      fmaf(kq.y, yj >= 1 ? u[1] : 0.f, fmaf(kq.x, u[0], f.g[yj] * x[0]))));
      if (s >= 4 && t0 + 4 * b + yj < len && in_bounds(yo, p.y_extent, p.err)) io<T>::st(y + yo, o);
      yo += 4 * p.ys;
    }
  }
  if (p.h_final) {
#pragma unroll
    for (int j = 0; j < E4; ++j)
      if (in_bounds(soff + 4 * LPR * j + 3, p.state_extent, p.err))
        *reinterpret_cast<float4 *>(p.h_final + soff + 4 * LPR * j) = make_float4(S[j][0].x, S[j][0].y, S[j][1].x, S[j][1].y);
  }
}

// One token per row, the state in place in a pool.  Bound by HBM: the state read and written once; 64 rows of 128
// heads x 64 x 128: 90 us, 0.91 of a copy's rate.  Four lanes a row and eight loads of 16 bytes in flight per
// lane; eight lanes: 99 to 100 us, 16: 121.
template <typename T, int LPR, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) delta_decode_kernel(const DeltaPlan p) {
  constexpr int R = WARPS * 32 / LPR;   // state rows of this CTA
  constexpr int E4 = kDState / LPR / 4; // float4s of a row per lane
  constexpr int NT = WARPS * 32;
  constexpr bool kStream = LPR == 4;    // a large batch
  __shared__ __align__(16) float sq[kDState], sk[kDState];
  __shared__ float s_kq;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int blocks_per_head = p.P / R;
  const int h = blockIdx.x / blocks_per_head, row0 = (blockIdx.x % blocks_per_head) * R;
  const int g = h / p.hpg;
  const long long seq = blockIdx.y;
  const int r = warp * (32 / LPR) + lane / LPR, s = lane % LPR;

  long long state_idx = seq;
  if (p.slots) {
    const int own = p.slots[seq];
    if (own < 0) return;
    bool twice = false;  // an earlier row of the batch has this slot
    for (int j = tid; j < seq; j += NT) twice |= p.slots[j] == own;
    if (__syncthreads_or(twice) || own >= p.n_slots) {
      if (tid == 0) latch_error(p.err, (int)SSD_ERR_DEVICE_BOUNDS);
      return;
    }
    state_idx = own;
  }
  const long long soff = ((state_idx * p.H + h) * p.P + row0 + r) * kDState + 4 * s;
  float S[E4][4];
#pragma unroll
  for (int j = 0; j < E4; ++j) load4(p.h_final + soff + 4 * LPR * j, S[j]);
  const float vr = io<T>::ld(static_cast<const T *>(p.v) + seq * p.vs + h * p.P + row0 + r);
  const float rdt = io<T>::ld(static_cast<const T *>(p.dt) + seq * p.ds + h);
  const float rb = io<T>::ld(static_cast<const T *>(p.b) + seq * p.bs + h);
  const float A = p.A[h], bias = p.dt_bias[h];
  if (warp == 0) {
    float rq[4], rk[4];
    load4(static_cast<const T *>(p.q) + seq * p.qs + g * kDState + 4 * lane, rq);
    load4(static_cast<const T *>(p.k) + seq * p.ks + g * kDState + 4 * lane, rk);
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qq = fmaf(rq[e], rq[e], qq);
      kk = fmaf(rk[e], rk[e], kk);
      qk = fmaf(rq[e], rk[e], qk);
    }
    float fq = p.q_scale, fk = 1.f;
    if (p.qk_norm) {
      fq *= 1.f / sqrtf(warp_sum(qq) + p.qk_eps);
      fk = 1.f / sqrtf(warp_sum(kk) + p.qk_eps);
    }
    qk = warp_sum(qk);
    *reinterpret_cast<float4 *>(&sq[4 * lane]) = make_float4(rq[0] * fq, rq[1] * fq, rq[2] * fq, rq[3] * fq);
    *reinterpret_cast<float4 *>(&sk[4 * lane]) = make_float4(rk[0] * fk, rk[1] * fk, rk[2] * fk, rk[3] * fk);
    if (lane == 0) s_kq = qk * fq * fk;
  }
  const float alpha = expf(A * step_of(rdt, bias, p)), beta = beta_of(rb, p);
  __syncthreads();
  float kv[E4][4], dk[2] = {0.f, 0.f}, dq[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < E4; ++j) {
    load4(&sk[4 * (j * LPR + s)], kv[j]);
    float qv[4];
    load4(&sq[4 * (j * LPR + s)], qv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dk[e & 1] = fmaf(S[j][e], kv[j][e], dk[e & 1]);
      dq[e & 1] = fmaf(S[j][e], qv[e], dq[e & 1]);
    }
  }
  float dk_ = dk[0] + dk[1], dq_ = dq[0] + dq[1];
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    dk_ += __shfl_xor_sync(0xffffffffu, dk_, o);
    dq_ += __shfl_xor_sync(0xffffffffu, dq_, o);
  }
  const float u = beta * (vr - alpha * dk_);
  if (s == 0) {
    const long long yo = seq * p.ys + (long long)h * p.P + row0 + r;
    if (in_bounds(yo, p.y_extent, p.err)) io<T>::st(static_cast<T *>(p.y) + yo, fmaf(u, s_kq, alpha * dq_));
  }
#pragma unroll
  for (int j = 0; j < E4; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) S[j][e] = fmaf(u, kv[j][e], alpha * S[j][e]);
    if (!in_bounds(soff + 4 * LPR * j + 3, p.state_extent, p.err)) continue;
    float4 *dst = reinterpret_cast<float4 *>(p.h_final + soff + 4 * LPR * j);
    const float4 x = make_float4(S[j][0], S[j][1], S[j][2], S[j][3]);
    // states beyond the L2 cache leave it first: 64 states of 128 heads 94.5 -> 90.3 us.  A small batch's stay, for
    // its next step.
    if (kStream) __stcs(dst, x);
    else *dst = x;
  }
}

// The rows of a CTA: as few as leave one CTA per SM, since the rows of an SM share its shared-memory reads, and
// as many as the registers allow once there are more.  Every choice gives the same bits.  256 tokens x H
// heads of 64 rows, fp32, in us with CW = 2, 4, 8:  H = 8: 31, 38, 60;  32: 44, 40, 61;  64: 79, 75, 61;
// 512: 527, 488, 392.
template <typename T, int CW>
cudaError_t launch_rows(const DeltaPlan &p, cudaStream_t s) {
  delta_recurrent_kernel<T, CW><<<dim3(p.H * p.P / (4 * CW), p.B), (kStageWarps + CW) * 32, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_recurrent(const DeltaPlan &p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.H * p.P;
  if (rows <= 8 * 148) return launch_rows<T, 2>(p, s);
  return rows <= 16 * 148 ? launch_rows<T, 4>(p, s) : launch_rows<T, 8>(p, s);
}
// Batches whose states stay in the L2 cache (64 MB of its 126) have eight lanes per row and 16 rows per CTA, which
// spreads a small one over more SMs; larger ones four lanes, 64 rows, and stores past the cache.  In us, the
// former and the latter: 1 row of 32 heads of 128 3.2 : 3.5, 5 rows 5.2 : 5.9, 20 rows (42 MB) 16.1 : 16.7; of 128
// heads of 64 16 rows (67 MB) 24.3 : 24.5, 64 rows (268 MB) 99 : 90.
template <typename T>
cudaError_t launch_decode(const DeltaPlan &p, cudaStream_t s) {
  if ((long long)p.B * p.H * p.P <= 131072) delta_decode_kernel<T, 8, 4><<<dim3(p.H * p.P / 16, p.B), 128, 0, s>>>(p);
  else delta_decode_kernel<T, 4, 8><<<dim3(p.H * p.P / 64, p.B), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <int N>
struct Ints {
  int v[N];
};
template <int N>
__global__ void put_ints_kernel(int *dst, const __grid_constant__ Ints<N> src, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src.v[i];
}
template <int N>
void put(int *dst, const int *host, int n, cudaStream_t s) {
  Ints<N> a;
  for (int i = 0; i < n; ++i) a.v[i] = host[i];
  put_ints_kernel<N><<<1, 256, 0, s>>>(dst, a, n);
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaPlan &p, cudaStream_t s) {
  return p.bf16 ? launch_recurrent<__nv_bfloat16>(p, s) : launch_recurrent<float>(p, s);
}
cudaError_t launch_delta_decode(const DeltaPlan &p, cudaStream_t s) {
  return p.bf16 ? launch_decode<__nv_bfloat16>(p, s) : launch_decode<float>(p, s);
}

// Through kernel parameters: a copy from the caller's memory could not be captured without keeping it.  A
// launch costs more the more parameters it has.
cudaError_t launch_put_ints(int *dst, const int *host, int n, cudaStream_t s) {
  for (; n > 960; n -= 960, dst += 960, host += 960) put<960>(dst, host, 960, s);
  if (n <= 64) put<64>(dst, host, n, s);
  else if (n <= 256) put<256>(dst, host, n, s);
  else put<960>(dst, host, n, s);
  return cudaGetLastError();
}

}  // namespace ssd
