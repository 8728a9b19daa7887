// delta_simt.cu -- the gated delta rule token by token in fp32: the decode step, short prefills and
// fp32 inputs.
//
// Per head and token, with S the P x N state and k^, q^ the normalised key and scaled query:
//   u = beta (v - alpha S k^),  y = alpha S q^ + u (k^.q^),  S <- alpha S + u k^^T.
// y is S_t q^ written with the old state, so both products with S come from one pass over it and
// one reduction, and k^.q^ is a scalar per token: the chain from token to token is one dot
// product, one reduction over a few lanes and one multiply-add.
//
// The rows of S are independent given k^, so LPR lanes hold a row (N / LPR elements each, in
// registers for the whole call) and a warp holds 32 / LPR rows.  The tokens are taken in tiles:
// the CTA reads a tile's q, k, v, dt and b into registers while it works on the tile before,
// then normalises q and k and puts all of it into shared memory, from which the token loop
// reads with broadcasts.
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

// kDecode: one token per row, the state in place in a pool; else whole sequences.
template <typename T, int LPR, int WARPS, int TT, bool kDecode>
__global__ void __launch_bounds__(WARPS * 32) delta_recurrent_kernel(const DeltaPlan p) {
  constexpr int R = WARPS * 32 / LPR;   // state rows of this CTA
  constexpr int E4 = kDState / LPR / 4; // float4s of a row per lane
  constexpr int NT = WARPS * 32;
  constexpr int TPW = (TT + WARPS - 1) / WARPS;  // tokens of a tile that a warp normalises
  constexpr int VPT = (TT * R + NT - 1) / NT;    // v elements of a tile per thread
  constexpr int NB = kDecode ? 1 : 2;
  __shared__ __align__(16) float sq[NB][TT][kDState], sk[NB][TT][kDState];
  __shared__ float sv[NB][TT][R];
  __shared__ float s_alpha[NB][TT], s_beta[NB][TT], s_kq[NB][TT];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int blocks_per_head = p.P / R;
  const int h = blockIdx.x / blocks_per_head, row0 = (blockIdx.x % blocks_per_head) * R;
  const int seq = p.order ? p.order[blockIdx.y] : (int)blockIdx.y;
  const int g = h / p.hpg;
  const int len = kDecode ? 1 : seq_len(p.cu, seq, p.L);
  const long long base = kDecode ? (long long)seq : seq_base(p.cu, seq, p.L);
  const int r = warp * (32 / LPR) + lane / LPR, s = lane % LPR;

  long long state_idx = seq;
  bool skip = false;
  if (kDecode && p.slots) {
    const int own = p.slots[seq];
    bool twice = false;  // an earlier row of the batch has this slot
    for (int j = tid; j < seq; j += NT) twice |= p.slots[j] == own;
    skip = own < 0;
    const bool bad = own >= p.n_slots || __syncthreads_or(twice && !skip);
    if (bad && !skip && tid == 0) latch_error(p.err, (int)SSD_ERR_DEVICE_BOUNDS);
    skip |= bad;
    if (skip) return;
    state_idx = own;
  }
  const long long soff = ((state_idx * p.H + h) * p.P + row0 + r) * kDState + 4 * s;

  float S[E4][4];
  const float *src = kDecode ? p.h_final : p.h0;
#pragma unroll
  for (int j = 0; j < E4; ++j) {
    if (src) {
      load4(src + soff + 4 * LPR * j, S[j]);
    } else {
      S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
    }
  }

  const float A = p.A[h], bias = p.dt_bias[h];
  const T *q = static_cast<const T *>(p.q) + g * kDState + 4 * lane;
  const T *k = static_cast<const T *>(p.k) + g * kDState + 4 * lane;
  const T *v = static_cast<const T *>(p.v) + h * p.P + row0;
  const T *dt = static_cast<const T *>(p.dt) + h;
  const T *bb = static_cast<const T *>(p.b) + h;
  float rq[TPW][4], rk[TPW][4], rv[VPT], rdt = 0.f, rb = 0.f;

  auto fetch = [&](int t0) {  // this thread's part of the tile at t0, into registers
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = t0 + warp + i * WARPS;
      if (warp + i * WARPS < TT && t < len) {
        load4(q + (base + t) * p.qs, rq[i]);
        load4(k + (base + t) * p.ks, rk[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = tid + i * NT, t = t0 + at / R;
      if (at < TT * R && t < len) rv[i] = io<T>::ld(v + (base + t) * p.vs + at % R);
    }
    if (tid < TT && t0 + tid < len) {
      rdt = io<T>::ld(dt + (base + t0 + tid) * p.ds);
      rb = io<T>::ld(bb + (base + t0 + tid) * p.bs);
    }
  };
  auto stage = [&](int t0, int buf) {  // the fetched tile into shared memory
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int at = warp + i * WARPS;
      if (at < TT && t0 + at < len) {
        float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qq = fmaf(rq[i][e], rq[i][e], qq);
          kk = fmaf(rk[i][e], rk[i][e], kk);
          qk = fmaf(rq[i][e], rk[i][e], qk);
        }
        float fq = p.q_scale, fk = 1.f;
        if (p.qk_norm) {
          fq *= 1.f / sqrtf(warp_sum(qq) + p.qk_eps);
          fk = 1.f / sqrtf(warp_sum(kk) + p.qk_eps);
        }
        qk = warp_sum(qk);
        *reinterpret_cast<float4 *>(&sq[buf][at][4 * lane]) =
            make_float4(rq[i][0] * fq, rq[i][1] * fq, rq[i][2] * fq, rq[i][3] * fq);
        *reinterpret_cast<float4 *>(&sk[buf][at][4 * lane]) =
            make_float4(rk[i][0] * fk, rk[i][1] * fk, rk[i][2] * fk, rk[i][3] * fk);
        if (lane == 0) s_kq[buf][at] = qk * fq * fk;
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = tid + i * NT;
      if (at < TT * R) sv[buf][at / R][at % R] = rv[i];
    }
    if (tid < TT) {
      float d = rdt + bias;
      if (p.softplus) d = d > 20.f ? d : log1pf(expf(d));
      d = fminf(fmaxf(d, p.dt_min), p.dt_max);
      s_alpha[buf][tid] = expf(A * d);
      s_beta[buf][tid] = p.beta_scale * (p.beta_sigmoid ? 1.f / (1.f + expf(-rb)) : rb);
    }
  };

  T *y = static_cast<T *>(p.y);
  const long long yoff = (long long)h * p.P + row0 + r;
  if (len > 0) fetch(0);
  for (int t0 = 0, buf = 0; t0 < len; t0 += TT, buf ^= NB - 1) {
    stage(t0, buf);
    __syncthreads();
    if (!kDecode && t0 + TT < len) fetch(t0 + TT);
    const int nt = min(TT, len - t0);
    for (int t = 0; t < nt; ++t) {
      float kv[E4][4], dk[2] = {0.f, 0.f}, dq[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < E4; ++j) {
        load4(&sk[buf][t][4 * (j * LPR + s)], kv[j]);
        float qv[4];
        load4(&sq[buf][t][4 * (j * LPR + s)], qv);
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
      const float alpha = s_alpha[buf][t];
      const float u = s_beta[buf][t] * (sv[buf][t][r] - alpha * dk_);
      if (s == 0) {
        const long long yo = (base + t0 + t) * p.ys + yoff;
        if (in_bounds(yo, p.y_extent, p.err)) io<T>::st(y + yo, fmaf(u, s_kq[buf][t], alpha * dq_));
      }
#pragma unroll
      for (int j = 0; j < E4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = fmaf(u, kv[j][e], alpha * S[j][e]);
    }
  }
  if (p.h_final) {
#pragma unroll
    for (int j = 0; j < E4; ++j)
      if (in_bounds(soff + 4 * LPR * j + 3, p.state_extent, p.err))
        *reinterpret_cast<float4 *>(p.h_final + soff + 4 * LPR * j) =
            make_float4(S[j][0], S[j][1], S[j][2], S[j][3]);
  }
}

template <typename T, bool kDecode>
cudaError_t launch(const DeltaPlan &p, cudaStream_t s) {
  constexpr int TT = kDecode ? 1 : 16;
  // 16 rows per CTA spread a small call over more SMs
  if ((long long)p.B * p.H * p.P <= 64 * 2 * 148) {
    delta_recurrent_kernel<T, 8, 4, TT, kDecode><<<dim3(p.H * p.P / 16, p.B), 128, 0, s>>>(p);
  } else {
    delta_recurrent_kernel<T, 4, 8, TT, kDecode><<<dim3(p.H * p.P / 64, p.B), 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

struct Ints {
  int v[960];
};
__global__ void put_ints_kernel(int *dst, const __grid_constant__ Ints src, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src.v[i];
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaPlan &p, cudaStream_t s) {
  return p.bf16 ? launch<__nv_bfloat16, false>(p, s) : launch<float, false>(p, s);
}
cudaError_t launch_delta_decode(const DeltaPlan &p, cudaStream_t s) {
  return p.bf16 ? launch<__nv_bfloat16, true>(p, s) : launch<float, true>(p, s);
}

cudaError_t launch_put_ints(int *dst, const int *host, int n, cudaStream_t s) {
  Ints a;
  for (int at = 0; at < n; at += 960) {
    const int m = n - at < 960 ? n - at : 960;
    for (int i = 0; i < m; ++i) a.v[i] = host[at + i];
    put_ints_kernel<<<1, 256, 0, s>>>(dst + at, a, m);
  }
  return cudaGetLastError();
}

}  // namespace ssd
