// delta_plan.h -- resolved launch parameters of the gated delta rule and of the 8-bit state cache.
#pragma once

#include <cuda_runtime.h>

#include "../../include/ssd.h"

namespace ssd {

// Tokens per chunk of the tensor-core kernel.
constexpr int kDeltaChunk = 64;
// One chunk's workspace records, written by the front end and read by the chunk kernel:
//  tile    per (chunk, group): the fp16 operand image of 64 key and 64 query rows, 16 of each in turn, two
//          halves of 64 columns, each 128 rows x 128 bytes with the 128-byte swizzle; then the row
//          factors rho_k[64], rho_q[64] (fp32)
//  record  per (chunk, head): the triangles of T~^T (its columns i >= its rows j) and A T (rows t >= columns j) as
//          operand images in blocks of 16 rows x 16 columns, 512 bytes: [row / 8][column / 8][row % 8][column % 8]
//          halves.  T~^T: for each 16 columns kb the row blocks 0 .. kb of hi, then of lo.  A T: for each 16
//          columns kb the row blocks kb .. 3.  Then u = beta rho_k [64], 2^cs [64] and w = u 2^{cs at the chunk's
//          end - cs} [64] (fp32).
constexpr long long kDeltaTileBytes = 32768 + 512;
constexpr int kDeltaTBytes = 20 * 512, kDeltaATBytes = 10 * 512;
constexpr long long kDeltaRecordBytes = kDeltaTBytes + kDeltaATBytes + 3 * 256;

struct DeltaPlan {
  int B, L, H, P, G, hpg;  // L: the longest sequence of a packed batch
  // packed batch: sequence b is token rows cu[b] .. cu[b+1]-1, its chunks are chunk0[b] ..,
  // and CTAs take the sequences in the order order[] (longest first); all on the device, null
  // for a uniform batch
  const int *cu, *chunk0, *order;
  long long rows;      // token rows
  long long n_chunks;  // over all sequences
  int heads_per_cta;   // of the front end
  int qk_norm;
  float qk_eps, q_scale;
  float dt_min, dt_max;
  int softplus, beta_sigmoid;
  float beta_scale;
  bool bf16;
  const void *q, *k, *v, *dt, *b;
  long long qs, ks, vs, ds, bs;  // row strides in elements
  const float *A, *dt_bias;
  const float *h0;
  float *h_final;      // null: not wanted
  void *y;
  long long ys;
  // decode: the pool of states, updated in place
  const int *slots;
  int n_slots;
  // workspace of the chunked kernel
  unsigned char *tiles, *records;
  int *err;
  // elements of the y and state buffers, for the debug build's index checks
  long long y_extent, state_extent;
};

// token recurrence in fp32 (delta_simt.cu)
cudaError_t launch_delta_recurrent(const DeltaPlan &p, cudaStream_t s);
cudaError_t launch_delta_decode(const DeltaPlan &p, cudaStream_t s);

// chunked on the tensor cores: the front end (delta_prep.cu) writes tiles and records, the chunks follow
// (delta_tc.cu)
cudaError_t launch_delta_front(const DeltaPlan &p, cudaStream_t s);
cudaError_t launch_delta_chunks(const DeltaPlan &p, cudaStream_t s);

struct StateCachePlan {
  ssd_state_format_t format;
  long long elems;
  int count, n_states, n_cache;
  const int *state_slots, *cache_slots;
  float *states;
  unsigned char *cache, *scales;
  int *err;
  long long cache_extent, states_extent;  // bytes and elements, for the debug build's index checks
};
cudaError_t launch_state_store(const StateCachePlan &p, cudaStream_t s);
cudaError_t launch_state_load(const StateCachePlan &p, cudaStream_t s);

// Writes n host ints to device memory from kernel parameters: the values are read before the call
// returns, in a stream capture too (a copy from pageable memory would be read at each replay).
cudaError_t launch_put_ints(int *dst, const int *host, int n, cudaStream_t s);

// shared with api.cu
int *device_error_ptr();
int bounds_denom();

}  // namespace ssd
