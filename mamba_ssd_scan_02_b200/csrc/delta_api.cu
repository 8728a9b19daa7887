// delta_api.cu -- the C ABI of the gated delta rule and of the 8-bit state cache: argument checks,
// workspace layout and launches.  Nothing here allocates device memory or synchronises.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "common.cuh"
#include "delta_plan.h"
#include "plan.h"

namespace ssd {
namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxGrid = 65535;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
ssd_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

bool ranges_overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return na && nb && pa < pb + nb && pb < pa + na;
}

// n rows of `width` bytes, `stride` bytes apart
struct Rows {
  const void *p;
  long long stride, width, n;
};
Rows dense(const void *p, long long bytes) { return Rows{p, bytes, bytes, 1}; }

// Whether two sets of rows share a byte.  Rows of equal stride may interleave (columns of one matrix); of different
// strides, overlapping spans count.
bool overlap(const Rows &a, const Rows &b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1 || a.width < 1 || b.width < 1) return false;
  if (!ranges_overlap(a.p, (size_t)((a.n - 1) * a.stride + a.width), b.p, (size_t)((b.n - 1) * b.stride + b.width))) return false;
  if (a.n == 1) {  // the first row of b that ends behind a's start, if it begins before a's end
    const long long d = (long long)(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
    const long long row = d < b.width ? 0 : (d - b.width) / b.stride + 1;
    return row < b.n && row * b.stride < d + a.width;
  }
  if (b.n == 1) return overlap(b, a);
  if (a.stride != b.stride) return true;
  long long d = (long long)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.stride;
  if (d < 0) d += a.stride;
  return d < a.width || d + b.width > a.stride;
}
// Whether `out` shares a byte with one of the others
bool overlaps_any(const Rows &out, const Rows *others, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(out, others[i])) return true;
  return false;
}

ssd_status_t check_config(const ssd_delta_config_t *c) {
  if (!c) return SSD_ERR_INVALID_ARG;
  if (c->batch < 1 || c->nheads < 1 || c->ngroups < 1 || c->seqlen < 0) return SSD_ERR_INVALID_ARG;
  if (c->nheads % c->ngroups != 0) return SSD_ERR_INVALID_ARG;
  if (c->io_dtype != SSD_F32 && c->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if ((c->headdim != 64 && c->headdim != 128) || c->dstate != kDState) return SSD_ERR_UNSUPPORTED;
  if (c->qk_norm != 0 && c->qk_norm != 1) return SSD_ERR_INVALID_ARG;
  if (c->qk_norm && !(c->qk_eps > 0.f && isfinite(c->qk_eps))) return SSD_ERR_INVALID_ARG;
  if (!isfinite(c->q_scale) || !isfinite(c->beta_scale)) return SSD_ERR_INVALID_ARG;
  if (!(c->dt_min <= c->dt_max)) return SSD_ERR_INVALID_ARG;
  if ((c->dt_softplus != 0 && c->dt_softplus != 1) || (c->beta_sigmoid != 0 && c->beta_sigmoid != 1))
    return SSD_ERR_INVALID_ARG;
  if (c->kernel != SSD_KERNEL_AUTO && c->kernel != SSD_KERNEL_SIMT && c->kernel != SSD_KERNEL_TENSOR)
    return SSD_ERR_INVALID_ARG;
  if (c->batch > kMaxGrid || c->nheads > kMaxGrid || c->seqlen > (1 << 30)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// A uniform batch, or packed sequences with host offsets cu[0..nseq].
struct Batch {
  const int *cu;
  int nseq, longest;
  long long rows, chunks;
};

Batch uniform(const ssd_delta_config_t *c) {
  const long long nc = (c->seqlen + kDeltaChunk - 1) / kDeltaChunk;
  return Batch{nullptr, c->batch, c->seqlen, (long long)c->batch * c->seqlen, c->batch * nc};
}

bool packed(const ssd_delta_config_t *c, const int *cu, int nseq, Batch *b) {
  if (!c || !cu || nseq < 1 || c->batch != 1 || cu[0] != 0 || cu[nseq] != c->seqlen) return false;
  *b = Batch{cu, nseq, 0, cu[nseq], 0};
  for (int i = 0; i < nseq; ++i) {
    const long long n = (long long)cu[i + 1] - cu[i];
    if (n < 0) return false;
    b->longest = std::max(b->longest, (int)n);
    b->chunks += (n + kDeltaChunk - 1) / kDeltaChunk;
  }
  return true;
}

// The longest sequence from which AUTO takes the chunked kernels.  They cost two launches and a chunk's latency
// (15 us); the recurrence costs its longest sequence, times its CTAs per SM once the state rows are more than
// one CTA per SM holds.  Both in us, bf16, at 64, 96, 128 tokens: 8 heads of 64 rows 9.3 : 15.0, 12.4 : 16.5,
// 15.6 : 16.6; at 16, 32, 64 tokens: 4 sequences of 32 heads 11.6 : 16.8, 18.4 : 16.9, 31.7 : 17.1.  Short sequences
// beside the longest change little, since a state in and out is most of what either costs them: 63 of one token
// and one of 28 tokens, 128 heads 387 : 324, 32 heads 94.5 : 97.3; 255 and one, 128 heads 1503 : 1212; 7 and one, 32
// heads 18.6 : 24.7, the most that the rule loses.
bool uses_chunks(const ssd_delta_config_t *c, const Batch &b) {
  if (b.rows == 0 || c->kernel == SSD_KERNEL_SIMT) return false;
  if (c->kernel == SSD_KERNEL_TENSOR) return true;
  // Their operands are bounded where beta |k|^2 is, by 2, and alpha, by 1; AUTO takes them where the configuration says
  // so.  (That A <= 0 is taken for granted: it is on the device.)
  const bool steps = c->dt_min >= 0.f || (c->dt_softplus && c->dt_max >= 0.f);  // dt >= 0
  const bool bounded = steps && c->qk_norm && c->beta_sigmoid && c->beta_scale >= 0.f && c->beta_scale <= 2.f;
  const bool one_each = (long long)b.nseq * c->nheads * c->headdim <= 16 * 148;
  return c->io_dtype == SSD_BF16 && bounded && b.longest >= (one_each ? 128 : 28) && tc_scan_available();
}

struct Layout {
  size_t tiles, records, ints, total;
};

Layout layout(const ssd_delta_config_t *c, const Batch &b) {
  Layout l{};
  size_t off = 0;
  if (uses_chunks(c, b)) {
    l.tiles = off;
    off = round_up(off + (size_t)(b.chunks * c->ngroups * kDeltaTileBytes), kAlign);
    l.records = off;
    off = round_up(off + (size_t)(b.chunks * c->nheads * kDeltaRecordBytes), kAlign);
  }
  l.ints = off;
  if (b.cu) off = round_up(off + (size_t)(3 * (long long)b.nseq + 2) * sizeof(int), kAlign);
  l.total = off;
  return l;
}

void fill(DeltaPlan &p, const ssd_delta_config_t *c) {
  p.H = c->nheads; p.P = c->headdim; p.G = c->ngroups; p.hpg = c->nheads / c->ngroups;
  p.qk_norm = c->qk_norm; p.qk_eps = c->qk_eps; p.q_scale = c->q_scale;
  p.dt_min = c->dt_min; p.dt_max = c->dt_max; p.softplus = c->dt_softplus;
  p.beta_sigmoid = c->beta_sigmoid; p.beta_scale = c->beta_scale;
  p.bf16 = c->io_dtype == SSD_BF16;
  p.err = device_error_ptr();
}

// The extent that the debug build's index checks allow for a buffer of n elements.
long long extent(long long n) { return n / bounds_denom(); }

template <class Args>
ssd_status_t check_rows(const ssd_delta_config_t *c, const Args *a, long long rows) {
  const long long qk = (long long)c->ngroups * kDState, w = (long long)c->nheads * c->headdim;
  if (!a->q || !a->k || !a->v || !a->dt || !a->b || !a->A || !a->dt_bias || !a->y) return SSD_ERR_INVALID_ARG;
  if (a->q_row_stride < qk || a->k_row_stride < qk || a->v_row_stride < w || a->dt_row_stride < c->nheads ||
      a->b_row_stride < c->nheads || a->y_row_stride < w)
    return SSD_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->y, 16) || a->q_row_stride % 8 ||
      a->k_row_stride % 8 || a->v_row_stride % 8 || a->y_row_stride % 8)
    return SSD_ERR_ALIGNMENT;
  const uintptr_t es = c->io_dtype == SSD_F32 ? 4 : 2;
  if (!aligned(a->dt, es) || !aligned(a->b, es) || !aligned(a->A, 4) || !aligned(a->dt_bias, 4)) return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}

// What a call reads but the states and slots, and y
constexpr int kInputs = 7;
template <class Args>
void input_rows(const ssd_delta_config_t *c, const Args *a, long long rows, Rows *in) {
  const long long e = c->io_dtype == SSD_F32 ? 4 : 2, qk = c->ngroups * kDState * e, H = c->nheads;
  in[0] = Rows{a->q, a->q_row_stride * e, qk, rows};
  in[1] = Rows{a->k, a->k_row_stride * e, qk, rows};
  in[2] = Rows{a->v, a->v_row_stride * e, H * c->headdim * e, rows};
  in[3] = Rows{a->dt, a->dt_row_stride * e, H * e, rows};
  in[4] = Rows{a->b, a->b_row_stride * e, H * e, rows};
  in[5] = dense(rows > 0 ? a->A : nullptr, 4 * H);
  in[6] = dense(rows > 0 ? a->dt_bias : nullptr, 4 * H);
}
template <class Args>
Rows y_rows(const ssd_delta_config_t *c, const Args *a, long long rows) {
  const long long e = c->io_dtype == SSD_F32 ? 4 : 2;
  return Rows{a->y, a->y_row_stride * e, (long long)c->nheads * c->headdim * e, rows};
}

template <class Args>
void fill_rows(DeltaPlan &p, const Args *a) {
  p.q = a->q; p.qs = a->q_row_stride; p.k = a->k; p.ks = a->k_row_stride; p.v = a->v; p.vs = a->v_row_stride;
  p.dt = a->dt; p.ds = a->dt_row_stride; p.b = a->b; p.bs = a->b_row_stride;
  p.A = a->A; p.dt_bias = a->dt_bias; p.y = a->y; p.ys = a->y_row_stride;
}

ssd_status_t run_prefill(const ssd_delta_config_t *c, const ssd_delta_args_t *a, const Batch &b, cudaStream_t s) {
  if (!a) return SSD_ERR_INVALID_ARG;
  if (c->kernel == SSD_KERNEL_TENSOR && (c->io_dtype != SSD_BF16 || !tc_scan_available())) return SSD_ERR_UNSUPPORTED;
  if (b.rows > 0) {
    const ssd_status_t st = check_rows(c, a, b.rows);
    if (st != SSD_OK) return st;
  }
  if (!aligned(a->h0, 16) || !aligned(a->h_final, 16)) return SSD_ERR_ALIGNMENT;
  const long long state = (long long)b.nseq * c->nheads * c->headdim * kDState * (long long)sizeof(float);
  Rows in[kInputs + 1];
  input_rows(c, a, b.rows, in);
  in[kInputs] = dense(a->h0, state);
  const Rows y = y_rows(c, a, b.rows), h_final = dense(a->h_final, state);
  if (overlaps_any(y, in, kInputs + 1) || overlap(y, h_final) || overlaps_any(h_final, in, kInputs) ||
      (a->h0 != a->h_final && overlap(h_final, in[kInputs])))
    return SSD_ERR_INVALID_ARG;
  if ((long long)b.nseq * c->nheads * (c->headdim / 64) > 1 << 30) return SSD_ERR_UNSUPPORTED;
  const Layout l = layout(c, b);
  if (l.total && (!a->workspace || a->workspace_bytes < l.total || !aligned(a->workspace, kAlign)))
    return SSD_ERR_WORKSPACE;
  const Rows scratch = dense(a->workspace, (long long)l.total);
  if (overlaps_any(scratch, in, kInputs + 1) || overlap(scratch, y) || overlap(scratch, h_final)) return SSD_ERR_INVALID_ARG;
  if (b.rows == 0 && !a->h_final) return SSD_OK;

  DeltaPlan p{};
  fill(p, c);
  fill_rows(p, a);
  p.B = b.nseq; p.L = b.longest; p.rows = b.rows; p.n_chunks = b.chunks;
  p.h0 = a->h0; p.h_final = a->h_final;
  p.y_extent = extent(b.rows > 0 ? (b.rows - 1) * a->y_row_stride + (long long)p.H * p.P : 0);
  p.state_extent = extent((long long)b.nseq * p.H * p.P * kDState);
  char *ws = static_cast<char *>(a->workspace);
  if (b.cu) {
    // offsets, first chunks, and the sequences by falling length: the longest start first
    std::vector<int> ints;
    try {
      ints.resize(3 * (size_t)b.nseq + 2);
    } catch (const std::bad_alloc &) {
      return SSD_ERR_INVALID_ARG;
    }
    int *cu = ints.data(), *first = cu + b.nseq + 1, *order = first + b.nseq + 1;
    first[0] = 0;
    for (int i = 0; i <= b.nseq; ++i) cu[i] = b.cu[i];
    for (int i = 0; i < b.nseq; ++i) {
      first[i + 1] = first[i] + (cu[i + 1] - cu[i] + kDeltaChunk - 1) / kDeltaChunk;
      order[i] = i;
    }
    std::sort(order, order + b.nseq, [&](int x, int y) {
      const int nx = cu[x + 1] - cu[x], ny = cu[y + 1] - cu[y];
      return nx != ny ? nx > ny : x < y;
    });
    int *dev = reinterpret_cast<int *>(ws + l.ints);
    const cudaError_t e = traced("ssd_put_ints", s, [&] { return launch_put_ints(dev, ints.data(), (int)ints.size(), s); });
    if (e != cudaSuccess) return SSD_ERR_CUDA;
    p.cu = dev; p.chunk0 = dev + b.nseq + 1; p.order = p.chunk0 + b.nseq + 1;
  }
  if (uses_chunks(c, b)) {
    p.tiles = reinterpret_cast<unsigned char *>(ws + l.tiles);
    p.records = reinterpret_cast<unsigned char *>(ws + l.records);
    const cudaError_t e = traced("ssd_delta_front", s, [&] { return launch_delta_front(p, s); });
    if (e != cudaSuccess) return SSD_ERR_CUDA;
    return from_cuda(traced("ssd_delta_chunks", s, [&] { return launch_delta_chunks(p, s); }));
  }
  return from_cuda(traced("ssd_delta_recurrent", s, [&] { return launch_delta_recurrent(p, s); }));
}

ssd_status_t run_decode(const ssd_delta_config_t *c, const ssd_delta_decode_args_t *a, cudaStream_t s) {
  ssd_status_t st = check_config(c);
  if (st != SSD_OK) return st;
  if (!a || !a->state) return SSD_ERR_INVALID_ARG;
  if ((st = check_rows(c, a, c->batch)) != SSD_OK) return st;
  if (a->n_slots < 1 || (!a->slots && a->n_slots < c->batch)) return SSD_ERR_INVALID_ARG;
  if (!aligned(a->state, 16) || !aligned(a->slots, 4)) return SSD_ERR_ALIGNMENT;
  Rows in[kInputs];
  input_rows(c, a, c->batch, in);
  const Rows y = y_rows(c, a, c->batch), slots = dense(a->slots, 4LL * c->batch);
  const Rows states = dense(a->state, (long long)a->n_slots * c->nheads * c->headdim * kDState * 4);
  if (overlaps_any(y, in, kInputs) || overlap(y, slots) || overlap(y, states) || overlaps_any(states, in, kInputs) ||
      overlap(states, slots))
    return SSD_ERR_INVALID_ARG;
  DeltaPlan p{};
  fill(p, c);
  fill_rows(p, a);
  p.B = c->batch; p.L = 1; p.rows = c->batch;
  p.h_final = a->state; p.slots = a->slots; p.n_slots = a->n_slots;
  p.y_extent = extent((p.rows - 1) * p.ys + (long long)p.H * p.P);
  p.state_extent = extent((long long)p.n_slots * p.H * p.P * kDState);
  return from_cuda(traced("ssd_delta_decode", s, [&] { return launch_delta_decode(p, s); }));
}

ssd_status_t run_state_cache(const ssd_state_cache_args_t *a, bool store, cudaStream_t s) {
  if (!a) return SSD_ERR_INVALID_ARG;
  if (a->format != SSD_STATE_E4M3 && a->format != SSD_STATE_INT8) return SSD_ERR_INVALID_ARG;
  if (a->count < 0 || a->state_elems < 128 || a->state_elems % 128 != 0) return SSD_ERR_INVALID_ARG;
  if (a->count == 0) return SSD_OK;
  if (!a->states || !a->cache || !a->scales || a->n_states < 1 || a->n_cache < 1) return SSD_ERR_INVALID_ARG;
  if ((!a->state_slots && a->n_states < a->count) || (!a->cache_slots && a->n_cache < a->count)) return SSD_ERR_INVALID_ARG;
  if (a->count > kMaxGrid || a->state_elems > (1LL << 40)) return SSD_ERR_UNSUPPORTED;
  if (!aligned(a->states, 16) || !aligned(a->cache, 16) || !aligned(a->scales, 4) || !aligned(a->state_slots, 4) ||
      !aligned(a->cache_slots, 4))
    return SSD_ERR_ALIGNMENT;
  // (below 2^62 bytes: sizes that no memory has would wrap around in the checks)
  if (a->state_elems > (1LL << 60) / std::max(a->n_states, a->n_cache)) return SSD_ERR_UNSUPPORTED;
  const Rows states = dense(a->states, 4 * a->state_elems * a->n_states), cache = dense(a->cache, a->state_elems * a->n_cache);
  const Rows scales = dense(a->scales, a->state_elems / 32 * a->n_cache);
  const Rows slots[] = {dense(a->state_slots, 4LL * a->count), dense(a->cache_slots, 4LL * a->count)};
  if (overlap(states, cache) || overlap(states, scales) || overlap(cache, scales)) return SSD_ERR_INVALID_ARG;
  if (store ? overlaps_any(cache, slots, 2) || overlaps_any(scales, slots, 2) : overlaps_any(states, slots, 2))
    return SSD_ERR_INVALID_ARG;
  StateCachePlan p{a->format, a->state_elems, a->count, a->n_states, a->n_cache, a->state_slots, a->cache_slots,
                   a->states, static_cast<unsigned char *>(a->cache), a->scales, device_error_ptr(),
                   extent(a->n_cache * a->state_elems), extent(a->n_states * a->state_elems)};
  if (store) return from_cuda(traced("ssd_state_store", s, [&] { return launch_state_store(p, s); }));
  return from_cuda(traced("ssd_state_load", s, [&] { return launch_state_load(p, s); }));
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_delta_workspace_size(const ssd_delta_config_t *cfg) {
  if (check_config(cfg) != SSD_OK) return 0;
  return layout(cfg, uniform(cfg)).total;
}

ssd_status_t ssd_delta_prefill(const ssd_delta_config_t *cfg, const ssd_delta_args_t *args, void *stream) {
  const ssd_status_t st = check_config(cfg);
  if (st != SSD_OK) return st;
  return run_prefill(cfg, args, uniform(cfg), static_cast<cudaStream_t>(stream));
}

size_t ssd_delta_varlen_workspace_size(const ssd_delta_config_t *cfg, const int *cu_seqlens, int nseq) {
  Batch b;
  if (check_config(cfg) != SSD_OK || !packed(cfg, cu_seqlens, nseq, &b)) return 0;
  return layout(cfg, b).total;
}

ssd_status_t ssd_delta_prefill_varlen(const ssd_delta_config_t *cfg, const ssd_delta_args_t *args,
                                      const int *cu_seqlens, int nseq, void *stream) {
  const ssd_status_t st = check_config(cfg);
  if (st != SSD_OK) return st;
  Batch b;
  if (!packed(cfg, cu_seqlens, nseq, &b)) return SSD_ERR_INVALID_ARG;
  if (nseq > kMaxGrid) return SSD_ERR_UNSUPPORTED;
  return run_prefill(cfg, args, b, static_cast<cudaStream_t>(stream));
}

ssd_status_t ssd_delta_decode_step(const ssd_delta_config_t *cfg, const ssd_delta_decode_args_t *args, void *stream) {
  return run_decode(cfg, args, static_cast<cudaStream_t>(stream));
}

ssd_status_t ssd_state_store(const ssd_state_cache_args_t *args, void *stream) {
  return run_state_cache(args, true, static_cast<cudaStream_t>(stream));
}

ssd_status_t ssd_state_load(const ssd_state_cache_args_t *args, void *stream) {
  return run_state_cache(args, false, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
