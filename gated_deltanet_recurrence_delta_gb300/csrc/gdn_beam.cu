// gdn_beam_select: the best continuations of each group's beams.
//
//   cand(w, x) = score_w + logit_wx - lse_w,  lse_w = log sum_x exp(logit_wx);
//   the best `beams` of a group, ties to the lowest (w, x)
//
// Memory-bound: each logit is read once. Within a row candidates rank as their
// logits do, so a slice of a row (at most 8192 logits, kept in registers)
// yields its maximum, its sum of exponentials and its best `beams` logits in
// one pass; a second kernel joins a group's slices and ranks its candidates in
// 64 bits, where alone different rows meet.
//
// A slice's best: a CTA's threads form 32 parts; every logit at or above the
// `beams`-th largest of the parts' maxima is a candidate. At least `beams` logits
// are, so the best are among them; for unordered logits hardly more than that
// are. Each counts how many of them are better. Equal logits in numbers beyond
// the list are taken one round of the whole CTA each.
#include <cuda_fp16.h>

#include "gdn_check.h"

namespace gdn {
namespace beam {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 32;                  // logits a thread holds
constexpr int kSlice = kThreads * kPer;   // logits of the largest slice
constexpr int kMaxBeams = 32;
constexpr int kParts = 32, kLanes = kThreads / kParts;
constexpr int kList = 1024;

struct Args {
  int groups, beams, V, eos, slices;
  long long stride;
  const void *logits;
  const float *scores;
  const uint8_t *done;
  int32_t *parent, *token;
  float *new_scores;
  uint8_t *new_done;
  float2 *stats;   // [rows][slices]: maximum, sum of exp(logit - maximum)
  float *best;     // [rows][slices][beams], best first; -inf where there are fewer
  int32_t *best_at;
};

__device__ __forceinline__ bool better(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

template <bool HALF>
__device__ __forceinline__ float logit(const void *p, long long i) {
  return HALF ? ldbf(static_cast<const bf16 *>(p) + i) : static_cast<const float *>(p)[i];
}

// Slice blockIdx.x of row blockIdx.y. A thread holds kPer / C runs of C logits
// (16 bytes), run k at C (k kThreads + tid) from the slice's start.
template <bool HALF>
__global__ void __launch_bounds__(kThreads) slice_kernel(const __grid_constant__ Args A) {
  constexpr int C = HALF ? 8 : 4, RUNS = kPer / C;
  __shared__ float s_max[kParts], s_red[kWarps], s_sum[kWarps], s_cut;
  __shared__ float s_val[kList];
  __shared__ int s_at[kList], s_n, s_pick[kWarps];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  const long long row = blockIdx.y;
  const float score = A.scores[row];
  if (!(score > -INFINITY) || (A.done && A.done[row])) return;  // its logits give no candidates
  const long long runs = (A.V + C - 1) / C;  // 16 bytes each, dealt out evenly
  const int i0 = C * (int)(runs * slice / A.slices), i1 = min(A.V, C * (int)(runs * (slice + 1) / A.slices));
  const long long base = row * A.stride;
  const char *p = static_cast<const char *>(A.logits) + base * (HALF ? 2 : 4);
  const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15) == 0;  // and so is every run then
  float v[kPer];
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const int i = i0 + C * (k * kThreads + tid);
    if (aligned && i + C <= i1) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p + (long long)i * (HALF ? 2 : 4)));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (HALF) {
          v[k * C + 2 * j] = __uint_as_float(w[j] << 16);
          v[k * C + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[k * C + j] = __uint_as_float(w[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) v[k * C + j] = i + j < i1 ? logit<HALF>(p, i + j) : -INFINITY;
    }
  }
  // ---- the slice's maximum and the parts' maxima (a NaN is no maximum, but reaches the sum)
  float top = v[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) top = fmaxf(top, v[j]);
  if (top != top) top = -INFINITY;
  if (tid == 0) s_n = 0;
  float part = top;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) part = fmaxf(part, __shfl_xor_sync(0xffffffffu, part, o));
  if (tid % kLanes == 0) s_max[tid / kLanes] = part;
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) part = fmaxf(part, __shfl_xor_sync(0xffffffffu, part, o));
  if (lane == 0) s_red[warp] = part;
  __syncthreads();
  float m = s_red[0];
#pragma unroll
  for (int j = 1; j < kWarps; ++j) m = fmaxf(m, s_red[j]);
  const float ref = m == -INFINITY ? 0.0f : m;
  if (warp == 0) {  // the part whose maximum has beams - 1 better ones
    static_assert(kParts == 32, "a part to a lane");
    const float x = s_max[lane];
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kParts; ++j) rank += better(__shfl_sync(0xffffffffu, x, j), j, x, lane);
    if (rank == A.beams - 1) s_cut = x;
  }
  __syncthreads();
  const float cut = s_cut;
  // ---- sum of exponentials, candidates
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    sum += exp2f((v[j] - ref) * 1.4426950408889634f);
    if (v[j] >= cut && v[j] > -INFINITY) {
      const int n = atomicAdd(&s_n, 1);
      if (n < kList) {
        s_val[n] = v[j];
        s_at[n] = i0 + C * (j / C * kThreads + tid) + j % C;
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  const long long at = row * A.slices + slice;
  if (tid == 0) {
    for (int j = 1; j < kWarps; ++j) sum += s_sum[j];
    A.stats[at] = make_float2(m, sum);
  }
  const int n = s_n;
  float *best = A.best + at * A.beams;
  int32_t *best_at = A.best_at + at * A.beams;
  if (n <= kList) {  // each candidate's rank among them
    for (int i = tid; i < n; i += kThreads) {
      const float x = s_val[i];
      const int ix = s_at[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += better(s_val[j], s_at[j], x, ix);
      if (rank < A.beams) {
        best[rank] = x;
        best_at[rank] = ix;
      }
    }
    for (int i = n + tid; i < A.beams; i += kThreads) {
      best[i] = -INFINITY;
      best_at[i] = -1;
    }
  } else {  // more candidates than the list holds: one after the other, the best behind the last one taken
    float last = INFINITY;
    int last_at = -1;
    for (int r = 0; r < A.beams; ++r) {
      float x = -INFINITY;
      int ix = 0x7fffffff;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int ij = i0 + C * (j / C * kThreads + tid) + j % C;
        if (v[j] > -INFINITY && better(last, last_at, v[j], ij) && better(v[j], ij, x, ix)) {
          x = v[j];
          ix = ij;
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        const int iy = __shfl_xor_sync(0xffffffffu, ix, o);
        if (better(y, iy, x, ix)) {
          x = y;
          ix = iy;
        }
      }
      __syncthreads();
      if (lane == 0) {
        s_red[warp] = x;
        s_pick[warp] = ix;
      }
      __syncthreads();
      for (int j = 0; j < kWarps; ++j)
        if (better(s_red[j], s_pick[j], x, ix)) {
          x = s_red[j];
          ix = s_pick[j];
        }
      last = x;
      last_at = ix;
      if (tid == 0) {
        best[r] = x;
        best_at[r] = x > -INFINITY ? ix : -1;
      }
    }
  }
}

// A score as a whole number of the same order; 0 is below every candidate's.
__device__ __forceinline__ unsigned long long key_of(double x) {
  const long long b = __double_as_longlong(x);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
__device__ __forceinline__ double score_of(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & 0x7fffffffffffffffull : ~k));
}

// Group blockIdx.x: joins its rows' slices, and takes its best candidates one
// after the other.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args A) {
  __shared__ double s_add[kMaxBeams];  // score - lse of a beam
  __shared__ unsigned long long s_key[kWarps];
  __shared__ int s_idx[kWarps];
  __shared__ uint8_t s_done[kMaxBeams];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = A.beams, S = A.slices;
  const long long row0 = (long long)blockIdx.x * W;
  for (int w = warp; w < W; w += kWarps) {
    const float score = A.scores[row0 + w];
    const bool over = A.done && A.done[row0 + w];
    double add = -INFINITY;
    if (over) {
      add = score;
    } else if (score > -INFINITY) {
      const float2 *st = A.stats + (row0 + w) * S;
      float m = -INFINITY;
      for (int i = lane; i < S; i += 32) m = fmaxf(m, st[i].x);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double sum = 0.0;
      for (int i = lane; i < S; i += 32) sum += (double)st[i].y * exp((double)st[i].x - (double)m);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      add = (double)score - ((double)m + log(sum));
    }
    if (lane == 0) {
      s_add[w] = add;
      s_done[w] = over;
    }
  }
  __syncthreads();
  // Candidate c < W S W: place c % W of slice c / W % S of beam c / (W S); its order among equals is (beam, token).
  const int N = W * S * W;
  unsigned long long last = ~0ull;  // the candidate taken last
  int last_at = -1;
  for (int r = 0; r < W; ++r) {
    unsigned long long key = 0;
    int at = 0x7fffffff;  // beam * 2^24 + token
    auto offer = [&](double x, int ix) {
      if (!(x > -INFINITY)) return;  // -inf, NaN
      const unsigned long long k = key_of(x);
      if ((k < last || (k == last && ix > last_at)) && (k > key || (k == key && ix < at))) {
        key = k;
        at = ix;
      }
    };
    for (int c = tid; c < N; c += kThreads) {
      const int w = c / (W * S);
      if (s_done[w]) continue;
      const int t = A.best_at[row0 * S * W + c];
      if (s_add[w] > -INFINITY && t >= 0) offer(s_add[w] + (double)A.best[row0 * S * W + c], (w << 24) + t);
    }
    if (tid < W && s_done[tid]) offer(s_add[tid], (tid << 24) + max(A.eos, 0));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
      const int i = __shfl_xor_sync(0xffffffffu, at, o);
      if (k > key || (k == key && i < at)) {
        key = k;
        at = i;
      }
    }
    __syncthreads();
    if (lane == 0) {
      s_key[warp] = key;
      s_idx[warp] = at;
    }
    __syncthreads();
    for (int j = 0; j < kWarps; ++j)
      if (s_key[j] > key || (s_key[j] == key && s_idx[j] < at)) {
        key = s_key[j];
        at = s_idx[j];
      }
    last = key;
    last_at = at;
    if (tid == 0) {
      const bool none = key == 0;
      const int w = none ? r : at >> 24, t = none ? -1 : s_done[w] ? A.eos : at & 0xffffff;
      A.parent[row0 + r] = (int)(row0 + w);
      A.token[row0 + r] = t;
      A.new_scores[row0 + r] = none ? -INFINITY : (float)score_of(key);
      if (A.new_done) A.new_done[row0 + r] = !none && (s_done[w] || t == A.eos);
    }
    if (key == 0) last = 0;  // nothing is left
  }
}

gdn_status check_dims(const gdn_beam_dims *d) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->beams < 1 || d->beams > kMaxBeams) return fail(GDN_ERR_SHAPE, "beams must be in [1, 32]");
  if (d->n_groups < 0 || (long long)d->n_groups * d->beams > 65535)
    return fail(GDN_ERR_SHAPE, "n_groups * beams must be in [0, 65535]");
  if (d->vocab < 1 || d->vocab > (1 << 24)) return fail(GDN_ERR_SHAPE, "vocab must be in [1, 2^24]");
  if (d->eos < -1 || d->eos >= d->vocab) return fail(GDN_ERR_SHAPE, "eos must be in [-1, vocab)");
  if (d->row_stride < d->vocab || d->row_stride >= (1LL << 40))
    return fail(GDN_ERR_SHAPE, "row_stride must be at least vocab, and below 2^40");
  return GDN_OK;
}

// Slices of a row: as few as the registers allow, more where the rows alone would leave SMs idle.
int slices_of(const gdn_beam_dims *d) {
  const long long rows = (long long)d->n_groups * d->beams;
  int n = (d->vocab + kSlice - 1) / kSlice;
  while (rows * n < 304 && d->vocab / (2 * n) >= 2048) n *= 2;
  return n;
}

}  // namespace beam
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_beam_workspace_size(const gdn_beam_dims *dims) {
  if (beam::check_dims(dims) != GDN_OK) return 0;
  return (size_t)dims->n_groups * dims->beams * beam::slices_of(dims) * (8 + 8 * (size_t)dims->beams);
}

extern "C" gdn_status gdn_beam_select(const gdn_beam_dims *dims, const void *logits, const float *scores,
                                      const uint8_t *done, int32_t *parent, int32_t *token, float *new_scores,
                                      uint8_t *new_done, void *workspace, size_t workspace_bytes, void *stream) {
  GDN_TRY(beam::check_dims(dims));
  if (dims->n_groups == 0) return GDN_OK;  // empty tensors may have no address
  GDN_TRY(check_ptr(logits, "logits", dims->half ? 2 : 4));
  GDN_TRY(check_ptr(scores, "scores", 4));
  GDN_TRY(check_ptr(parent, "parent", 4));
  GDN_TRY(check_ptr(token, "token", 4));
  GDN_TRY(check_ptr(new_scores, "new_scores", 4));
  if ((done == nullptr) != (new_done == nullptr))
    return fail(GDN_ERR_ARG, "done and new_done must both be given or both be NULL");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < gdn_beam_workspace_size(dims))
    return fail(GDN_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdn_beam_workspace_size");
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  (void)dev;
  beam::Args A = {};
  A.groups = dims->n_groups;
  A.beams = dims->beams;
  A.V = dims->vocab;
  A.eos = dims->eos;
  A.slices = beam::slices_of(dims);
  A.stride = dims->row_stride;
  A.logits = logits;
  A.scores = scores;
  A.done = done;
  A.parent = parent;
  A.token = token;
  A.new_scores = new_scores;
  A.new_done = new_done;
  const size_t rows = (size_t)dims->n_groups * dims->beams;
  A.stats = static_cast<float2 *>(workspace);
  A.best = reinterpret_cast<float *>(A.stats + rows * A.slices);
  A.best_at = reinterpret_cast<int32_t *>(A.best + rows * A.slices * dims->beams);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(A.slices, (unsigned)rows), block(beam::kThreads);
  if (launch_pdl(dims->half ? beam::slice_kernel<true> : beam::slice_kernel<false>, grid, block, 0, st, A) != cudaSuccess)
    return check_launch("beam_select");
  launch_pdl(beam::join_kernel, dim3(A.groups), block, 0, st, A);
  return check_launch("beam_select");
}
