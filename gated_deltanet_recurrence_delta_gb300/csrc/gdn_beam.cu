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
// A slice's best: a CTA's threads form P >= `beams` parts (8, 16 or 32); every logit
// at or above the smallest of the parts' maxima is a candidate. That is one a part
// at least, so the best `beams` are among them, and P ln P or so of unordered
// logits. Each counts how many of them are better. Equal logits in numbers beyond
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 in one register pair, and the paired instructions.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 bytes of logits: 4 fp32, or 8 bf16 that stay packed.
template <bool HALF>
struct Run {
  static constexpr int C = HALF ? 8 : 4;
  uint4 w;
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (HALF)
      return __uint_as_float(i & 1 ? word(i / 2) & 0xffff0000u : word(i / 2) << 16);
    else
      return __uint_as_float(word(i));
  }
  __device__ __forceinline__ float top() const {  // a NaN is no maximum unless all are
    if constexpr (HALF) {
      auto h = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
      const __nv_bfloat162 m = __hmax2(__hmax2(h(w.x), h(w.y)), __hmax2(h(w.z), h(w.w)));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3)));
    }
  }
};

// Slice blockIdx.x of row blockIdx.y: run k of a thread is run k kThreads + tid of the slice.
template <bool HALF>
__global__ void __launch_bounds__(kThreads, HALF ? 5 : 4) slice_kernel(const __grid_constant__ Args A) {
  constexpr int C = Run<HALF>::C, RUNS = kPer / C, B = HALF ? 2 : 4;
  __shared__ float s_max[kParts], s_red[kWarps], s_sum[kWarps];
  __shared__ uint4 s_run[kList / C];
  __shared__ int s_run_at[kList / C], s_runs, s_n, s_pick[kWarps];
  __shared__ float s_val[kList];
  __shared__ int s_at[kList];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  const long long row = blockIdx.y;
  const float score = A.scores[row];
  if (!(score > -INFINITY) || (A.done && A.done[row])) return;  // its logits give no candidates
  const long long runs = (A.V + C - 1) / C;  // 16 bytes each, dealt out evenly
  const int i0 = C * (int)(runs * slice / A.slices), i1 = min(A.V, C * (int)(runs * (slice + 1) / A.slices));
  const char *p = static_cast<const char *>(A.logits) + row * A.stride * B;
  const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15) == 0;  // and so is every run then
  Run<HALF> v[RUNS];
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    const int i = i0 + C * (k * kThreads + tid);
    if (aligned && i + C <= i1) {
      v[k].w = __ldcs(reinterpret_cast<const uint4 *>(p + (long long)i * B));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if constexpr (HALF) {
          const uint32_t x = i + j < i1 ? *reinterpret_cast<const unsigned short *>(p + (long long)(i + j) * 2) : 0xff80u;
          w[j / 2] = j & 1 ? w[j / 2] | x << 16 : x;
        } else {
          w[j] = i + j < i1 ? *reinterpret_cast<const uint32_t *>(p + (long long)(i + j) * 4) : 0xff800000u;
        }
      }
      v[k].w = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // ---- the slice's maximum and the parts' maxima (a NaN is no maximum, but reaches the sum)
  float most[RUNS], top = -INFINITY;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    most[k] = v[k].top();
    top = fmaxf(top, most[k]);
  }
  float part = top;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) part = fmaxf(part, __shfl_xor_sync(0xffffffffu, part, o));
  if (tid % kLanes == 0) s_max[tid / kLanes] = part;
  if (tid == 0) s_n = s_runs = 0;
  __syncthreads();
  float m = s_max[lane];
  static_assert(kParts == 32, "a part to a lane");
  float cut = m;  // every warp finds it: the smallest maximum of 8, 16 or 32 parts
  if (A.beams <= 16) cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, 1));
  if (A.beams <= 8) cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, 2));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) cut = fminf(cut, __shfl_xor_sync(0xffffffffu, cut, o));
  if (cut == -INFINITY) {  // some parts hold nothing: the maximum that beams - 1 others of the 32 exceed
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < kParts; ++j) rank += better(__shfl_sync(0xffffffffu, m, j), j, m, lane);
    cut = __shfl_sync(0xffffffffu, m, __ffs(__ballot_sync(0xffffffffu, rank == A.beams - 1)) - 1);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.0f : m;
  // ---- the runs that hold candidates (few do), the sum of exponentials
#pragma unroll
  for (int k = 0; k < RUNS; ++k)
    if (most[k] >= cut && most[k] > -INFINITY) {
      const int n = atomicAdd(&s_runs, 1);
      if (n < kList / C) {
        s_run[n] = v[k].w;
        s_run_at[n] = i0 + C * (k * kThreads + tid);
      }
    }
  // 2^(v log2(e) + shift): what the shift's rounding loses is the same for all and put right in the sum
  constexpr float log2e = 1.4426950408889634f;
  const float shift = __fmul_rn(-ref, log2e), lost = fmaf(-ref, log2e, -shift);
  const f2 slope = pair(log2e, log2e), shifts = pair(shift, shift);
  f2 sums[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
  for (int k = 0; k < RUNS; ++k)
#pragma unroll
    for (int j = 0; j < C; j += 2) {
      const float2 x = halves(fma2(pair(v[k].at(j), v[k].at(j + 1)), slope, shifts));
      sums[j / 2 & 1] = add2(sums[j / 2 & 1], pair(ex2(x.x), ex2(x.y)));
    }
  const float2 both = halves(add2(sums[0], sums[1]));
  float sum = both.x + both.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  const long long at = row * A.slices + slice;
  if (tid == 0) {
    for (int j = 1; j < kWarps; ++j) sum += s_sum[j];
    A.stats[at] = make_float2(m, sum * ex2(lost));
  }
  float *best = A.best + at * A.beams;
  int32_t *best_at = A.best_at + at * A.beams;
  const int listed = s_runs;
  if (listed <= kList / C) {  // each candidate's rank among them
    for (int i = tid; i < listed * C; i += kThreads) {
      const Run<HALF> r = {s_run[i / C]};
      float x = -INFINITY;
#pragma unroll
      for (int j = 0; j < C; ++j) x = i % C == j ? r.at(j) : x;
      if (x >= cut && x > -INFINITY) {
        const int n = atomicAdd(&s_n, 1);
        s_val[n] = x;
        s_at[n] = s_run_at[i / C] + i % C;
      }
    }
    __syncthreads();
    const int n = s_n;
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
      for (int k = 0; k < RUNS; ++k)
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int ij = i0 + C * (k * kThreads + tid) + j;
          const float y = v[k].at(j);
          if (y > -INFINITY && better(last, last_at, y, ij) && better(y, ij, x, ix)) {
            x = y;
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

// log(x) of a float x >= 1 as a sum of two floats, to about 2^-40. x = 2^e m with m in
// [2/3, 4/3): log m = 2 artanh(t), t = (m - 1) / (m + 1), |t| <= 1/5: 2 t is kept in two
// floats, the rest of the series, below 2 t / 70, in one.
__device__ __forceinline__ double log_of(float x) {
  const int e = (int)((__float_as_uint(x) - 0x3f2aaaabu) >> 23);
  const float m = __uint_as_float(__float_as_uint(x) - ((uint32_t)e << 23));
  const float a = __fsub_rn(m, 1.0f);            // exact
  const float b = __fadd_rn(m, 1.0f), bl = __fsub_rn(m, __fsub_rn(b, 1.0f));  // m + 1 = b + bl
  const float t = __fdiv_rn(a, b);
  const float tl = __fdiv_rn(__fsub_rn(fmaf(-t, b, a), __fmul_rn(t, bl)), b);  // what the quotient is short of
  const float s = __fmul_rn(t, t);
  float p = 2.0f / 13;
  p = fmaf(p, s, 2.0f / 11);
  p = fmaf(p, s, 2.0f / 9);
  p = fmaf(p, s, 2.0f / 7);
  p = fmaf(p, s, 2.0f / 5);
  p = fmaf(p, s, 2.0f / 3);
  const float rest = fmaf(__fmul_rn(p, s), t, 2.0f * tl);
  return (double)e * 0.6931471805599453 + ((double)(2.0f * t) + (double)rest);
}

// A score as a whole number of the same order; 0 is below every candidate's.
__device__ __forceinline__ unsigned long long key_of(double x) {
  const long long b = __double_as_longlong(x + 0.0);  // -0 is 0
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
__device__ __forceinline__ double score_of(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ uint32_t key_of(float x) {  // 0 for -inf; x is a logit that is a number
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 is 0
  return x == -INFINITY ? 0 : b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Place {  // of a row's list
  float x;
  int at;
};

// Group blockIdx.x. A warp joins a row's slices: their lists are in order, so the
// row's best is always one of 32 heads (lists of higher tokens in higher lanes:
// equal logits go to the lowest). Then the rows' lists meet, in 64 bits: the
// fp64 units do two operations a cycle per SM, so that only the beams^2 scores are
// formed there. Candidates below the worst of the
// rows' best are no one's, the others count how many are better.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args A) {
  extern __shared__ Place s_lists[];  // [kWarps][32][beams]: lane 0's is what has been joined so far
  __shared__ Place s_row[kMaxBeams * kMaxBeams];
  __shared__ unsigned long long s_key[kMaxBeams * kMaxBeams];
  __shared__ int s_at[kMaxBeams * kMaxBeams], s_n;
  __shared__ double s_add[kMaxBeams];  // score - lse of a beam
  __shared__ uint8_t s_done[kMaxBeams];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = A.beams, S = A.slices;
  const long long row0 = (long long)blockIdx.x * W;
  Place *mine = s_lists + warp * 32 * W;
  for (int w = warp; w < W; w += kWarps) {
    const long long row = row0 + w;
    const float score = A.scores[row];
    const bool over = A.done && A.done[row];
    if (lane == 0) {
      s_done[w] = over;
      s_add[w] = over ? (double)score : -INFINITY;
    }
    if (over || !(score > -INFINITY)) {
      for (int i = lane; i < W; i += 32) s_row[w * W + i] = {-INFINITY, -1};
      continue;
    }
    const float2 *st = A.stats + row * S;
    float m = -INFINITY, sum = 0.0f;
    const int n0 = min(31, S) * W;  // the first slices' lists
    const float *bx0 = A.best + row * S * W;
    const int32_t *bi0 = A.best_at + row * S * W;
    for (int i = lane; i < W; i += 32) mine[i] = {-INFINITY, -1};
#pragma unroll 4
    for (int i = lane; i < n0; i += 32) mine[W + i] = {bx0[i], bi0[i]};
    for (int i = lane; i < S; i += 32) m = fmaxf(m, st[i].x);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int i = lane; i < S; i += 32) {
      const float2 x = st[i];
      sum += x.y * ex2((x.x - m) * 1.4426950408889634f);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // a sum that is not finite, or of nothing, makes every candidate NaN; else it is at least 1
    if (lane == 0) s_add[w] = sum >= 0.75f && sum < INFINITY ? (double)score - ((double)m + log_of(sum)) : (double)NAN;
    for (int s0 = 0; s0 < S; s0 += 31) {  // 31 slices at a time
      const int n = min(31, S - s0) * W;
      if (s0 > 0) {
        const float *bx = bx0 + s0 * W;
        const int32_t *bi = bi0 + s0 * W;
        for (int i = lane; i < n; i += 32) mine[W + i] = {bx[i], bi[i]};
        for (int i = lane; i < W; i += 32) mine[i] = s_row[w * W + i];
      }
      __syncwarp();
      const bool list = lane == 0 || (lane - 1) * W < n;
      int at = 0;
      Place head = list ? mine[lane * W] : Place{-INFINITY, -1};
      for (int r = 0; r < W; ++r) {
        const uint32_t key = key_of(head.x), top = __reduce_max_sync(0xffffffffu, key);
        const int from = __ffs(__ballot_sync(0xffffffffu, key == top)) - 1;
        if (lane == from) {
          s_row[w * W + r] = top ? head : Place{-INFINITY, -1};
          ++at;
          head = top && at < W ? mine[lane * W + at] : Place{-INFINITY, -1};
        }
      }
      __syncwarp();
    }
  }
  if (tid == 0) s_n = 0;
  __syncthreads();
  auto key_at = [&](int w, int r) -> unsigned long long {  // 0: no candidate
    double x = s_add[w];
    if (s_done[w]) {
      if (r > 0) return 0;
    } else {
      if (s_row[w * W + r].at < 0) return 0;
      x += (double)s_row[w * W + r].x;
    }
    return x > -INFINITY ? key_of(x) : 0;  // not -inf, not NaN
  };
  unsigned long long cut = lane < W ? key_at(lane, 0) : ~0ull;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) cut = min(cut, __shfl_xor_sync(0xffffffffu, cut, o));
  for (int c = tid; c < W * W; c += kThreads) {
    const int w = c / W, r = c - w * W;
    const unsigned long long k = key_at(w, r);
    if (k > 0 && k >= cut) {
      const int i = atomicAdd(&s_n, 1);
      s_key[i] = k;
      s_at[i] = (w << 24) + (s_done[w] ? max(A.eos, 0) : s_row[c].at);
    }
  }
  __syncthreads();
  const int n = s_n;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long k = s_key[i];
    const int at = s_at[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += s_key[j] > k || (s_key[j] == k && s_at[j] < at);
    if (rank >= W) continue;
    const int w = at >> 24, t = s_done[w] ? A.eos : at & 0xffffff;
    A.parent[row0 + rank] = (int)(row0 + w);
    A.token[row0 + rank] = t;
    A.new_scores[row0 + rank] = (float)score_of(k);
    if (A.new_done) A.new_done[row0 + rank] = s_done[w] || t == A.eos;
  }
  for (int r = n + tid; r < W; r += kThreads) {  // places without a candidate
    A.parent[row0 + r] = (int)(row0 + r);
    A.token[row0 + r] = -1;
    A.new_scores[row0 + r] = -INFINITY;
    if (A.new_done) A.new_done[row0 + r] = 0;
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
  const size_t lists = (size_t)beam::kWarps * 32 * A.beams * sizeof(beam::Place);
  static std::atomic<uint64_t> ready{0};  // a bit a device: the attribute holds for the process
  const uint64_t bit = 1ull << dev->id;
  if (lists > 16384 && !(ready.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(beam::join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             beam::kWarps * 32 * beam::kMaxBeams * (int)sizeof(beam::Place)) != cudaSuccess)
      return check_launch("beam_select");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  launch_pdl(beam::join_kernel, dim3(A.groups), block, lists, st, A);
  return check_launch("beam_select");
}
