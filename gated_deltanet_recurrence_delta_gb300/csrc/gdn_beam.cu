// gdn_beam_select: the best continuations of each group's beams.
//
//   cand(w, x) = score_w + logit_wx - lse_w,  lse_w = log sum_x exp(logit_wx);
//   the best `beams` of a group, ties to the lowest (w, x)
//
// Memory-bound: each logit is read once. Within a row candidates rank as their
// logits do, so a slice of a row yields its maximum, its sum of exponentials (each
// thread's own, against its own maximum so far) and its best `beams` logits in one
// pass; a second kernel joins a group's slices and ranks its candidates in 64
// bits, where alone different rows meet. (As the work of a group's last CTA the join
// cost more: 16 x 8 beams of 131072 bf16 logits took 22 to 28 us in the variants
// tried, 15.6 to 22 as two kernels. Its code is new to that SM, and the registers
// of both parts are the slices'.)
//
// A slice's best: a CTA's threads form P >= `beams` parts (8, 16 or 32). At least
// `beams` logits reach the smallest of the parts' maxima over the first runs, so
// only runs that reach it are listed. At the end the parts' maxima over the whole
// slice give a tighter cut, which P ln P or so of unordered logits reach: each
// counts how many of them are better. Equal logits in numbers beyond the list are
// taken one after the other.
//
// 16 x 8 beams of 131072 bf16 logits (33.6 MB, 4.9 us at the copy rate): 15.6 us as a
// graph, 2.2 TB/s; the logits' stream 5.7 of them, a slice's start and end 3, join 3.4. A slice's cuts, lists and
// ranking and the join are latency: dependent loads, barriers, code that is new to its
// SM.
// 4 x 4 beams of 32000 fp32 logits: 6.9 us, of which the two launches are 4.
// Slow, and right: logits of which all but a few are one finite number (masks of the type's lowest value), whose lists
// overflow (16 x 8 beams of 131072: 199 us fp32, 125 us bf16); 32 beams, whose cuts are low: some slices' lists overflow,
// and in the join, where 32 divides the threads, a part sees a few places of all slices only (4 x 32 beams of 131072:
// slices 500 us, join 290).
#include <cuda_fp16.h>

#include "gdn_check.h"

namespace gdn {
namespace beam {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// 16 bytes of logits each that a thread works on at a time, and the next in flight: what three CTAs' registers hold (4 x 4
// beams of 32000 fp32 logits 7.05 us, 16 x 8 of 131072 bf16 ones 15.6; 4 runs 7.6 and 15.6, 5 7.0 and 16.2, 8 7.3 and more)
constexpr int kRuns = 6;
constexpr int kLeast = 4096;  // logits that are worth a CTA
constexpr int kMaxBeams = 32;
constexpr int kParts = 32, kLanes = kThreads / kParts;
constexpr int kList = 512;

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
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_min(float x) {
  float y;
  asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float part_max(float x) {  // over the lanes of a part
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// A number that `beams` of the parts' maxima reach, by every warp: the smallest of 8, 16 or 32 parts, or, where some
// parts hold nothing, the one that beams - 1 others exceed.
__device__ __forceinline__ float cut_of(const float (&most)[kParts], int beams, int lane) {
  static_assert(kParts == 32, "a part to a lane");
  const float m = most[lane];
  float cut = m;
  if (beams <= 16) cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, 1));
  if (beams <= 8) cut = fmaxf(cut, __shfl_xor_sync(0xffffffffu, cut, 2));
  cut = warp_min(cut);
  if (cut == -INFINITY) {
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < kParts; ++j) rank += better(most[j], j, m, lane);
    cut = __shfl_sync(0xffffffffu, m, __ffs(__ballot_sync(0xffffffffu, rank == beams - 1)) - 1);
  }
  return cut;
}

constexpr int kFinal = 1024;  // candidates that are ranked in 64 bits

// Group blockIdx.x. A warp sums up a row's slices; then all candidates of the rows'
// slices are compared in fp32 against the smallest maximum of as many parts of the
// threads as there are beams, with what fp32 may be off by: what remains, a few more
// than `beams`, counts in 64 bits how many are better. (The fp64 units do two
// operations a cycle per SM.) Where more remain than the list holds (rows of equal
// logits) they are taken one after the other.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args A) {
  __shared__ unsigned long long s_key[kFinal];
  __shared__ int s_at[kFinal], s_n, s_pick[kWarps];
  __shared__ float s_best[kFinal];     // the candidates' logits
  __shared__ double s_add[kMaxBeams];  // score - lse
  __shared__ float s_close[kMaxBeams], s_off[kMaxBeams];  // that in fp32, and what it may be off by
  __shared__ float s_row[3][kMaxBeams];                   // score, maximum, sum of exponentials
  __shared__ uint8_t s_none[kMaxBeams];                   // the beam has no candidates
  __shared__ unsigned long long s_top[kWarps];
  __shared__ float s_max[32];
  __shared__ uint8_t s_done[kMaxBeams];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = A.beams, S = A.slices;
  const long long row0 = (long long)blockIdx.x * W;
  const int each = S * W, N = W * each;  // candidates of a row, of all
  const float *best = A.best + row0 * each;
  const int32_t *best_at = A.best_at + row0 * each;
  const int c0 = min(tid, N - 1);
  const float x0 = __ldcg(best + c0);  // in flight meanwhile
  const int at0 = __ldcg(best_at + c0);
  if (tid == 0) s_n = 0;
#pragma unroll 1
  for (int w = warp; w < W; w += kWarps) {
    const long long row = row0 + w;
    const float2 *st = A.stats + row * S;
    const float score = A.scores[row];
    const bool over = A.done && A.done[row];
    float2 x = lane < S ? __ldcg(st + lane) : make_float2(-INFINITY, 0.0f);
    for (int i = lane + 32; i < S; i += 32) {
      const float2 y = __ldcg(st + i);
      const float m = fmaxf(x.x, y.x), r = m == -INFINITY ? 0.0f : m;
      x = make_float2(m, x.y * ex2((x.x - r) * 1.4426950408889634f) + y.y * ex2((y.x - r) * 1.4426950408889634f));
    }
    const float m = warp_max(x.x);
    float sum = x.y * ex2((x.x - m) * 1.4426950408889634f);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_done[w] = over;
      // a sum that is not finite, or of nothing, makes every candidate NaN; else it is at least 1
      s_none[w] = !(score > -INFINITY && (over || (sum >= 0.75f && sum < INFINITY)));
      s_row[0][w] = score;
      s_row[1][w] = m;
      s_row[2][w] = sum;
      // log2 is 2^-22 off, of itself or of 1, and each of three roundings 2^-24; too large for fp32: by anything
      const float log = __log2f(fmaxf(sum, 0.75f)) * 0.693147182f;
      const float size = fabsf(score) + (over ? 0.0f : fabsf(m) + fabsf(log) + 1.0f);
      s_close[w] = over ? score : score - (m + log);
      s_off[w] = size < 1e37f ? 3.6e-7f * size : INFINITY;
    }
  }
  __syncthreads();
  if (warp == kWarps - 1 && lane < W) {  // one warp, the one with the fewest candidates, while the others look at theirs
    // (an operation in 64 bits takes 16 cycles of the SM, however few lanes it has)
    const double lse = s_done[lane] ? 0.0 : (double)s_row[1][lane] + log_of(s_row[2][lane]);
    s_add[lane] = (double)s_row[0][lane] - lse;
  }
  // A candidate: c < N is place c % W of slice c / W % S of beam c / (W S), and stands for a finished beam if it is its
  // first. false: it is none.
  auto candidate = [&](int c, float &x, int t, int &w, int &at) {
    w = c / each;
    if (s_done[w]) x = 0.0f;
    at = (w << 24) + (s_done[w] ? max(A.eos, 0) : t);
    return !s_none[w] && (s_done[w] ? c == w * each : t >= 0);
  };
  auto exact = [&](int w, float x) {
    const double y = s_add[w] + (double)x;
    return y > -INFINITY ? key_of(y) : 0ull;
  };
  auto close = [&](int w, float x, float side) {  // the score less (side -1) or more (1) than fp32 may be off by, or NaN
    const float a = s_close[w];
    return a + x + side * (s_off[w] + 2.4e-7f * (fabsf(a) + fabsf(x)));  // 2^-22
  };
  float top = -INFINITY;
#pragma unroll 1
  for (int c = tid; c < N; c += kThreads) {
    float x = c == tid ? x0 : __ldcg(best + c);
    int w, at;
    if (candidate(c, x, c == tid ? at0 : __ldcg(best_at + c), w, at))
      top = fmaxf(top, close(w, x, -1.0f));  // a NaN is no maximum
  }
  top = part_max(top);
  if (tid % kLanes == 0) s_max[tid / kLanes] = top;
  __syncthreads();
  const float cut = cut_of(s_max, W, lane);
#pragma unroll 1
  for (int c = tid; c < N; c += kThreads) {
    float x = c == tid ? x0 : __ldcg(best + c);
    int w, at;
    if (!candidate(c, x, c == tid ? at0 : __ldcg(best_at + c), w, at)) continue;
    if (close(w, x, 1.0f) < cut) continue;
    const int i = atomicAdd(&s_n, 1);
    if (i < kFinal) {
      s_best[i] = x;
      s_at[i] = at;
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n <= kFinal) {
    for (int i = tid; i < n; i += kThreads) s_key[i] = exact(s_at[i] >> 24, s_best[i]);
    __syncthreads();
  }
  auto put = [&](int place, unsigned long long k, int at) {
    const int w = at >> 24, t = s_done[w] ? A.eos : at & 0xffffff;
    A.parent[row0 + place] = (int)(row0 + w);
    A.token[row0 + place] = t;
    A.new_scores[row0 + place] = (float)score_of(k);
    if (A.new_done) A.new_done[row0 + place] = s_done[w] || t == A.eos;
  };
  if (n <= kFinal) {
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = s_key[i];
      const int at = s_at[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += s_key[j] > k || (s_key[j] == k && s_at[j] < at);
      if (rank < W) put(rank, k, at);
    }
  } else {
    unsigned long long last = ~0ull;  // the candidate taken last
    int last_at = -1;
#pragma unroll 1
    for (int r = 0; r < W; ++r) {
      unsigned long long key = 0;
      int at = 0x7fffffff;
#pragma unroll 1
      for (int c = tid; c < N; c += kThreads) {
        float x = __ldcg(best + c);
        int w, i;
        if (!candidate(c, x, __ldcg(best_at + c), w, i)) continue;
        const unsigned long long k = exact(w, x);
        if (k > 0 && (k < last || (k == last && i > last_at)) && (k > key || (k == key && i < at))) {
          key = k;
          at = i;
        }
      }
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
        s_top[warp] = key;
        s_pick[warp] = at;
      }
      __syncthreads();
      for (int j = 0; j < kWarps; ++j)
        if (s_top[j] > key || (s_top[j] == key && s_pick[j] < at)) {
          key = s_top[j];
          at = s_pick[j];
        }
      last = key;  // n > kFinal >= W: there is one
      last_at = at;
      if (tid == 0) put(r, key, at);
    }
  }
  for (int r = n + tid; r < W; r += kThreads) {  // places without a candidate
    A.parent[row0 + r] = (int)(row0 + r);
    A.token[row0 + r] = -1;
    A.new_scores[row0 + r] = -INFINITY;
    if (A.new_done) A.new_done[row0 + r] = 0;
  }
}

// Slice blockIdx.x of row blockIdx.y, kRuns runs of a thread at a time, the next in
// flight.
template <bool HALF>
__global__ void __launch_bounds__(kThreads, 3) slice_kernel(const __grid_constant__ Args A) {
  constexpr int C = Run<HALF>::C, B = HALF ? 2 : 4, LIST = 512;
  __shared__ float s_max[kParts], s_red[kWarps], s_sum[kWarps];
  __shared__ uint4 s_run[LIST];  // the runs that may hold candidates, and where they begin
  __shared__ int s_run_at[LIST], s_runs;
  __shared__ float s_val[kList];  // the candidates
  __shared__ int s_at[kList], s_n, s_pick[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  if (tid == 0) s_runs = s_n = 0;
  griddep_wait();
  griddep_trigger();
  const long long row = blockIdx.y;
  const int all = (A.V + C - 1) / C;  // 16 bytes each, dealt out evenly
  const int r0 = (int)((long long)all * slice / A.slices), r1 = (int)((long long)all * (slice + 1) / A.slices);
  const char *p = static_cast<const char *>(A.logits) + row * A.stride * B;
  const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15) == 0;  // and so is every run then
  auto fetch = [&](int r) {  // run r, -inf behind the row's end
    Run<HALF> x;
    if (aligned && r < r1 && (r + 1) * C <= A.V) {
      x.w = __ldcs(reinterpret_cast<const uint4 *>(p) + r);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int i = r * C + j;
        const bool in = r < r1 && i < A.V;
        if constexpr (HALF) {
          const uint32_t u = in ? *reinterpret_cast<const unsigned short *>(p + (long long)i * 2) : 0xff80u;
          w[j / 2] = j & 1 ? w[j / 2] | u << 16 : u;
        } else {
          w[j] = in ? *reinterpret_cast<const uint32_t *>(p + (long long)i * 4) : 0xff800000u;
        }
      }
      x.w = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
  };
  Run<HALF> ahead[kRuns];
  const float score = A.scores[row];
  const bool over = A.done && A.done[row];
#pragma unroll
  for (int k = 0; k < kRuns; ++k) ahead[k] = fetch(r0 + k * kThreads + tid);
  if (score > -INFINITY && !over) {  // else its logits give no candidates
    constexpr float log2e = 1.4426950408889634f;
    float m = -INFINITY, cut = -INFINITY;  // the thread's maximum so far; at least `beams` logits reach the cut
    f2 sums = pair(0.0f, 0.0f);            // of exp(logit - m)
    int turn = 0;
    for (int rb = r0; rb < r1; rb += kRuns * kThreads, ++turn) {
      Run<HALF> v[kRuns];
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        v[k] = ahead[k];
        if (rb + kRuns * kThreads < r1) ahead[k] = fetch(rb + (kRuns + k) * kThreads + tid);
      }
      float most[kRuns], top = m;  // a NaN is no maximum, but reaches the sum
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        most[k] = v[k].top();
        top = fmaxf(top, most[k]);
      }
      if ((turn & (turn + 1)) == 0 || cut == -INFINITY) {  // again each time that twice as much has been seen
        const float part = part_max(top);
        if (tid % kLanes == 0) s_max[tid / kLanes] = part;
        __syncthreads();
        cut = cut_of(s_max, A.beams, lane);
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
        if (most[k] >= cut && most[k] > -INFINITY) {  // few do
          const int n = atomicAdd(&s_runs, 1);
          if (n < LIST) {
            s_run[n] = v[k].w;
            s_run_at[n] = (rb + k * kThreads + tid) * C;
          }
        }
      const float ref = top == -INFINITY ? 0.0f : top, fade = ex2((m - ref) * log2e);
      m = top;
      sums = mul2(sums, pair(fade, fade));
      const f2 less = pair(-ref, -ref), slope = pair(log2e, log2e);
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int j = 0; j < C; j += 2) {
          const float2 x = halves(mul2(add2(pair(v[k].at(j), v[k].at(j + 1)), less), slope));
          sums = add2(sums, pair(ex2(x.x), ex2(x.y)));
        }
    }
    // ---- the slice's maximum and sum; the cut of all its logits
    const float part = part_max(m);
    if (tid % kLanes == 0) s_max[tid / kLanes] = part;
    __syncthreads();
    const float most = warp_max(s_max[lane]);
    cut = cut_of(s_max, A.beams, lane);
    const float2 both = halves(sums);
    float sum = (both.x + both.y) * ex2((m - (most == -INFINITY ? 0.0f : most)) * log2e);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const long long at = row * A.slices + slice;
    if (tid == 0) {
      for (int j = 1; j < kWarps; ++j) sum += s_sum[j];
      A.stats[at] = make_float2(most, sum);
    }
    float *best = A.best + at * A.beams;
    int32_t *best_at = A.best_at + at * A.beams;
    const int listed = s_runs;
    if (listed <= LIST) {  // the candidates
#pragma unroll 1
      for (int i = tid; i - lane < listed * C; i += kThreads) {
        float x = -INFINITY;
        if (i < listed * C) {
          const Run<HALF> r = {s_run[i / C]};
#pragma unroll
          for (int j = 0; j < C; ++j) x = i % C == j ? r.at(j) : x;
        }
        const bool in = x >= cut && x > -INFINITY;
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (who == 0) continue;
        int k = 0;
        if (lane == 0) k = atomicAdd(&s_n, __popc(who));
        k = __shfl_sync(0xffffffffu, k, 0) + __popc(who & ((1u << lane) - 1));
        if (in && k < kList) {
          s_val[k] = x;
          s_at[k] = s_run_at[i / C] + i % C;
        }
      }
      __syncthreads();
    }
    const int n = listed <= LIST ? s_n : kList + 1;
    if (n <= kList) {
      for (int i = tid; i < n; i += kThreads) {  // each one's rank among them
        const float x = s_val[i];
        const int ix = s_at[i];
        int rank = 0;
#pragma unroll 8
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
    } else {  // more than the lists hold (equal logits): one after the other, the best behind the last one taken
      float last = INFINITY;
      int last_at = -1;
#pragma unroll 1
      for (int r = 0; r < A.beams; ++r) {
        float x = -INFINITY;
        int ix = 0x7fffffff;
#pragma unroll 1
        for (int k = r0 + tid; k < r1; k += kThreads) {
          const Run<HALF> v = fetch(k);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const float y = v.at(j);
            if (y > -INFINITY && better(last, last_at, y, k * C + j) && better(y, k * C + j, x, ix)) {
              x = y;
              ix = k * C + j;
            }
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

// Slices of a row: about three CTAs for each of 152 SMs in all (16 x 8 rows of 131072 bf16 logits: 608 CTAs 22 us, 456
// 15.7 us, 304 16.4 us: what a slice costs besides its logits, the cuts and the ranking, is a third of it).
int slices_of(const gdn_beam_dims *d) {
  const int rows = d->n_groups * d->beams, want = rows > 0 ? 456 / rows : 1, most = d->vocab / kLeast;
  return want < 1 || most < 1 ? 1 : want < most ? want : most;
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
  static std::atomic<uint64_t> ready{0};  // a bit a device: the attributes hold for the process
  const uint64_t bit = 1ull << dev->id;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    // one split of an SM's memory for both kernels, which follow one another on it: with the driver's own choices for
    // each 16 x 8 beams take 19.1 us, with half of it shared 15.6, all 16.3
    bool ok = true;
    for (auto *k : {beam::slice_kernel<true>, beam::slice_kernel<false>, beam::join_kernel})
      ok &= cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 50) == cudaSuccess;
    if (!ok) return check_launch("beam_select");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (launch_pdl(dims->half ? beam::slice_kernel<true> : beam::slice_kernel<false>, grid, block, 0, st, A) != cudaSuccess)
    return check_launch("beam_select");
  launch_pdl(beam::join_kernel, dim3(A.groups), block, 0, st, A);
  return check_launch("beam_select");
}
