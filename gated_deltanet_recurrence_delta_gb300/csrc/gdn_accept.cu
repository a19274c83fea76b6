// gdn_accept_draft: drafted tokens tested against the target's probabilities,
// and the draw of the token that follows, from given random numbers.
//
// generate.py (sparkle, mlx_streaming/mtp), accept_prefix: the verify forward's
// distributions decide how many drafted tokens stand; the accept length feeds
// the commit of the recurrent states. Here the test keeps the target's
// distribution for any draft distribution:
//   draft x stands iff u draft(x) < target(x)   (exact: the product of two
//   floats fits a double)
//   next ~ max(target - draft, 0) at the first refusal, ~ target after the last
//
// Memory-bound by the one or two rows of V probabilities the draw is made
// from. A cluster of CTAs shares one batch row: each sums its slice of the
// vocabulary, the slice sums meet in distributed shared memory, and the CTA
// whose slice holds the drawn point finds the index in the one warp's share
// (an eighth of the slice) that holds it. The drawn index is a comparison of
// running sums, so sums are carried as two floats (~48 bits): plain fp32 sums
// would move ~1% of the draws to a neighbouring token.
#include "gdn_launch.h"

namespace gdn {
namespace accept {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;

struct Args {
  int T, V;
  const int32_t *tokens;
  const float *target, *draft, *uniform;
  const int32_t *n_tokens;
  int32_t *accept_len, *next;
  unsigned int *status;
};

// The weight of a token: max(p - q, 0), or max(p, 0) without q; exact as hi + lo.
struct Weight {
  float hi, lo;
};
__device__ __forceinline__ Weight weight(float p, float q) {
  Weight w;
  w.hi = __fsub_rn(p, q);
  const float b = __fsub_rn(p, w.hi);  // two-difference
  w.lo = __fadd_rn(__fsub_rn(p, __fadd_rn(w.hi, b)), __fsub_rn(b, q));
  if (!(p > q)) w.hi = w.lo = 0.0f;  // NaN counts as zero
  return w;
}
// (hi, lo) += w, the rounding of the leading sum kept in lo
__device__ __forceinline__ void add(float &hi, float &lo, Weight w) {
  const float s = __fadd_rn(hi, w.hi), z = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, z)), __fsub_rn(w.hi, z));
  hi = s;
  lo = __fadd_rn(lo, __fadd_rn(e, w.lo));
}

// The row that is drawn from. `taken`: a token whose draft probability is 1.
struct Row {
  const float *p, *q;
  int taken;
  __device__ __forceinline__ Weight at(int i) const {
    return weight(p[i], q ? q[i] : i == taken ? 3.4e38f : 0.0f);
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ double ld_cluster(const double *p, uint32_t rank) {
  uint32_t a;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ Args A) {
  __shared__ int s_kept, s_bad, s_pick;
  __shared__ double s_warp[kWarps], s_total;
  griddep_wait();
  griddep_trigger();
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long b = blockIdx.x / kCluster;
  const int n = A.n_tokens ? A.n_tokens[b] : A.T;

  // ---- the drafts: lane t tests token t + 1; every CTA of the cluster alike
  if (warp == 0) {
    bool bad = n < 0 || n > A.T, stands = false;
    if (!bad && lane < n - 1) {
      const int x = A.tokens[b * A.T + lane + 1];
      if (x < 0 || x >= A.V) {
        bad = true;
      } else {
        const float p = A.target[(b * A.T + lane) * A.V + x];
        const float q = A.draft ? A.draft[(b * (A.T - 1) + lane) * A.V + x] : 1.0f;
        stands = (double)A.uniform[b * A.T + lane] * (double)q < (double)p;
      }
    }
    const unsigned ok = __ballot_sync(0xffffffffu, stands);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s_kept = __ffs(~ok) - 1;  // T <= 32: at most 31 drafts, so a zero bit is there
      s_bad = bad;
      s_pick = -1;
    }
  }
  __syncthreads();
  const int kept = s_kept;
  if (s_bad || n == 0) {  // the same for every CTA of the cluster
    if (rank == 0 && tid == 0) {
      if (s_bad) set_status(A.status, GDN_ERR_INDEX);
      A.accept_len[b] = 0;
      A.next[b] = -1;
    }
    return;
  }
  const bool refused = kept < n - 1;
  Row R;
  R.p = A.target + (b * A.T + kept) * A.V;
  R.q = refused && A.draft ? A.draft + (b * (A.T - 1) + kept) * A.V : nullptr;
  R.taken = refused && !A.draft ? A.tokens[b * A.T + kept + 1] : -1;

  // ---- this warp's contiguous share of the row
  const long long W = (long long)kCluster * kWarps, w = (long long)rank * kWarps + warp;
  const int i0 = (int)(A.V * w / W), i1 = (int)(A.V * (w + 1) / W);
  double total = 0.0, before = 0.0, mine = 0.0;
  for (int again = 0; again < 2; ++again) {
    float hi = 0.0f, lo = 0.0f;
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) add(hi, lo, R.at(i));
    const double s = warp_sum((double)hi + (double)lo);
    if (lane == 0) s_warp[warp] = s;
    __syncthreads();
    if (tid == 0) {
      double x = 0.0;
      for (int j = 0; j < kWarps; ++j) x += s_warp[j];
      s_total = x;
    }
    cluster_sync();
    total = before = 0.0;
    for (uint32_t r = 0; r < kCluster; ++r) {
      const double x = ld_cluster(&s_total, r);
      if (r < rank) before += x;
      if (r == rank) mine = x;
      total += x;
    }
    if (total > 0.0 || !refused) break;  // the same for every CTA
    cluster_sync();  // every CTA has read the sums that the next pass overwrites
    R.q = nullptr;  // no mass is left: draw from the target itself
    R.taken = -1;
  }

  // ---- the CTA that holds the drawn point: the first whose running sum
  // exceeds it, else (the sums' last bits) the last that has any mass
  const double spot = (double)A.uniform[b * A.T + A.T - 1] * total;
  int owner = -1, last = -1;
  {
    double run = 0.0;
    for (uint32_t r = 0; r < kCluster; ++r) {
      const double x = ld_cluster(&s_total, r);
      run += x;
      if (x > 0.0) {
        last = (int)r;
        if (owner < 0 && run > spot) owner = (int)r;
      }
    }
    if (owner < 0) owner = last;
  }
  if (rank == 0 && tid == 0) {
    A.accept_len[b] = kept + 1;
    if (owner < 0) A.next[b] = -1;  // no mass at all
  }
  if (owner == (int)rank) {
    // the warp's share, by the same rule
    double run = before;
    int pick = -1, tail = -1;
    double pick_at = 0.0, tail_at = 0.0;
    for (int j = 0; j < kWarps; ++j) {
      const double x = s_warp[j];
      if (x > 0.0) {
        tail = j;
        tail_at = run;
        if (pick < 0 && run + x > spot) {
          pick = j;
          pick_at = run;
        }
      }
      run += x;
    }
    if (pick < 0) {
      pick = tail;
      pick_at = tail_at;
    }
    // its tokens, a contiguous run for each thread of the CTA
    const long long v = (long long)rank * kWarps + pick;
    const int j0 = (int)(A.V * v / W), j1 = (int)(A.V * (v + 1) / W);
    const int per = (j1 - j0 + kThreads - 1) / kThreads;
    const int a = min(j0 + tid * per, j1), z = min(a + per, j1);
    double s = 0.0;
    for (int i = a; i < z; ++i) {
      const Weight x = R.at(i);
      s += (double)x.hi + (double)x.lo;
    }
    double incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();  // s_warp has been read
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    double at = pick_at + incl - s;
    for (int j = 0; j < warp; ++j) at += s_warp[j];
    // the lowest token whose running sum exceeds the point, else the last with mass
    int found = 0x7fffffff, heavy = -1;
    for (int i = a; i < z; ++i) {
      const Weight x = R.at(i);
      at += (double)x.hi + (double)x.lo;
      if (x.hi > 0.0f) {
        heavy = i;
        if (found == 0x7fffffff && at > spot) found = i;
      }
    }
    found = __reduce_min_sync(0xffffffffu, found);
    heavy = __reduce_max_sync(0xffffffffu, heavy);
    __shared__ int s_found[kWarps], s_heavy[kWarps];
    if (lane == 0) {
      s_found[warp] = found;
      s_heavy[warp] = heavy;
    }
    __syncthreads();
    if (tid == 0) {
      for (int j = 0; j < kWarps; ++j) {
        found = min(found, s_found[j]);
        heavy = max(heavy, s_heavy[j]);
      }
      A.next[b] = found < 0x7fffffff ? found : heavy;
    }
  }
  cluster_sync();  // no CTA leaves while another reads its sums
}

}  // namespace accept
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_accept_draft(int32_t B, int32_t T, int32_t V, const int32_t *tokens,
                                       const float *target_probs, const float *draft_probs, const float *uniform,
                                       const int32_t *n_tokens, int32_t *accept_len, int32_t *next_token,
                                       void *stream) {
  if (B < 0 || B > (1 << 20)) return fail(GDN_ERR_SHAPE, "B must be in [0, 2^20]");
  if (T < 1 || T > 32) return fail(GDN_ERR_SHAPE, "T must be in [1, 32]");
  if (V < 1 || V > (1 << 30)) return fail(GDN_ERR_SHAPE, "V must be in [1, 2^30]");
  if (B == 0) return GDN_OK;  // empty tensors may have no address
  GDN_TRY(check_ptr(tokens, "tokens", 4));
  GDN_TRY(check_ptr(target_probs, "target_probs", 4));
  if (draft_probs) GDN_TRY(check_ptr(draft_probs, "draft_probs", 4));
  GDN_TRY(check_ptr(uniform, "uniform", 4));
  if (n_tokens) GDN_TRY(check_ptr(n_tokens, "n_tokens", 4));
  GDN_TRY(check_ptr(accept_len, "accept_len", 4));
  GDN_TRY(check_ptr(next_token, "next_token", 4));
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  accept::Args A = {T, V, tokens, target_probs, draft_probs, uniform, n_tokens, accept_len, next_token, dev->status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * accept::kCluster);
  cfg.blockDim = dim3(accept::kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = accept::kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  (void)cudaLaunchKernelEx(&cfg, accept::accept_kernel, A);
  return check_launch("accept_draft");
}
