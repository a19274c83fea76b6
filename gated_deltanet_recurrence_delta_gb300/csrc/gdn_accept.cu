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
// vocabulary, a share for each of its warps, the 64 shares' sums meet in
// distributed shared memory, and the CTA whose share holds the drawn point
// finds the index in it. The drawn index is a comparison of
// running sums, so sums are carried as two floats (~46 bits): plain fp32 sums
// would move ~1% of the draws to a neighbouring token.
//
// 64 rows of 8 tokens over 131072 (67 MB of draft and target rows): 18.0 us, 56%
// of the measured copy rate; the rest is the chain of the drafts' loads (2 us),
// the exchange and the search (2 us) and the launch. 8 rows, certain drafts over
// 32000: 6.4 us. 33 rows of 5 over 99991, whose draft and target rows differ in
// their address modulo 16 and are read 4 bytes at a time: 14.2 us.
#include "gdn_check.h"

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

// The weight of a token, max(p - q, 0), exact as hi + lo. Negative and NaN p
// count as zero, a NaN q as no more than p. p >= q >= 0 makes the subtraction's
// error (p - hi) - q exact.
struct Weight {
  float hi, lo;
};
__device__ __forceinline__ Weight weight(float p, float q) {
  p = fmaxf(p, 0.0f);
  q = fminf(q, p);
  Weight w;
  w.hi = __fsub_rn(p, q);
  w.lo = __fsub_rn(__fsub_rn(p, w.hi), q);
  return w;
}

// A number as hi + lo, hi the nearest float: ~48 bits from the fp32 units. (The
// chip's fp64 units do two operations a cycle per SM: sums in doubles took half
// the kernel's time.)
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two plus(Two a, Two b) {
  const float s = __fadd_rn(a.hi, b.hi), z = __fsub_rn(s, a.hi);
  float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, z)), __fsub_rn(b.hi, z));
  e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  const float h = __fadd_rn(s, e);
  return {h, __fsub_rn(e, __fsub_rn(h, s))};
}
__device__ __forceinline__ bool above(Two a, Two b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// A sum as two floats. hi starts at kBase, above every weight, so that each
// addition's error w - (s - hi) is exact; lo collects the errors, which are
// below 2^-22, to about 2^-46.
constexpr float kBase = 2.0f;
struct Sum {
  float hi = kBase, lo = 0.0f;
  __device__ __forceinline__ void add(Weight w) {
    const float s = __fadd_rn(hi, w.hi);
    const float e = __fsub_rn(w.hi, __fsub_rn(s, hi));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, w.lo));
  }
  __device__ __forceinline__ Two value() const;
};

__device__ __forceinline__ Two Sum::value() const {
  const float h = __fsub_rn(hi, kBase), s = __fadd_rn(h, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, h))};
}

// The row that is drawn from. `taken`: a token whose draft probability is 1.
struct Row {
  const float *p, *q;
  int taken;
  __device__ __forceinline__ Weight at(int i) const {
    return weight(p[i], q ? q[i] : i == taken ? __int_as_float(0x7f800000) : 0.0f);
  }
};

// This lane's part of the mass of tokens [i0, i1). TWO: a draft row beside the
// target's; VEC: 16-byte loads (both rows' addresses leave the same rest to 16).
template <bool TWO, bool VEC>
__device__ __forceinline__ Two lane_mass(const Row &R, int i0, int i1, int lane) {
  Sum sum[4];
  if (VEC) {
    const int a = min(i1, i0 + (int)(((16 - (reinterpret_cast<uintptr_t>(R.p + i0) & 15)) & 15) / 4));
    if (i0 + lane < a) sum[0].add(R.at(i0 + lane));
    const int z = a + (i1 - a) / 4 * 4;
    constexpr int kBatch = 4;  // 16-byte loads of each row in flight
    int i = a + 4 * lane;
    for (; i + 128 * (kBatch - 1) < z; i += 128 * kBatch) {
      float4 p[kBatch], q[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        p[k] = __ldcs(reinterpret_cast<const float4 *>(R.p + i + 128 * k));
        if (TWO) q[k] = __ldcs(reinterpret_cast<const float4 *>(R.q + i + 128 * k));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        sum[0].add(weight(p[k].x, TWO ? q[k].x : 0.0f));
        sum[1].add(weight(p[k].y, TWO ? q[k].y : 0.0f));
        sum[2].add(weight(p[k].z, TWO ? q[k].z : 0.0f));
        sum[3].add(weight(p[k].w, TWO ? q[k].w : 0.0f));
      }
    }
    for (; i < z; i += 128)
      for (int k = 0; k < 4; ++k) sum[k].add(R.at(i + k));
    if (z + lane < i1) sum[0].add(R.at(z + lane));
  } else {
    constexpr int kBatch = 16;
    int i = i0 + lane;
    for (; i + 32 * (kBatch - 1) < i1; i += 32 * kBatch) {
      float p[kBatch], q[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        p[k] = __ldcs(R.p + i + 32 * k);
        q[k] = TWO ? __ldcs(R.q + i + 32 * k) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) sum[k & 3].add(weight(p[k], q[k]));
    }
    for (; i < i1; i += 32) sum[0].add(R.at(i));
  }
  return plus(plus(sum[0].value(), sum[1].value()), plus(sum[2].value(), sum[3].value()));
}
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = plus(x, {__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
  return x;
}
__device__ __forceinline__ Two warp_scan(Two x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if (lane >= o) x = plus(y, x);
  }
  return x;
}
__device__ __forceinline__ Two ld_cluster(const Two *p, uint32_t rank) {
  uint32_t a;
  Two v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(a));
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ Args A) {
  __shared__ int s_kept, s_bad, s_pick;
  __shared__ __align__(8) Two s_warp[kWarps], s_part[kWarps], s_at, s_spot;
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
    }
  }
  __syncthreads();
  const int kept = s_kept;
  const float u_draw = A.uniform[b * A.T + A.T - 1];
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
  constexpr int W = kCluster * kWarps;
  const int w = (int)rank * kWarps + warp;
  const int i0 = (int)((long long)A.V * w / W), i1 = (int)((long long)A.V * (w + 1) / W);
  for (int again = 0; again < 2; ++again) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(R.p), qa = reinterpret_cast<uintptr_t>(R.q);
    Two s;  // the branches are the same for a warp
    if (R.q)
      s = (pa & 15) == (qa & 15) ? lane_mass<true, true>(R, i0, i1, lane) : lane_mass<true, false>(R, i0, i1, lane);
    else if (R.taken < i0 || R.taken >= i1)
      s = lane_mass<false, true>(R, i0, i1, lane);
    else  // around the taken token
      s = plus(lane_mass<false, true>(R, i0, R.taken, lane), lane_mass<false, true>(R, R.taken + 1, i1, lane));
    s = warp_sum(s);
    if (lane == 0) s_warp[warp] = s;
    cluster_sync();
    if (warp == 0) {
      // the share that holds the drawn point: the first whose running sum
      // exceeds it, else (the sums' last bits) the last that has any mass.
      // Two shares to a lane; every CTA finds the same.
      static_assert(W == 64, "two shares to a lane");
      const Two x0 = ld_cluster(&s_warp[(2 * lane) % kWarps], 2 * lane / kWarps);
      const Two x1 = ld_cluster(&s_warp[(2 * lane + 1) % kWarps], (2 * lane + 1) / kWarps);
      const Two incl = warp_scan(plus(x0, x1), lane);
      Two before = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      if (lane == 0) before = {0.0f, 0.0f};
      const Two mid = plus(before, x0);
      const float th = __shfl_sync(0xffffffffu, incl.hi, 31), tl = __shfl_sync(0xffffffffu, incl.lo, 31);
      const double at_mass = (double)u_draw * ((double)th + (double)tl);
      const Two spot = {(float)at_mass, (float)(at_mass - (double)(float)at_mass)};
      const bool h0 = x0.hi > 0.0f && above(mid, spot), h1 = x1.hi > 0.0f && above(incl, spot);
      const unsigned hit = __ballot_sync(0xffffffffu, h0 || h1);
      const unsigned mass = __ballot_sync(0xffffffffu, x0.hi > 0.0f || x1.hi > 0.0f);
      int pick = -1;
      if (hit) {
        const int l = __ffs(hit) - 1;
        pick = 2 * l + (__shfl_sync(0xffffffffu, (int)h0, l) ? 0 : 1);
      } else if (mass) {
        const int l = 31 - __clz(mass);
        pick = 2 * l + (__shfl_sync(0xffffffffu, (int)(x1.hi > 0.0f), l) ? 1 : 0);
      }
      if (lane == max(pick, 0) / 2) {
        s_pick = pick;
        s_at = (pick & 1) ? mid : before;
        s_spot = spot;
      }
    }
    __syncthreads();
    if (s_pick >= 0 || !refused || again) break;  // the same for every CTA
    cluster_sync();  // every CTA has read the sums that the next pass overwrites
    R.q = nullptr;   // no mass is left: draw from the target itself
    R.taken = -1;
  }
  const int pick = s_pick;
  const Two spot = s_spot;
  if (rank == 0 && tid == 0) {
    A.accept_len[b] = kept + 1;
    if (pick < 0) A.next[b] = -1;  // no mass at all
  }
  cluster_sync_arrive();  // this CTA no longer reads the others' sums
  if (pick >= 0 && pick / kWarps == (int)rank) {
    // its tokens, a contiguous run for each thread of the CTA
    const int j0 = (int)((long long)A.V * pick / W), j1 = (int)((long long)A.V * (pick + 1) / W);
    const int per = (j1 - j0 + kThreads - 1) / kThreads;
    const int a = min(j0 + tid * per, j1), z = min(a + per, j1);
    Two s = {0.0f, 0.0f};
    for (int i = a; i < z; ++i) {
      const Weight x = R.at(i);
      s = plus(s, {x.hi, x.lo});
    }
    const Two incl = warp_scan(s, lane);
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    Two at = s_at;
    for (int j = 0; j < warp; ++j) at = plus(at, s_part[j]);
    const Two ahead = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    if (lane > 0) at = plus(at, ahead);
    // the lowest token whose running sum exceeds the point, else the last with mass
    int found = 0x7fffffff, heavy = -1;
    for (int i = a; i < z; ++i) {
      const Weight x = R.at(i);
      at = plus(at, {x.hi, x.lo});
      if (x.hi > 0.0f) {
        heavy = i;
        if (found == 0x7fffffff && above(at, spot)) found = i;
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
  cluster_sync_wait();  // no CTA leaves while another reads its sums
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
