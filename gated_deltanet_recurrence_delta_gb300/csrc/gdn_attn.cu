// Causal attention over a pool of cached keys and values: packed prompts
// (gdn_attn_prefill) and rows that share prefixes (gdn_attn_shared_prefix).
//
// statecache.py (squad-0.8b, qev_fast), CacheQwen35's attention layers: a
// chunk's queries attend over the cached prefix and, causally, the chunk.
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// One warp per (query token, head), one pass over its keys with the running
// maximum and sum of the softmax.
#include "gdn_launch.h"

namespace gdn {
namespace attn {

struct Args {
  int B, T, n_tokens, n_groups, hq, hk, G;
  float scale;
  long long qs, kvs, kv_rows;
  const bf16 *q, *k, *v;
  bf16 *out;
  const int32_t *cu, *kv_start, *kv_len;                      // prefill
  const int32_t *group_rows, *prefix_start, *prefix_len;      // shared prefix
  const int32_t *suffix_start, *suffix_len, *q_len;
  unsigned int *status;
};

// The largest i in [0, n) with a[i] <= x, or -1.
__device__ __forceinline__ int find_row(const int32_t *a, int n, int x) {
  int lo = -1, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

struct Extent {
  long long start;
  int len;
};
__device__ __forceinline__ bool inside(long long start, long long len, long long rows) {
  return start >= 0 && len >= 0 && start + len <= rows;
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(128) attn_rows_kernel(const __grid_constant__ Args A) {
  constexpr int E = D / 32;  // channels of a lane
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  if (!SHARED && blockIdx.x == 0)
    for (int b = threadIdx.x; b < A.B; b += 128)
      if (A.cu[b] < 0 || A.cu[b] > A.cu[b + 1] || A.cu[b + 1] > A.n_tokens) set_status(A.status, GDN_ERR_INDEX);
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / A.hq), h = (int)(unit - (long long)t * A.hq);
  if (t >= A.n_tokens) return;
  Extent ext[2] = {{0, 0}, {0, 0}};
  bool real = true;
  if (SHARED) {
    const int b = t / A.T, i = t - b * A.T;
    if (A.n_groups > 0) {
      const int g = find_row(A.group_rows, A.n_groups, b);
      const bool ok = A.group_rows[0] == 0 && A.group_rows[A.n_groups] == A.B && g >= 0 && b < A.group_rows[g + 1];
      if (!ok || !inside(A.prefix_start[g], A.prefix_len[g], A.kv_rows)) {
        set_status(A.status, GDN_ERR_INDEX);
        return;
      }
      ext[0] = {A.prefix_start[g], A.prefix_len[g]};
    }
    const int ql = A.q_len ? A.q_len[b] : A.T;
    if (!inside(A.suffix_start[b], A.suffix_len[b], A.kv_rows) || ql < 0 || ql > A.T) {
      set_status(A.status, GDN_ERR_INDEX);
      return;
    }
    real = i < ql;
    ext[1] = {A.suffix_start[b], max(0, A.suffix_len[b] - ql + i + 1)};
    if (!real) ext[0].len = ext[1].len = 0;
  } else {
    const int b = find_row(A.cu, A.B, t);
    if (b < 0 || t >= A.cu[b + 1]) return;
    const int n = A.cu[b + 1] - A.cu[b], i = t - A.cu[b];
    const long long start = A.kv_start ? A.kv_start[b] : A.cu[b];
    const int m = A.kv_len ? A.kv_len[b] : n;
    if (A.cu[b] < 0 || A.cu[b + 1] > A.n_tokens || !inside(start, m, A.kv_rows)) {
      set_status(A.status, GDN_ERR_INDEX);
      return;
    }
    ext[1] = {start, max(0, m - n + i + 1)};
  }
  float q[E], o[E], top = -INFINITY, sum = 0.0f;
  const bf16 *qp = A.q + t * A.qs + (long long)h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = ldbf(qp + e) * A.scale;
    o[e] = 0.0f;
  }
  for (int x = 0; x < 2; ++x) {
    const long long base = ext[x].start * A.kvs + (long long)(h / A.G) * D + lane * E;
    for (int j = 0; j < ext[x].len; ++j) {
      const bf16 *kp = A.k + base + j * A.kvs, *vp = A.v + base + j * A.kvs;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], ldbf(kp + e), s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      const float m = fmaxf(top, s), old = top == m ? 1.0f : __expf(top - m), p = __expf(s - m);
      top = m;
      sum = sum * old + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(p, ldbf(vp + e), o[e] * old);
    }
  }
  bf16 *op = A.out + ((long long)t * A.hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) op[e] = __float2bfloat16_rn(sum > 0.0f ? o[e] / sum : 0.0f);
}

gdn_status check(const gdn_attn_dims *d) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->B < 0 || d->n_tokens < 0 || d->n_groups < 0 || d->n_groups > d->B)
    return fail(GDN_ERR_SHAPE, "B and n_tokens must be >= 0 and n_groups in [0, B]");
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->n_q_heads % d->n_kv_heads != 0 ||
      d->n_q_heads / d->n_kv_heads > 64 || d->n_kv_heads > 4096)
    return fail(GDN_ERR_SHAPE, "n_q_heads must be a multiple of n_kv_heads, at most 64 per key head");
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (d->scale != d->scale) return fail(GDN_ERR_ARG, "scale must be a number");
  if (d->q_stride % 8 != 0 || d->kv_stride % 8 != 0)
    return fail(GDN_ERR_SHAPE, "token strides must be multiples of 8 elements");
  if (d->q_stride < (long long)d->n_q_heads * d->head_dim || d->kv_stride < (long long)d->n_kv_heads * d->head_dim)
    return fail(GDN_ERR_SHAPE, "token strides must cover the heads");
  if (d->q_stride > (1LL << 32) || d->kv_stride > (1LL << 32))
    return fail(GDN_ERR_SHAPE, "token strides must be at most 2^32 elements");
  if (d->kv_rows < 0 || d->kv_rows > (1LL << 31) - 1) return fail(GDN_ERR_SHAPE, "kv_rows must be in [0, 2^31)");
  return GDN_OK;
}

Args make_args(const gdn_attn_dims *d, const void *q, const void *k, const void *v, void *out) {
  Args A = {};
  A.B = d->B;
  A.T = d->T;
  A.n_tokens = d->n_tokens;
  A.n_groups = d->n_groups;
  A.hq = d->n_q_heads;
  A.hk = d->n_kv_heads;
  A.G = d->n_q_heads / d->n_kv_heads;
  A.scale = d->scale;
  A.qs = d->q_stride;
  A.kvs = d->kv_stride;
  A.kv_rows = d->kv_rows;
  A.q = static_cast<const bf16 *>(q);
  A.k = static_cast<const bf16 *>(k);
  A.v = static_cast<const bf16 *>(v);
  A.out = static_cast<bf16 *>(out);
  return A;
}

template <bool SHARED>
gdn_status launch(Args &A, int D, cudaStream_t st) {
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  A.status = dev->status;
  const dim3 grid((unsigned)(((long long)A.n_tokens * A.hq + 3) / 4));
  if (D == 64) launch_pdl(attn_rows_kernel<64, SHARED>, grid, dim3(128), 0, st, A);
  if (D == 128) launch_pdl(attn_rows_kernel<128, SHARED>, grid, dim3(128), 0, st, A);
  if (D == 256) launch_pdl(attn_rows_kernel<256, SHARED>, grid, dim3(128), 0, st, A);
  return check_launch(SHARED ? "attn_shared_prefix" : "attn_prefill");
}

}  // namespace attn
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_attn_prefill(const gdn_attn_dims *d, const void *q, const void *k, const void *v,
                            const int32_t *cu_seqlens, const int32_t *kv_start, const int32_t *kv_len, void *out,
                            void *stream) {
  GDN_TRY(attn::check(d));
  if (d->B == 0 || d->n_tokens == 0) return GDN_OK;  // empty tensors may have no address
  if ((kv_start == nullptr) != (kv_len == nullptr))
    return fail(GDN_ERR_ARG, "kv_start and kv_len must both be given or both be NULL");
  GDN_TRY(check_ptr(q, "q"));
  GDN_TRY(check_ptr(k, "k"));
  GDN_TRY(check_ptr(v, "v"));
  GDN_TRY(check_ptr(out, "out"));
  GDN_TRY(check_ptr(cu_seqlens, "cu_seqlens", 4));
  if (kv_start) {
    GDN_TRY(check_ptr(kv_start, "kv_start", 4));
    GDN_TRY(check_ptr(kv_len, "kv_len", 4));
  }
  attn::Args A = attn::make_args(d, q, k, v, out);
  A.cu = cu_seqlens;
  A.kv_start = kv_start;
  A.kv_len = kv_len;
  return attn::launch<false>(A, d->head_dim, static_cast<cudaStream_t>(stream));
}

size_t gdn_attn_workspace_size(const gdn_attn_dims *d) {
  if (attn::check(d) != GDN_OK) return 0;
  return 256;
}

gdn_status gdn_attn_shared_prefix(const gdn_attn_dims *d, const void *q, const void *k, const void *v,
                                  const int32_t *group_rows, const int32_t *prefix_start, const int32_t *prefix_len,
                                  const int32_t *suffix_start, const int32_t *suffix_len, const int32_t *q_len,
                                  void *out, void *workspace, size_t workspace_bytes, void *stream) {
  GDN_TRY(attn::check(d));
  if (d->T < 1 || d->T > 64) return fail(GDN_ERR_SHAPE, "T must be in [1, 64]");
  if ((long long)d->B * d->T != d->n_tokens) return fail(GDN_ERR_SHAPE, "n_tokens must be B * T");
  if (d->B == 0) return GDN_OK;
  GDN_TRY(check_ptr(q, "q"));
  GDN_TRY(check_ptr(k, "k"));
  GDN_TRY(check_ptr(v, "v"));
  GDN_TRY(check_ptr(out, "out"));
  if (d->n_groups > 0) {
    GDN_TRY(check_ptr(group_rows, "group_rows", 4));
    GDN_TRY(check_ptr(prefix_start, "prefix_start", 4));
    GDN_TRY(check_ptr(prefix_len, "prefix_len", 4));
  }
  GDN_TRY(check_ptr(suffix_start, "suffix_start", 4));
  GDN_TRY(check_ptr(suffix_len, "suffix_len", 4));
  if (q_len) GDN_TRY(check_ptr(q_len, "q_len", 4));
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < gdn_attn_workspace_size(d))
    return fail(GDN_ERR_WORKSPACE, "workspace missing, not 256-byte aligned, or too small");
  attn::Args A = attn::make_args(d, q, k, v, out);
  A.group_rows = group_rows;
  A.prefix_start = prefix_start;
  A.prefix_len = prefix_len;
  A.suffix_start = suffix_start;
  A.suffix_len = suffix_len;
  A.q_len = q_len;
  return attn::launch<true>(A, d->head_dim, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
