// gdn_attn_kv4: attention of decode and verify rows over a paged cache held in
// 4 bits.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max), over the keys
//   that the token sees, with K and V read from their codes and scales.
//
// One CTA a query head of a token: 128 keys at a time, a thread forms one key's
// score, then the threads share the channels of the output.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "gdn_check.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace attn_kv4 {

using namespace kv4;

struct Args {
  int B, T, hq, hk, n_pages, max_pages;
  float scale, out_mul;  // the pool's exponents are in them
  long long qs;
  const bf16 *q;
  const uint8_t *pool;
  const int32_t *table, *kv_len, *q_len;
  bf16 *out;
  unsigned int *status;
};

constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3(uint8_t b) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3))); }

template <int D>
__device__ __forceinline__ float value_at(const uint8_t *block, int kind, int token, int c) {
  const uint8_t byte = block[codes_at(D, kind) + swizzle(token * (D / 2) + c / 2)];
  const int g = c / kGroup;
  const float s = e4m3(block[scales_at(D, kind) + (kind == 0 ? token * (D / kGroup) + g : g * kPage + token)]);
  return (float)((c & 1 ? byte >> 4 : byte & 15) - 8) * s;
}

template <int D>
__global__ void __launch_bounds__(kThreads) simple_kernel(const __grid_constant__ Args A) {
  __shared__ float s_q[D], s_p[kThreads], s_red[4];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
  const int len = A.kv_len[b], ql = A.q_len ? A.q_len[b] : A.T;
  bool bad = len < 0 || len > (long long)A.max_pages * kPage || ql < 0 || ql > A.T;
  const int32_t *table = A.table + (long long)b * A.max_pages;
  if (!bad)
    for (int i = tid; i < (len + kPage - 1) / kPage; i += kThreads) bad |= table[i] < 0 || table[i] >= A.n_pages;
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(A.status, GDN_ERR_INDEX);
    return;
  }
  const int sees = t < ql ? min(len, max(0, len - ql + t + 1)) : 0;
  const bf16 *q = A.q + ((long long)b * A.T + t) * A.qs + h * D;
  for (int c = tid; c < D; c += kThreads) s_q[c] = ldbf(q + c);
  const int hk = h / (A.hq / A.hk);
  float m = -INFINITY, l = 0.0f, o[(D + kThreads - 1) / kThreads] = {};
  for (int j0 = 0; j0 < sees; j0 += kThreads) {
    __syncthreads();
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j < sees) {
      const uint8_t *block = A.pool + ((long long)table[j / kPage] * A.hk + hk) * block_bytes(D);
      s = 0.0f;
      for (int c = 0; c < D; ++c) s += s_q[c] * value_at<D>(block, 0, j % kPage, c);
      s *= A.scale;
    }
    float top = s;
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float next = fmaxf(m, top), ref = next == -INFINITY ? 0.0f : next;
    const float fade = exp2f(m - ref);
    s_p[tid] = exp2f(s - ref);
    m = next;
    l *= fade;
    __syncthreads();
    const int n = min(kThreads, sees - j0);
    for (int i = 0; i < n; ++i) l += s_p[i];
    for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k) {
      const int c = tid + k * kThreads;
      o[k] *= fade;
      if (c < D)
        for (int i = 0; i < n; ++i)
          o[k] += s_p[i] * value_at<D>(A.pool + ((long long)table[(j0 + i) / kPage] * A.hk + hk) * block_bytes(D), 1,
                                       (j0 + i) % kPage, c);
    }
  }
  bf16 *out = A.out + (((long long)b * A.T + t) * A.hq + h) * D;
  for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k)
    if (tid + k * kThreads < D) out[tid + k * kThreads] = __float2bfloat16(sees > 0 ? o[k] / l * A.out_mul : 0.0f);
}

gdn_status check_dims(const gdn_attn_kv4_dims *d) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->B < 0 || d->B > (1 << 20)) return fail(GDN_ERR_SHAPE, "B must be in [0, 2^20]");
  if (d->T < 1 || d->T > 64) return fail(GDN_ERR_SHAPE, "T must be in [1, 64]");
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads / d->n_kv_heads > 64 ||
      d->n_q_heads > 4096)
    return fail(GDN_ERR_SHAPE, "n_q_heads must be a multiple of n_kv_heads, at most 64 times it and at most 4096");
  const int D = d->head_dim;
  if (D != 64 && D != 128 && D != 256) return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (d->n_pages < 0 || d->n_pages >= (1 << 25)) return fail(GDN_ERR_SHAPE, "n_pages must be in [0, 2^25)");
  if (d->max_pages < 0 || d->max_pages >= (1 << 25)) return fail(GDN_ERR_SHAPE, "max_pages must be in [0, 2^25)");
  if (d->k_exp < -32 || d->k_exp > 32 || d->v_exp < -32 || d->v_exp > 32)
    return fail(GDN_ERR_SHAPE, "k_exp and v_exp must be in [-32, 32]");
  if (d->q_stride % 8 != 0 || d->q_stride < (long long)d->n_q_heads * D || d->q_stride >= (1LL << 32))
    return fail(GDN_ERR_SHAPE, "q_stride must be a multiple of 8 elements that covers the heads, below 2^32");
  if (!(fabs(ldexp((double)d->scale, d->k_exp) * 1.4426950408889634) <= 3.4e38))
    return fail(GDN_ERR_ARG, "|scale| 2^k_exp log2(e) must be finite");
  return GDN_OK;
}

}  // namespace attn_kv4
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_attn_kv4_workspace_size(const gdn_attn_kv4_dims *dims) {
  return attn_kv4::check_dims(dims) == GDN_OK ? 256 : 0;
}

extern "C" gdn_status gdn_attn_kv4(const gdn_attn_kv4_dims *dims, const void *q, const void *pool,
                                   const int32_t *page_table, const int32_t *kv_len, const int32_t *q_len, void *out,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  GDN_TRY(attn_kv4::check_dims(dims));
  if (dims->B == 0) return GDN_OK;  // empty tensors may have no address
  GDN_TRY(check_ptr(q, "q"));
  GDN_TRY(check_ptr(out, "out"));
  GDN_TRY(check_ptr(kv_len, "kv_len", 4));
  if (dims->n_pages > 0) GDN_TRY(check_ptr(pool, "pool"));
  if (dims->max_pages > 0) GDN_TRY(check_ptr(page_table, "page_table", 4));
  if (q_len) GDN_TRY(check_ptr(q_len, "q_len", 4));
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
      workspace_bytes < gdn_attn_kv4_workspace_size(dims))
    return fail(GDN_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdn_attn_kv4_workspace_size");
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  attn_kv4::Args A = {};
  A.B = dims->B;
  A.T = dims->T;
  A.hq = dims->n_q_heads;
  A.hk = dims->n_kv_heads;
  A.n_pages = dims->n_pages;
  A.max_pages = dims->max_pages;
  A.scale = (float)(ldexp((double)dims->scale, dims->k_exp) * 1.4426950408889634);
  A.out_mul = ldexpf(1.0f, dims->v_exp);
  A.qs = dims->q_stride;
  A.q = static_cast<const bf16 *>(q);
  A.pool = static_cast<const uint8_t *>(pool);
  A.table = page_table;
  A.kv_len = kv_len;
  A.q_len = q_len;
  A.out = static_cast<bf16 *>(out);
  A.status = dev->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dims->B > 65535) return fail(GDN_ERR_SHAPE, "B");
  const dim3 grid(A.hq, A.T, A.B), block(attn_kv4::kThreads);
  const int D = dims->head_dim;
  if (D == 64) launch_pdl(attn_kv4::simple_kernel<64>, grid, block, 0, st, A);
  if (D == 128) launch_pdl(attn_kv4::simple_kernel<128>, grid, block, 0, st, A);
  if (D == 256) launch_pdl(attn_kv4::simple_kernel<256>, grid, block, 0, st, A);
  return check_launch("attn_kv4");
}
