// gdn_kv4_store / gdn_kv4_load: tokens' keys and values into 4-bit pages, and
// back to bf16.
//
// Per 16 channels x of a token's head, y = x 2^-exp:
//   s = e4m3(max|y| / 7, in [2^-9, 240]),  u = 8 + rint(y / s) in [1, 15]
//
// Memory-bound in a prompt: 4 bytes a channel pair in, 9/8 out. 8192 tokens of 4 heads
// of 256 stored and loaded: 15.7 us, 86 MB at 5.5 TB/s (79% of a copy's rate, where the
// pages are still in L2 when they are read back); two thirds of the store's issue slots
// are used. 64 tokens of 8 heads of 128: 3 us for both calls, the launches' latency.
//
// A lane takes the 16 channels of one scale of the keys and of the values: 32 bytes of
// bf16, 8 bytes of codes, one scale each. A warp takes 8 groups of 4 tokens, so that a token's 8 code
// pieces and key scales are contiguous, and the value scales of neighbouring tokens
// (which lie together, [d/16][64]) meet in one sector.
//
// The quotient is rounded exactly without a division per channel. y has 8
// significant bits, s at most 4: y/s is either k + 1/2 exactly or at least 2^-10
// from it (y and (k + 1/2) s are both whole multiples of y's last place, which
// is at least 2^-10 s where |y| > 0.4 s). y times the reciprocal of s is off by
// less than 2^-19 (|y/s| < 8), so rounding it to multiples of 2^-16 gives k + 1/2
// exactly where the quotient is, and stays on the right side elsewhere; then it
// is rounded to whole numbers, ties to even: two operations, 192 + q first. max|y| / 7 is a true division: its
// ties (max|y| = 7 times a number of 5 bits) are exact in fp32.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "gdn_check.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {

constexpr int kThreads = 128;

struct Args {
  int n, hk, groups;  // tokens, heads, scales of a token (hk d / 16)
  bool wide;          // k and v allow accesses of 32 bytes
  long long rows;     // of the pool
  long long ks, vs;
  float k_mul, v_mul;  // 2^-exp (store), 2^exp (load)
  bf16 *k, *v;
  const int32_t *index;
  uint8_t *pool;
  unsigned int *status;
};

// This lane's token and group; false where there is none.
struct Place {
  int t, group;
};
__device__ __forceinline__ bool place_of(const Args &A, Place &p) {
  const int lane = threadIdx.x & 31;
  const uint32_t octets = (uint32_t)(A.groups + 7) / 8, w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const uint32_t quad = w / octets;
  const long long t = (long long)quad * 4 + (lane >> 3);
  p.group = (int)(w - quad * octets) * 8 + (lane & 7);
  p.t = (int)t;
  return t < A.n && p.group < A.groups;
}

// The token's pool row, or -1.
__device__ __forceinline__ long long row_of(const Args &A, int t) {
  const long long r = A.index[t];
  if (r < -1 || r >= A.rows) {
    set_status(A.status, GDN_ERR_INDEX);
    return -1;
  }
  return r;
}

// The block of the group's head, and in it the 8 bytes of its keys' codes and their scale byte, and the values'.
template <int D>
struct Where {
  uint8_t *codes, *k_scale, *v_scale;
  __device__ __forceinline__ Where(const Args &A, const Place &p, long long row) {
    constexpr int G = D / kGroup;
    const int head = p.group / G, g = p.group % G, token = (int)(row % kPage);
    uint8_t *block = A.pool + ((row / kPage) * A.hk + head) * (long long)block_bytes(D);
    codes = block + swizzle(token * (D / 2) + g * 8);
    k_scale = block + scales_at(D, 0) + token * G + g;
    v_scale = block + scales_at(D, 1) + g * kPage + token;
  }
};

// 32 bytes, as one access where every token's heads begin on such a boundary.
__device__ __forceinline__ void load32(const bf16 *p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    *reinterpret_cast<uint4 *>(w) = __ldcs(reinterpret_cast<const uint4 *>(p));
    *reinterpret_cast<uint4 *>(w + 4) = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
  }
}
__device__ __forceinline__ void store32(bf16 *p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *(reinterpret_cast<uint4 *>(p) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ float scale_of(uint8_t byte) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3))); }

// 16 channels to their codes; returns the scale byte.
__device__ __forceinline__ uint8_t quantise(const uint32_t (&w)[8], float mul, uint32_t (&code)[2]) {
  uint32_t top2 = 0;  // the largest magnitude's bits: an infinity or NaN is at least 0x7f80
#pragma unroll
  for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, w[i] & 0x7fff7fffu);
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  const float amax = __uint_as_float(top << 16) * mul;
  const float wide = fminf(fmaxf(__fdiv_rn(amax, 7.0f), 0.001953125f), 240.0f);
  const __nv_fp8_storage_t byte = __nv_cvt_float_to_fp8(wide, __NV_SATFINITE, __NV_E4M3);
  const float s = scale_of(byte), r = mul * (1.0f / s);
  // In fp32 1.5 * 2^23 + 8 + q has the code 8 + q as its last bits: the codes are shifted together as they are, and
  // what the numbers' other bits add up to (modulo 2^32) is taken off at the end.
  constexpr float kWhole = 12582912.0f;
  constexpr uint32_t kRest = 0x4b400000u * 0x11111111u;
  const auto code_of = [&](int i) {
    const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    return __fmaf_rn(x, r, 192.0f);  // 192 + q, to multiples of 2^-16
  };
  code[0] = code[1] = 0;
  if (wide > 0.015625f && wide < 240.0f) {  // s is off by at most a 16th: |q| < 7.5
#pragma unroll
    for (int i = 0; i < 16; ++i)
      code[i / 8] += __float_as_uint(__fadd_rn(code_of(i), kWhole + 8.0f - 192.0f)) << (4 * (i % 8));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      code[i / 8] += __float_as_uint(__fadd_rn(fminf(fmaxf(code_of(i), 185.0f), 199.0f), kWhole + 8.0f - 192.0f)) << (4 * (i % 8));
  }
  code[0] -= kRest;
  code[1] -= kRest;
  if (top >= 0x7f80u) {
    code[0] = code[1] = 0x99999999u;
    return 0x7f;  // e4m3 NaN: the group reads back as NaN
  }
  return byte;
}

template <int D>
__global__ void __launch_bounds__(kThreads) store_kernel(const __grid_constant__ Args A) {
  griddep_wait();
  griddep_trigger();
  Place p;
  if (!place_of(A, p)) return;
  uint32_t k[8], v[8], code[2];
  load32(A.k + p.t * A.ks + p.group * kGroup, A.wide, k);
  load32(A.v + p.t * A.vs + p.group * kGroup, A.wide, v);
  const long long row = row_of(A, p.t);
  if (row < 0) return;
  const Where<D> at(A, p, row);
  *at.k_scale = quantise(k, A.k_mul, code);
  *reinterpret_cast<uint2 *>(at.codes + codes_at(D, 0)) = make_uint2(code[0], code[1]);
  *at.v_scale = quantise(v, A.v_mul, code);
  *reinterpret_cast<uint2 *>(at.codes + codes_at(D, 1)) = make_uint2(code[0], code[1]);
}

// 16 codes times their scale to bf16. A nibble at the mantissa's bit 3 of 16 makes 16 + u; times s, less 24 s, that is
// (u - 8) s exactly.
__device__ __forceinline__ void expand(bf16 *to, bool wide, uint2 code, float s) {
  auto bits = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t *>(&h); };
  const __nv_bfloat162 mul = __float2bfloat162_rn(s), add = __float2bfloat162_rn(-24.0f * s);
  uint32_t w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = h ? code.y : code.x;
    uint32_t v[4];  // channels i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = ((i == 0 ? c << 3 : c >> (4 * i - 3)) & 0x00780078u) | 0x41804180u;
      v[i] = bits(__hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x), mul, add));
    }
    w[4 * h] = __byte_perm(v[0], v[1], 0x5410);
    w[4 * h + 1] = __byte_perm(v[2], v[3], 0x5410);
    w[4 * h + 2] = __byte_perm(v[0], v[1], 0x7632);
    w[4 * h + 3] = __byte_perm(v[2], v[3], 0x7632);
  }
  store32(to, wide, w);
}

template <int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const __grid_constant__ Args A) {
  griddep_wait();
  griddep_trigger();
  Place p;
  if (!place_of(A, p)) return;
  const long long row = row_of(A, p.t);
  if (row < 0) return;
  const Where<D> at(A, p, row);
  const uint2 k = *reinterpret_cast<const uint2 *>(at.codes + codes_at(D, 0));
  const uint2 v = *reinterpret_cast<const uint2 *>(at.codes + codes_at(D, 1));
  const uint8_t sk = *at.k_scale, sv = *at.v_scale;
  expand(A.k + p.t * A.ks + p.group * kGroup, A.wide, k, scale_of(sk) * A.k_mul);
  expand(A.v + p.t * A.vs + p.group * kGroup, A.wide, v, scale_of(sv) * A.v_mul);
}

// The checks of both calls; A.n stays 0 where there is nothing to do.
gdn_status arguments(const gdn_kv4_dims *d, const void *k, const void *v, const int32_t *kv_index, const void *pool,
                     bool store, Args &A) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->n_tokens < 0 || d->n_kv_heads < 1 || d->n_kv_heads > 4096)
    return fail(GDN_ERR_SHAPE, "n_tokens must be >= 0 and n_kv_heads in [1, 4096]");
  const int D = d->head_dim;
  if (D != 64 && D != 128 && D != 256) return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (d->n_pages < 0 || d->n_pages >= (1 << 25)) return fail(GDN_ERR_SHAPE, "n_pages must be in [0, 2^25)");
  if (d->k_exp < -32 || d->k_exp > 32 || d->v_exp < -32 || d->v_exp > 32)
    return fail(GDN_ERR_SHAPE, "k_exp and v_exp must be in [-32, 32]");
  if (d->k_stride % 8 != 0 || d->v_stride % 8 != 0)
    return fail(GDN_ERR_SHAPE, "token strides must be multiples of 8 elements");
  const long long width = (long long)d->n_kv_heads * D;
  if (d->k_stride < width || d->v_stride < width) return fail(GDN_ERR_SHAPE, "token strides must cover the heads");
  if (d->k_stride >= (1LL << 32) || d->v_stride >= (1LL << 32))
    return fail(GDN_ERR_SHAPE, "token strides must be below 2^32 elements");
  const long long warps = ((long long)d->n_tokens + 3) / 4 * ((width / kGroup + 7) / 8);
  if (warps > 0x7fffffffLL) return fail(GDN_ERR_SHAPE, "more tokens and heads than a grid holds");
  A = {};
  if (d->n_tokens == 0) return GDN_OK;  // empty tensors may have no address
  GDN_TRY(check_ptr(k, "k"));
  GDN_TRY(check_ptr(v, "v"));
  GDN_TRY(check_ptr(kv_index, "kv_index", 4));
  if (d->n_pages > 0) GDN_TRY(check_ptr(pool, "pool"));
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  A.n = d->n_tokens;
  A.hk = d->n_kv_heads;
  A.groups = (int)(width / kGroup);
  A.rows = (long long)d->n_pages * kPage;
  A.ks = d->k_stride;
  A.vs = d->v_stride;
  A.k_mul = ldexpf(1.0f, store ? -d->k_exp : d->k_exp);
  A.v_mul = ldexpf(1.0f, store ? -d->v_exp : d->v_exp);
  A.k = static_cast<bf16 *>(const_cast<void *>(k));
  A.v = static_cast<bf16 *>(const_cast<void *>(v));
  A.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 | A.ks % 16 | A.vs % 16) == 0;
  A.index = kv_index;
  A.pool = static_cast<uint8_t *>(const_cast<void *>(pool));
  A.status = dev->status;
  return GDN_OK;
}

void launch(const Args &A, int D, bool store, void *stream) {
  const long long warps = ((long long)A.n + 3) / 4 * ((A.groups + 7) / 8);
  const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))), block(kThreads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D == 64) launch_pdl(store ? store_kernel<64> : load_kernel<64>, grid, block, 0, st, A);
  if (D == 128) launch_pdl(store ? store_kernel<128> : load_kernel<128>, grid, block, 0, st, A);
  if (D == 256) launch_pdl(store ? store_kernel<256> : load_kernel<256>, grid, block, 0, st, A);
}

}  // namespace kv4
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_kv4_store(const gdn_kv4_dims *dims, const void *k, const void *v, const int32_t *kv_index,
                                    void *pool, void *stream) {
  kv4::Args A;
  GDN_TRY(kv4::arguments(dims, k, v, kv_index, pool, true, A));
  if (A.n == 0) return GDN_OK;
  kv4::launch(A, dims->head_dim, true, stream);
  return check_launch("kv4_store");
}

extern "C" gdn_status gdn_kv4_load(const gdn_kv4_dims *dims, const void *pool, const int32_t *kv_index, void *k, void *v,
                                   void *stream) {
  kv4::Args A;
  GDN_TRY(kv4::arguments(dims, k, v, kv_index, pool, false, A));
  if (A.n == 0) return GDN_OK;
  kv4::launch(A, dims->head_dim, false, stream);
  return check_launch("kv4_load");
}
