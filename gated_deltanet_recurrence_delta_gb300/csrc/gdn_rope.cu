// gdn_head_norm_rope: per-head RMS norms of queries and keys, the position
// rotation and the writing of K and V to their pool rows, in one pass.
//
// statecache.py (squad-0.8b, qev_fast), CacheQwen35's attention layers: q and
// k are RMS-normalised per head, rotated by the token's position (rotary
// offset of the cached prefix) and k, v appended to the layer's cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (y0, y1) -> (y0 cos - y1 sin, y1 cos + y0 sin)
//
// Memory-bound: every element is read and written once, 4 bytes for ~8 flops.
// 8192 tokens, 16 + 4 + 4 heads of 256: 38.4 us, 5.3 TB/s or 79% of the measured
// copy rate; 4095 video tokens, 32 + 8 + 8 heads of 128: 20.8 us, 73%; 64 tokens:
// 3.1 us of latency on the device. What keeps it from the copy rate is latency:
// 126 registers leave two CTAs an SM, 22% of its warps, which wait for their
// loads; issue slots are at 47%. Pairs of channels go through paired fp32
// instructions with the weights folded into the rotation (48 -> 38 us).
// A head lies over D/8 lanes of a warp, 16 bytes per lane, so a warp load
// covers 32/(D/8) heads and the norm is a sum over the head's lanes. The
// angles depend on the token only: a warp forms its lanes' cosines and sines
// once and applies them to all the heads it takes of that token. The next four
// heads' loads are in flight while four are computed.
//
// Angles: positions reach 2^31 while the result needs ~2^-20 of a turn, so the
// turns pos * inv_freq / (2 pi) modulo 1 are formed in 64-bit fixed point:
// F = frac(inv_freq / (2 pi)) * 2^64, and pos * F wraps modulo 2^64 exactly as
// turns wrap modulo 1. The only errors are F's own rounding (2^-54 of a turn
// from the fp64 division, times |pos| < 2^31) and the final fp32 rounding.
#include "gdn_check.h"

namespace gdn {
namespace rope {

struct Args {
  int n, hq, hk, rot, axes, adjacent, slices, items;
  float eps;
  long long qs, ks, vs, kv_rows;
  const bf16 *q, *k, *v, *qw, *kw;
  const int32_t *pos;
  const double *inv_freq;
  const uint8_t *axis;
  const int32_t *kv_index;
  bf16 *qo, *ko, *vo;
  unsigned int *status;
};

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
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 unpack2(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t pack2(f2 x) {
  const float2 v = halves(x);
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads a lane has in flight

// A lane holds 8 channels of a head as two groups of four, lo and hi:
//   pairs (i, i + rot/2): lane c < rot/8 takes channels 4c.. and rot/2 + 4c..,
//     so both halves of its four pairs are its own and no shuffle moves them;
//   adjacent pairs, and channels that do not rotate: channels 8c.. in a row.
// Either way a lane has four angles.
template <int D, bool ADJ>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_kernel(const __grid_constant__ Args A) {
  constexpr int LPH = D / 8, HPI = 32 / LPH;  // lanes of a head, heads of one warp load
  __shared__ uint64_t s_freq[D / 2];
  __shared__ uint8_t s_axis[D / 2];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, half = A.rot / 2;
  if (tid < half) {
    const double t = A.inv_freq[tid] * 0.15915494309189535;  // turns per position
    s_freq[tid] = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
    int a = A.axis ? A.axis[tid] : 0;
    if (a >= A.axes) {
      set_status(A.status, GDN_ERR_INDEX);
      a = 0;
    }
    s_axis[tid] = (uint8_t)a;
  }
  __syncthreads();
  const int c = lane % LPH, sub = lane / LPH;  // this lane's place in the head, the head's place in the load
  const bool rotates = c * 8 < A.rot;
  const int lo = !ADJ && rotates ? 4 * c : 8 * c, hi = !ADJ && rotates ? half + 4 * c : 8 * c + 4;
  auto load = [&](const bf16 *p) {  // 16 bytes of a head
    uint4 x;
    if (ADJ) {
      x = *reinterpret_cast<const uint4 *>(p + lo);
    } else {
      const uint2 a = *reinterpret_cast<const uint2 *>(p + lo), b = *reinterpret_cast<const uint2 *>(p + hi);
      x = make_uint4(a.x, a.y, b.x, b.y);
    }
    return x;
  };
  auto store = [&](bf16 *p, uint4 x) {
    if (ADJ) {
      *reinterpret_cast<uint4 *>(p + lo) = x;
    } else {
      *reinterpret_cast<uint2 *>(p + lo) = make_uint2(x.x, x.y);
      *reinterpret_cast<uint2 *>(p + hi) = make_uint2(x.z, x.w);
    }
  };
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint4 wq = A.qw ? load(A.qw) : ones, wk = A.kw ? load(A.kw) : ones;
  // A token's batches of up to kBatch loads, each of one kind: q, then k, then v.
  constexpr int HPB = HPI * kBatch;  // heads of a batch
  const int bq = (A.hq + HPB - 1) / HPB, bk = (A.hk + HPB - 1) / HPB;
  struct Cursor {  // batch b of token t, up to b1
    unsigned u;
    int t, b, b1;
  };
  const unsigned units = (unsigned)A.n * (unsigned)A.slices, stride = gridDim.x * (kThreads / 32);
  auto enter = [&](Cursor &x) {  // the first batch of unit u: a token, or a slice of its batches
    if (x.u >= units) return;
    x.t = (int)(x.u / (unsigned)A.slices);
    const int slice = (int)(x.u - (unsigned)x.t * (unsigned)A.slices);
    x.b = A.items * slice / A.slices;
    x.b1 = A.items * (slice + 1) / A.slices;
  };
  auto advance = [&](Cursor &x) {
    if (++x.b >= x.b1) {
      x.u += stride;
      enter(x);
    }
  };
  auto kind_of = [&](int b) { return b < bq ? 0 : b < bq + bk ? 1 : 2; };
  auto head_of = [&](int b) { return (b < bq ? b : b < bq + bk ? b - bq : b - bq - bk) * HPB + sub; };
  auto fetch = [&](const Cursor &x, uint4 (&v)[kBatch]) {
    const int kind = kind_of(x.b), h = head_of(x.b), heads = kind == 0 ? A.hq : A.hk;
    const bf16 *src = (kind == 0 ? A.q + x.t * A.qs : kind == 1 ? A.k + x.t * A.ks : A.v + x.t * A.vs) + h * D;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      v[j] = h + j * HPI < heads ? load(src + j * HPI * D) : make_uint4(0, 0, 0, 0);
  };

  Cursor cur = {blockIdx.x * (kThreads / 32) + (tid >> 5), 0, 0, 0};
  if (cur.u >= units) return;
  enter(cur);
  uint4 x[kBatch], ahead[kBatch];
  fetch(cur, x);
  int seen = -1, coef_kind = -1;
  long long row = 0;
  float cs[4], sn[4];
  // pair k of the results is (own pair k) P_k + (partner) Q_k, over the rms: the weights are in the coefficients.
  // Adjacent pairs: the partner is the pair itself, swapped; else pair k ^ 2.
  f2 P[4], Q[4];
  while (cur.u < units) {
    Cursor next = cur;
    advance(next);
    if (next.u < units) fetch(next, ahead);  // in flight while this batch is computed
    if (cur.t != seen) {
      seen = cur.t;
      coef_kind = -1;
      row = A.kv_index ? A.kv_index[cur.t] : cur.t;
      if (row < -1 || row >= A.kv_rows) {
        if (lane == 0) set_status(A.status, GDN_ERR_INDEX);
        row = -1;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = 1.0f;
        sn[e] = 0.0f;
      }
      if (rotates) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * c + e;
          const uint64_t turns = (uint64_t)(int64_t)A.pos[(long long)s_axis[i] * A.n + cur.t] * s_freq[i];
          sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31: half turns
        }
      }
    }
    const int kind = kind_of(cur.b), h0 = head_of(cur.b), heads = kind == 0 ? A.hq : A.hk;
    bf16 *dst = (kind == 0 ? A.qo + (long long)cur.t * A.hq * D : (kind == 1 ? A.ko : A.vo) + row * A.hk * D) + h0 * D;
    const bool kept = kind == 0 || row >= 0;
    if (kind == 2) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (kept && h0 + j * HPI < heads) store(dst + j * HPI * D, x[j]);
    } else {
      if (kind != coef_kind) {
        coef_kind = kind;
        const uint4 wv = kind == 0 ? wq : wk;
        const f2 w[4] = {unpack2(wv.x), unpack2(wv.y), unpack2(wv.z), unpack2(wv.w)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // (y0, y1) -> (y0 cos - y1 sin, y1 cos + y0 sin), y = x w
          if (ADJ) {
            const float2 v = halves(w[k]);
            P[k] = mul2(w[k], pair(cs[k], cs[k]));
            Q[k] = mul2(pair(v.y, v.x), pair(-sn[k], sn[k]));
          } else {
            const int e = 2 * (k & 1);
            P[k] = mul2(w[k], pair(cs[e], cs[e + 1]));
            Q[k] = mul2(w[k ^ 2], k < 2 ? pair(-sn[e], -sn[e + 1]) : pair(sn[e], sn[e + 1]));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const f2 y[4] = {unpack2(x[j].x), unpack2(x[j].y), unpack2(x[j].z), unpack2(x[j].w)};
        const float2 sq = halves(fma2(y[3], y[3], fma2(y[2], y[2], fma2(y[1], y[1], mul2(y[0], y[0])))));
        float ss = sq.x + sq.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.0f / D) + A.eps);
        const f2 scale = pair(inv, inv);
        uint32_t z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f2 far = y[k ^ 2];
          if (ADJ) {
            const float2 v = halves(y[k]);
            far = pair(v.y, v.x);
          }
          z[k] = pack2(mul2(fma2(y[k], P[k], mul2(far, Q[k])), scale));
        }
        if (kept && h0 + j * HPI < heads) store(dst + j * HPI * D, make_uint4(z[0], z[1], z[2], z[3]));
      }
    }
    cur = next;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) x[j] = ahead[j];
  }
}

}  // namespace rope
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_head_norm_rope(const gdn_rope_dims *d, const void *q, const void *k, const void *v,
                                         const void *q_weight, const void *k_weight, const int32_t *positions,
                                         const double *inv_freq, const uint8_t *axis, const int32_t *kv_index,
                                         void *q_out, void *k_out, void *v_out, void *stream) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->n_tokens < 0 || d->n_q_heads < 1 || d->n_kv_heads < 1 || d->n_q_heads > 4096 || d->n_kv_heads > 4096)
    return fail(GDN_ERR_SHAPE, "n_tokens must be >= 0 and head counts in [1, 4096]");
  const int D = d->head_dim;
  if (D != 64 && D != 128 && D != 256) return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (d->rot_dim < 0 || d->rot_dim > D || d->rot_dim % 16 != 0)
    return fail(GDN_ERR_SHAPE, "rot_dim must be a multiple of 16 in [0, head_dim]");
  if (d->n_axes < 1 || d->n_axes > 8) return fail(GDN_ERR_SHAPE, "n_axes must be in [1, 8]");
  if (!(d->eps >= 0.0f)) return fail(GDN_ERR_ARG, "eps must be >= 0");
  if (d->q_stride % 8 != 0 || d->k_stride % 8 != 0 || d->v_stride % 8 != 0)
    return fail(GDN_ERR_SHAPE, "token strides must be multiples of 8 elements");
  if (d->q_stride < (long long)d->n_q_heads * D || d->k_stride < (long long)d->n_kv_heads * D ||
      (v && d->v_stride < (long long)d->n_kv_heads * D))
    return fail(GDN_ERR_SHAPE, "token strides must cover the heads");
  if (d->kv_rows < 0 || (!kv_index && d->kv_rows < d->n_tokens))
    return fail(GDN_ERR_SHAPE, "kv_rows must hold the tokens");
  if (d->n_tokens == 0) return GDN_OK;  // empty tensors may have no address
  GDN_TRY(check_ptr(q, "q"));
  GDN_TRY(check_ptr(k, "k"));
  GDN_TRY(check_ptr(q_out, "q_out"));
  GDN_TRY(check_ptr(k_out, "k_out"));
  if ((v == nullptr) != (v_out == nullptr)) return fail(GDN_ERR_ARG, "v and v_out must both be given or both be NULL");
  if (v) {
    GDN_TRY(check_ptr(v, "v"));
    GDN_TRY(check_ptr(v_out, "v_out"));
  }
  if (q_weight) GDN_TRY(check_ptr(q_weight, "q_weight"));
  if (k_weight) GDN_TRY(check_ptr(k_weight, "k_weight"));
  if (d->rot_dim > 0) {
    GDN_TRY(check_ptr(positions, "positions", 4));
    GDN_TRY(check_ptr(inv_freq, "inv_freq", 8));
  }
  if (kv_index) GDN_TRY(check_ptr(kv_index, "kv_index", 4));
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  rope::Args A = {};
  A.n = d->n_tokens;
  A.hq = d->n_q_heads;
  A.hk = d->n_kv_heads;
  A.rot = d->rot_dim;
  A.axes = d->n_axes;
  A.adjacent = d->adjacent != 0;
  A.eps = d->eps;
  A.qs = d->q_stride;
  A.ks = d->k_stride;
  A.vs = d->v_stride;
  A.kv_rows = d->kv_rows;
  A.q = static_cast<const bf16 *>(q);
  A.k = static_cast<const bf16 *>(k);
  A.v = static_cast<const bf16 *>(v);
  A.qw = static_cast<const bf16 *>(q_weight);
  A.kw = static_cast<const bf16 *>(k_weight);
  A.pos = positions;
  A.inv_freq = inv_freq;
  A.axis = axis;
  A.kv_index = kv_index;
  A.qo = static_cast<bf16 *>(q_out);
  A.ko = static_cast<bf16 *>(k_out);
  A.vo = static_cast<bf16 *>(v_out);
  A.status = dev->status;
  const int per_batch = 32 / (D / 8) * rope::kBatch;
  A.items = (A.hq + per_batch - 1) / per_batch + (v ? 2 : 1) * ((A.hk + per_batch - 1) / per_batch);
  // a token's heads go to several warps where the tokens alone would leave SMs idle
  const long long want = (long long)dev->sms * 32 / A.n;
  A.slices = (int)(want < 1 ? 1 : want > A.items ? A.items : want);
  const long long ctas = ((long long)A.n * A.slices + 7) / 8;
  const dim3 grid((unsigned)(ctas < dev->sms * 2 ? ctas : dev->sms * 2));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 block(rope::kThreads);
  if (D == 64) launch_pdl(A.adjacent ? rope::norm_rope_kernel<64, true> : rope::norm_rope_kernel<64, false>, grid, block, 0, st, A);
  if (D == 128) launch_pdl(A.adjacent ? rope::norm_rope_kernel<128, true> : rope::norm_rope_kernel<128, false>, grid, block, 0, st, A);
  if (D == 256) launch_pdl(A.adjacent ? rope::norm_rope_kernel<256, true> : rope::norm_rope_kernel<256, false>, grid, block, 0, st, A);
  return check_launch("head_norm_rope");
}
