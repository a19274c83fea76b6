// gdn_attn_kv4: attention of decode and verify rows over a paged cache held in
// 4 bits.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max), over the keys
//   that the token sees, with K and V read from their codes and scales.
//
// Bound by the cache's bytes, 9/8 of one a key channel pair, as long as turning
// 4 bits into fp16 costs less than reading them. So the codes become matrix
// operands in registers: the keys (and, for the second product, the channels)
// are the 16 rows of a warp-level product and the queries its 8 columns, and
// nothing dequantised is ever stored. tcgen05 takes its operands from shared
// memory, where a tile of 128 keys in fp16 would be written and read again for at
// most 8 useful columns out of a decode step's handful of queries.
//
//   - Scores S^T = K Q^T: a lane holds a quarter of two keys' channels. The order
//     of the channels in the product is free, so the eight codes of a 32-bit word
//     go where they come out: nibble i and i + 4 form a pair. (w << 2) and (w >> 6)
//     put two nibbles each at the mantissa's bits 2 and 6; with the exponents of 256
//     and 16 that is 256 + u and 16 + u, and one paired fp16 multiply-add with s and
//     -264 s or -24 s gives (u - 8) s exactly (s has 4 significant bits, 264 = 33 * 8):
//     10 instructions for 8 numbers.
//   - Output O^T = V^T P^T: a lane holds 4 keys of an eighth of the channels;
//     byte permutes put two keys' nibbles of one channel into one register. The
//     probabilities move from the scores' layout to the operand's by 8x8
//     transposes between lanes.
//   - The running maximum is a reference that is only moved when a score exceeds
//     it by 2^8 (fp16 holds the probabilities up to there): most tiles need one
//     vote and no exchange between lanes.
//
// A page's block of one head is contiguous: one bulk copy into a ring of stages.
// The warps issue them in turn, two pages behind the slowest, from a list of the
// share's blocks that all threads write 128 at a time (a fifth warp for the copies
// would take a quarter of the registers of an SM's partition). Four warps take 16
// keys of a page each, with statistics and accumulators of their own that meet at
// the end of a segment. The (row, key head, query tile, page) sequence is dealt out
// in equal shares to a CTA each, so a share may begin and end inside a row: a second
// kernel joins those rows' parts.
#include <cuda_fp16.h>
#include <math.h>

#include "gdn_check.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace attn_kv4 {

using namespace kv4;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxCtas = 640;
constexpr float kNone = -3.0e38f;              // a reference below every score
constexpr float kLag = 8.0f;                   // scores may exceed the reference by 2^8
constexpr int kLeast = 2;                      // pages that are worth a CTA

struct Header {  // of the row part that a CTA's share begins and does not end
  int b, unit, last, pad;  // last: the CTA that ends it; -1: none
};

struct Args {
  int B, T, hq, hk, G, n_pages, max_pages, tiles;  // tiles: query tiles of a key head
  float scale, out_mul;  // the pool's exponents are in them
  long long qs;
  const bf16 *q;
  const uint8_t *pool;
  const int32_t *table, *kv_len, *q_len;
  bf16 *out;
  Header *header;  // [gridDim.x]
  float *stats;    // [2 gridDim.x][columns][2]: reference, sum; a NaN reference: the row is bad
  float *part;     // [2 gridDim.x][columns / 8][D / 64][8][64]
  unsigned int *status;
};

template <int D, int NT>
struct Shape {
  static constexpr int N = 8 * NT;              // query columns
  static constexpr bool kQRegs = NT * D <= 128; // the queries stay in registers
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 4 : 6;
  static constexpr int kBlock = block_bytes(D);
  static constexpr int kSteps = D / 16;         // products of 16 channels
  static constexpr int kMeetD = D == 128 ? 128 : 64;  // channels of the warps' meeting at a time
  static constexpr int kPad = kMeetD + 4;
  static constexpr int kMeet = kWarps * 8 * kPad * 4;
  static constexpr int kQ = kQRegs ? 0 : kSteps * NT * 32 * 8;
  static constexpr int kBytes = kStages * kBlock + kMeet + kQ;
  static constexpr int kCtas = NT * D >= 512 ? 2 : NT > 1 || D > 128 ? 3 : 4;  // on an SM, as the accumulators' registers allow
};

// A row's tokens of the cache, -1 where its numbers are bad.
__device__ __forceinline__ int row_len(const Args &A, int b, int &ql) {
  const int len = A.kv_len[b];
  ql = A.q_len ? A.q_len[b] : A.T;
  return len < 0 || len > (long long)A.max_pages * kPage || ql < 0 || ql > A.T ? -1 : len;
}
__device__ __forceinline__ int row_pages(const Args &A, int b) {
  int ql;
  return (max(row_len(A, b, ql), 0) + kPage - 1) / kPage;
}

// This CTA's share: X in [x0, x1) of the sequence of all rows' units' pages.
struct Share {
  long long x, x1, row0;  // row0: where row b begins
  int b, n;               // the row, its pages
};
// One row's part of the share: pages [p, p + count) of `unit`; moves on.
struct Segment {
  int b, unit, p, count, n;
  long long end;  // where the unit ends
};
__device__ __forceinline__ bool next_segment(const Args &A, int units, Share &s, Segment &g) {
  if (s.x >= s.x1) return false;
  while (s.x >= s.row0 + (long long)s.n * units) {  // rows without pages are passed over
    s.row0 += (long long)s.n * units;
    s.n = row_pages(A, ++s.b);
  }
  const long long at = s.x - s.row0;
  g.b = s.b;
  g.n = s.n;
  g.unit = (int)(at / s.n);
  g.p = (int)(at - (long long)g.unit * s.n);
  g.count = (int)min((long long)(s.n - g.p), s.x1 - s.x);
  g.end = s.row0 + (long long)(g.unit + 1) * s.n;
  s.x += g.count;
  return true;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose(uint32_t x) {  // of an 8 x 8 fp16 matrix, a row to 4 lanes
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }
// Two e4m3 numbers (the low 16 bits).
__device__ __forceinline__ __half2 e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)w));
  return half2_of(h);
}

// A pair of scales, and what they make of the bias and the exponents.
struct Scale {
  __half2 s, at2, at6;
  __device__ __forceinline__ explicit Scale(__half2 x) : s(x) {
    at2 = __hmul2(x, __float2half2_rn(-264.0f));
    at6 = __hmul2(x, __float2half2_rn(-24.0f));
  }
};
__device__ __forceinline__ __half2 field(uint32_t x, uint32_t mask, uint32_t exponent) {  // (x & mask) | exponent
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(exponent));
  return half2_of(y);
}
// Nibble i of each half of w, times its scale, in v[i]: at the mantissa's bit 2 of 256 it is 256 + u, at bit 6 of 16
// it is 16 + u.
__device__ __forceinline__ void unpack(uint32_t w, const Scale &s, uint32_t (&v)[4]) {
  const uint32_t x = w << 2, y = w >> 6;
  constexpr uint32_t e2 = 0x5c005c00u, e6 = 0x4c004c00u, m2 = 0x003c003cu, m6 = 0x03c003c0u;
  v[0] = bits(__hfma2(field(x, m2, e2), s.s, s.at2));
  v[1] = bits(__hfma2(field(x, m6, e6), s.s, s.at6));
  v[2] = bits(__hfma2(field(y, m2, e2), s.s, s.at2));
  v[3] = bits(__hfma2(field(y, m6, e6), s.s, s.at6));
}

// Where key r of a warp's 16 (as rows of the first product) stands among its tokens, so that the shared-memory reads
// of the second product's lanes, keys 2t, 2t + 1, 2t + 8 and 2t + 9, fall on different banks.
template <int D>
__device__ __forceinline__ constexpr int key_of(int r) {
  return D == 256 ? r : 4 * ((r & 7) >> 1) + (r & 1) + (r >> 3) * 2;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kCtas) attn_kernel(const __grid_constant__ Args A) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  float *s_meet = reinterpret_cast<float *>(smem + S::kStages * S::kBlock);
  uint2 *s_q = reinterpret_cast<uint2 *>(smem + S::kStages * S::kBlock + S::kMeet);
  __shared__ __align__(8) uint64_t s_full[S::kStages], s_empty[S::kStages];
  __shared__ int s_bad[S::kStages];   // the stage's page does not exist
  __shared__ float s_ref[kWarps][S::N], s_sum[kWarps][S::N];
  __shared__ long long s_scan[kWarps], s_row0;
  __shared__ int s_b, s_n;
  __shared__ long long s_list[2 * kThreads];  // where the share's blocks stand in the pool; -1: no such page

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kWarps);
    }
    fence_mbar_init();
  }
  griddep_wait();
  griddep_trigger();

  // ---- the share
  const int units = A.hk * A.tiles, N = gridDim.x, cta = blockIdx.x;
  const int per = (A.B + kThreads - 1) / kThreads;
  const int r0 = min(A.B, tid * per), r1 = min(A.B, r0 + per);
  long long mine = 0;
  for (int b = r0; b < r1; ++b) mine += row_pages(A, b);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) s_scan[warp] = upto;
  if (tid == 0) s_b = -1;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_scan[w];
    total += s_scan[w];
  }
  const long long all = total * units;
  const int used = (int)min((long long)N, (all + kLeast - 1) / kLeast);  // CTAs that get a share
  Share share;
  share.x = cta < used ? all * cta / used : 0;
  share.x1 = cta < used ? all * (cta + 1) / used : 0;
  if (share.x < share.x1) {
    long long row0 = upto - mine;
    if (share.x >= row0 * units && share.x < upto * units) {
      for (int b = r0; b < r1; ++b) {
        const int n = row_pages(A, b);
        if (share.x < (row0 + n) * units) {
          s_b = b;
          s_n = n;
          s_row0 = row0 * units;
          break;
        }
        row0 += n;
      }
    }
  }
  // ---- rows without keys: zeros, dealt out evenly
  for (int b = (int)((long long)A.B * cta / N); b < (int)((long long)A.B * (cta + 1) / N); ++b) {
    int ql;
    const int len = row_len(A, b, ql);
    if (len < 0 && tid == 0) set_status(A.status, GDN_ERR_INDEX);
    if (len != 0) continue;
    uint4 *o = reinterpret_cast<uint4 *>(A.out + (long long)b * A.T * A.hq * D);
    for (int i = tid; i < A.T * A.hq * D / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
  }
  if (tid == 0) A.header[cta].last = -1;
  __syncthreads();
  share.b = s_b;
  share.n = s_n;
  share.row0 = s_row0;
  if (s_b < 0) return;

  // ---- the blocks of the share: entry e is page e of it
  const long long x0 = share.x;
  const uint32_t count = (uint32_t)(share.x1 - x0);  // pages of the share
  Share walk = share;
  auto list = [&](uint32_t e0) {  // entries [e0, e0 + kThreads)
    walk.x = x0 + e0 + tid;
    Segment at;
    long long block = -1;
    if (walk.x < walk.x1) {
      next_segment(A, units, walk, at);
      const int page = A.table[(long long)at.b * A.max_pages + at.p];
      if (page >= 0 && page < A.n_pages) block = (long long)page * A.hk + at.unit / A.tiles;
    }
    s_list[(e0 + tid) % (2 * kThreads)] = block;
  };
  auto copy = [&](uint32_t e, int stage) {  // one thread; the stage is empty
    const long long block = s_list[e % (2 * kThreads)];
    s_bad[stage] = block < 0;
    if (block < 0) {
      set_status(A.status, GDN_ERR_INDEX);
      mbar_arrive(&s_full[stage]);
    } else {
      mbar_arrive_expect_tx(&s_full[stage], S::kBlock);
      bulk_g2s(ring + stage * S::kBlock, A.pool + block * S::kBlock, S::kBlock, &s_full[stage]);
    }
  };
  list(0);
  __syncthreads();
  if (tid == 0)
    for (uint32_t e = 0; e < S::kStages - 2 && e < count; ++e) copy(e, e);

  // ---- the products
  const int row = lane >> 2, t = lane & 3;  // the lane's place in the operands
  const int k_a = key_of<D>(row), k_b = key_of<D>(row + 8);
  Segment g;
  int stage = 0;
  uint32_t parity = 0;  // of the ring's round
  uint32_t done = 0;    // pages of the share
  bool dead = false;
  while (next_segment(A, units, share, g)) {
    int ql;
    const int len = row_len(A, g.b, ql);
    const int head = g.unit / A.tiles, col0 = (g.unit - head * A.tiles) * S::N, cols = A.T * A.G;
    // ---- the queries: column `row` of tile j, channels t D/4 .. of it
    uint2 qf[S::kQRegs ? S::kSteps * NT : 1];
    float f[NT][2];      // scale of columns 2t, 2t + 1
    int sees[NT][2], least = len;  // keys that they see; the fewest of the tile
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float mul = A.scale;
      {
        const int c = col0 + 8 * j + row;
        const bool real = c < cols;
        const int tok = real ? c / A.G : 0;
        const bf16 *q = A.q + ((long long)g.b * A.T + tok) * A.qs + (head * A.G + (real ? c - tok * A.G : 0)) * D + t * (D / 4);
        uint32_t x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 y = real ? *(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0, 0, 0, 0);
          x[4 * i] = y.x;
          x[4 * i + 1] = y.y;
          x[4 * i + 2] = y.z;
          x[4 * i + 3] = y.w;
        }
        uint32_t top2 = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) top2 = __vmaxu2(top2, x[i] & 0x7fff7fffu);
        uint32_t top = max(top2 & 0xffffu, top2 >> 16) >> 7;  // the largest channel's exponent field
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(1, min(253, (int)top));  // 2^(e - 127) and its inverse are both normal
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        mul *= __uint_as_float((uint32_t)e << 23);
        if (S::kQRegs || j % kWarps == warp) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {  // 8 channels, two products
            const uint32_t *y = x + 4 * i;
            float ch[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ch[2 * k] = __uint_as_float(y[k] << 16) * down;
              ch[2 * k + 1] = __uint_as_float(y[k] & 0xffff0000u) * down;
            }
            uint2 b[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              b[k].x = bits(__floats2half2_rn(ch[2 * k], ch[2 * k + 4]));
              b[k].y = bits(__floats2half2_rn(ch[2 * k + 1], ch[2 * k + 5]));
              if constexpr (S::kQRegs)
                qf[(2 * i + k) * NT + j] = b[k];
              else
                s_q[((2 * i + k) * NT + j) * 32 + lane] = b[k];
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[j][k] = __shfl_sync(0xffffffffu, mul, 4 * (2 * t + k));
        const int c = col0 + 8 * j + 2 * t + k, tok = c / A.G;
        sees[j][k] = c < cols && tok < ql ? min(len, max(0, len - ql + tok + 1)) : 0;
      }
    }
    // the tile's first token sees the fewest keys, unless columns or tokens are missing
    const int tok0 = col0 / A.G, tok1 = (min(cols, col0 + S::N) - 1) / A.G;
    least = col0 + S::N <= cols && tok1 < ql ? max(0, len - ql + tok0 + 1) : 0;
    if (!S::kQRegs) __syncthreads();

    float acc[D / 16][NT][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      ref[j][0] = ref[j][1] = kNone;
      sum[j][0] = sum[j][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
    }
    bool bad = false;

    for (int i = 0; i < g.count; ++i, ++done) {
      const int key0 = (g.p + i) * kPage + warp * 16;  // the warp's first key
      if (done % kThreads == kThreads - 16) {
        list(done + 16);
        __syncthreads();
      }
      if ((int)(done % kWarps) == warp && lane == 0 && done + S::kStages - 2 < count && !dead) {
        // the stage that all warps left two pages ago (fresh ones in the first round)
        const int to = stage >= 2 ? stage - 2 : stage + S::kStages - 2;
        if (done + S::kStages - 2 >= S::kStages && !mbar_wait_bounded(&s_empty[to], stage >= 2 ? parity : parity ^ 1)) {
          set_status(A.status, GDN_ERR_TIMEOUT);
          dead = true;
        } else {
          copy(done + S::kStages - 2, to);
        }
      }
      __syncwarp();
      if (!dead && !mbar_wait_bounded(&s_full[stage], parity)) {
        if (lane == 0) set_status(A.status, GDN_ERR_TIMEOUT);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      bad |= dead || s_bad[stage];
      const uint8_t *block = ring + stage * S::kBlock;
      if (!bad && key0 < len) {
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
        const int ka = warp * 16 + k_a, kb = warp * 16 + k_b;
        // ---- scores: a chunk of up to 32 channels (16 bytes) of each key at a time
        constexpr int CH = D < 128 ? 16 : 32, CHUNKS = D / 4 / CH;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          uint32_t wa[CH / 8], wb[CH / 8];
          const int byte = t * (D / 8) + c * 16;
          __half2 sa, sb;
          if constexpr (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2 *>(block + swizzle(ka * 32 + byte));
            const uint2 y = *reinterpret_cast<const uint2 *>(block + swizzle(kb * 32 + byte));
            wa[0] = x.x, wa[1] = x.y, wb[0] = y.x, wb[1] = y.y;
            sa = e4m3x2(block[scales_at(D, 0) + ka * 4 + t] * 0x101u);
            sb = e4m3x2(block[scales_at(D, 0) + kb * 4 + t] * 0x101u);
          } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(block + swizzle(ka * (D / 2) + byte));
            const uint4 y = *reinterpret_cast<const uint4 *>(block + swizzle(kb * (D / 2) + byte));
            wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
            wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
            const int at = t * (D / 64) + c * 2;
            sa = e4m3x2(*reinterpret_cast<const unsigned short *>(block + scales_at(D, 0) + ka * (D / 16) + at));
            sb = e4m3x2(*reinterpret_cast<const unsigned short *>(block + scales_at(D, 0) + kb * (D / 16) + at));
          }
#pragma unroll
          for (int gr = 0; gr < CH / 16; ++gr) {
            const Scale za(gr ? __high2half2(sa) : __low2half2(sa)), zb(gr ? __high2half2(sb) : __low2half2(sb));
#pragma unroll
            for (int w = 2 * gr; w < 2 * gr + 2; ++w) {
              uint32_t va[4], vb[4];
              unpack(wa[w], za, va);
              unpack(wb[w], zb, vb);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int step = c * (CH / 4) + 2 * w + k;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  uint2 b;
                  if constexpr (S::kQRegs)
                    b = qf[step * NT + j];
                  else
                    b = s_q[(step * NT + j) * 32 + lane];
                  mma(s[j], va[2 * k], vb[2 * k], va[2 * k + 1], vb[2 * k + 1], b.x, b.y);
                }
              }
            }
          }
        }
        // ---- probabilities
        const bool edge = key0 + 16 > least;
        const int ja = key0 + k_a, jb = key0 + k_b;
        bool over = false;
        float y[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[j][k] = fmaf(s[j][k], f[j][k & 1], -ref[j][k & 1]);
            if (edge && (k < 2 ? ja : jb) >= sees[j][k & 1]) y[j][k] = -INFINITY;
            over |= y[j][k] > kLag;
          }
        }
        if (__any_sync(0xffffffffu, over)) {  // the references move to the columns' maxima so far
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float fade[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float top = kNone;
              if (!edge || ja < sees[j][k]) top = fmaxf(top, s[j][k] * f[j][k]);
              if (!edge || jb < sees[j][k]) top = fmaxf(top, s[j][k + 2] * f[j][k]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              top = fmaxf(top, ref[j][k]);
              fade[k] = ex2(ref[j][k] - top);
              ref[j][k] = top;
              sum[j][k] *= fade[k];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[j][k] = fmaf(s[j][k], f[j][k & 1], -ref[j][k & 1]);
              if (edge && (k < 2 ? ja : jb) >= sees[j][k & 1]) y[j][k] = -INFINITY;
            }
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[m][j][k] *= fade[k & 1];
          }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[j][k] = ex2(y[j][k]);
          sum[j][0] += y[j][0] + y[j][2];
          sum[j][1] += y[j][1] + y[j][3];
          p[j][0] = transpose(bits(__floats2half2_rn(y[j][0], y[j][1])));
          p[j][1] = transpose(bits(__floats2half2_rn(y[j][2], y[j][3])));
        }
        // ---- output: a word of 8 channels of 4 keys at a time
        const uint8_t *codes = block + codes_at(D, 1), *scales = block + scales_at(D, 1);
        int kv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) kv[k] = warp * 16 + key_of<D>(2 * t + (k & 1) + (k >> 1) * 8);
        uint32_t wv[4][D / 64];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t *at = codes + swizzle(kv[k] * (D / 2) + row * (D / 16));
          if constexpr (D == 64) {
            wv[k][0] = *reinterpret_cast<const uint32_t *>(at);
          } else if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2 *>(at);
            wv[k][0] = x.x, wv[k][1] = x.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(at);
            wv[k][0] = x.x, wv[k][1] = x.y, wv[k][2] = x.z, wv[k][3] = x.w;
          }
        }
        constexpr int GR = D == 256 ? 2 : 1;  // scales of the lane's channels
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          uint32_t e;  // 4 keys' scales
          if constexpr (D == 256) {
            const uint8_t *at = scales + (2 * row + gr) * kPage + warp * 16 + 2 * t;
            e = *reinterpret_cast<const unsigned short *>(at) | (uint32_t)*reinterpret_cast<const unsigned short *>(at + 8) << 16;
          } else {
            e = *reinterpret_cast<const uint32_t *>(scales + (D == 64 ? row >> 1 : row) * kPage + warp * 16 + 4 * t);
          }
          if (key0 + 16 > len) {  // what the page holds behind the row's tokens may be anything
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 - warp * 16 + kv[k] >= len) e &= ~(0xffu << (8 * k));
          }
          const Scale z0(e4m3x2(e)), z1(e4m3x2(e >> 16));
#pragma unroll
          for (int w = gr * (D / 64 / GR); w < (gr + 1) * (D / 64 / GR); ++w) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v0[4], v1[4];
              unpack(__byte_perm(wv[0][w], wv[1][w], h ? 0x7632 : 0x5410), z0, v0);
              unpack(__byte_perm(wv[2][w], wv[3][w], h ? 0x7632 : 0x5410), z1, v1);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                  mma(acc[4 * w + 2 * h + k][j], v0[2 * k], v0[2 * k + 1], v1[2 * k], v1[2 * k + 1], p[j][0], p[j][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[stage]);
      if (++stage == S::kStages) {
        stage = 0;
        parity ^= 1;
      }
    }

    // ---- the four warps meet: 8 columns, kMeetD channels at a time
    const bool whole = g.p == 0 && g.p + g.count == g.n;
    const int slot = 2 * cta + (g.p == 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[j][k] += __shfl_xor_sync(0xffffffffu, sum[j][k], o);
        if (row == 0) {
          s_ref[warp][8 * j + 2 * t + k] = bad ? __int_as_float(0x7fffffff) : ref[j][k];
          s_sum[warp][8 * j + 2 * t + k] = sum[j][k];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float own[2];  // 2^(reference - the warps' largest)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ref[w][8 * j + 2 * t + k]);
        own[k] = ex2(ref[j][k] - top);
      }
      const int c = tid >> 4, part = tid & 15;  // the column and channels that this thread finishes
      float top = kNone, total_sum = 0.0f;
      bool lost = false;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lost |= s_ref[w][8 * j + c] != s_ref[w][8 * j + c];
        top = fmaxf(top, s_ref[w][8 * j + c]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total_sum += s_sum[w][8 * j + c] * ex2(s_ref[w][8 * j + c] - top);
#pragma unroll
      for (int h = 0; h < D / S::kMeetD; ++h) {
        constexpr int ROWS = 8 * S::kMeetD / D;  // a lane holds the D/8 channels from row D/8 on
        if (row / ROWS == h) {
          const int d0 = row % ROWS * (D / 8);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int m = 0; m < D / 16; m += 2)
              *reinterpret_cast<float4 *>(s_meet + (warp * 8 + 2 * t + k) * S::kPad + d0 + 2 * m) =
                  make_float4(acc[m][j][k] * own[k], acc[m][j][k + 2] * own[k], acc[m + 1][j][k] * own[k],
                              acc[m + 1][j][k + 2] * own[k]);
        }
        __syncthreads();
        constexpr int PER = S::kMeetD / 16;  // channels a thread finishes
        float o[PER];
#pragma unroll
        for (int k = 0; k < PER; k += 4) {
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 z = *reinterpret_cast<const float4 *>(s_meet + (w * 8 + c) * S::kPad + part * PER + k);
            x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
          }
          o[k] = x.x, o[k + 1] = x.y, o[k + 2] = x.z, o[k + 3] = x.w;
        }
        const int ch = h * S::kMeetD + part * PER;  // the first of them
        if (whole) {
          const int col = col0 + 8 * j + c;
          if (col < cols && !lost) {
            const int tok = col / A.G;
            const float inv = total_sum == 0.0f ? 0.0f : A.out_mul / total_sum;
            bf16 *out = A.out + (((long long)g.b * A.T + tok) * A.hq + head * A.G + col - tok * A.G) * D + ch;
            uint32_t z[PER / 2];
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
              z[k] = *reinterpret_cast<const uint32_t *>(&x);
            }
            if constexpr (PER == 8)
              *reinterpret_cast<uint4 *>(out) = make_uint4(z[0], z[1], z[2], z[3]);
            else
              *reinterpret_cast<uint2 *>(out) = make_uint2(z[0], z[1]);
          }
        } else {
          float *to = A.part + ((((long long)slot * NT + j) * (D / 64) + ch / 64) * 8 + c) * 64 + ch % 64;
#pragma unroll
          for (int k = 0; k < PER; k += 4) *reinterpret_cast<float4 *>(to + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          if (part == 0 && h == 0)
            *reinterpret_cast<float2 *>(A.stats + ((long long)slot * S::N + 8 * j + c) * 2) =
                make_float2(lost ? __int_as_float(0x7fffffff) : top, total_sum);
        }
        __syncthreads();  // the meeting place and the queries are free again
      }
    }
    if (!whole && g.p == 0 && tid == 0) {
      const int last = (int)((g.end * used + all - 1) / all) - 1;  // the last CTA whose share begins before the unit's end
      A.header[cta] = {g.b, g.unit, last, 0};
    }
  }
}

// The parts of a row that several shares held: CTA (i, slab) joins the one that
// share i began; 8 columns by 64 channels, a part to a warp.
template <int D, int NT>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args A) {
  constexpr int SLABS = NT * (D / 64);
  __shared__ float s_top[8], s_wt[8][8];
  __shared__ float4 s_o[8][128];
  griddep_wait();
  griddep_trigger();
  const int i = blockIdx.x, slab = blockIdx.y, j = slab / (D / 64);
  const Header H = A.header[i];
  if (H.last < 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = H.last - i + 1;
  auto slot_of = [&](int k) { return k == 0 ? 2 * i + 1 : 2 * (i + k); };
  // ---- the columns' largest reference: 8 lanes a part, warps over the parts
  float top = kNone;
  bool lost = false;
  for (int k = tid >> 3; k < n; k += 32) {
    const float r = A.stats[((long long)slot_of(k) * (8 * NT) + 8 * j + (tid & 7)) * 2];
    lost |= r != r;
    top = fmaxf(top, r);
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane < 8) s_wt[warp][lane] = top;
  if (__syncthreads_or(lost)) return;
  if (tid < 8) {
    for (int w = 0; w < 8; ++w) top = fmaxf(top, s_wt[w][tid]);
    s_top[tid] = top;
  }
  __syncthreads();
  // ---- lane: columns lane / 16 + 2 m, channels 4 (lane % 16)
  float4 o[4];
  float l[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    o[m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l[m] = 0.0f;
  }
#pragma unroll 2
  for (int k = warp; k < n; k += 8) {
    const long long slot = slot_of(k);
    const float4 *from = reinterpret_cast<const float4 *>(A.part + (slot * SLABS + slab) * 512);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int c = lane / 16 + 2 * m;
      const float2 st = *reinterpret_cast<const float2 *>(A.stats + (slot * (8 * NT) + 8 * j + c) * 2);
      const float4 x = from[32 * m + lane];
      const float w = ex2(st.x - s_top[c]);
      l[m] += st.y * w;
      o[m].x += x.x * w, o[m].y += x.y * w, o[m].z += x.z * w, o[m].w += x.w * w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    s_o[warp][32 * m + lane] = o[m];
    if (lane % 16 == 0) s_wt[warp][lane / 16 + 2 * m] = l[m];
  }
  __syncthreads();
  if (tid < 128) {
    float4 x = s_o[0][tid];
    const int c = tid / 16;
    float total = s_wt[0][c];
    for (int w = 1; w < 8; ++w) {
      const float4 z = s_o[w][tid];
      x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
      total += s_wt[w][c];
    }
    const int head = H.unit / A.tiles, col = (H.unit - head * A.tiles) * (8 * NT) + 8 * j + c;
    if (col < A.T * A.G) {
      const int tok = col / A.G;
      const float inv = total == 0.0f ? 0.0f : A.out_mul / total;
      bf16 *out = A.out + (((long long)H.b * A.T + tok) * A.hq + head * A.G + col - tok * A.G) * D +
                  slab % (D / 64) * 64 + tid % 16 * 4;
      const __nv_bfloat162 a = __floats2bfloat162_rn(x.x * inv, x.y * inv), b = __floats2bfloat162_rn(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2 *>(out) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
  }
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
  if ((double)d->B * d->T * d->n_q_heads * d->max_pages > 1099511627776.0)
    return fail(GDN_ERR_SHAPE, "B * T * n_q_heads * max_pages must be at most 2^40");
  if (!(fabs(ldexp((double)d->scale, d->k_exp) * 1.4426950408889634) <= 3.4e38))
    return fail(GDN_ERR_ARG, "|scale| 2^k_exp log2(e) must be finite");
  return GDN_OK;
}

// Query tiles of 8 columns that a CTA takes at once: what the columns fill, and the registers hold.
int tiles_at_once(const gdn_attn_kv4_dims *d) {
  const int cols = d->T * (d->n_q_heads / d->n_kv_heads);
  return cols <= 8 ? 1 : cols <= 16 || d->head_dim == 256 ? 2 : 4;
}
size_t part_bytes(int D, int NT) { return (size_t)2 * kMaxCtas * 8 * NT * D * 4; }
size_t stats_bytes(int NT) { return (size_t)2 * kMaxCtas * 8 * NT * 8; }

template <int D, int NT>
gdn_status launch(Args A, int sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  if (cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess)
    return check_launch("attn_kv4");
  // no more CTAs than the rows could fill with pages
  const long long most = (long long)A.B * A.hk * A.tiles * A.max_pages;
  int ctas = sms * S::kCtas < kMaxCtas ? sms * S::kCtas : kMaxCtas;
  if (most < (long long)ctas * kLeast) ctas = most < 2 * kLeast ? 2 : (int)((most + kLeast - 1) / kLeast);
  if (launch_pdl(attn_kernel<D, NT>, dim3(ctas), dim3(kThreads), S::kBytes, stream, A) != cudaSuccess)
    return check_launch("attn_kv4");
  launch_pdl(join_kernel<D, NT>, dim3(ctas, NT * (D / 64)), dim3(256), 0, stream, A);
  return check_launch("attn_kv4");
}

}  // namespace attn_kv4
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_attn_kv4_workspace_size(const gdn_attn_kv4_dims *dims) {
  if (attn_kv4::check_dims(dims) != GDN_OK) return 0;
  const int NT = attn_kv4::tiles_at_once(dims);
  return attn_kv4::kMaxCtas * sizeof(attn_kv4::Header) + attn_kv4::stats_bytes(NT) +
         attn_kv4::part_bytes(dims->head_dim, NT);
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
  const int D = dims->head_dim, NT = attn_kv4::tiles_at_once(dims);
  attn_kv4::Args A = {};
  A.B = dims->B;
  A.T = dims->T;
  A.hq = dims->n_q_heads;
  A.hk = dims->n_kv_heads;
  A.G = A.hq / A.hk;
  A.n_pages = dims->n_pages;
  A.max_pages = dims->max_pages;
  A.tiles = (A.T * A.G + 8 * NT - 1) / (8 * NT);
  A.scale = (float)(ldexp((double)dims->scale, dims->k_exp) * 1.4426950408889634);
  A.out_mul = ldexpf(1.0f, dims->v_exp);
  A.qs = dims->q_stride;
  A.q = static_cast<const bf16 *>(q);
  A.pool = static_cast<const uint8_t *>(pool);
  A.table = page_table;
  A.kv_len = kv_len;
  A.q_len = q_len;
  A.out = static_cast<bf16 *>(out);
  A.header = static_cast<attn_kv4::Header *>(workspace);
  A.stats = reinterpret_cast<float *>(A.header + attn_kv4::kMaxCtas);
  A.part = A.stats + attn_kv4::stats_bytes(NT) / 4;
  A.status = dev->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D == 64)
    return NT == 1 ? attn_kv4::launch<64, 1>(A, dev->sms, st)
                   : NT == 2 ? attn_kv4::launch<64, 2>(A, dev->sms, st) : attn_kv4::launch<64, 4>(A, dev->sms, st);
  if (D == 128)
    return NT == 1 ? attn_kv4::launch<128, 1>(A, dev->sms, st)
                   : NT == 2 ? attn_kv4::launch<128, 2>(A, dev->sms, st) : attn_kv4::launch<128, 4>(A, dev->sms, st);
  return NT == 1 ? attn_kv4::launch<256, 1>(A, dev->sms, st) : attn_kv4::launch<256, 2>(A, dev->sms, st);
}
