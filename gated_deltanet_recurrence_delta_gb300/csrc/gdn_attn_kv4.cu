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
//   - Scores S^T = K Q^T: a warp takes 16 or 32 keys of a page; a lane holds a
//     quarter of two keys' channels. The order of the channels in the product is
//     free, so the eight codes of a 32-bit word go where they come out: nibble i
//     and i + 4 form a pair. (w << 2) and (w >> 6) put two nibbles each at the
//     mantissa's bits 2 and 6; with the exponents of 256 and 16 that is 256 + u and
//     16 + u, and one paired fp16 multiply-add with s and -264 s or -24 s gives
//     (u - 8) s exactly (s has 4 significant bits, 264 = 33 * 8): 10 instructions
//     for 8 numbers.
//   - Output O^T = V^T P^T: a warp takes a share of the channels for all 64 keys,
//     so that a row's output is one warp's alone; the probabilities go through
//     shared memory, moved from the scores' layout to the operand's by 8x8
//     transposes between lanes. A lane holds 4 keys of 8 channels; byte permutes put
//     two keys' nibbles of one channel into one register.
//   - The running maximum is a reference that is only moved, after the first page,
//     when a probability would exceed 2^15 (fp16 ends at 2^16): the barrier that hands
//     the probabilities over also says whether any did. It is moved to 7 below the
//     maximum: fp16 rounds numbers to no finer than half of 2^-24, which is then 2^-32 of
//     the largest probability. The factor 2^7 is in the products and the sums alike.
//
// A page's block of one head is contiguous: one bulk copy into a ring of stages. At
// a page's barrier all warps have left the page before it, so its stage is filled
// again right behind it. The (row, key head, query tile, page) sequence is dealt out
// in equal shares to a CTA each, a unit's set-up counting as a few pages, so a share
// may begin and end inside a unit, whose parts a second kernel joins. (Joined by the
// last CTA to finish, 16 verify rows take 35 us in place of 28.7, 8 decode rows 12.0 in
// place of 10.8: one SM then reads all of a unit's parts, behind an exchange of
// counters; 64 long decode rows, of few parts, are 1 us faster that way.)
//
// 64 decode rows of 8192 tokens, 32/8 heads of 128 (605 MB): 121.3 us, 5.0 TB/s, 74% of
// a copy's rate. A page of a head is 650 instructions of each of two warps, half of
// them the codes' way into operands; 63% of the issue slots and half the ALU pipe's are
// used, the rest goes to the page's chain (wait, scores, maximum, barrier, output),
// which 16 warps an SM do not hide entirely. 16 verify rows of 8 tokens, 16/4 heads of
// 256 (41.6 MB, 4.5 GFLOP): 28.3 us: 32 query columns take 244 registers, so that 8
// warps an SM are all there are. 8 decode rows of up to 2048 tokens: 10.8 us: start,
// two pages and the join in turn, all latency.
#include <cuda_fp16.h>
#include <math.h>

#include "gdn_check.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace attn_kv4 {

using namespace kv4;

constexpr int kMaxCtas = 1536;
constexpr float kNone = -3.0e38f;  // below every score
constexpr float kTop = 7.0f;       // where a move of the reference leaves the largest score
constexpr float kLag = 15.0f;      // scores may lie above it by this much: fp16 holds probabilities up to 2^16
constexpr int kLeast = 2;          // pages that are worth a CTA (8 and 45 decode rows: 1, 3 the same, 4 a us more)
// Pages that a unit's queries and output are worth (45 odd decode rows 10.0 us with 1, 10.6 with 2; 16 verify rows, of four
// tiles, 30.6 and 28.7, with 3 28.2).
template <int NT>
constexpr int kSetup = NT == 4 ? 3 : NT;
constexpr int kMostParts = 64;     // of a unit, on the average
constexpr int kJoin = 256;         // threads of a join, each with 4 channels of a column
constexpr int kFan = 16;           // parts whose loads it has in flight: a lane of 16 has the statistics of each
constexpr int kMargin = 16;        // positions that the copies may be ahead

struct Args {
  int B, T, hq, hk, G, n_pages, max_pages, tiles;  // tiles: query tiles of a key head
  float scale, out_mul;  // the pool's exponents are in them
  long long qs;
  const bf16 *q;
  const uint8_t *pool;
  const int32_t *table, *kv_len, *q_len;
  bf16 *out;
  int ctas;      // of the attention kernel
  float *stats;  // [2 gridDim.x][columns][2]: reference, sum; a NaN reference: the row is bad
  float *part;   // [2 gridDim.x][columns][D]
  unsigned int *status;
};

// The variant for head size D and tiles of 8 NT query columns (tiles_at_once: as few as hold a key head's columns,
// since a page's codes are turned into operands once for all of them).
// Stages and CTAs of an SM share its memory and registers. One column tile of 128: 2 stages and 8 CTAs (64 rows of
// 8192 tokens 123 us; 3 stages and 6 CTAs 126; 7 CTAs 136; 9, whose registers spill, 140). Four tiles of 256: 3 stages and
// 2 CTAs of 244 registers (16 verify rows 29 us; 3 CTAs, which spill, twice that).
template <int D, int NT>
struct Shape {
  static constexpr int W = D == 256 ? 4 : 2;     // warps: each holds D / W channels' outputs in registers
  static constexpr int kThreads = 32 * W;
  static constexpr int kSubs = 4 / W;            // 16 keys each that a warp scores
  static constexpr int N = 8 * NT;               // query columns
  static constexpr bool kQRegs = NT == 1;        // the queries stay in registers
  static constexpr int kTiles = kQRegs ? 1 : (NT + W - 1) / W;  // query tiles that a warp brings in
  static constexpr int kStages = D == 128 && NT == 1 ? 2 : 3;
  static constexpr int kBlock = block_bytes(D);
  static constexpr int kSteps = D / 16;          // products of 16 channels
  static constexpr int kSlice = D / W;           // channels of a warp's output
  static constexpr int kMt = kSlice / 16;        // tiles of 16 of them
  static constexpr int kP = 2 * 4 * NT * 32 * 8;
  static constexpr int kQ = kQRegs ? 0 : kSteps * NT * 32 * 8;
  static constexpr int kBytes = kStages * kBlock + kP + kQ;
  // on an SM, as shared memory and registers allow
  static constexpr int kCtas = D == 256 ? (NT == 1 ? 3 : NT == 2 ? 3 : 2) : D == 128 ? (NT == 1 ? 8 : NT == 2 ? 6 : 4) : (NT == 1 ? 10 : NT == 2 ? 8 : 5);
};

// A row's tokens of the cache, -1 where its numbers are bad.
__device__ __forceinline__ int row_len(const Args &A, int b, int &ql) {
  const int len = A.kv_len[b];
  ql = A.q_len ? A.q_len[b] : A.T;
  return len < 0 || len > (long long)A.max_pages * kPage || ql < 0 || ql > A.T ? -1 : len;
}
// Positions of each of a row's units: its pages and the set-up, none for a row without tokens.
template <int SETUP>
__device__ __forceinline__ int row_cost(const Args &A, int b) {
  int ql;
  const int len = row_len(A, b, ql);
  return len > 0 ? (len + kPage - 1) / kPage + SETUP : 0;
}

// A walk over positions [x, x1) of the sequence of all rows' units.
template <int SETUP>
struct Walk {
  int x, x1, row0;  // row0: where row b begins
  int b, cost;      // the row, the positions of each of its units
  __device__ __forceinline__ void find_row(const Args &A, int units) {
    while (x >= row0 + cost * units) {  // rows without tokens are passed over
      row0 += cost * units;
      cost = row_cost<SETUP>(A, ++b);
    }
  }
};
// One unit's part of a share: pages [p, p + count), the first at position x.
struct Segment {
  int b, unit, p, count, x;
  int first, end;  // the unit's first page's position, and behind its last
};
template <int SETUP>
__device__ __forceinline__ bool next_segment(const Args &A, int units, Walk<SETUP> &w, Segment &g) {
  while (w.x < w.x1) {
    w.find_row(A, units);
    g.b = w.b;
    g.unit = (w.x - w.row0) / w.cost;
    g.first = w.row0 + g.unit * w.cost + SETUP;
    g.end = g.first - SETUP + w.cost;
    g.x = max(w.x, g.first);
    const int to = min(g.end, w.x1);
    w.x = to;
    g.p = g.x - g.first;
    g.count = to - g.x;
    if (g.count > 0) return true;
  }
  return false;
}

// How `total` positions are dealt out to `used` CTAs.
struct Deal {
  int used, base, rem;
  __device__ __forceinline__ Deal(int total, int n) : used(n), base(n > 0 ? total / n : 0), rem(n > 0 ? total - base * n : 0) {}
  __device__ __forceinline__ int start(int cta) const { return cta * base + min(cta, rem); }
  __device__ __forceinline__ int owner(int x) const {
    const int y = x - rem * (base + 1);
    return y < 0 ? x / (base + 1) : rem + y / base;
  }
};

// What all rows cost, found by each warp alone: 32 rows at a time, of which a lane keeps the sums of `per` in a row. (With
// neighbouring rows to a lane each load is 32 lines: 1000 rows of 150 tokens 84 us in place of 59, 20000 of 60 557 in
// place of 341.)
template <int SETUP>
struct Rows {
  int chunks, per, c0, mine, upto, real;  // the lane's cost in the first 32; its sums, and all before; rows of any cost
  __device__ __forceinline__ int cost(const Args &A, int i, int lane) const {
    const int b = 32 * i + lane;
    return b < A.B ? row_cost<SETUP>(A, b) : 0;
  }
  __device__ __forceinline__ static int scan(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  __device__ __forceinline__ Rows(const Args &A, int lane) {
    chunks = (A.B + 31) / 32;
    per = (chunks + 31) / 32;
    c0 = cost(A, 0, lane);
    mine = __reduce_add_sync(0xffffffffu, c0);
    if (lane > 0) mine = 0;
    int some = c0 > 0;
    if (per == 1) {
#pragma unroll 4
      for (int i = 1; i < chunks; ++i) {
        const int c = cost(A, i, lane), sum = __reduce_add_sync(0xffffffffu, c);
        some += c > 0;
        if (lane == i) mine = sum;
      }
    } else {
      for (int g = 0; g * per < chunks; ++g) {
        int c = 0;
#pragma unroll 4
        for (int i = max(1, g * per); i < min(chunks, (g + 1) * per); ++i) {
          const int x = cost(A, i, lane);
          c += x;
          some += x > 0;
        }
        const int sum = __reduce_add_sync(0xffffffffu, c);
        if (lane == g) mine += sum;
      }
    }
    real = __reduce_add_sync(0xffffffffu, some);
    upto = scan(mine, lane);
  }
  __device__ __forceinline__ Deal deal(const Args &A, int units, int ctas) const {
    const int total = __shfl_sync(0xffffffffu, upto, 31) * units;
    return Deal(total, min(min(ctas, total / kLeast), (int)min((long long)real * units * kMostParts, (long long)ctas)));
  }
  // The row of position w.x, which is one of the sequence's.
  __device__ __forceinline__ void find(const Args &A, int units, int lane, Walk<SETUP> &w) const {
    const int owner = __ffs(__ballot_sync(0xffffffffu, w.x < upto * units)) - 1;
    int first = __shfl_sync(0xffffffffu, upto - mine, owner);
    for (int i = owner * per; i < chunks; ++i) {
      const int c = i == 0 ? c0 : cost(A, i, lane), sum = scan(c, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, w.x < (first + sum) * units);
      if (hit) {
        const int l = __ffs(hit) - 1;
        w.b = 32 * i + l;
        w.cost = __shfl_sync(0xffffffffu, c, l);
        w.row0 = (first + __shfl_sync(0xffffffffu, sum, l) - w.cost) * units;
        return;
      }
      first += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  // Row w.b: its cost and where it begins.
  __device__ __forceinline__ void place(const Args &A, int units, int lane, Walk<SETUP> &w) const {
    const int at = w.b / 32, owner = at / per, l = w.b % 32;
    int first = __shfl_sync(0xffffffffu, upto - mine, owner);
    for (int i = owner * per; i < at; ++i) first += __reduce_add_sync(0xffffffffu, cost(A, i, lane));
    const int c = at == 0 ? c0 : cost(A, at, lane);
    w.cost = __shfl_sync(0xffffffffu, c, l);
    w.row0 = (first + __reduce_add_sync(0xffffffffu, lane < l ? c : 0)) * units;
  }
};

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

// Where key r of 16 (as rows of the first product) stands among its tokens: a lane of the second product, with keys
// 2t, 2t + 1, 2t + 8 and 2t + 9, then holds four tokens in a row, whose scales are one word.
__device__ __forceinline__ constexpr int key_of(int r) { return 4 * ((r & 7) >> 1) + (r & 1) + (r >> 3) * 2; }

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, Shape<D, NT>::kCtas) attn_kernel(const __grid_constant__ Args A) {
  using S = Shape<D, NT>;
  constexpr int W = S::W, kThreads = S::kThreads, SETUP = kSetup<NT>;
  constexpr long long kNoPage = -1, kNothing = -2;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  uint2 *s_p = reinterpret_cast<uint2 *>(smem + S::kStages * S::kBlock);  // [2][4][NT][32]
  uint2 *s_q = s_p + S::kP / 8;                                          // [kSteps][NT][32]
  __shared__ __align__(8) uint64_t s_full[S::kStages];
  __shared__ long long s_list[2 * kThreads];  // where the blocks of the share's positions begin
  __shared__ int s_bad[S::kStages];           // the stage's page does not exist
  __shared__ float s_top[W][S::N], s_sum[W][S::N], s_f[S::N];

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(&s_full[i], 1);
    fence_mbar_init();
  }
  griddep_wait();
  griddep_trigger();

  // ---- the share
  const int units = A.hk * A.tiles, N = gridDim.x, cta = blockIdx.x;
  const Rows<SETUP> rows(A, lane);
  const Deal deal = rows.deal(A, units, N);
  Walk<SETUP> share;
  share.x = cta < deal.used ? deal.start(cta) : 0;
  share.x1 = cta < deal.used ? deal.start(cta + 1) : 0;
  const int x0 = share.x, x1 = share.x1;
  const bool any_share = x0 < x1;
  if (any_share) rows.find(A, units, lane, share);

  // ---- the blocks of the share, kThreads positions at a time
  Walk<SETUP> walk = share;
  auto list = [&](int i0) {
    long long block = kNothing;
    walk.x = x0 + i0 + tid;
    if (walk.x < x1) {
      walk.find_row(A, units);
      const int unit = (walk.x - walk.row0) / walk.cost, p = walk.x - walk.row0 - unit * walk.cost - SETUP;
      if (p >= 0) {
        const int page = A.table[(long long)walk.b * A.max_pages + p];
        block = page >= 0 && page < A.n_pages ? ((long long)page * A.hk + unit / A.tiles) * S::kBlock : kNoPage;
      }
    }
    s_list[(i0 + tid) % (2 * kThreads)] = block;
  };
  uint32_t ahead = 0;  // thread 0: the position whose block is copied next
  const uint32_t span = x1 - x0;
  bool dead = false;   // a wait has run out: no copy is started any more
  auto copy = [&](int stage) {  // thread 0; the stage is free
    long long block;
    do {
      if (ahead >= span || dead) return;
      block = s_list[ahead++ % (2 * kThreads)];
    } while (block == kNothing);
    s_bad[stage] = block < 0;
    if (block < 0) {
      set_status(A.status, GDN_ERR_INDEX);
      mbar_arrive(&s_full[stage]);
    } else {
      mbar_arrive_expect_tx(&s_full[stage], S::kBlock);
      bulk_g2s(ring + stage * S::kBlock, A.pool + block, S::kBlock, &s_full[stage]);
    }
  };
  // ---- the queries of a unit's tile: column `row`, channels t D/4 .. of it; the first unit's as early as may be
  const int row = lane >> 2, t = lane & 3;  // the lane's place in the operands
  const int cols = A.T * A.G;
  uint32_t xq[D / 8];
  auto load_q = [&](const Segment &g, int j) {
    const int head = g.unit / A.tiles, c = (g.unit - head * A.tiles) * S::N + 8 * j + row, tok = c / A.G;
    const bf16 *q = A.q + ((long long)g.b * A.T + tok) * A.qs + (head * A.G + c - tok * A.G) * D + t * (D / 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 y = c < cols ? *(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0, 0, 0, 0);
      xq[4 * i] = y.x;
      xq[4 * i + 1] = y.y;
      xq[4 * i + 2] = y.z;
      xq[4 * i + 3] = y.w;
    }
  };
  Segment g;
  bool more = false;
  if (any_share) {
    list(0);
    more = next_segment(A, units, share, g);
    if (more && (S::kQRegs || warp < NT)) load_q(g, S::kQRegs ? 0 : warp);
    __syncthreads();
    if (tid == 0)
      for (int i = 0; i < S::kStages - 1; ++i) copy(i);
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
  if (!any_share) return;

  // ---- the products
  const int k_a = key_of(row), k_b = key_of(row + 8);
  // offsets inside a block: the lane's codes of its two keys of the warp's first 16, and of its four keys of any 16 (the
  // swizzle of D >= 128 does not depend on which 16)
  const int sub0 = warp * S::kSubs;  // the warp's first 16 keys
  constexpr int LB = D / (16 * W);   // a lane's bytes of a key's row in the second product: 8 channels, or 4
  constexpr int k16 = 8 * D;         // bytes of 16 keys
  const int at_a = sub0 * k16 + swizzle(k_a * (D / 2) + t * (D / 8)), at_b = sub0 * k16 + swizzle(k_b * (D / 2) + t * (D / 8));
  const int at_s = scales_at(D, 0) + (sub0 * 16 + k_a) * (D / 16) + t * (D / 64);  // and the first key's scales
  int at_v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) at_v[k] = codes_at(D, 1) + swizzle((4 * t + k) * (D / 2) + warp * (D / 2 / W) + row * LB);
  const int at_z = scales_at(D, 1) + (warp * S::kSlice + row * (S::kSlice / 8)) / kGroup * kPage + 4 * t;
  int stage = 0, buf = 0, listed = kThreads;  // listed: positions whose blocks are known
  uint32_t parity = 0;  // of the ring's round
  for (bool first = true; more; first = false) {
    int ql;
    const int len = row_len(A, g.b, ql);
    const int head = g.unit / A.tiles, col0 = (g.unit - head * A.tiles) * S::N;
    // ---- the queries in fp16
    uint2 qf[S::kQRegs ? S::kSteps : 1];
    float f[NT][2];    // scale of columns 2t, 2t + 1
    int sees[NT][2];   // keys that they see
    if (!S::kQRegs) __syncthreads();  // the last unit's queries are used no more
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i) {
      const int j = S::kQRegs ? i : i * W + warp;  // each warp its own, or the tiles dealt out
      if (j >= NT) break;
      if (i > 0 || !first) load_q(g, j);
      uint32_t top2 = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top2 = __vmaxu2(top2, xq[i] & 0x7fff7fffu);
      uint32_t top = max(top2 & 0xffffu, top2 >> 16) >> 7;  // the largest channel's exponent field
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max(1, min(253, (int)top));  // 2^(e - 127) and its inverse are both normal
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);
      const float mul = A.scale * __uint_as_float((uint32_t)e << 23);
#pragma unroll
      for (int m = 0; m < D / 32; ++m) {  // 8 channels, two products
        const uint32_t *y = xq + 4 * m;
        float ch[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ch[2 * k] = __uint_as_float(y[k] << 16) * down;
          ch[2 * k + 1] = __uint_as_float(y[k] & 0xffff0000u) * down;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint2 b;
          b.x = bits(__floats2half2_rn(ch[2 * k], ch[2 * k + 4]));
          b.y = bits(__floats2half2_rn(ch[2 * k + 1], ch[2 * k + 5]));
          if constexpr (S::kQRegs)
            qf[2 * m + k] = b;
          else
            s_q[((2 * m + k) * NT + j) * 32 + lane] = b;
        }
      }
      if constexpr (S::kQRegs) {
#pragma unroll
        for (int k = 0; k < 2; ++k) f[0][k] = __shfl_sync(0xffffffffu, mul, 4 * (2 * t + k));
      } else if (t == 0) {
        s_f[8 * j + row] = mul;
      }
    }
    if (!S::kQRegs) __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!S::kQRegs) f[j][k] = s_f[8 * j + 2 * t + k];
        const int c2 = col0 + 8 * j + 2 * t + k, tok2 = c2 / A.G;
        sees[j][k] = c2 >= cols ? len : tok2 < ql ? max(0, len - ql + tok2 + 1) : 0;  // a column of nobody's sees all
      }
    }
    // the tile's first token sees the fewest keys, unless tokens are missing
    const int least = (min(cols, col0 + S::N) - 1) / A.G < ql ? max(0, len - ql + col0 / A.G + 1) : 0;

    float acc[S::kMt][NT][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      ref[j][0] = ref[j][1] = 0.0f;
      sum[j][0] = sum[j][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < S::kMt; ++i) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
    }
    bool bad = false, first_page = true;

    for (int i = 0; i < g.count; ++i) {
      const int key0 = (g.p + i) * kPage;  // the page's first key
      if (!dead && !mbar_wait_bounded(&s_full[stage], parity)) {
        if (lane == 0) set_status(A.status, GDN_ERR_TIMEOUT);
        dead = true;
        // let copies already in flight land before the CTA's memory is released
        for (int k = 0; k < S::kStages - 1 && g.x + i + k < x1; ++k)
          (void)mbar_wait_bounded(&s_full[(stage + k) % S::kStages], parity ^ (stage + k >= S::kStages));
      }
      dead = __any_sync(0xffffffffu, dead);
      bad |= dead || s_bad[stage];
      const uint8_t *block = ring + stage * S::kBlock;

      if (key0 + kPage > len) {  // what the page holds behind the row's tokens may be anything: values of zero
        uint8_t *z = ring + stage * S::kBlock + scales_at(D, 1);
        for (int k = tid; k < D / kGroup * kPage; k += kThreads)
          if (key0 + k % kPage >= len) z[k] = 0;
        fence_proxy_async_smem();  // before the stage is filled again
      }
      // ---- scores, times their scale, less the reference
      float y[S::kSubs][NT][4];
      bool over = first_page;
      if (!bad) {
#pragma unroll
        for (int u = 0; u < S::kSubs; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j) y[u][j][0] = y[u][j][1] = y[u][j][2] = y[u][j][3] = 0.0f;
        // a chunk of up to 32 channels (16 bytes) of each key at a time
        constexpr int CH = D < 128 ? 16 : 32, CHUNKS = D / 4 / CH;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          uint32_t wa[S::kSubs][CH / 8], wb[S::kSubs][CH / 8];
          __half2 sa[S::kSubs], sb[S::kSubs];
          const uint8_t *pa = block + (c ? at_a ^ 16 : at_a), *pb = block + (c ? at_b ^ 16 : at_b), *ps = block + at_s + 2 * c;
#pragma unroll
          for (int u = 0; u < S::kSubs; ++u) {
            if constexpr (D == 64) {  // 16 keys further on the swizzle's bit 9 is the other one
              const int other = (u & 1) << 6;
              const uint2 x = *reinterpret_cast<const uint2 *>(block + ((at_a + u * k16) ^ other));
              const uint2 y = *reinterpret_cast<const uint2 *>(block + ((at_b + u * k16) ^ other));
              wa[u][0] = x.x, wa[u][1] = x.y, wb[u][0] = y.x, wb[u][1] = y.y;
              sa[u] = e4m3x2(ps[u * D] * 0x101u);
              sb[u] = e4m3x2(ps[u * D + 2 * (D / 16)] * 0x101u);
            } else {
              const uint4 x = *reinterpret_cast<const uint4 *>(pa + u * k16);
              const uint4 y = *reinterpret_cast<const uint4 *>(pb + u * k16);
              wa[u][0] = x.x, wa[u][1] = x.y, wa[u][2] = x.z, wa[u][3] = x.w;
              wb[u][0] = y.x, wb[u][1] = y.y, wb[u][2] = y.z, wb[u][3] = y.w;
              sa[u] = e4m3x2(*reinterpret_cast<const unsigned short *>(ps + u * D));
              sb[u] = e4m3x2(*reinterpret_cast<const unsigned short *>(ps + u * D + 2 * (D / 16)));
            }
          }
#pragma unroll
          for (int gr = 0; gr < CH / 16; ++gr) {
#pragma unroll
            for (int w = 2 * gr; w < 2 * gr + 2; ++w) {
              uint32_t va[S::kSubs][4], vb[S::kSubs][4];
#pragma unroll
              for (int u = 0; u < S::kSubs; ++u) {
                unpack(wa[u][w], Scale(gr ? __high2half2(sa[u]) : __low2half2(sa[u])), va[u]);
                unpack(wb[u][w], Scale(gr ? __high2half2(sb[u]) : __low2half2(sb[u])), vb[u]);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int step = c * (CH / 4) + 2 * w + k;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  uint2 b;
                  if constexpr (S::kQRegs)
                    b = qf[step];
                  else
                    b = s_q[(step * NT + j) * 32 + lane];
#pragma unroll
                  for (int u = 0; u < S::kSubs; ++u)
                    mma(y[u][j], va[u][2 * k], vb[u][2 * k], va[u][2 * k + 1], vb[u][2 * k + 1], b.x, b.y);
                }
              }
            }
          }
        }
#pragma unroll
        for (int u = 0; u < S::kSubs; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[u][j][k] = fmaf(y[u][j][k], f[j][k & 1], -ref[j][k & 1]);
        if (key0 + kPage > least) {
#pragma unroll
          for (int u = 0; u < S::kSubs; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (key0 + (sub0 + u) * 16 + (k < 2 ? k_a : k_b) >= sees[j][k & 1]) y[u][j][k] = -INFINITY;
        }
        float top = y[0][0][0];
#pragma unroll
        for (int u = 0; u < S::kSubs; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, y[u][j][k]);
        over = __any_sync(0xffffffffu, top > kLag) || first_page;
      }
      // ---- probabilities, to the warps that need them
      uint2 *to = s_p + buf * (4 * NT * 32);
      float add[NT][2];  // the lane's share of the sums
      auto hand_over = [&] {
#pragma unroll
        for (int j = 0; j < NT; ++j) add[j][0] = add[j][1] = 0.0f;
#pragma unroll
        for (int u = 0; u < S::kSubs; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = ex2(y[u][j][k]);
            add[j][0] += e[0] + e[2];
            add[j][1] += e[1] + e[3];
            uint2 p;
            p.x = transpose(bits(__floats2half2_rn(e[0], e[1])));
            p.y = transpose(bits(__floats2half2_rn(e[2], e[3])));
            to[((sub0 + u) * NT + j) * 32 + lane] = p;
          }
      };
      if (!bad && !over) hand_over();
      const bool moved = __syncthreads_or(over);
      if (tid == 0) copy(stage == 0 ? S::kStages - 1 : stage - 1);  // all warps have left the page before
      if (moved) {  // the references move to kTop below the columns' maxima so far, always at a unit's first page here
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = first_page ? kNone : kTop;
            if (!bad) {
#pragma unroll
              for (int u = 0; u < S::kSubs; ++u) top = fmaxf(top, fmaxf(y[u][j][k], y[u][j][k + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if (row == 0) s_top[warp][8 * j + 2 * t + k] = top;
          }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float fade[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float up = s_top[0][8 * j + 2 * t + k];
#pragma unroll
            for (int w = 1; w < W; ++w) up = fmaxf(up, s_top[w][8 * j + 2 * t + k]);
            // a column that sees no key of a first page sees none at all
            up = up == kNone ? 0.0f : up - kTop;
            fade[k] = first_page ? 1.0f : ex2(-up);
            ref[j][k] += up;
#pragma unroll
            for (int u = 0; u < S::kSubs; ++u) {
              y[u][j][k] -= up;
              y[u][j][k + 2] -= up;
            }
          }
#pragma unroll
          for (int m = 0; m < S::kMt; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[m][j][k] *= fade[k & 1];
          sum[j][0] *= fade[0];
          sum[j][1] *= fade[1];
        }
        if (!bad) hand_over();
        __syncthreads();
      }
      first_page = false;
      // ---- output: the warp's channels of 16 keys at a time
      if (!bad) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          sum[j][0] += add[j][0];
          sum[j][1] += add[j][1];
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint2 p[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) p[j] = to[(ks * NT + j) * 32 + lane];
          uint32_t wv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint8_t *at = block + (D == 64 && ks & 1 ? (at_v[k] + ks * k16) ^ 64 : at_v[k] + ks * k16);
            if constexpr (LB == 4)
              wv[k] = *reinterpret_cast<const uint32_t *>(at);
            else
              wv[k] = *reinterpret_cast<const unsigned short *>(at);
          }
          const uint32_t e = *reinterpret_cast<const uint32_t *>(block + at_z + 16 * ks);  // 4 keys' scales
          const Scale z0(e4m3x2(e)), z1(e4m3x2(e >> 16));
#pragma unroll
          for (int h = 0; h < LB / 2; ++h) {
            uint32_t v0[4], v1[4];
            unpack(__byte_perm(wv[0], wv[1], h ? 0x7632 : 0x5410), z0, v0);
            unpack(__byte_perm(wv[2], wv[3], h ? 0x7632 : 0x5410), z1, v1);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                mma(acc[2 * h + k][j], v0[2 * k], v0[2 * k + 1], v1[2 * k], v1[2 * k + 1], p[j].x, p[j].y);
          }
        }
      }
      buf ^= 1;
      if (++stage == S::kStages) {
        stage = 0;
        parity ^= 1;
      }
      if (g.x + i - x0 >= listed - kMargin && x0 + listed < x1) {  // the same for all threads
        list(listed);
        listed += kThreads;
        __syncthreads();
      }
    }

    // ---- the sums over all warps' keys
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[j][k] += __shfl_xor_sync(0xffffffffu, sum[j][k], o);
        if (row == 0) s_sum[warp][8 * j + 2 * t + k] = sum[j][k];
      }
    const Segment g0 = g;
    more = next_segment(A, units, share, g);
    bad = __syncthreads_or(bad);
    const int ch = warp * S::kSlice + row * (S::kSlice / 8);  // the lane's first channel
    const bool whole = g0.p == 0 && g0.x + g0.count == g0.end;
    if (whole && bad) continue;
    const int slot = 2 * cta + (g0.p == 0);
    bf16 *out = A.out + (long long)g0.b * A.T * A.hq * D + head * A.G * D;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = 8 * j + 2 * t + k, col = col0 + c;
        if (col >= cols) continue;
        float all = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) all += s_sum[w][c];
        if (whole) {
          const int tok = col / A.G;
          const float inv = all == 0.0f ? 0.0f : A.out_mul / all;
          bf16 *to = out + (tok * A.hq + col - tok * A.G) * D + ch;
          uint32_t z[S::kMt];
#pragma unroll
          for (int m = 0; m < S::kMt; ++m) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc[m][j][k] * inv, acc[m][j][k + 2] * inv);
            z[m] = *reinterpret_cast<const uint32_t *>(&x);
          }
          if constexpr (S::kMt == 4)
            *reinterpret_cast<uint4 *>(to) = make_uint4(z[0], z[1], z[2], z[3]);
          else
            *reinterpret_cast<uint2 *>(to) = make_uint2(z[0], z[1]);
        } else {
          float *part = A.part + ((long long)slot * S::N + c) * D + ch;
#pragma unroll
          for (int m = 0; m < S::kMt; m += 2)
            __stcg(reinterpret_cast<float4 *>(part + 2 * m),
                   make_float4(acc[m][j][k], acc[m][j][k + 2], acc[m + 1][j][k], acc[m + 1][j][k + 2]));
          if (row == 0 && warp == 0)
            __stcg(reinterpret_cast<float2 *>(A.stats + ((long long)slot * S::N + c) * 2),
                   make_float2(bad ? __int_as_float(0x7fffffff) : all == 0.0f ? kNone : ref[j][k], all));
        }
      }
  }
}

// The parts of a unit that several CTAs worked on. Where there are more units than CTAs, job blockIdx.x is the unit that
// CTA blockIdx.x begins and does not finish, else it is a unit; kJoin pieces of 4 channels of its columns. Which unit,
// and whose parts, is found while the attention kernel still runs: this one is launched when every CTA of that one has
// passed its own wait, so that whatever wrote the lengths is complete, and no kernel of the call writes them.
template <int D, int NT>
__global__ void __launch_bounds__(kJoin, 3) join_kernel(const __grid_constant__ Args A) {
  constexpr int N = 8 * NT, E = D / 4, SETUP = kSetup<NT>;
  __shared__ int s_job[4];  // the row, its unit, the CTA with the first part, and how many there are
  const int lane = threadIdx.x & 31, units = A.hk * A.tiles;
  if (threadIdx.x < 32) {
    const int job = blockIdx.x;
    const Rows<SETUP> rows(A, lane);
    const Deal deal = rows.deal(A, units, A.ctas);
    Walk<SETUP> w;
    w.b = 0;
    int unit = 0, i0 = 0, n = 0;
    if (A.B * (long long)units <= A.ctas) {
      w.b = job / units;
      unit = job - w.b * units;
      rows.place(A, units, lane, w);
      if (w.cost > 0) {
        i0 = deal.owner(w.row0 + unit * w.cost + SETUP);
        n = deal.owner(w.row0 + (unit + 1) * w.cost - 1) - i0 + 1;
      }
    } else if (job + 1 < deal.used) {
      w.x = deal.start(job + 1);
      rows.find(A, units, lane, w);
      unit = (w.x - w.row0) / w.cost;
      i0 = job;
      const int first = w.row0 + unit * w.cost + SETUP;
      if (first >= deal.start(job) && first < w.x) n = deal.owner(first - SETUP + w.cost - 1) - i0 + 1;
    }
    if (lane == 0) {
      s_job[0] = w.b;
      s_job[1] = unit;
      s_job[2] = i0;
      s_job[3] = n;
    }
  }
  __syncthreads();
  const int b = s_job[0], unit = s_job[1], i0 = s_job[2], n = s_job[3];
  griddep_wait();
  griddep_trigger();
  if (n < 2) return;
#pragma unroll 1
  for (int piece = blockIdx.y * kJoin; piece < N * E; piece += gridDim.y * kJoin) {
    const int head = unit / A.tiles, e = piece + threadIdx.x, c = e / E, col = (unit - head * A.tiles) * N + c;
    if (c - lane / E >= N || col - lane / E >= A.T * A.G) return;  // the warp's first column
    const bool real = c < N && col < A.T * A.G;
    const float4 *part = reinterpret_cast<const float4 *>(A.part) + e;
    const float2 *stats = reinterpret_cast<const float2 *>(A.stats) + c;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = kNone, l = 0.0f;
    bool lost = false;
    auto slot = [&](int k) { return 2 * (i0 + k) + (k == 0); };
#pragma unroll 1
    for (int k = 0; k < n; k += kFan) {
      float4 x[kFan];
      float2 st = make_float2(kNone, 0.0f);  // lane: its column of part k + lane % kFan
      if (real && k + lane % kFan < n) st = __ldcg(stats + slot(k + lane % kFan) * N);
#pragma unroll
      for (int h = 0; h < kFan; ++h) {
        x[h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (real && k + h < n) x[h] = __ldcg(part + slot(k + h) * (N * E));
      }
      lost |= st.x != st.x;
      float next = fmaxf(top, st.x);
#pragma unroll
      for (int m = 1; m < kFan; m <<= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, m));
      const float fade = ex2(top - next), mul = ex2(st.x - next);
      top = next;
      l = l * fade + mul * st.y;
      o.x *= fade, o.y *= fade, o.z *= fade, o.w *= fade;
#pragma unroll
      for (int h = 0; h < kFan; ++h) {
        const float y = __shfl_sync(0xffffffffu, mul, (lane & 16) + h);
        o.x += x[h].x * y, o.y += x[h].y * y, o.z += x[h].z * y, o.w += x[h].w * y;
      }
    }
#pragma unroll
    for (int m = 1; m < kFan; m <<= 1) l += __shfl_xor_sync(0xffffffffu, l, m);
    if (__any_sync(0xffffffffu, lost)) return;  // the row is bad: all its columns are
    if (!real) continue;
    const int tok = col / A.G;
    const float inv = l == 0.0f ? 0.0f : A.out_mul / l;
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), y1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    bf16 *out = A.out + (((long long)b * A.T + tok) * A.hq + head * A.G + col - tok * A.G) * D + e % E * 4;
    *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
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
  const double tiles = (d->T * (d->n_q_heads / d->n_kv_heads) + 7) / 8;
  if (d->B * tiles * d->n_kv_heads * (d->max_pages + 2.0) > 1073741824.0)
    return fail(GDN_ERR_SHAPE, "B * n_kv_heads * ceil(T * n_q_heads / n_kv_heads / 8) * (max_pages + 2) must be at most 2^30");
  if (!(fabs(ldexp((double)d->scale, d->k_exp) * 1.4426950408889634) <= 3.4e38))
    return fail(GDN_ERR_ARG, "|scale| 2^k_exp log2(e) must be finite");
  return GDN_OK;
}

// Query tiles of 8 columns that a CTA takes at once, as the columns fill them (8 tokens of 4 heads a key head, 64 rows of
// 8192 tokens: 234 us with four tiles, 294 with two at a time).
int tiles_at_once(const gdn_attn_kv4_dims *d) {
  const int cols = d->T * (d->n_q_heads / d->n_kv_heads);
  return cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
}
size_t stats_bytes(int NT) { return (size_t)2 * kMaxCtas * 8 * NT * 8; }
size_t part_bytes(int D, int NT) { return (size_t)2 * kMaxCtas * 8 * NT * D * 4; }

template <int D, int NT>
gdn_status launch(Args A, int sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  static std::atomic<uint64_t> ready{0};  // a bit a device: the attribute holds for the process
  const uint64_t bit = 1ull << device_info().id;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess)
      return check_launch("attn_kv4");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  // no more CTAs than the rows could fill
  const long long units = (long long)A.B * A.hk * A.tiles, most = units * (A.max_pages + kSetup<NT>) / kLeast;
  int ctas = sms * S::kCtas < kMaxCtas ? sms * S::kCtas : kMaxCtas;
  if (most < ctas) ctas = most < 1 ? 1 : (int)most;
  A.ctas = ctas;
  if (launch_pdl(attn_kernel<D, NT>, dim3(ctas), dim3(S::kThreads), S::kBytes, stream, A) != cudaSuccess)
    return check_launch("attn_kv4");
  // a CTA takes several pieces of a unit where all would not be on the SMs at once
  const int jobs = units < ctas ? (int)units : ctas, pieces = (S::N * D / 4 + kJoin - 1) / kJoin, fit = 3 * sms / jobs;
  launch_pdl(join_kernel<D, NT>, dim3(jobs, fit < 1 ? 1 : fit < pieces ? fit : pieces), dim3(kJoin), 0, stream, A);
  return check_launch("attn_kv4");
}

}  // namespace attn_kv4
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_attn_kv4_workspace_size(const gdn_attn_kv4_dims *dims) {
  if (attn_kv4::check_dims(dims) != GDN_OK) return 0;
  const int NT = attn_kv4::tiles_at_once(dims);
  return attn_kv4::stats_bytes(NT) + attn_kv4::part_bytes(dims->head_dim, NT);
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
  A.stats = static_cast<float *>(workspace);
  A.part = A.stats + attn_kv4::stats_bytes(NT) / 4;
  A.status = dev->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto pick = [&](auto one, auto two, auto four) { return (NT == 1 ? one : NT == 2 ? two : four)(A, dev->sms, st); };
  if (D == 64) return pick(attn_kv4::launch<64, 1>, attn_kv4::launch<64, 2>, attn_kv4::launch<64, 4>);
  if (D == 128) return pick(attn_kv4::launch<128, 1>, attn_kv4::launch<128, 2>, attn_kv4::launch<128, 4>);
  return pick(attn_kv4::launch<256, 1>, attn_kv4::launch<256, 2>, attn_kv4::launch<256, 4>);
}
