// Causal attention over a pool of cached keys and values on the tcgen05 tensor
// cores: packed prompts (gdn_attn_prefill) and rows that share prefixes
// (gdn_attn_shared_prefix).
//
// statecache.py (squad-0.8b, qev_fast), CacheQwen35's attention layers: a
// chunk's queries attend over the cached prefix and, causally, the chunk;
// generate.py (sparkle, mlx_streaming/mtp), tree_verify_step: several drafted
// paths of one sequence over its one cached prompt.
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// One pass over the keys in blocks of 128 with the running maximum and sum of
// the softmax. The query heads that share a key head are packed into the rows
// of one tile: row r of a tile is (token r / G, head r % G), so 128 / G tokens
// fill the M = 128 of the tensor cores and one kernel serves prompts, drafted
// tokens and single tokens alike. A CTA has
//   - one TMA warp: Q tiles, then K and V blocks through a ring of units of
//     128 keys x min(D, 128) channels, in the order the products take them;
//   - one MMA warp: S = Q K^T into TMEM, O += P V with P read from TMEM;
//   - one warp that clears the rows of V that lie past an extent's end;
//   - one or two softmax groups of four warps, a thread per row: S from TMEM
//     to registers, exponentials, P (bf16) back over S.
// D = 64, 128: two S tiles and two O tiles fill the TMEM's 512 columns, and two
// softmax groups work in turn with the tensor cores. They take either two query
// tiles against the same keys, or (one tile of rows only) the even and the odd
// key blocks, each with its own running maximum, joined at the end.
// D = 256: one O tile of 256 columns and two S tiles in turn, one group.
//
// Running maximum: O is rescaled only where a row's maximum grew by more than
// 2^8 since the value it is measured against; probabilities then reach 2^8 at
// most, which fp32 sums and bf16's exponent carry without loss.
//
// What bounds it. A 128 x 128 x 128 product takes 512 cycles, the softmax of a
// 128 x 128 tile ~1200 of one group (512 of them the exponentials' own), so two
// groups keep up with two S and two O products, 2048 cycles for two tiles and
// a block; measured 2900, as S reads both operands from shared memory at its
// full rate while the copies write there too. One prompt of 8192 tokens, 32/8
// heads, D = 128: 379 us, 1450 TFLOP/s or 75% of the measured bf16 rate; 512
// tokens after 7680 (128 of 152 SMs have a tile): 55 us, 63%; 32 packed prompts
// of 16 to 2048 tokens, D = 256: 340 us, 46%, half of it the start and end of
// each CTA (5 blocks on average between them). Steps that carried it: one
// elected thread issues the products (all lanes waiting and lane 0 issuing
// cost 700 cycles a block: 512 -> 404 us); the block's maximum found beside its
// probabilities instead of before them (404 -> 377 us).
#include <float.h>

#include "gdn_check.h"
#include "gdn_umma.cuh"

namespace gdn {
namespace attn {

constexpr int kMaxCtas = 152;  // CTAs of a shared-prefix call: one per SM
constexpr int BN = 128;        // keys of a block
constexpr float kLog2e = 1.4426950408889634f;
// Rows with T G <= 16 queries per key head have at most so many keys of their own attended in the join, longer extents
// as lines split over the SMs. Join against lines, us a call with L2 flushed, all rows of one length:
//   keys of a row                              64      256      512     1024     1536     2048
//   64 rows, 8 key heads of 128               16/43   25/39    37/49    61/76    82/98  100/117
//   64 rows, 4 key heads of 256               18/40   27/41    41/53    64/81   84/102  101/121
//   8 rows, 4 key heads of 256                12/36   14/27    18/29    25/33    31/35    37/37
//   1 row, 4 key heads of 256                 10/32   12/27    16/28    23/31    29/32    35/33
//   1 row, 8 key heads of 128                 10/29   12/19    14/21    21/24    25/23    30/23
// So the join is the faster one up to here but for a call of one row, whose few CTAs lose up to a third at the end.
constexpr int kOwnKeys = 2048;
constexpr int kLeast = 2;      // blocks of a CTA's stretch at least
// a segment's queries, first latency and stores, in blocks' time: 1, 2, 4 gave 29.4, 27.7, 27.2 us for 8 x 8 verify
// tokens over 8192 keys (D = 256) and 22, 18.3, 17.4 us for 45 rows in 7 groups
constexpr int kSetup = 4;

struct Args {
  int B, T, n_tokens, n_groups, hq, hk, G;
  int TQ;           // tokens of one 128-row tile
  int tile_tokens;  // tokens of one CTA's tiles (TQ, or 2 TQ for two query tiles)
  int max_tiles;    // prefill: tiles the grid covers
  bool out32;       // out is 32-byte aligned
  float c, c_signed;  // |scale| log2(e), and with the sign
  uint32_t idesc_s; // instruction descriptor of S (the sign of scale)
  long long kv_rows, qs, kvs;
  const bf16 *q, *k, *v;  // for the join's own loads
  bf16 *out;
  const int32_t *cu, *kv_start, *kv_len;                  // prefill
  const int32_t *group_rows, *prefix_start, *prefix_len;  // shared prefix
  const int32_t *suffix_start, *suffix_len, *q_len;
  unsigned int *status;
  // shared prefix: partial results. A slot of the prefix region holds 2 (D = 256: 1) tiles of prefix_rows rows,
  // of the suffix region 2 (1) tiles of suffix_rows rows: D/4 times 16 bytes of every row, and (maximum, sum) pairs.
  int prefix_rows, suffix_rows;
  float *prefix_o, *suffix_o;
  float2 *prefix_ml, *suffix_ml;
  int own_keys;     // rows with at most so many keys of their own have them attended in the join (0: none)
  long long *plan;  // cost per CTA, whether the groups are in order, then per entry (first cost, first line)
};

__device__ __forceinline__ bool inside(long long start, long long len, long long rows) {
  return start >= 0 && len >= 0 && start + len <= rows;
}
__device__ __forceinline__ int blocks_of(int keys) { return keys <= 0 ? 0 : (int)(((long long)keys + BN - 1) / BN); }

// ------------------------------------------------------------ what a CTA does
// One segment: the query tokens [t0, t0 + ntok) of one key head over the key
// blocks [b0, b1) of one extent. Token i sees keys below lim0 + step * i.
struct Seg {
  int t0, ntok, head, kv0, len, b0, b1, lim0, step;
  bool pair;  // two query tiles; else one tile, whose blocks alternate between the S tiles
  int slot;   // of the partial results; prefix and suffix lines are told apart by `own`
  bool own;
};

// Entry e of a shared-prefix call: a group's prefix (e < n_groups) or a row's own extent.
struct Entry {
  int first, ntok;  // query tokens
  int kv0, len, lim0, step;
  int tiles, blocks;
  bool ok;
  __device__ long long line_cost() const { return blocks > 0 ? blocks + kSetup : 0; }
  __device__ long long cost(int hk) const { return line_cost() * tiles * hk; }
};

// The group of row b (-1 without groups); the offsets are in order.
__device__ __forceinline__ int group_of(const Args &A, int b) {
  if (A.n_groups == 0) return -1;
  int lo = 0, hi = A.n_groups;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (A.group_rows[m] <= b) lo = m; else hi = m;
  }
  return lo;
}
__device__ __forceinline__ Entry entry_at(const Args &A, int e, bool all_ok) {
  Entry x = {};
  if (e < A.n_groups) {
    const int a = all_ok ? A.group_rows[e] : 0, z = all_ok ? A.group_rows[e + 1] : 0;
    x.kv0 = A.prefix_start[e];
    x.len = A.prefix_len[e];
    x.ok = all_ok && inside(x.kv0, x.len, A.kv_rows);
    x.first = a * A.T;
    x.ntok = (z - a) * A.T;
    x.lim0 = x.len;
  } else {
    const int b = e - A.n_groups;
    const int ql = A.q_len ? A.q_len[b] : A.T;
    x.kv0 = A.suffix_start[b];
    x.len = A.suffix_len[b];
    x.ok = all_ok && ql >= 0 && ql <= A.T && inside(x.kv0, x.len, A.kv_rows);
    x.first = b * A.T;
    x.ntok = x.ok ? ql : 0;
    x.lim0 = x.len - ql + 1;
    x.step = 1;
  }
  if (x.ok && x.ntok > 0) {
    x.tiles = (x.ntok + A.tile_tokens - 1) / A.tile_tokens;
    x.blocks = e >= A.n_groups && x.len <= A.own_keys ? 0 : blocks_of(x.len);
  }
  return x;
}

// A CTA of a shared-prefix call takes the stretch [pos, end) of all lines' cost
// laid end to end (a line: one tile of one key head over one extent), so every
// SM gets the same work whatever the lengths. A line that crosses a border
// leaves partial results in both CTAs; slot (line + CTA) is unique, since each
// next segment moves to the next line or the next CTA.
struct Walk {
  const Args &A;
  bool all_ok;
  int e;
  Entry x;
  long long first_cost, first_line, pos, end;
  int cta;
  __device__ Walk(const Args &a) : A(a) {}
  __device__ bool next(Seg &s) {
    while (pos < end) {
      const long long lc = x.line_cost();
      if (pos >= first_cost + x.cost(A.hk)) {  // the next entry
        first_cost += x.cost(A.hk);
        first_line += (long long)x.tiles * A.hk;
        if (++e >= A.n_groups + A.B) return false;
        x = entry_at(A, e, all_ok);
        continue;
      }
      const long long off = pos - first_cost;  // a 64-bit division takes hundreds of cycles
      const long long li = off < (1LL << 31) ? (long long)((unsigned)off / (unsigned)lc) : off / lc;
      const long long a = first_cost + li * lc;
      const long long z = min(end, a + lc);
      const int tile = (int)(li / A.hk);
      s.head = (int)(li - (long long)tile * A.hk);
      s.b0 = (int)max(pos - a - kSetup, 0LL);
      s.b1 = (int)(z - a - kSetup);
      pos = z;
      if (s.b1 <= s.b0) continue;
      s.t0 = x.first + tile * A.tile_tokens;
      s.ntok = min(A.tile_tokens, x.ntok - tile * A.tile_tokens);
      s.kv0 = x.kv0;
      s.len = x.len;
      s.step = x.step;
      s.lim0 = x.lim0 + x.step * tile * A.tile_tokens;
      s.pair = s.ntok > A.TQ;
      s.own = e >= A.n_groups;
      s.slot = (int)(first_line + li) + cta;
      return true;
    }
    return false;
  }
};

// The block-wide exclusive sum of (a, b) over the threads; totals in ta, tb.
template <int NT>
__device__ void block_scan(long long &a, long long &b, long long &ta, long long &tb, long long (*sm)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += x;
      ib += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sm[warp][0] = ia;
    sm[warp][1] = ib;
  }
  __syncthreads();
  long long pa = 0, pb = 0;
  ta = tb = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) {
      pa = ta;
      pb = tb;
    }
    ta += sm[w][0];
    tb += sm[w][1];
  }
  a = pa + ia - a;
  b = pb + ib - b;
}

constexpr int kSegs = 4;  // segments found ahead
struct Start {  // where the CTA's work begins
  int e, any;
  long long first_cost, first_line;
  Entry entry;
  Seg seg;  // prefill
};

// Prefill: the CTA's one segment. Tiles are numbered through the sequences; the
// grid's first CTAs take the last tiles, which see the most keys.
__device__ bool prefill_seg(const Args &A, Seg &s) {
  const int lane = threadIdx.x & 31;
  s.head = blockIdx.x % A.hk;
  const int want = A.max_tiles - 1 - (int)(blockIdx.x / A.hk);
  int seen = 0;
  for (int b0 = 0; b0 < A.B; b0 += 32) {  // a warp looks at 32 sequences at a time
    const int b = b0 + lane;
    int a = 0, n = 0, kv0 = 0, m = 0;
    if (b < A.B) {
      a = A.cu[b];
      n = A.cu[b + 1] - a;
      kv0 = A.kv_start ? A.kv_start[b] : a;
      m = A.kv_len ? A.kv_len[b] : n;
      if (a < 0 || n < 0 || (long long)a + n > A.n_tokens) {
        set_status(A.status, GDN_ERR_INDEX);
        n = 0;
      }
    }
    const int tiles = (n + A.tile_tokens - 1) / A.tile_tokens;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, want < seen + incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int tile = want - seen - __shfl_sync(0xffffffffu, incl - tiles, l);
      a = __shfl_sync(0xffffffffu, a, l);
      n = __shfl_sync(0xffffffffu, n, l);
      const long long start = __shfl_sync(0xffffffffu, kv0, l);
      m = __shfl_sync(0xffffffffu, m, l);
      if (!inside(start, m, A.kv_rows)) {
        if (lane == 0) set_status(A.status, GDN_ERR_INDEX);
        return false;
      }
      s.t0 = a + tile * A.tile_tokens;
      s.ntok = min(A.tile_tokens, n - tile * A.tile_tokens);
      s.kv0 = (int)start;
      s.len = m;
      s.step = 1;
      s.lim0 = m - n + tile * A.tile_tokens + 1;
      s.b0 = 0;
      s.b1 = blocks_of(min(m, s.lim0 + s.ntok - 1));
      s.pair = s.ntok > A.TQ;
      s.slot = 0;
      s.own = false;
      return true;
    }
    seen += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// ------------------------------------------------------------------- kernel

template <int D>
struct Cfg {
  static constexpr int NS = D == 256 ? 1 : 2;               // query tiles = softmax groups = O tiles
  static constexpr int UC = D < 128 ? D : 128;              // channels of a ring unit
  static constexpr int HB = D / UC;                         // units of a K or V block
  static constexpr int UB = BN * UC * 2;                    // bytes of a unit
  static constexpr int NU = D == 64 ? 10 : 5;               // units of the ring
  static constexpr int QB = 128 * D * 2;                    // bytes of a Q tile
  static constexpr int kBar = NS * QB + NU * UB;
  static constexpr int kBytes = kBar + 8 * (2 * NU + 13 + 2 * kSegs) + 1024;
  static constexpr int kThreads = NS * 128 + 128;
  static constexpr int kO = 256;                            // TMEM column of the first O tile
};

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B over one K = 16 step; A's rows are the TMEM lanes, two bf16 per column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(db), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 32 columns of this warp's lanes, in flight until tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 bytes of one row: each lane of a warp has another row, and the memory pipe takes as long for 16.
__device__ __forceinline__ void st_32bytes(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 at once: (x0, x1) * c + a
__device__ __forceinline__ void fma2(float &x0, float &x1, float c, float a) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mov.b64 z, {%3, %3};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(c), "f"(a));
}
__device__ __forceinline__ void add2(float &s0, float &s1, float x0, float x1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Every wait is bounded; one that runs out raises the CTA's abort flag, which ends the others.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned int *status) {
  if (mbar_try_wait(bar, parity)) return true;
  for (uint32_t i = 0; i < (1u << 22); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *abort) return false;
  }
  *abort = 1;
  set_status(status, GDN_ERR_TIMEOUT);
  return false;
}

// The same by all lanes of a warp, with one outcome.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned int *status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort, status));
}

// Where unit `u` of a segment's K or V block lies in the order of the loads.
// Two query tiles: K0 V0 K1 V1 ...; one tile: K0 K1 V0 K2 V1 ... (S runs two blocks ahead).
__device__ __forceinline__ int k_place(bool pair, int j) { return pair ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_place(bool pair, int j, int n) { return pair ? 2 * j + 1 : j < n - 1 ? 2 * j + 2 : 2 * n - 1; }

// The key blocks that query tile q of the segment sees.
__device__ __forceinline__ int tile_blocks(const Args &A, const Seg &s, int q) {
  const int last = min(s.ntok, (q + 1) * A.TQ) - 1;  // the tile's last token sees the most keys
  return max(0, min(s.b1, blocks_of(min(s.len, s.lim0 + s.step * last))) - s.b0);
}

// Which query slots a segment's tiles take: two tiles both, one tile each slot in turn, so that the next tile can land
// while this one is in use.
struct QSlots {
  int used[2] = {0, 0}, turn = 0;
  __device__ __forceinline__ int first(bool pair, int slots) {
    if (pair || slots == 1) return 0;
    turn ^= 1;
    return turn;
  }
};
// The segment's block whose last rows lie past the extent, if it is among the first n; else -1.
__device__ __forceinline__ int tail_block(const Seg &s, int n) {
  return n > 0 && (long long)(s.b0 + n) * BN > s.len ? n - 1 : -1;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args A) {
  using C = Cfg<D>;
  constexpr int NS = C::NS, NU = C::NU, HB = C::HB, NT = C::kThreads;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char *sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::kBar), *empty = full + NU;
  uint64_t *q_full = empty + NU, *q_empty = q_full + 2, *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 2, *handed = o_full + 2,
           *clean = handed + 1, *dirty = clean + 1, *seg_full = dirty + 1, *seg_empty = seg_full + kSegs;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Start s_start;
  __shared__ Seg s_seg[kSegs];
  __shared__ long long s_scan[NT / 32][2];
  __shared__ float2 s_ml[NS == 2 && !SHARED ? 128 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMma = NS * 4, kTma = NS * 4 + 1, kClean = NS * 4 + 2, kQ = NS * 4 + 3;

  if (tid == 0) {
    for (int i = 0; i < NU; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], NS * 4 + 3);  // the softmax warps, the loads, the products, the cleaning warp
    }
    mbar_init(handed, 4);
    mbar_init(clean, 1);
    mbar_init(dirty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // the four warps of a softmax group
      mbar_init(&o_full[i], 1);
    }
    fence_mbar_init();
    s_abort = 0;
  }
  if (warp == kMma) tmem_alloc(&s_tmem, 512);
  if (tid == kTma * 32) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  griddep_trigger();  // after this CTA's TMEM is allocated: a dependent kernel cannot take it first

  // ---- what this CTA does
  Walk walk(A);
  bool any;
  if (SHARED) {
    const int n = A.n_groups + A.B;
    // the groups' offsets run from 0 to B without a step back, or no row is touched (and no slot used)
    Entry mine = entry_at(A, min(tid, n - 1), true);  // this thread's first entry: its loads run beside the offsets' own
    bool broken = false;
    if (A.n_groups > 0) {
      const int from = A.group_rows[0], to = A.group_rows[A.n_groups];  // two loads in flight at once
      broken = (from != 0) | (to != A.B);
      for (int g = tid; g < A.n_groups; g += NT) broken |= A.group_rows[g] > A.group_rows[g + 1];
    }
    const bool all_ok = !__syncthreads_or(broken);
    if (!all_ok && blockIdx.x == 0 && tid == 0) set_status(A.status, GDN_ERR_INDEX);
    long long total = 0, lines = 0, ta, tb;
    long long my_cost = 0, my_first = 0, my_line = 0;  // of the last entry looked at
    for (int e0 = 0; e0 < n; e0 += NT) {
      const int e = e0 + tid;
      long long a = 0, b = 0;
      if (e < n) {
        if (e0 > 0 || !all_ok) mine = entry_at(A, e, all_ok);
        if (!mine.ok && blockIdx.x == 0) set_status(A.status, GDN_ERR_INDEX);
        a = mine.cost(A.hk);
        b = (long long)mine.tiles * A.hk;
      }
      my_cost = a;
      block_scan<NT>(a, b, ta, tb, s_scan);
      my_first = total + a;
      my_line = lines + b;
      if (blockIdx.x == 0 && e < n) {  // for the join
        A.plan[2 + 2 * e] = my_first;
        A.plan[3 + 2 * e] = my_line;
      }
      total += ta;
      lines += tb;
    }
    const long long up = total + gridDim.x - 1;  // a 64-bit division takes hundreds of cycles
    const long long share = max(up < (1LL << 31) ? (long long)((unsigned)up / gridDim.x) : up / gridDim.x, (long long)kSetup + kLeast);
    if (blockIdx.x == 0 && tid == 0) {
      A.plan[0] = share;
      A.plan[1] = all_ok;
    }
    walk.pos = blockIdx.x * share;
    walk.end = min(walk.pos + share, total);
    any = walk.pos < walk.end;
    if (any) {
      // the entry that holds pos; more entries than threads are gone through again
      long long before = 0, before_lines = 0;
      for (int e0 = 0; e0 < n; e0 += NT) {
        const int e = e0 + tid;
        if (n > NT) {
          long long a = 0, b = 0;
          if (e < n) {
            mine = entry_at(A, e, all_ok);
            a = mine.cost(A.hk);
            b = (long long)mine.tiles * A.hk;
          }
          my_cost = a;
          block_scan<NT>(a, b, ta, tb, s_scan);
          my_first = before + a;
          my_line = before_lines + b;
          before += ta;
          before_lines += tb;
        }
        if (my_first <= walk.pos && walk.pos < my_first + my_cost) {
          s_start.e = e;
          s_start.first_cost = my_first;
          s_start.first_line = my_line;
          s_start.entry = mine;
        }
        if (n > NT && walk.pos < before) break;  // the same for every thread
      }
      __syncthreads();
      walk.all_ok = all_ok;
      walk.e = s_start.e;
      walk.first_cost = s_start.first_cost;
      walk.first_line = s_start.first_line;
      walk.x = s_start.entry;
      walk.cta = blockIdx.x;
    }
  } else {
    if (warp == 0) {
      Seg s = {};
      const bool got = prefill_seg(A, s);
      if (lane == 0) {
        s_start.any = got;
        s_start.seg = s;
      }
    }
    __syncthreads();
    any = s_start.any;
  }
  // The segments one after the other: one thread finds them (its divisions and
  // loads would cost every other thread registers and time) and hands them on
  // through a ring of shared memory. A prefill CTA has one.
  uint32_t seg_count = 0;
  auto next_seg = [&](Seg &s, bool whole_warp) -> bool {
    const uint32_t k = seg_count++;
    if (!SHARED) {
      s = s_start.seg;
      return k == 0;
    }
    const int i = k % kSegs;
    const uint32_t phase = (k / kSegs) & 1;
    if (!(whole_warp ? warp_wait(&seg_full[i], phase, &s_abort, A.status)
                     : wait_or_abort(&seg_full[i], phase, &s_abort, A.status)))
      return false;
    s = s_seg[i];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(&seg_empty[i]);
    return s.ntok > 0;
  };

  if (any) {
    Seg s;
    if (warp == kTma) {
      if (lane == 0) {
        // ---- K and V blocks
        int u = 0;  // units issued
        bool ok = true;
        while (ok && next_seg(s, false)) {
          const int n = tile_blocks(A, s, s.pair ? 1 : 0);
          for (int i = 0; ok && i < 2 * n; ++i) {  // K and V blocks in the order of the products
            bool is_v;
            int j;
            if (s.pair) {
              is_v = i & 1;
              j = i >> 1;
            } else {
              is_v = i == 2 * n - 1 || (i >= 2 && !(i & 1));
              j = i == 2 * n - 1 ? n - 1 : is_v ? i / 2 - 1 : (i + 1) / 2;
            }
            for (int h = 0; h < HB; ++h, ++u) {
              const int st = u % NU;
              if (u >= NU && !wait_or_abort(&empty[st], ((u / NU) - 1) & 1, &s_abort, A.status)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&full[st], C::UB);
              const uint32_t dst = smem_u32(sm) + NS * C::QB + st * C::UB;
#pragma unroll
              for (int c = 0; c < C::UC / 64; ++c)
                tma_load_3d(dst + c * BN * 128, is_v ? &vmap : &kmap, h * C::UC + c * 64, s.head,
                            s.kv0 + (s.b0 + j) * BN, &full[st]);
            }
          }
        }
        // the copies this thread issued have landed before the CTA's memory is released
        for (int i = max(0, u - NU); i < u; ++i) (void)mbar_wait_bounded(&full[i % NU], (i / NU) & 1);
      }
    } else if (warp == kQ) {
      if (lane == 0) {
        // ---- query tiles: a warp of its own, so that the next segment's keys do not wait for this one's queries
        QSlots slots;
        uint32_t found = 0;
        bool ok = true, more = true;
        while (ok && more) {
          more = SHARED ? walk.next(s) : found == 0;
          if (SHARED) {
            const int i = found % kSegs;
            if (found >= kSegs && !wait_or_abort(&seg_empty[i], ((found / kSegs) - 1) & 1, &s_abort, A.status)) break;
            if (!more) s.ntok = 0;  // the end
            s_seg[i] = s;
            mbar_arrive(&seg_full[i]);
          } else {
            s = s_start.seg;
          }
          ++found;
          if (!more) break;
          if (tile_blocks(A, s, s.pair ? 1 : 0) == 0) continue;
          const int first = slots.first(s.pair, NS), tiles = s.pair ? 2 : 1;
          for (int t = 0; ok && t < tiles; ++t) {
            const int q = first + t;
            if (slots.used[q] > 0) ok = wait_or_abort(&q_empty[q], (slots.used[q] - 1) & 1, &s_abort, A.status);
            if (!ok) break;
            ++slots.used[q];
            mbar_arrive_expect_tx(&q_full[q], (uint32_t)((D / 64) * A.TQ * A.G * 128));
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(smem_u32(sm) + q * C::QB + c * 128 * 128, &qmap, c * 64, s.head * A.G, s.t0 + t * A.TQ, &q_full[q]);
          }
        }
        for (int q = 0; q < NS; ++q)
          if (slots.used[q] > 0) (void)mbar_wait_bounded(&q_full[q], (slots.used[q] - 1) & 1);
      }
    } else if (warp == kMma) {
      // ---- products: one thread issues them all
      if (elect_one()) {
        int base = 0;  // units of earlier segments
        QSlots slots;
        uint32_t pc[2] = {0, 0}, cleaned = 0;  // P tiles taken from each buffer, blocks with cleaned tails
        bool ok = true;
        const uint64_t q_desc = umma_desc(smem_u32(sm)), k_desc = umma_desc(smem_u32(sm) + NS * C::QB),
                       v_desc = umma_desc_mn(smem_u32(sm) + NS * C::QB, BN * 128);
        constexpr uint32_t idesc_o = idesc_bf16(128, C::UC) | (1u << 16);  // B (V) is read MN-major
        while (ok && next_seg(s, false)) {
          const int nb0 = tile_blocks(A, s, 0), nb1 = s.pair ? tile_blocks(A, s, 1) : 0;
          const int n = s.pair ? nb1 : nb0;
          if (n == 0) continue;
          const int q_first = slots.first(s.pair, NS);
          for (int q = q_first; ok && q < q_first + (s.pair ? 2 : 1); ++q)
            ok = wait_or_abort(&q_full[q], slots.used[q]++ & 1, &s_abort, A.status);
          if (!ok) break;
          const int tail = tail_block(s, n);  // the block whose V rows past the extent are cleaned first
          bool handed_over = false;
          auto unit_ready = [&](int g) {
            if (ok) ok = wait_or_abort(&full[g % NU], (g / NU) & 1, &s_abort, A.status);
          };
          // S tile `buf` = query tile q times block j; done: the block's last use
          auto issue_s = [&](int q, int buf, int j, bool done) {
            const int g0 = base + k_place(s.pair, j) * HB;
#pragma unroll
            for (int h = 0; h < HB; ++h) {
              unit_ready(g0 + h);
              if (!ok) return;
              tc_fence_after();
              const uint64_t a = q_desc + (uint32_t)((q * C::QB + h * (C::UC / 64) * 128 * 128) >> 4);
              const uint64_t b = k_desc + (uint32_t)(((g0 + h) % NU) * (C::UB >> 4));
#pragma unroll
              for (int x = 0; x < C::UC / 16; ++x) {
                const uint32_t step = (uint32_t)(((x >> 2) * 128 * 128 + (x & 3) * 32) >> 4);
                umma_f16(tmem + buf * 128, a + step, b + step, A.idesc_s, h > 0 || x > 0);
              }
            }
            umma_commit(&s_full[buf]);
            if (done)
              for (int h = 0; h < HB; ++h) umma_commit(&empty[(g0 + h) % NU]);
          };
          // O tile o += P tile `buf` times block j
          auto issue_o = [&](int o, int buf, int j, bool first, bool done) {
            const int g0 = base + v_place(s.pair, j, n) * HB;
            if (j == tail) {  // landed: hand the units to the cleaning warp
              for (int h = 0; h < HB; ++h) unit_ready(g0 + h);
              if (ok && !handed_over) mbar_arrive(dirty);
              handed_over = true;
            }
            if (ok) ok = wait_or_abort(&p_full[buf], pc[buf] & 1, &s_abort, A.status);
            if (!ok) return;
            ++pc[buf];
#pragma unroll
            for (int h = 0; h < HB; ++h) {
              unit_ready(g0 + h);
              if (ok && j == tail && h == 0) ok = wait_or_abort(clean, cleaned & 1, &s_abort, A.status);
              if (!ok) return;
              tc_fence_after();
              const uint64_t b = v_desc + (uint32_t)(((g0 + h) % NU) * (C::UB >> 4));
#pragma unroll
              for (int x = 0; x < BN / 16; ++x)
                umma_ts(tmem + C::kO + o * D + h * C::UC, tmem + buf * 128 + x * 8, b + (uint32_t)(x * 2048 >> 4), idesc_o,
                        !first || x > 0);
            }
            if (done)
              for (int h = 0; h < HB; ++h) umma_commit(&empty[(g0 + h) % NU]);
          };
          if (s.pair) {
            if (nb0 > 0) issue_s(0, 0, 0, false);
            if (ok) issue_s(1, 1, 0, true);
            for (int j = 0; ok && j < n; ++j) {
              if (j < nb0) {
                issue_o(0, 0, j, j == 0, false);
                if (j + 1 == nb0 && ok) umma_commit(&o_full[0]);
                if (j + 1 < nb0 && ok) issue_s(0, 0, j + 1, false);
              }
              if (ok) issue_o(1, 1, j, j == 0, true);
              if (j + 1 == n && ok) umma_commit(&o_full[1]);
              if (j + 1 < n && ok) issue_s(1, 1, j + 1, true);
            }
          } else {
            issue_s(q_first, 0, 0, true);
            if (ok && n > 1) issue_s(q_first, 1, 1, true);
            for (int j = 0; ok && j < n; ++j) {
              const int o = NS == 2 ? (j & 1) : 0;
              issue_o(o, j & 1, j, NS == 2 ? j < 2 : j == 0, true);
              if (ok && (NS == 1 || j + 2 >= n)) umma_commit(&o_full[o]);
              if (ok && j + 2 < n) issue_s(q_first, j & 1, j + 2, true);
            }
          }
          for (int q = q_first; ok && q < q_first + (s.pair ? 2 : 1); ++q) umma_commit(&q_empty[q]);
          if (tail >= 0) ++cleaned;
          base += 2 * n * HB;
        }
      }
    } else if (warp == kClean) {
      // ---- V rows past an extent's end hold anything, and 0 * NaN must not enter the product: zeros over them
      // (lane 0 of the MMA warp says when they have landed: a parity alone does not tell a ring unit's later phases apart)
      int base = 0;
      uint32_t cleaned = 0;
      bool ok = true;
      while (ok && next_seg(s, true)) {
        const int n = tile_blocks(A, s, s.pair ? 1 : 0), tail = tail_block(s, n);
        if (tail >= 0) {
          const int g0 = base + v_place(s.pair, tail, n) * HB, valid = s.len - (s.b0 + tail) * BN;
          ok = warp_wait(dirty, cleaned & 1, &s_abort, A.status);
          if (!ok) break;
          ++cleaned;
          for (int h = 0; h < HB; ++h) {
            const int g = g0 + h;
            (void)mbar_try_wait(&full[g % NU], (g / NU) & 1);  // complete: acquires the copy's writes
            unsigned char *p = sm + NS * C::QB + (g % NU) * C::UB;
            for (int i = valid * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
              for (int c = 0; c < C::UC / 64; ++c)
                *reinterpret_cast<uint4 *>(p + c * BN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(clean);
        }
        base += 2 * n * HB;
      }
    } else if (warp < kMma) {
      // ---- softmax: thread = row of a tile
      const int grp = warp >> 2, wq = warp & 3, row = (wq << 5) + lane;
      uint32_t sc[2] = {0, 0}, oc = 0;  // S tiles taken from each buffer, O tiles waited for
      bool ok = true;
      while (ok && next_seg(s, true)) {
        const int q = s.pair ? grp : 0;
        const int nb = tile_blocks(A, s, q);
        const int tok = row / A.G + q * A.TQ, gh = row - (row / A.G) * A.G;
        const bool real = row < A.TQ * A.G && tok < s.ntok;
        const bool busy = __any_sync(0xffffffffu, real);  // few query rows leave warps without any
        const int lim = real ? min(s.len, s.lim0 + s.step * tok) : 0x7fffffff;
        const int j0 = (!s.pair && NS == 2) ? grp : 0, dj = (!s.pair && NS == 2) ? 2 : 1;
        float top = -INFINITY, sum = 0.0f;  // the maximum that O is measured against (before scaling), the sum
        const uint32_t o_tmem = tmem_at(tmem, wq, C::kO + (NS == 2 ? grp : 0) * D);
        for (int j = j0; j < nb; j += dj) {
          const int buf = NS == 2 ? grp : (j & 1);
          const uint32_t s_tmem_at = tmem_at(tmem, wq, buf * 128);
          ok = warp_wait(&s_full[buf], sc[buf] & 1, &s_abort, A.status);
          if (!ok) break;
          ++sc[buf];
          if (!busy) {  // its rows of P stay whatever they are: they reach its rows of O only
            if (lane == 0) mbar_arrive(&p_full[buf]);
            continue;
          }
          tc_fence_after();
          const int key0 = (s.b0 + j) * BN;
          const bool masked = __any_sync(0xffffffffu, lim < key0 + BN);
          auto load_scores = [&](float (&x)[128]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32_async(s_tmem_at + 32 * i, x + 32 * i);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 128; ++i) x[i] = key0 + i < lim ? x[i] : -INFINITY;
            }
          };
          if (j == j0) {  // the first block: its maximum is the one to measure against
            float x[128];
            load_scores(x);
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(x[k], x[k + 4]);
#pragma unroll
            for (int i = 8; i < 128; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], fmaxf(x[i + k], x[i + k + 4]));
            top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          }
          // Probabilities against the maximum so far, while the block's own maximum is found beside them (one
          // after the other costs a third more). A row that outgrew it is rare after the first blocks: O is
          // rescaled and the block's probabilities formed again.
          uint32_t p[64];
          float part;
          while (true) {
            float x[128];
            load_scores(x);
            const float shift = top == -INFINITY ? 0.0f : -top * A.c;
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float sm4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              float &a = x[2 * i], &b = x[2 * i + 1];
              mx[i & 3] = fmaxf(mx[i & 3], fmaxf(a, b));
              fma2(a, b, A.c, shift);
              a = ex2(a);
              b = ex2(b);
              add2(sm4[2 * (i & 1)], sm4[2 * (i & 1) + 1], a, b);
              // a probability's rounding to bf16 is at most 2^-8 of itself, as the output's own is, and on average
              // zero: outputs are 2.0e-3 to 2.3e-3 off in place of 1.6e-3 (relative 2-norm), and the product runs at
              // bf16's rate; the sum is of the unrounded values
              p[i] = pack_bf16(a, b);
            }
            part = (sm4[0] + sm4[1]) + (sm4[2] + sm4[3]);
            const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grew = m > top && ((m - top) * A.c > 8.0f || top == -INFINITY);
            if (!__any_sync(0xffffffffu, grew)) break;
            const float keep = grew ? ex2((top - m) * A.c) : 1.0f;  // 0 from -inf
            if (grew) top = m;
            sum *= keep;
            if (NS == 1) {  // the product before may still be adding to O
              ok = warp_wait(&o_full[0], (oc + j - 1) & 1, &s_abort, A.status);
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              float v[32];
              tmem_ld32_async(o_tmem + i, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= keep;
              tmem_st32(o_tmem + i, reinterpret_cast<const uint32_t *>(v));
            }
          }
          if (!ok) break;
          tmem_st32(s_tmem_at, p);
          tmem_st32(s_tmem_at + 32, p + 32);
          sum += part;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        if (!ok) break;
        const int mine = nb > j0 ? (nb - j0 + dj - 1) / dj : 0;  // blocks this group took
        if (mine > 0) {
          // D = 256 completes a phase with every product: a parity tells only neighbouring phases apart, and
          // the last S tile vouches for the products up to two before the last
          const uint32_t ph = NS == 1 ? oc + nb - 1 : oc;
          if (NS == 1 && nb > 1) ok = warp_wait(&o_full[0], (ph - 1) & 1, &s_abort, A.status);
          if (!ok) break;
          ok = warp_wait(&o_full[NS == 2 ? grp : 0], ph & 1, &s_abort, A.status);
          if (!ok) break;
          oc += NS == 1 ? nb : 1;
          tc_fence_after();
        }
        // ---- the segment's results
        if (SHARED) {
          const int rows = s.own ? A.suffix_rows : A.prefix_rows;
          const long long r = ((long long)s.slot * NS + grp) * rows + row;
          if (real)  // a group that took no block says so: (-inf, 0)
            (s.own ? A.suffix_ml : A.prefix_ml)[r] = make_float2(top == -INFINITY ? -INFINITY : top * A.c, sum);
          // 16 bytes of each row side by side: a warp's stores and the join's loads are contiguous
          float4 *dst = reinterpret_cast<float4 *>(s.own ? A.suffix_o : A.prefix_o) +
                        ((long long)s.slot * NS + grp) * rows * (D / 4) + row;
          if (mine > 0 && busy) {
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              float v[32];
              tmem_ld32_async(o_tmem + i, v);
              tmem_wait_ld();
              if (real) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  dst[(i + k) / 4 * rows] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
              }
            }
          }
        } else {
          const bool split = NS == 2 && !s.pair;  // the groups took alternate blocks of the same rows
          float *far = reinterpret_cast<float *>(sm + NS * C::QB);
          float w0 = 1.0f, w1 = 0.0f;
          if (split) {
            // group 1 hands its rows over in the ring's memory, which every product has read by then
            const int n0 = (nb + 1) / 2, n1 = nb / 2;
            if (grp == 1) {
              if (n0 > 0) ok = warp_wait(&o_full[0], 0, &s_abort, A.status);
              if (!ok) break;
              s_ml[row] = make_float2(top, sum);
              if (n1 > 0) {
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                  float v[32];
                  tmem_ld32_async(o_tmem + i, v);
                  tmem_wait_ld();
#pragma unroll
                  for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<float4 *>(far + ((i + k) / 4 * 128 + row) * 4) =
                        make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                }
              }
            }
            if (grp == 1) {
              __syncwarp();
              if (lane == 0) mbar_arrive(handed);
              break;
            }
            ok = warp_wait(handed, 0, &s_abort, A.status);
            if (!ok) break;
            const float2 o = s_ml[row];
            if (o.y != 0.0f) {  // a sum of zero saw no key; a NaN counts
              const float m = fmaxf(top, o.x);
              w0 = sum > 0.0f ? ex2((top - m) * A.c) : 0.0f;
              w1 = ex2((o.x - m) * A.c);
              sum = sum * w0 + o.y * w1;
            }
          }
          const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
          w0 *= inv;
          w1 *= inv;
          bf16 *dst = A.out + ((long long)(s.t0 + tok) * A.hq + s.head * A.G + gh) * D;
#pragma unroll 1
          for (int i = 0; i < D; i += 64) {
            float v[64];
            if (mine > 0) {
              tmem_ld32_async(o_tmem + i, v);
              tmem_ld32_async(o_tmem + i + 32, v + 32);
              tmem_wait_ld();
            }
            if (real) {
              if (mine == 0 || inv == 0.0f) {
#pragma unroll
                for (int k = 0; k < 64; ++k) v[k] = 0.0f;
              }
              if (w1 != 0.0f) {
#pragma unroll
                for (int k = 0; k < 64; k += 4) {
                  const float4 f = *reinterpret_cast<const float4 *>(far + ((i + k) / 4 * 128 + row) * 4);
                  v[k] = fmaf(v[k], w0, f.x * w1);
                  v[k + 1] = fmaf(v[k + 1], w0, f.y * w1);
                  v[k + 2] = fmaf(v[k + 2], w0, f.z * w1);
                  v[k + 3] = fmaf(v[k + 3], w0, f.w * w1);
                }
              } else {
#pragma unroll
                for (int k = 0; k < 64; ++k) v[k] *= w0;
              }
              uint32_t w[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                if (A.out32) {
                  st_32bytes(dst + i + 2 * k, w + k);
                } else {
                  *reinterpret_cast<uint4 *>(dst + i + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                  *reinterpret_cast<uint4 *>(dst + i + 2 * k + 8) = make_uint4(w[k + 4], w[k + 5], w[k + 6], w[k + 7]);
                }
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

// One part of a row's result: the maximum (in powers of two), the sum and four channels.
struct Part {
  float top, sum;
  float4 o;
  __device__ __forceinline__ void add(float m, float l, float4 v) {
    if (l == 0.0f) return;  // saw no key; its channels were not written
    const float best = fmaxf(top, m), a = top == -INFINITY ? 0.0f : ex2(top - best), w = ex2(m - best);
    top = best;
    sum = fmaf(l, w, sum * a);
    o.x = fmaf(v.x, w, o.x * a);
    o.y = fmaf(v.y, w, o.y * a);
    o.z = fmaf(v.z, w, o.z * a);
    o.w = fmaf(v.w, w, o.w * a);
  }
};

// Where an entry's lines begin in the plan.
struct Place {
  long long cost, line;
};
__device__ __forceinline__ Place place_of(const Args &A, int e) { return {A.plan[2 + 2 * e], A.plan[3 + 2 * e]}; }

// Adds the partial results that the attention kernel left of one entry for channels 4c.. of (token t, head), in
// order, kParts of them loaded at once.
constexpr int kParts = 8;
template <int D>
__device__ __forceinline__ void add_line(const Args &A, Part &P, const Entry &x, Place at_line, bool own, int t, int head,
                                         int gh, int c, long long share) {
  constexpr int NS = Cfg<D>::NS;
  if (x.blocks == 0) return;
  const int ti = t - x.first, tile = ti / A.tile_tokens, i = ti - tile * A.tile_tokens;
  const bool pair = min(A.tile_tokens, x.ntok - tile * A.tile_tokens) > A.TQ;
  const long long li = (long long)tile * A.hk + head, a = at_line.cost + li * x.line_cost(), z = a + x.line_cost();
  const int rows = own ? A.suffix_rows : A.prefix_rows;
  const int streams = NS == 2 && !pair ? 2 : 1, s0 = pair ? i / A.TQ : 0, row = (pair ? i % A.TQ : i) * A.G + gh;
  const float4 *po = reinterpret_cast<const float4 *>(own ? A.suffix_o : A.prefix_o) + (long long)c * rows + row;
  const float2 *pml = (own ? A.suffix_ml : A.prefix_ml) + row;
  // the CTAs that took some of the line's blocks
  const bool small = z < (1LL << 31) && share < (1LL << 31);
  const int c0 = small ? (unsigned)(a + kSetup) / (unsigned)share : (int)((a + kSetup) / share);
  const int c1 = small ? (unsigned)(z - 1) / (unsigned)share : (int)((z - 1) / share), n = (c1 - c0 + 1) * streams;
  const long long first = (at_line.line + li + c0) * NS + s0;
  const int stride = NS / streams;
  for (int p0 = 0; p0 < n; p0 += kParts) {
    float2 ml[kParts];
    float4 v[kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const long long at = (first + (long long)min(p0 + k, n - 1) * stride) * rows;
      ml[k] = pml[at];
      v[k] = po[at * (D / 4)];
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (p0 + k < n) P.add(ml[k].x, ml[k].y, v[k]);
  }
}

// Joins the partial results of a shared-prefix call: a thread takes four
// channels of one (query token, head).
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args A) {
  griddep_wait();
  griddep_trigger();
  // items: (token, key head, channel group, head of the group), the last fastest
  const long long item = (long long)blockIdx.x * 128 + threadIdx.x;
  const long long per_token = (long long)(D / 4) * A.hq;
  const bool few = item < (1LL << 31);
  const int t = few ? (unsigned)item / (unsigned)per_token : (int)(item / per_token);
  const int of_token = (int)(item - t * per_token), head = of_token / ((D / 4) * A.G);
  const int in = of_token - head * ((D / 4) * A.G), c = in / A.G, gh = in - c * A.G;
  if (t >= A.n_tokens) return;
  const int b = t / A.T, g = group_of(A, b);
  const long long share = A.plan[0], in_order = A.plan[1];
  const Place own_at = place_of(A, A.n_groups + b), shared_at = place_of(A, max(g, 0));
  const Entry own = entry_at(A, A.n_groups + b, true), shared = g >= 0 ? entry_at(A, g, true) : own;
  if (!in_order || !own.ok || !shared.ok) return;
  Part P = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (t - own.first < own.ntok) {
    if (g >= 0) add_line<D>(A, P, shared, shared_at, false, t, head, gh, c, share);
    add_line<D>(A, P, own, own_at, true, t, head, gh, c, share);
  }
  const float inv = 1.0f / P.sum;
  uint2 r = make_uint2(0u, 0u);
  if (P.sum != 0.0f) r = make_uint2(pack_bf16(P.o.x * inv, P.o.y * inv), pack_bf16(P.o.z * inv, P.o.w * inv));
  *reinterpret_cast<uint2 *>(A.out + ((long long)t * A.hq + head * A.G + gh) * D + 4 * c) = r;
}

// The join of rows with few query rows per key head (T G <= 16: decode steps,
// short verifies), which attends over the row's own keys itself. A tile of
// tcgen05 has 128 rows: with 4 of them real, a segment of the kernel above took
// 4 us of latencies for 1 us of bytes. Here a CTA of four warps takes one (row,
// key head); each warp copies tiles of 16 keys and values to stages of its own
// (cp.async) and multiplies them with the 16-row products of the warp-level
// tensor instruction, whose fragments stay in registers from the scores to the
// values. The job is bytes, not products: ~6 instructions a key of 512 bytes
// (on the fp32 units ~60, which bounded it at half the memory rate).
// None of this reads what the kernel before wrote, so it runs before the wait
// for it, on the SMs which that kernel leaves; only then the parts are joined.
// 64 rows x 8 key heads, ~550 keys of 128 channels each: 37 us (147 MB of keys
// and values, 4 TB/s; ~7 us of each CTA are latencies at its start and join).
constexpr int kJoinWarps = 4, kRows = 16, kTileKeys = 16;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// c[16][8] += a[16][16] b[16][8]
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct JoinSmem {
  static constexpr int kTile = kTileKeys * D * 2;             // bytes of a tile's keys, and of its values
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int kWarp = kStages * 2 * kTile;           // a warp's ring
  static constexpr int kMl = kJoinWarps * kWarp;              // float2 [warps][kRows]
  static constexpr int kBytes = kMl + kJoinWarps * kRows * 8;
  static_assert(kRows * D * 4 <= kWarp, "a warp's results fit over its ring");
};

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) join_rows_kernel(const __grid_constant__ Args A) {
  using S = JoinSmem<D>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  float2 *s_ml = reinterpret_cast<float2 *>(smem_raw + S::kMl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / A.hk, head = blockIdx.x - b * A.hk, R = A.T * A.G;
  const Entry own = entry_at(A, A.n_groups + b, true);
  const int g = group_of(A, b);
  const Entry shared = g >= 0 ? entry_at(A, g, true) : own;
  const bool here = own.ok && own.len <= A.own_keys;
  unsigned char *ring = smem_raw + warp * S::kWarp;

  // this thread's rows of a product: lane / 4 and lane / 4 + 8
  float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] = 0.0f;
  if (here && own.ntok > 0) {
    const bf16 *kp = A.k + (long long)own.kv0 * A.kvs + (long long)head * D;
    const bf16 *vp = A.v + (long long)own.kv0 * A.kvs + (long long)head * D;
    const int tiles = (own.len + kTileKeys - 1) / kTileKeys, mine = (tiles - warp + kJoinWarps - 1) / kJoinWarps;
    auto fetch = [&](int i) {  // this warp's i-th tile; 16-byte chunk c of key j at place c ^ (j % 8)
      if (i < mine) {
        const int j0 = (warp + i * kJoinWarps) * kTileKeys;
        const uint32_t dst = smem_u32(ring) + (i % S::kStages) * 2 * S::kTile;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int at = x * 32 + lane, key = at / (D / 8), c = at % (D / 8);
          const bool in = j0 + key < own.len;  // rows past the end arrive as zeros
          const long long src = (long long)(in ? j0 + key : 0) * A.kvs + c * 8;
          const uint32_t to = dst + key * D * 2 + ((c ^ (key & 7)) << 4);
          cp_async16(to, kp + src, in);
          cp_async16(to + S::kTile, vp + src, in);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) fetch(i);
    // query fragments: rows lane / 4 (+ 8), channels 2 (lane % 4) (+ 8) of each 16
    uint32_t q[D / 16][4];
    int lim[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = lane / 4 + 8 * h, t = row / A.G;
      const bool in = row < R && t < own.ntok;
      lim[h] = in ? min(own.len, own.lim0 + t) : 0;
      const bf16 *src = A.q + (long long)(own.first + (in ? t : 0)) * A.qs +
                        (long long)(head * A.G + (in ? row - t * A.G : 0)) * D + 2 * (lane & 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][h] = in ? *reinterpret_cast<const uint32_t *>(src + 16 * k) : 0u;
        q[k][h + 2] = in ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 8) : 0u;
      }
    }
    const int m = lane >> 3, mr = lane & 7;  // the matrix of an ldmatrix that this lane addresses, and its row
    for (int i = 0; i < mine; ++i) {
      fetch(i + S::kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");  // tile i has landed
      __syncwarp();
      const uint32_t kt = smem_u32(ring) + (i % S::kStages) * 2 * S::kTile, vt = kt + S::kTile;
      float sc[2][4] = {};  // keys 0-7 and 8-15: rows lane / 4 and + 8, keys 2 (lane % 4) and + 1
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t f[4];
        ldmatrix4(f, kt + ((m >> 1) * 8 + mr) * D * 2 + (((2 * k + (m & 1)) ^ mr) << 4));
        mma16816(sc[0], q[k], f[0], f[1]);
        mma16816(sc[1], q[k], f[2], f[3]);
      }
      const int j = (warp + i * kJoinWarps) * kTileKeys + 2 * (lane & 3);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float &x = sc[n][2 * h + e];
            x = j + 8 * n + e < lim[h] ? x * A.c_signed : -INFINITY;
            mx[h] = fmaxf(mx[h], x);
          }
      // as above: the maximum moves only when a row outgrew it by 2^8
      if (__any_sync(0xffffffffu, mx[0] - top[0] > 8.0f || mx[1] - top[1] > 8.0f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float best = fmaxf(top[h], mx[h]);
          best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
          best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
          const float keep = best > top[h] ? ex2(top[h] - best) : 1.0f;
          top[h] = best;
          sum[h] *= keep;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * h] *= keep;
            o[n][2 * h + 1] *= keep;
          }
        }
      }
      uint32_t p[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float shift = top[h] == -INFINITY ? 0.0f : top[h];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float a = ex2(sc[n][2 * h] - shift), e = ex2(sc[n][2 * h + 1] - shift);
          sum[h] += a + e;
          p[h + 2 * n] = pack_bf16(a, e);
        }
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t f[4];
        ldmatrix4_trans(f, vt + ((m & 1) * 8 + mr) * D * 2 + (((2 * n + (m >> 1)) ^ mr) << 4));
        mma16816(o[2 * n], p, f[0], f[1]);
        mma16816(o[2 * n + 1], p, f[2], f[3]);
      }
      __syncwarp();  // the stage may be overwritten
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  // the warp's results over its ring: fp32 [kRows][D]
  float *s_o = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = lane / 4 + 8 * h;
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
    if ((lane & 3) == 0) s_ml[warp * kRows + row] = make_float2(top[h], sum[h]);
    if (row < R)
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2 *>(s_o + row * D + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
  }
  __syncthreads();
  griddep_wait();
  griddep_trigger();

  // ---- the parts of four channels of a query row: the warps', then the prefix's (and the row's own, if the kernel
  // before took it)
  const long long share = A.plan[0], in_order = A.plan[1];
  const Place own_at = place_of(A, A.n_groups + b), shared_at = place_of(A, max(g, 0));
  if (!in_order || !own.ok || !shared.ok) return;
  for (int item = tid; item < R * (D / 4); item += kJoinWarps * 32) {
    const int c = item / R, row = item - c * R, t = row / A.G, gh = row - t * A.G;
    Part P = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    if (t < own.ntok) {
      for (int w = 0; here && w < kJoinWarps; ++w) {
        const float2 ml = s_ml[w * kRows + row];
        P.add(ml.x, ml.y, *reinterpret_cast<const float4 *>(smem_raw + w * S::kWarp + (row * D + 4 * c) * 4));
      }
      if (g >= 0) add_line<D>(A, P, shared, shared_at, false, own.first + t, head, gh, c, share);
      add_line<D>(A, P, own, own_at, true, own.first + t, head, gh, c, share);
    }
    uint2 r = make_uint2(0u, 0u);
    const float inv = 1.0f / P.sum;
    if (P.sum != 0.0f) r = make_uint2(pack_bf16(P.o.x * inv, P.o.y * inv), pack_bf16(P.o.z * inv, P.o.w * inv));
    *reinterpret_cast<uint2 *>(A.out + ((long long)(own.first + t) * A.hq + head * A.G + gh) * D + 4 * c) = r;
  }
}

template <int D>
gdn_status launch_join_rows(const Args &A, cudaStream_t st) {
  constexpr int bytes = JoinSmem<D>::kBytes;
  const DeviceInfo &dev = device_info();
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[dev.id].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(join_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return fail(GDN_ERR_CUDA, "attention: cannot reserve shared memory");
    ready[dev.id].store(true, std::memory_order_release);
  }
  launch_pdl(join_rows_kernel<D>, dim3((unsigned)(A.B * A.hk)), dim3(kJoinWarps * 32), bytes, st, A);
  return check_launch("attention");
}

// --------------------------------------------------------------------- host

gdn_status check(const gdn_attn_dims *d) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->B < 0 || d->n_tokens < 0 || d->n_groups < 0 || d->n_groups > d->B)
    return fail(GDN_ERR_SHAPE, "B and n_tokens must be >= 0 and n_groups in [0, B]");
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->n_q_heads % d->n_kv_heads != 0 ||
      d->n_q_heads / d->n_kv_heads > 64 || d->n_kv_heads > 4096)
    return fail(GDN_ERR_SHAPE, "n_q_heads must be a multiple of n_kv_heads, at most 64 per key head");
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (!(fabsf(d->scale) * kLog2e <= FLT_MAX)) return fail(GDN_ERR_ARG, "scale, and scale * log2(e), must be finite");
  if (d->q_stride % 8 != 0 || d->kv_stride % 8 != 0)
    return fail(GDN_ERR_SHAPE, "token strides must be multiples of 8 elements");
  if (d->q_stride < (long long)d->n_q_heads * d->head_dim || d->kv_stride < (long long)d->n_kv_heads * d->head_dim)
    return fail(GDN_ERR_SHAPE, "token strides must cover the heads");
  if (d->q_stride > (1LL << 32) || d->kv_stride > (1LL << 32))
    return fail(GDN_ERR_SHAPE, "token strides must be at most 2^32 elements");
  if (d->kv_rows < 0 || d->kv_rows > (1LL << 31) - 1) return fail(GDN_ERR_SHAPE, "kv_rows must be in [0, 2^31)");
  return GDN_OK;
}


using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [rows][heads][D] with `stride` elements between rows; boxes of 64 channels x box_heads x box_rows, 128-byte swizzle.
gdn_status encode(CUtensorMap *map, const void *base, int D, int heads, long long rows, long long stride, int box_heads,
                  int box_rows) {
  static const EncodeTiled fn = []() -> EncodeTiled {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  if (!fn) return fail(GDN_ERR_CUDA, "attention: cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)(rows > 0 ? rows : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  if (fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(GDN_ERR_CUDA, "attention: cannot encode a tensor map");
  return GDN_OK;
}

Args make_args(const gdn_attn_dims *d, void *out, unsigned int *status) {
  Args A = {};
  A.B = d->B;
  A.T = d->T;
  A.n_tokens = d->n_tokens;
  A.n_groups = d->n_groups;
  A.hq = d->n_q_heads;
  A.hk = d->n_kv_heads;
  A.G = d->n_q_heads / d->n_kv_heads;
  A.TQ = 128 / A.G;
  A.tile_tokens = (d->head_dim == 256 ? 1 : 2) * A.TQ;
  // masked scores are -inf: times a scale of exactly zero they would be NaN
  A.c = fmaxf(fabsf(d->scale) * kLog2e, 1e-30f);
  A.c_signed = d->scale * kLog2e;
  // kind::f16, bf16 A and B, fp32 D, N = 128, M = 128; bit 13 negates A for a negative scale
  A.idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24) | (d->scale < 0.0f ? 1u << 13 : 0u);
  A.kv_rows = d->kv_rows;
  A.out = static_cast<bf16 *>(out);
  A.out32 = reinterpret_cast<uintptr_t>(out) % 32 == 0;
  A.status = status;
  return A;
}

template <int D, bool SHARED>
gdn_status launch_t(const gdn_attn_dims *d, const void *q, const void *k, const void *v, const Args &A, int grid,
                    cudaStream_t st) {
  CUtensorMap qm, km, vm;
  GDN_TRY(encode(&qm, q, D, A.hq, A.n_tokens, d->q_stride, A.G, A.TQ));
  GDN_TRY(encode(&km, k, D, A.hk, A.kv_rows, d->kv_stride, 1, BN));
  GDN_TRY(encode(&vm, v, D, A.hk, A.kv_rows, d->kv_stride, 1, BN));
  const DeviceInfo &dev = device_info();
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[dev.id].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attn_kernel<D, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kBytes) !=
        cudaSuccess)
      return fail(GDN_ERR_CUDA, "attention: cannot reserve shared memory");
    ready[dev.id].store(true, std::memory_order_release);
  }
  launch_pdl(attn_kernel<D, SHARED>, dim3((unsigned)grid), dim3(Cfg<D>::kThreads), Cfg<D>::kBytes, st, qm, km, vm, A);
  GDN_TRY(check_launch("attention"));
  if (SHARED) {
    const long long items = (long long)A.n_tokens * A.hq * (D / 4);
    if (A.own_keys > 0) return launch_join_rows<D>(A, st);
    launch_pdl(join_kernel<D>, dim3((unsigned)((items + 127) / 128)), dim3(128), 0, st, A);
  }
  return check_launch("attention");
}

template <bool SHARED>
gdn_status launch(const gdn_attn_dims *d, const void *q, const void *k, const void *v, const Args &A, int grid,
                  cudaStream_t st) {
  if (d->head_dim == 64) return launch_t<64, SHARED>(d, q, k, v, A, grid, st);
  if (d->head_dim == 128) return launch_t<128, SHARED>(d, q, k, v, A, grid, st);
  return launch_t<256, SHARED>(d, q, k, v, A, grid, st);
}

// The workspace of a shared-prefix call; base NULL: its size only.
size_t carve(const gdn_attn_dims *d, Args &A, unsigned char *base) {
  const int D = d->head_dim, ns = D == 256 ? 1 : 2;
  const long long prefix_lines = (long long)A.hk * ((long long)d->B * d->T / A.tile_tokens + d->n_groups);
  const long long own_lines = (long long)A.hk * d->B * ((d->T + A.tile_tokens - 1) / A.tile_tokens);
  A.prefix_rows = A.TQ * A.G;
  A.suffix_rows = (d->T < A.TQ ? d->T : A.TQ) * A.G;
  const long long ps = d->n_groups > 0 ? (prefix_lines + kMaxCtas) * ns * A.prefix_rows : 0;
  const long long ss = ((d->n_groups > 0 ? prefix_lines : 0) + own_lines + kMaxCtas) * ns * A.suffix_rows;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char *p = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  A.plan = reinterpret_cast<long long *>(take(16 * ((size_t)d->n_groups + d->B + 1)));
  A.prefix_ml = reinterpret_cast<float2 *>(take((size_t)ps * 8));
  A.suffix_ml = reinterpret_cast<float2 *>(take((size_t)ss * 8));
  A.prefix_o = reinterpret_cast<float *>(take((size_t)ps * D * 4));
  A.suffix_o = reinterpret_cast<float *>(take((size_t)ss * D * 4));
  return at;
}

gdn_status check_shared(const gdn_attn_dims *d) {
  GDN_TRY(check(d));
  if (d->T < 1 || d->T > 64) return fail(GDN_ERR_SHAPE, "T must be in [1, 64]");
  if ((long long)d->B * d->T != d->n_tokens) return fail(GDN_ERR_SHAPE, "n_tokens must be B * T");
  if ((long long)d->B * d->n_kv_heads > (1LL << 31) - 1 ||
      (long long)d->n_tokens * d->n_q_heads * (d->head_dim / 4) / 128 >= (1LL << 31) - 1)
    return fail(GDN_ERR_SHAPE, "too many rows in one call");
  return GDN_OK;
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
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  attn::Args A = attn::make_args(d, out, dev->status);
  A.cu = cu_seqlens;
  A.kv_start = kv_start;
  A.kv_len = kv_len;
  // fewer two-tile CTAs than SMs: one tile each, its keys shared between the two groups
  if ((long long)d->n_tokens * d->n_kv_heads < (long long)dev->sms * A.tile_tokens) A.tile_tokens = A.TQ;
  const long long tiles = (long long)d->n_tokens / A.tile_tokens + d->B;
  if (tiles * A.hk > (1LL << 31) - 1) return fail(GDN_ERR_SHAPE, "too many tokens in one call");
  A.max_tiles = (int)tiles;
  return attn::launch<false>(d, q, k, v, A, (int)(tiles * A.hk), static_cast<cudaStream_t>(stream));
}

size_t gdn_attn_workspace_size(const gdn_attn_dims *d) {
  if (attn::check_shared(d) != GDN_OK) return 0;
  attn::Args A = attn::make_args(d, nullptr, nullptr);
  return attn::carve(d, A, nullptr);
}

gdn_status gdn_attn_shared_prefix(const gdn_attn_dims *d, const void *q, const void *k, const void *v,
                                  const int32_t *group_rows, const int32_t *prefix_start, const int32_t *prefix_len,
                                  const int32_t *suffix_start, const int32_t *suffix_len, const int32_t *q_len,
                                  void *out, void *workspace, size_t workspace_bytes, void *stream) {
  GDN_TRY(attn::check_shared(d));
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
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  attn::Args A = attn::make_args(d, out, dev->status);
  (void)attn::carve(d, A, static_cast<unsigned char *>(workspace));
  A.group_rows = group_rows;
  A.prefix_start = prefix_start;
  A.prefix_len = prefix_len;
  A.suffix_start = suffix_start;
  A.suffix_len = suffix_len;
  A.q_len = q_len;
  A.q = static_cast<const bf16 *>(q);
  A.k = static_cast<const bf16 *>(k);
  A.v = static_cast<const bf16 *>(v);
  A.qs = d->q_stride;
  A.kvs = d->kv_stride;
  A.own_keys = d->T * A.G <= attn::kRows && (long long)d->B * A.hk < (1LL << 31) ? attn::kOwnKeys : 0;
  const int grid = dev->sms < attn::kMaxCtas ? dev->sms : attn::kMaxCtas;
  return attn::launch<true>(d, q, k, v, A, grid, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
