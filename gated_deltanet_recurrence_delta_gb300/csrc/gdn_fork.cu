// gdn_cache_fork: rows of a paged cache become copies of other rows and get
// room for new tokens; gdn_slots_copy: the copies that this takes.
//
// cache_fork is bookkeeping of a few thousand numbers between dependent steps
// (which pages are used -> which are free -> who gets which -> where the tokens
// go), so one CTA does it without leaving the SM: what is used stands as one bit
// a page in shared memory, free pages are ranked by a scan of the bits' counts,
// and the page of rank k goes to the row whose needs cover k. Latency bounds it:
// seven barriers, and the chain parent -> length -> last page of dependent loads.
// 64 rows of 4000 to 8192 tokens: 6.8 us (14 as one barrier after the other and pages
// handed out row by row); 30 rows of up to 700: 5.2 us.
//
// slots_copy is an HBM copy of 16-byte vectors; a CTA takes one piece of one
// slot of one layer, and a skipped pair's CTAs end at once. States and conv tails
// of 8 layers (446 MB read and written): 57 us, 7.8 TB/s: sources that several rows
// copy are in L2 after the first.
#include "gdn_check.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace fork {

constexpr int kThreads = 1024, kWarps = 32;
constexpr int kMaxRows = 1024, kMaxPages = 1 << 20;
constexpr int kPage = kv4::kPage;

struct Args {
  int rows, T, width, n_pages;
  const int32_t *parent, *n_new, *table, *len;
  const uint8_t *pinned;
  int32_t *table_out, *len_out, *index, *page_src, *page_dst;
  const int32_t *state;
  int32_t *state_out, *state_src, *state_dst;
  unsigned int *status;
};

constexpr int kFresh = 2048;  // new pages that shared memory holds (more: through the table)

__device__ __forceinline__ int pages(int tokens) { return (tokens + kPage - 1) / kPage; }

__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ Args A) {
  extern __shared__ uint32_t s_used[];  // a bit a page
  __shared__ int s_par[kMaxRows], s_len[kMaxRows], s_new[kMaxRows], s_first[kMaxRows];
  __shared__ int s_tail[kMaxRows];  // the row's partly filled last page
  __shared__ int s_need[kMaxRows];  // pages of the rows up to this one
  __shared__ int s_dead[kMaxRows];  // rows without children, in order
  __shared__ int s_state[kMaxRows];
  __shared__ int s_fresh[kFresh];   // the new pages, in order
  __shared__ uint8_t s_copy[kMaxRows];
  __shared__ int s_part[4][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = A.rows;
  s_first[tid] = kMaxRows;
  s_copy[tid] = 0;
  griddep_wait();
  griddep_trigger();
  const int words = (A.n_pages + 31) / 32;
  const long long most = (long long)A.width * kPage;

  // ---- the rows, their last pages; pinned pages
  bool bad = false;
  int par = -1, len = 0, take = 0, tail = -1;
  if (tid < R) {
    par = A.parent ? A.parent[tid] : tid;
    take = A.n_new ? A.n_new[tid] : A.T;
    if (par < -1 || par >= R) {
      bad = true;
      par = -1;
    }
    if (take < 0 || take > A.T) {
      bad = true;
      take = 0;
    }
    if (par >= 0) {
      len = A.len[par];
      if (len < 0 || len > most) {
        bad = true;
        len = 0;
      }
    }
    if (len % kPage) {
      tail = A.table[(long long)par * A.width + len / kPage];
      if (tail < 0 || tail >= A.n_pages) tail = -1;
    }
    s_par[tid] = par;
    s_len[tid] = len;
    s_new[tid] = take;
    s_tail[tid] = tail;
    if (A.state) s_state[tid] = A.state[tid];
  }
#pragma unroll 4
  for (int w = warp; w < words; w += kWarps) {  // a page to a lane
    const int page = 32 * w + lane;
    const bool taken = page >= A.n_pages || (A.pinned && A.pinned[page]);
    const uint32_t bits = __ballot_sync(0xffffffffu, taken);
    if (lane == 0) s_used[w] = bits;
  }
  __syncthreads();
  if (take > 0 && tail >= 0 && (s_used[tail >> 5] >> (tail & 31) & 1)) s_copy[tid] = 1;  // pinned
  if (par >= 0) atomicMin(&s_first[par], tid);                                            // the lowest child
  __syncthreads();  // what the votes below read of other rows is written in front of it
  // ---- the rows' pages: handed on and marked, 128 of each of two rows at a time
  for (int ra = warp; ra < R; ra += 2 * kWarps) {
    const int rb = ra + kWarps, na = pages(s_len[ra]), nb = rb < R ? pages(s_len[rb]) : 0;
    const int32_t *from_a = A.table + (long long)max(s_par[ra], 0) * A.width;
    const int32_t *from_b = nb ? A.table + (long long)s_par[rb] * A.width : from_a;
    int32_t *to_a = A.table_out + (long long)ra * A.width, *to_b = A.table_out + (long long)rb * A.width;
    for (int j0 = lane; j0 - lane < max(na, nb); j0 += 128) {
      int x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + 32 * (k & 3);
        x[k] = j < (k < 4 ? na : nb) ? (k < 4 ? from_a : from_b)[j] : -2;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + 32 * (k & 3);
        if (j >= (k < 4 ? na : nb)) continue;
        (k < 4 ? to_a : to_b)[j] = x[k];
        if (x[k] < 0 || x[k] >= A.n_pages)
          bad = true;
        else
          atomicOr(&s_used[x[k] >> 5], 1u << (x[k] & 31));
      }
    }
  }
  // ---- partly filled last pages that are to be written, and are not the row's alone: two rows at a time
  for (int r0 = warp; r0 < R; r0 += 2 * kWarps) {
    bool look[2], other[2] = {false, false};
    int n[2], page[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = min(r0 + q * kWarps, R - 1);
      n[q] = s_len[r];
      page[q] = s_tail[r];
      look[q] = r0 + q * kWarps < R && s_new[r] > 0 && page[q] >= 0 && !s_copy[r];
    }
    if (!look[0] && !look[1]) continue;
    for (int x0 = lane; x0 < R; x0 += 64) {  // the loads of two others each together
      int there[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = k & 1, r = r0 + q * kWarps, at = n[q] / kPage, x = x0 + 32 * (k >> 1), m = x < R ? s_len[x] : 0;
        there[k] = -1;
        if (!look[q] || x == r || pages(m) <= at || !(m > n[q] || (m == n[q] && x < r))) continue;
        // the row's own last page stands there, or a full one
        there[k] = m / kPage == at ? s_tail[x] : A.table[(long long)s_par[x] * A.width + at];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) other[k & 1] |= there[k] == page[k & 1];
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (__any_sync(0xffffffffu, look[q] && other[q]) && lane == 0) s_copy[r0 + q * kWarps] = 1;
  }
  if (bad) set_status(A.status, GDN_ERR_INDEX);
  __syncthreads();
  // ---- what each row needs, who has a state slot to give and to find, which pages are free: four scans at once
  int need = 0;
  bool wide = false;  // more than a line of the table holds
  if (take > 0) {
    const long long after = (long long)len + take;
    wide = after > most;
    if (!wide) need = s_copy[tid] + pages((int)after) - pages(len);
  }
  const bool again = tid < R && (par < 0 || s_first[par] != tid), dead = tid < R && s_first[tid] == kMaxRows;
  const int per = (words + kThreads - 1) / kThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += 32 - __popc(s_used[w]);
  int upto = need, ahead = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o), z = __shfl_up_sync(0xffffffffu, ahead, o);
    if (lane >= o) {
      upto += y;
      ahead += z;
    }
  }
  const uint32_t agains = __ballot_sync(0xffffffffu, again), deads = __ballot_sync(0xffffffffu, dead);
  if (lane == 31) {
    s_part[0][warp] = upto;
    s_part[1][warp] = ahead;
    s_part[2][warp] = __popc(agains);
    s_part[3][warp] = __popc(deads);
  }
  __syncthreads();
  auto before = [&](int q) { return (int)__reduce_add_sync(0xffffffffu, lane < warp ? s_part[q][lane] : 0); };
  upto += before(0);
  ahead += before(1);
  const int nth = before(2) + __popc(agains & ((1u << lane) - 1)), nth_dead = before(3) + __popc(deads & ((1u << lane) - 1));
  const int wanted = __reduce_add_sync(0xffffffffu, s_part[0][lane]), total = __reduce_add_sync(0xffffffffu, s_part[1][lane]);
  s_need[tid] = upto;
  if (dead) s_dead[nth_dead] = tid;
  __syncthreads();
  // ---- the free pages: listed by rank. Beyond the list rank k goes to the first row whose needs reach beyond k
  auto give = [&](int k, int page) {
    int lo = 0, hi = R - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (s_need[mid] > k) hi = mid;
      else lo = mid + 1;
    }
    if (s_need[lo] > total) return;  // its pages do not all exist
    const int j = k - (lo > 0 ? s_need[lo - 1] : 0) - s_copy[lo];  // -1: the copy
    A.table_out[(long long)lo * A.width + pages(s_len[lo]) + j] = page;
    if (j < 0) A.page_dst[lo] = page;
  };
  int first = ahead - mine;  // the rank of the first free page of this thread's words
  for (int j = 0; j < per; ++j) {  // a warp takes its lanes' words one after the other, a page to a lane
    const int w = w0 + j;
    const uint32_t open = w < w1 ? ~s_used[w] : 0;
    uint32_t turn = __ballot_sync(0xffffffffu, open && first < wanted);
    for (; turn; turn &= turn - 1) {
      const int who = __ffs(turn) - 1;
      const uint32_t theirs = __shfl_sync(0xffffffffu, open, who);
      const int page = 32 * __shfl_sync(0xffffffffu, w, who) + lane;
      const int k = __shfl_sync(0xffffffffu, first, who) + __popc(theirs & ((1u << lane) - 1));
      if (!(theirs >> lane & 1) || k >= wanted) continue;
      if (k < kFresh) s_fresh[k] = page;
      else give(k, page);
    }
    first += __popc(open);
  }
  __syncthreads();
  const bool full = wide || (need > 0 && upto > total);
  const int listed = full ? 0 : max(0, min(need, kFresh - (upto - need)));  // of the row's new pages
  auto place = [&](int r, int k, int j, int copied) {  // new page j of row r, which is the list's k-th; a copy comes first
    A.table_out[(long long)r * A.width + pages(s_len[r]) + j - copied] = s_fresh[k];
    if (j < copied) A.page_dst[r] = s_fresh[k];
  };
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (j < listed) place(tid, upto - need + j, j, s_copy[tid]);
  for (uint32_t turn = __ballot_sync(0xffffffffu, listed > 2); turn; turn &= turn - 1) {  // many: a warp
    const int who = __ffs(turn) - 1, r = 32 * warp + who, n = __shfl_sync(0xffffffffu, listed, who);
    const int k = __shfl_sync(0xffffffffu, upto - need, who);
    for (int j = 2 + lane; j < n; j += 32) place(r, k + j, j, s_copy[r]);
  }
  // ---- the rows' lengths and copies, the state slots
  if (tid < R) {
    if (full) {
      set_status(A.status, GDN_ERR_FULL);
      s_new[tid] = 0;
    }
    A.len_out[tid] = len + (full ? 0 : take);
    const bool copy = s_copy[tid] && !full;
    A.page_src[tid] = copy ? tail : -1;
    if (!copy) A.page_dst[tid] = -1;
    if (A.state) {
      const int from = par < 0 ? -1 : s_state[par], to = again ? s_state[s_dead[nth]] : from;
      A.state_out[tid] = to;
      A.state_src[tid] = again ? from : -1;
      A.state_dst[tid] = again && par >= 0 ? to : -1;
    }
  }
  __syncthreads();
  // ---- the pool rows of the new tokens
  for (long long i = tid; i < (long long)R * A.T; i += kThreads) {
    const int r = (int)(i / A.T), t = (int)(i - (long long)r * A.T), n = s_len[r], place = n + t;
    int row = -1;
    if (t < s_new[r]) {
      const int at = place / kPage - pages(n) + s_copy[r];  // of the row's new pages; below 0: its last page
      const int page = at < 0 ? s_tail[r]
                       : wanted <= kFresh ? s_fresh[(r > 0 ? s_need[r - 1] : 0) + at]
                                          : A.table_out[(long long)r * A.width + place / kPage];
      if (page >= 0) row = page * kPage + place % kPage;
    }
    A.index[i] = row;
  }
}

}  // namespace fork

namespace slots {

constexpr int kThreads = 256, kPiece = 8;  // 16-byte vectors a thread moves

struct Pool {
  uint4 *base;
  const int32_t *src, *dst;
  long long vec, first;  // vectors of a slot; first CTA
  int n, layers, slots, pieces;
};
struct Args {
  Pool pool[GDN_MAX_SLOT_POOLS];
  int n;
  unsigned int *status;
};

__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ Args A) {
  griddep_wait();
  griddep_trigger();
  int k = 0;
  while (k + 1 < A.n && blockIdx.x >= A.pool[k + 1].first) ++k;
  const Pool &P = A.pool[k];
  long long i = blockIdx.x - P.first;  // [pair][layer][piece]
  const int piece = (int)(i % P.pieces);
  i /= P.pieces;
  const int layer = (int)(i % P.layers), pair = (int)(i / P.layers);
  const int s = P.src[pair], d = P.dst[pair];
  if (s == -1) return;
  if (s < 0 || s >= P.slots || d < 0 || d >= P.slots) {
    if (threadIdx.x == 0) set_status(A.status, GDN_ERR_INDEX);
    return;
  }
  const uint4 *from = P.base + ((long long)layer * P.slots + s) * P.vec;
  uint4 *to = P.base + ((long long)layer * P.slots + d) * P.vec;
  const long long e0 = (long long)piece * (kThreads * kPiece) + threadIdx.x;
  uint4 x[kPiece];
#pragma unroll
  for (int j = 0; j < kPiece; ++j)
    if (e0 + j * kThreads < P.vec) x[j] = __ldcs(from + e0 + j * kThreads);
#pragma unroll
  for (int j = 0; j < kPiece; ++j)
    if (e0 + j * kThreads < P.vec) __stcs(to + e0 + j * kThreads, x[j]);
}

}  // namespace slots
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_cache_fork(const gdn_fork_dims *d, const int32_t *parent, const int32_t *n_new,
                                     const int32_t *page_table, const int32_t *kv_len, const uint8_t *pinned,
                                     int32_t *page_table_out, int32_t *kv_len_out, int32_t *kv_index, int32_t *page_src,
                                     int32_t *page_dst, const int32_t *state_idx, int32_t *state_idx_out,
                                     int32_t *state_src, int32_t *state_dst, void *stream) {
  if (!d) return fail(GDN_ERR_ARG, "dims is NULL");
  if (d->n_rows < 0 || d->n_rows > fork::kMaxRows) return fail(GDN_ERR_SHAPE, "n_rows must be in [0, 1024]");
  if (d->T < 0 || d->T > (1 << 20)) return fail(GDN_ERR_SHAPE, "T must be in [0, 2^20]");
  if (d->n_pages < 0 || d->n_pages > fork::kMaxPages) return fail(GDN_ERR_SHAPE, "n_pages must be in [0, 2^20]");
  if (d->max_pages < 0 || d->max_pages > fork::kMaxPages) return fail(GDN_ERR_SHAPE, "max_pages must be in [0, 2^20]");
  if (d->n_rows == 0) return GDN_OK;  // empty tensors may have no address
  if (parent) GDN_TRY(check_ptr(parent, "parent", 4));
  if (n_new) GDN_TRY(check_ptr(n_new, "n_new", 4));
  if (d->max_pages > 0) {
    GDN_TRY(check_ptr(page_table, "page_table", 4));
    GDN_TRY(check_ptr(page_table_out, "page_table_out", 4));
  }
  GDN_TRY(check_ptr(kv_len, "kv_len", 4));
  GDN_TRY(check_ptr(kv_len_out, "kv_len_out", 4));
  if (d->T > 0) GDN_TRY(check_ptr(kv_index, "kv_index", 4));
  GDN_TRY(check_ptr(page_src, "page_src", 4));
  GDN_TRY(check_ptr(page_dst, "page_dst", 4));
  if (page_table && page_table == page_table_out) return fail(GDN_ERR_ARG, "page_table_out must be another buffer than page_table");
  if (kv_len == kv_len_out) return fail(GDN_ERR_ARG, "kv_len_out must be another buffer than kv_len");
  const bool states = state_idx != nullptr;
  if (states != (state_idx_out != nullptr) || states != (state_src != nullptr) || states != (state_dst != nullptr))
    return fail(GDN_ERR_ARG, "state_idx, state_idx_out, state_src and state_dst must all be given or all be NULL");
  if (states) {
    GDN_TRY(check_ptr(state_idx, "state_idx", 4));
    GDN_TRY(check_ptr(state_idx_out, "state_idx_out", 4));
    GDN_TRY(check_ptr(state_src, "state_src", 4));
    GDN_TRY(check_ptr(state_dst, "state_dst", 4));
    if (state_idx == state_idx_out) return fail(GDN_ERR_ARG, "state_idx_out must be another buffer than state_idx");
  }
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  fork::Args A = {d->n_rows, d->T, d->max_pages, d->n_pages, parent, n_new, page_table, kv_len, pinned, page_table_out,
                  kv_len_out, kv_index, page_src, page_dst, state_idx, state_idx_out, state_src, state_dst, dev->status};
  const size_t smem = (size_t)(d->n_pages + 31) / 32 * 4;
  static std::atomic<uint64_t> ready{0};  // a bit a device: the attribute holds for the process
  const uint64_t bit = 1ull << dev->id;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {  // beside the kernel's own 41 KB the default allows 6
    if (cudaFuncSetAttribute(fork::fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, fork::kMaxPages / 8) !=
        cudaSuccess)
      return check_launch("cache_fork");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  launch_pdl(fork::fork_kernel, dim3(1), dim3(fork::kThreads), smem, static_cast<cudaStream_t>(stream), A);
  return check_launch("cache_fork");
}

extern "C" gdn_status gdn_slots_copy(const gdn_slot_pool *pools, int32_t n_pools, void *stream) {
  if (n_pools < 0 || n_pools > GDN_MAX_SLOT_POOLS) return fail(GDN_ERR_SHAPE, "n_pools must be in [0, 4]");
  if (n_pools == 0) return GDN_OK;
  if (!pools) return fail(GDN_ERR_ARG, "pools is NULL");
  slots::Args A = {};
  long long ctas = 0;
  for (int k = 0; k < n_pools; ++k) {
    const gdn_slot_pool &p = pools[k];
    if (p.slot_bytes < 0 || p.slot_bytes % 16 != 0 || p.slot_bytes > (1LL << 40))
      return fail(GDN_ERR_SHAPE, "slot_bytes must be a multiple of 16 in [0, 2^40]");
    if (p.n < 0 || p.n_layers < 0 || p.n_slots < 0 || (long long)p.n * p.n_layers > (1 << 20))
      return fail(GDN_ERR_SHAPE, "n, n_layers and n_slots must be >= 0, n * n_layers at most 2^20");
    if (p.n == 0 || p.n_layers == 0 || p.slot_bytes == 0) continue;
    GDN_TRY(check_ptr(p.base, "base"));
    GDN_TRY(check_ptr(p.src, "src", 4));
    GDN_TRY(check_ptr(p.dst, "dst", 4));
    slots::Pool &q = A.pool[A.n++];
    q.base = static_cast<uint4 *>(p.base);
    q.src = p.src;
    q.dst = p.dst;
    q.vec = p.slot_bytes / 16;
    q.first = ctas;
    q.n = p.n;
    q.layers = p.n_layers;
    q.slots = p.n_slots;
    const long long pieces = (q.vec + slots::kThreads * slots::kPiece - 1) / (slots::kThreads * slots::kPiece);
    if (pieces * p.n * p.n_layers > 0x7fffffffLL - ctas) return fail(GDN_ERR_SHAPE, "more copies than a grid holds");
    q.pieces = (int)pieces;
    ctas += pieces * p.n * p.n_layers;
  }
  if (ctas == 0) return GDN_OK;
  const DeviceInfo *dev;
  GDN_TRY(current_device(&dev));
  A.status = dev->status;
  launch_pdl(slots::copy_kernel, dim3((unsigned)ctas), dim3(slots::kThreads), 0, static_cast<cudaStream_t>(stream), A);
  return check_launch("slots_copy");
}
