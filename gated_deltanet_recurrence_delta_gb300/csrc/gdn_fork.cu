// gdn_cache_fork: rows of a paged cache become copies of other rows and get
// room for new tokens; gdn_slots_copy: the copies that this takes.
//
// cache_fork is bookkeeping of a few thousand numbers between dependent steps
// (which pages are used -> which are free -> who gets which -> where the tokens
// go), so one CTA does it without leaving the SM: what is used stands as one bit
// a page in shared memory, free pages are ranked by a scan of the bits' counts,
// and the page of rank k goes to the row whose needs cover k. Latency bounds it.
//
// slots_copy is an HBM copy of 16-byte vectors; a CTA takes one piece of one
// slot of one layer, and a skipped pair's CTAs end at once.
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

// Inclusive scan over the CTA; `part` holds kWarps numbers.
__device__ __forceinline__ int scan(int x, int *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // part may still be read by an earlier scan
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int y = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  y = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  return x + (warp > 0 ? y : 0);
}

__device__ __forceinline__ int pages(int tokens) { return (tokens + kPage - 1) / kPage; }

__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ Args A) {
  extern __shared__ uint32_t s_used[];  // a bit a page
  __shared__ int s_par[kMaxRows], s_len[kMaxRows], s_new[kMaxRows], s_first[kMaxRows];
  __shared__ int s_need[kMaxRows];  // pages of the rows up to this one
  __shared__ int s_dead[kMaxRows];  // rows without children, in order
  __shared__ uint8_t s_copy[kMaxRows];
  __shared__ int s_part[kWarps], s_total;
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = A.rows;
  const int words = (A.n_pages + 31) / 32;
  const long long most = (long long)A.width * kPage;

  // ---- the rows
  bool bad = false;
  if (tid < R) {
    int p = A.parent ? A.parent[tid] : tid, n = A.n_new ? A.n_new[tid] : A.T, len = 0;
    if (p < -1 || p >= R) {
      bad = true;
      p = -1;
    }
    if (p >= 0) {
      len = A.len[p];
      if (len < 0 || len > most) {
        bad = true;
        len = 0;
      }
    }
    if (n < 0 || n > A.T) {
      bad = true;
      n = 0;
    }
    s_par[tid] = p;
    s_len[tid] = len;
    s_new[tid] = n;
    s_first[tid] = kMaxRows;
    s_copy[tid] = 0;
  }
  // ---- pinned pages
  for (int w = tid; w < words; w += kThreads) {
    uint32_t bits = w == words - 1 && A.n_pages % 32 ? ~0u << (A.n_pages % 32) : 0u;
    if (A.pinned)
      for (int i = 0; i < 32 && 32 * w + i < A.n_pages; ++i) bits |= (uint32_t)(A.pinned[32 * w + i] != 0) << i;
    s_used[w] = bits;
  }
  __syncthreads();
  if (tid < R && s_par[tid] >= 0) atomicMin(&s_first[s_par[tid]], tid);  // the lowest child
  // ---- the rows' pages: handed on and marked
  for (int r = warp; r < R; r += kWarps) {
    const int p = s_par[r], n = pages(s_len[r]);
    if (p < 0) continue;
    const int32_t *from = A.table + (long long)p * A.width;
    int32_t *to = A.table_out + (long long)r * A.width;
    for (int j = lane; j < n; j += 32) {
      const int page = from[j];
      to[j] = page;
      if (page < 0 || page >= A.n_pages)
        bad = true;
      else
        atomicOr(&s_used[page >> 5], 1u << (page & 31));
    }
  }
  // ---- partly filled last pages that are to be written, and are not the row's alone
  for (int r = warp; r < R; r += kWarps) {
    const int len = s_len[r], at = len / kPage;
    if (s_new[r] == 0 || len % kPage == 0) continue;
    const int page = A.table[(long long)s_par[r] * A.width + at];
    if (page < 0 || page >= A.n_pages) continue;
    bool other = A.pinned && A.pinned[page];
    for (int x = lane; x < R; x += 32)
      other |= x != r && pages(s_len[x]) > at && (s_len[x] > len || (s_len[x] == len && x < r)) &&
               A.table[(long long)s_par[x] * A.width + at] == page;
    if (__any_sync(0xffffffffu, other) && lane == 0) s_copy[r] = 1;
  }
  __syncthreads();
  // ---- what each row needs
  int need = 0;
  if (tid < R && s_new[tid] > 0) {
    const long long after = (long long)s_len[tid] + s_new[tid];
    if (after > most) {
      need = -1;
    } else {
      need = s_copy[tid] + pages((int)after) - pages(s_len[tid]);
    }
  }
  const bool wide = need < 0;  // more than a line of the table holds
  need = max(need, 0);
  const int upto = scan(need, s_part);
  if (tid < R) s_need[tid] = upto;
  // ---- free pages: this thread's run of words
  const int per = (words + kThreads - 1) / kThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += 32 - __popc(s_used[w]);
  const int ahead = scan(mine, s_part);
  if (tid == kThreads - 1) s_total = ahead;
  __syncthreads();
  const int total = s_total, wanted = R > 0 ? s_need[R - 1] : 0;
  int k = ahead - mine;  // rank of this thread's first free page
  if (k < wanted) {
    int r = -1;
    for (int w = w0; w < w1 && k < wanted; ++w) {
      for (uint32_t free = ~s_used[w]; free && k < wanted; free &= free - 1, ++k) {
        const int page = 32 * w + __ffs(free) - 1;
        if (r < 0 || k >= s_need[r]) {  // the first row whose needs reach beyond k
          int lo = r + 1, hi = R - 1;
          while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (s_need[mid] > k) hi = mid;
            else lo = mid + 1;
          }
          r = lo;
        }
        if (s_need[r] > total) continue;  // its pages do not all exist
        const int j = k - (r > 0 ? s_need[r - 1] : 0) - s_copy[r];  // -1: the copy
        const int at = pages(s_len[r]) + j;
        A.table_out[(long long)r * A.width + at] = page;
        if (j < 0) A.page_dst[r] = page;
      }
    }
  }
  // ---- the rows' lengths and copies, the state slots
  bool full = false;
  int taken = 0, again = 0, dead = 0;
  if (tid < R) {
    taken = s_new[tid];
    full = wide || (taken > 0 && need > 0 && upto > total);
    if (full) taken = 0;
    A.len_out[tid] = s_len[tid] + taken;
    const bool copy = s_copy[tid] && !full;
    A.page_src[tid] = copy ? A.table[(long long)s_par[tid] * A.width + s_len[tid] / kPage] : -1;
    if (!copy) A.page_dst[tid] = -1;
    again = s_par[tid] < 0 || s_first[s_par[tid]] != tid;
    dead = s_first[tid] == kMaxRows;
  }
  if (A.state) {
    const int nth_dead = scan(dead, s_part);
    if (dead) s_dead[nth_dead - 1] = tid;
    const int nth = scan(again, s_part);
    __syncthreads();
    if (tid < R) {
      const int from = s_par[tid] < 0 ? -1 : A.state[s_par[tid]];
      const int to = again ? A.state[s_dead[nth - 1]] : from;
      A.state_out[tid] = to;
      A.state_src[tid] = again ? from : -1;
      A.state_dst[tid] = again && from >= 0 ? to : -1;
    }
  }
  if (__syncthreads_or(bad) && tid == 0) set_status(A.status, GDN_ERR_INDEX);
  if (__syncthreads_or(full) && tid == 0) set_status(A.status, GDN_ERR_FULL);
  // ---- the pool rows of the new tokens
  if (tid < R) s_new[tid] = taken;
  __syncthreads();
  for (long long i = tid; i < (long long)R * A.T; i += kThreads) {
    const int r = (int)(i / A.T), t = (int)(i - (long long)r * A.T), place = s_len[r] + t;
    int row = -1;
    if (t < s_new[r]) {
      const int page = A.table_out[(long long)r * A.width + place / kPage];
      if (page >= 0 && page < A.n_pages) row = page * kPage + place % kPage;
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
  if (smem > 16384) {  // always to the most, so that calls of several threads agree
    if (cudaFuncSetAttribute(fork::fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, fork::kMaxPages / 8) !=
        cudaSuccess)
      return check_launch("cache_fork");
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
