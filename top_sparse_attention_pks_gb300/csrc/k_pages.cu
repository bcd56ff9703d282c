// Pages of a block table on the device: reference counts, fork, growth with
// copy-on-write, truncation and compaction.
//
// "Paged KV cache, or why reserving for the maximum length is wasteful",
// "Paging" and "Page sharing": rows of the table point at fixed-size pages and
// rows with the same prefix point at the same ones; "What this table does not
// say": somebody has to keep the list of free pages.  Here that is a count of
// holders per page and a bitmap of the pages nobody holds, both in device
// memory, so a decode loop changes its table without a host round trip.
//
// All results are whole numbers that do not depend on the order of the
// threads: counts change by atomic adds, a page becomes free when its count
// reaches zero, and pages are taken lowest id first (a prefix sum over the
// rows' needs against a prefix sum over the bitmap), so no list order exists
// that atomics could disturb.  The bitmap is what keeps the allocating scans
// small: 131,072 pages are 16 KB.
//
// The calls on small tables are bound by latency (a launch and a few dependent
// L2 round trips); the data movement of k_pages_move is bound by HBM.

#include "pks_internal.h"

namespace pks {
namespace {

// header words of the state
constexpr int kHdrPages = 0, kHdrPageSize = 1, kHdrFree = 2, kHdrErr = 3, kHdrMoves = 4,
              kHdrMagic = 5, kHdrGrant = 6, kHdrUsed = 7, kHdrCalls = 8;

constexpr int kRowThreads = 256;    // fork, free: a block a row
constexpr int kRowUnroll = 8;       // entries of a row a thread has in flight
constexpr int kPlanThreads = 1024;  // extend and compact: the one planning block
constexpr int kMaxRows = 4096;
constexpr int kTakenShared = 1024;  // taken pages that extend keeps in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;  // units a thread has in flight
// blocks an SM of the moving kernels (compact, 367 MB moved: 134 us with 4, 128 with
// 8, 123 with 16; tails take the same from 4 on)
constexpr int kMoveBlocks = 16;

struct PageState {
  int32_t* hdr;
  int32_t* ref;
  uint32_t* free_map;
  int4* moves;      // (source page, destination page, tokens, -)
  int32_t* taken;   // extend: the pages taken, ascending
  int32_t* cnt;     // extend: growing holders of a shared last page, zero between calls
  int32_t* last;    // extend: the highest of them + 1, zero between calls
  uint64_t* stamp;  // compact: (call << 32) | counterpart page
};

PageState page_state(void* state, const PagesLayout& L) {
  uint8_t* s = static_cast<uint8_t*>(state);
  PageState p;
  p.hdr = reinterpret_cast<int32_t*>(s);
  p.ref = reinterpret_cast<int32_t*>(s + L.ref);
  p.free_map = reinterpret_cast<uint32_t*>(s + L.free_map);
  p.moves = reinterpret_cast<int4*>(s + L.moves);
  p.taken = reinterpret_cast<int32_t*>(s + L.taken);
  p.cnt = reinterpret_cast<int32_t*>(s + L.cnt);
  p.last = reinterpret_cast<int32_t*>(s + L.last);
  p.stamp = reinterpret_cast<uint64_t*>(s + L.stamp);
  return p;
}

__device__ __forceinline__ void flag_error(int32_t* hdr, int code) {
  atomicCAS(hdr + kHdrErr, 0, code);
}

// the state is one that pks_pages_init filled for these pages
__device__ __forceinline__ bool state_ok(const PageState& st, int num_pages, int page_size) {
  const int2 of = *reinterpret_cast<const int2*>(st.hdr + kHdrPages);
  return (st.hdr[kHdrMagic] == kPagesMagic) & (of.x == num_pages) & (of.y == page_size);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return (int)(((int64_t)tokens + page_size - 1) / page_size);
}

// inclusive scan over the block of one value a thread; s_warp holds NT / 32 ints
template <int NT>
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp may still be read from an earlier scan
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  static_assert(NT == 1024, "one warp scans the warps' sums");
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return x + (warp > 0 ? before : 0);
}

// ---- init: holders of every page, from the tables
__global__ void __launch_bounds__(kRowThreads)
k_pages_count(PageState st, const int32_t* __restrict__ seq_lens,
              const int32_t* __restrict__ block_table, int num_pages, int page_size,
              int max_pages) {
  const int b = blockIdx.x;
  const int len = seq_lens[b];
  if (len < 0 || len > max_pages * page_size) {
    if (threadIdx.x == 0) flag_error(st.hdr, kErrLen);
    return;
  }
  const int n = pages_of(len, page_size);
  for (int p = threadIdx.x; p < n; p += kRowThreads) {
    const int page = block_table[(int64_t)b * max_pages + p];
    if ((unsigned)page < (unsigned)num_pages) atomicAdd(&st.ref[page], 1);
    else flag_error(st.hdr, kErrPage);
  }
}

__global__ void __launch_bounds__(256)
k_pages_map(PageState st, int num_pages, int page_size) {
  const int p = blockIdx.x * 256 + threadIdx.x;
  const bool is_free = p < num_pages && st.ref[p] == 0;
  const uint32_t m = __ballot_sync(0xffffffffu, is_free);
  if ((threadIdx.x & 31) == 0 && p < num_pages) {
    st.free_map[p >> 5] = m;
    if (m) atomicAdd(&st.hdr[kHdrFree], __popc(m));
  }
  if (p == 0) {
    st.hdr[kHdrPages] = num_pages;
    st.hdr[kHdrPageSize] = page_size;
    st.hdr[kHdrMagic] = kPagesMagic;
  }
}

// ---- fork: a block a fork.  Every block decides from the lists and from rows
// that no fork of this call writes, so the outcome does not depend on the
// order of the blocks.
__global__ void __launch_bounds__(kRowThreads)
k_pages_fork(PageState st, int32_t* seq_lens, int32_t* block_table, int num_pages, int page_size,
             int B, int max_pages, int n, const int32_t* __restrict__ src_rows,
             const int32_t* __restrict__ dst_rows, const int32_t* __restrict__ n_tokens) {
  const int i = blockIdx.x, tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait(src_rows, dst_rows, n_tokens);
  const bool known = state_ok(st, num_pages, page_size);
  const int src = src_rows[i], dst = dst_rows[i];
  bool bad = (unsigned)src >= (unsigned)B || (unsigned)dst >= (unsigned)B || src == dst;
  for (int j = tid; j < n; j += kRowThreads) {
    const int d = dst_rows[j], s = src_rows[j];
    // an earlier fork has this destination; a row on both sides
    bad |= (j < i && d == dst) || d == src || s == dst;
  }
  if (__syncthreads_or(bad) || !known) {
    if (tid == 0) flag_error(st.hdr, known ? kErrRow : kErrState);
    return;
  }
  if (seq_lens[dst] != 0) {
    if (tid == 0) flag_error(st.hdr, kErrRow);
    return;
  }
  const int len = seq_lens[src];
  int tok = n_tokens ? n_tokens[i] : len;
  if (tok < 0) tok = len;
  if (len < 0 || len > max_pages * page_size || tok > len) {
    if (tid == 0) flag_error(st.hdr, kErrLen);
    return;
  }
  const int np = pages_of(tok, page_size);
  const int32_t* from = block_table + (int64_t)src * max_pages;
  int32_t* to = block_table + (int64_t)dst * max_pages;
  bool bad_page = false;
  for (int p0 = tid; p0 < np; p0 += kRowThreads * kRowUnroll) {
    int page[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int p = p0 + u * kRowThreads;
      page[u] = p < np ? from[p] : 0;
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) bad_page |= (unsigned)page[u] >= (unsigned)num_pages;
  }
  if (__syncthreads_or(bad_page)) {  // also: every thread has read the destination's length
    if (tid == 0) flag_error(st.hdr, kErrPage);
    return;
  }
  for (int p0 = tid; p0 < np; p0 += kRowThreads * kRowUnroll) {
    int page[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int p = p0 + u * kRowThreads;
      page[u] = p < np ? from[p] : -1;
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u)
      if (page[u] >= 0) {
        to[p0 + u * kRowThreads] = page[u];
        atomicAdd(&st.ref[page[u]], 1);
      }
  }
  if (tid == 0) seq_lens[dst] = tok;
}

// ---- free: a block a row
__global__ void __launch_bounds__(kRowThreads)
k_pages_free(PageState st, int32_t* seq_lens, int32_t* block_table, int num_pages, int page_size,
             int B, int max_pages, int n, const int32_t* __restrict__ rows,
             const int32_t* __restrict__ keep) {
  const int i = blockIdx.x, tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait(rows, keep);
  const bool known = state_ok(st, num_pages, page_size);
  const int row = rows[i];
  bool bad = (unsigned)row >= (unsigned)B;
  for (int j = tid; j < i; j += kRowThreads) bad |= rows[j] == row;
  if (__syncthreads_or(bad) || !known) {
    if (tid == 0) flag_error(st.hdr, known ? kErrRow : kErrState);
    return;
  }
  const int len = seq_lens[row];
  const int tok = keep ? keep[i] : 0;
  if (len < 0 || len > max_pages * page_size || tok < 0 || tok > len) {
    if (tid == 0) flag_error(st.hdr, kErrLen);
    return;
  }
  const int p1 = pages_of(len, page_size);
  int32_t* row_t = block_table + (int64_t)row * max_pages;
  int freed = 0;
  for (int p0 = pages_of(tok, page_size) + tid; p0 < p1; p0 += kRowThreads * kRowUnroll) {
    int page[kRowUnroll], had[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int p = p0 + u * kRowThreads;
      page[u] = p < p1 ? row_t[p] : -1;
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      if (p0 + u * kRowThreads >= p1) continue;
      row_t[p0 + u * kRowThreads] = -1;
      if ((unsigned)page[u] < (unsigned)num_pages) had[u] = atomicSub(&st.ref[page[u]], 1);
      else flag_error(st.hdr, kErrPage);
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      if ((unsigned)page[u] >= (unsigned)num_pages) continue;
      if (had[u] <= 0) {  // the tables hold it more often than its count says
        atomicAdd(&st.ref[page[u]], 1);
        flag_error(st.hdr, kErrState);
      } else if (had[u] == 1) {
        atomicOr(&st.free_map[page[u] >> 5], 1u << (page[u] & 31));
        ++freed;
      }
    }
  }
  freed = __reduce_add_sync(0xffffffffu, freed);
  if ((tid & 31) == 0 && freed) atomicAdd(&st.hdr[kHdrFree], freed);
  __syncthreads();  // every thread has read the length
  if (tid == 0) seq_lens[row] = tok;
}

// ---- extend: one block plans the growth of every row
__global__ void __launch_bounds__(kPlanThreads)
k_pages_extend(PageState st, int32_t* seq_lens, int32_t* block_table, int num_pages,
               int page_size, int B, int max_pages, const int32_t* __restrict__ add) {
  constexpr int kPer = kMaxRows / kPlanThreads;
  __shared__ int s_warp[32];
  __shared__ int s_start[kMaxRows + 1];  // first taken page of each row
  __shared__ int s_had[kMaxRows];        // the row's pages before
  __shared__ int s_taken[kTakenShared];  // the first taken pages (the rest: st.taken)
  __shared__ unsigned s_need[kPlanThreads / 32];
  const int tid = threadIdx.x;
  const int max_len = max_pages * page_size;
  pdl_launch_dependents();  // the copies' blocks may come in and wait
  pdl_wait(add);
  const int n_free = st.hdr[kHdrFree];
  const bool known = state_ok(st, num_pages, page_size);
  const int words = (num_pages + 31) / 32;
  // the bitmap's first words, on their way while the rows are looked at
  uint4 first_words = make_uint4(0, 0, 0, 0);
  if (tid * 4 < words) first_words = *reinterpret_cast<const uint4*>(st.free_map + tid * 4);
  int len[kPer], inc[kPer], tail[kPer], holders[kPer];
  bool bad_len = false, bad_page = false;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int b = tid + u * kPlanThreads;
    len[u] = inc[u] = 0;
    if (b < B) {
      len[u] = seq_lens[b];
      inc[u] = add[b];
    }
  }
  if (!known) {
    if (tid == 0) {
      flag_error(st.hdr, kErrState);
      st.hdr[kHdrGrant] = st.hdr[kHdrMoves] = 0;
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int b = tid + u * kPlanThreads;
    tail[u] = -1;  // the partly filled last page of a growing row
    holders[u] = 0;
    if (b >= B) continue;
    if (len[u] < 0 || len[u] > max_len || inc[u] < 0 || inc[u] > max_len - len[u]) {
      bad_len = true;
      inc[u] = 0;
    } else if (inc[u] > 0 && len[u] % page_size) {
      tail[u] = block_table[(int64_t)b * max_pages + len[u] / page_size];
      if ((unsigned)tail[u] >= (unsigned)num_pages) {
        bad_page = true;
        tail[u] = -1;
      } else {
        atomicAdd(&st.cnt[tail[u]], 1);
        atomicMax(&st.last[tail[u]], b + 1);
        holders[u] = st.ref[tail[u]];
      }
    }
  }
  const bool any_len = __syncthreads_or(bad_len), any_page = __syncthreads_or(bad_page);
  int need[kPer];
  bool copy[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int b = tid + u * kPlanThreads;
    copy[u] = false;
    need[u] = 0;
    if (inc[u] > 0) {
      // the last growing holder keeps the page when every holder grows
      if (tail[u] >= 0)
        copy[u] = holders[u] > 1 && !(__ldcg(&st.cnt[tail[u]]) == holders[u] &&
                                      __ldcg(&st.last[tail[u]]) == b + 1);
      need[u] = pages_of(len[u] + inc[u], page_size) - pages_of(len[u], page_size) + copy[u];
    }
  }
  // the rows' needs may sum up past 32 bits before they are refused (a warp's do
  // not: 128 rows of up to 2^24 pages)
  unsigned mine = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) mine += need[u];
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((tid & 31) == 0) s_need[tid >> 5] = mine;
  __syncthreads();
  unsigned long long all = s_need[tid & 31];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  const bool enough = n_free >= 0 && all <= (unsigned long long)n_free;
  // prefix sums of needs and copies over the rows, 1024 rows at a time
  int at[kPer], c_at[kPer], total = 0, copies = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    at[u] = c_at[u] = 0;
    if (u * kPlanThreads >= B || !enough) continue;  // (the whole block)
    int t0, t1;
    at[u] = total + block_scan<kPlanThreads>(need[u], s_warp, t0) - need[u];
    c_at[u] = copies + block_scan<kPlanThreads>(copy[u], s_warp, t1) - copy[u];
    total += t0;
    copies += t1;
  }
  const bool granted = !any_len && !any_page && enough;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {  // (all threads have read the counts)
    if (tail[u] >= 0) st.cnt[tail[u]] = st.last[tail[u]] = 0;
    const int b = tid + u * kPlanThreads;
    if (b < B) {
      s_start[b] = at[u];
      s_had[b] = pages_of(len[u], page_size) - copy[u];
    }
  }
  if (tid == 0) {
    s_start[B] = total;
    st.hdr[kHdrGrant] = granted;
    if (!granted) {
      st.hdr[kHdrMoves] = 0;
      flag_error(st.hdr, any_len ? kErrLen : any_page ? kErrPage : kErrNoPages);
    }
  }
  if (!granted) return;
  // the lowest `total` free pages: rank every thread's words of the bitmap
  int rank0 = 0;
  for (int w0 = 0; rank0 < total && w0 < words; w0 += kPlanThreads * 4) {
    uint4 m = first_words;
    const int w = w0 + tid * 4;  // the map is padded to whole uint4s
    if (w0 > 0) m = make_uint4(0, 0, 0, 0);
    if (w0 > 0 && w < words) m = *reinterpret_cast<const uint4*>(st.free_map + w);
    const int mine = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
    int in_pass;
    int r = rank0 + block_scan<kPlanThreads>(mine, s_warp, in_pass) - mine;
    if (mine && r < total) {
      uint32_t x[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        while (x[j] && r < total) {
          const int bit = __ffs(x[j]) - 1;
          x[j] &= x[j] - 1;
          const int page = (w + j) * 32 + bit;
          if (r < kTakenShared) s_taken[r] = page;
          else st.taken[r] = page;
          ++r;
        }
      *reinterpret_cast<uint4*>(st.free_map + w) = make_uint4(x[0], x[1], x[2], x[3]);
    }
    rank0 += in_pass;
  }
  __syncthreads();
  auto taken = [&](int r) { return r < kTakenShared ? s_taken[r] : st.taken[r]; };
  if (rank0 < total) {  // the bitmap has fewer pages than the count of free ones:
    for (int r = tid; r < rank0; r += kPlanThreads) {  // those found go back
      const int page = taken(r);
      atomicOr(&st.free_map[page >> 5], 1u << (page & 31));
    }
    if (tid == 0) {
      flag_error(st.hdr, kErrState);
      st.hdr[kHdrGrant] = st.hdr[kHdrMoves] = 0;
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int b = tid + u * kPlanThreads;
    if (b >= B) continue;
    if (copy[u]) {  // numbered in row order
      st.moves[c_at[u]] = make_int4(tail[u], taken(at[u]), len[u] % page_size, 0);
      atomicSub(&st.ref[tail[u]], 1);
    }
    if (inc[u] > 0) seq_lens[b] = len[u] + inc[u];
  }
  // the table: entry j of a row's taken pages follows the pages it had (its
  // copy, if any, replaces the last of them)
  for (int r = tid; r < total; r += kPlanThreads) {
    int lo = 0, hi = B - 1;  // the last row with s_start <= r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_start[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const int page = taken(r);
    block_table[(int64_t)lo * max_pages + s_had[lo] + (r - s_start[lo])] = page;
    st.ref[page] = 1;
  }
  if (tid == 0) {
    st.hdr[kHdrMoves] = copies;
    st.hdr[kHdrFree] = n_free - total;
  }
}

// ---- compact: one block pairs the held pages at or above n_used with the free
// pages below it, both in ascending order
__global__ void __launch_bounds__(kPlanThreads)
k_pages_pair(PageState st, int num_pages, int page_size) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x;
  pdl_launch_dependents();  // the moving blocks may come in and wait
  pdl_wait();
  if (!state_ok(st, num_pages, page_size)) {
    if (tid == 0) flag_error(st.hdr, kErrState);
    return;
  }
  const int n_free = st.hdr[kHdrFree];
  const bool in_range = n_free >= 0 && n_free <= num_pages;
  const int n_used = in_range ? num_pages - n_free : 0;
  const int words = in_range ? (num_pages + 31) / 32 : 0;
  const uint32_t call = (uint32_t)st.hdr[kHdrCalls] + 1;
  int holes = 0, high = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + tid;
    uint32_t hole = 0, held = 0;
    if (w < words) {
      const uint32_t m = st.free_map[w];
      const int below = n_used - w * 32;  // bits under n_used
      const uint32_t lo = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1u;
      const int valid = num_pages - w * 32;
      const uint32_t in = valid >= 32 ? 0xffffffffu : (1u << valid) - 1u;
      hole = m & lo & in;
      held = ~m & ~lo & in;
    }
    int t0, t1;
    int r0 = holes + block_scan<kPlanThreads>(__popc(hole), s_warp, t0) - __popc(hole);
    int r1 = high + block_scan<kPlanThreads>(__popc(held), s_warp, t1) - __popc(held);
    for (; hole; hole &= hole - 1) st.moves[r0++].y = w * 32 + __ffs(hole) - 1;
    for (; held; held &= held - 1) st.moves[r1++].x = w * 32 + __ffs(held) - 1;
    holes += t0;
    high += t1;
  }
  __syncthreads();
  // both counts agree while the map and n_free do; else nothing moves
  const bool agree = in_range && holes == high;
  const int n = agree ? high : 0;
  for (int r = tid; r < n; r += kPlanThreads) {
    const int src = st.moves[r].x, dst = st.moves[r].y;
    st.stamp[src] = ((uint64_t)call << 32) | (uint32_t)dst;
    st.stamp[dst] = ((uint64_t)call << 32) | (uint32_t)src;
  }
  if (tid == 0) {
    if (!agree) flag_error(st.hdr, kErrState);
    st.hdr[kHdrMoves] = n;
    st.hdr[kHdrUsed] = agree ? n_used : -1;
    if (agree) st.hdr[kHdrCalls] = (int32_t)call;
  }
}

// ---- data movement of extend (part of a page) and compact (whole pages), and
// compact's pass over counts, bitmap, page map and table
struct MovePools {
  uint8_t* data[PKS_PAGES_MAX_POOLS];
  int64_t token_bytes[PKS_PAGES_MAX_POOLS];
  int n;
};

template <typename V>
__device__ __forceinline__ void move_units(const PageState& st, const MovePools& pools,
                                           int page_size, bool whole, int64_t jobs_per_pool) {
  const int n = st.hdr[kHdrMoves];
  constexpr int64_t kJob = (int64_t)kMoveThreads * kMoveUnroll;  // units of a job
  const int64_t jobs = (int64_t)n * pools.n * jobs_per_pool;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int64_t piece = j % jobs_per_pool;
    const int pool = (int)(j / jobs_per_pool % pools.n);
    const int4 mv = st.moves[j / jobs_per_pool / pools.n];
    const int64_t tb = pools.token_bytes[pool];
    const int64_t units = (whole ? page_size : mv.z) * tb / (int64_t)sizeof(V);
    const int64_t page_bytes = page_size * tb;
    const V* src = reinterpret_cast<const V*>(pools.data[pool] + mv.x * page_bytes);
    V* dst = reinterpret_cast<V*>(pools.data[pool] + mv.y * page_bytes);
    const int64_t u0 = piece * kJob + threadIdx.x;
    V v[kMoveUnroll];
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
      const int64_t u = u0 + k * kMoveThreads;
      if (u < units) v[k] = src[u];
    }
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
      const int64_t u = u0 + k * kMoveThreads;
      if (u < units) dst[u] = v[k];
    }
  }
}

template <typename V>
__global__ void __launch_bounds__(kMoveThreads)
k_pages_copy_tails(PageState st, MovePools pools, int num_pages, int page_size,
                   int64_t jobs_per_pool) {
  pdl_launch_dependents();
  pdl_wait();
  if (!state_ok(st, num_pages, page_size)) return;
  move_units<V>(st, pools, page_size, false, jobs_per_pool);
}

template <typename V>
__global__ void __launch_bounds__(kMoveThreads)
k_pages_move(PageState st, MovePools pools, const int32_t* __restrict__ seq_lens,
             int32_t* __restrict__ block_table, int32_t* __restrict__ page_map, int num_pages,
             int page_size, int B, int max_pages, int64_t jobs_per_pool) {
  pdl_launch_dependents();
  pdl_wait(seq_lens);
  if (!state_ok(st, num_pages, page_size)) return;
  const int n_used = st.hdr[kHdrUsed];
  if (n_used < 0) return;  // refused
  const uint32_t call = (uint32_t)st.hdr[kHdrCalls];
  const int t0 = blockIdx.x * kMoveThreads + threadIdx.x, step = gridDim.x * kMoveThreads;
  // one thread a page; a pair's counts are written by its source's thread alone
  for (int p = t0; p < num_pages; p += step) {
    const uint64_t s = st.stamp[p];
    const bool moved = (uint32_t)(s >> 32) == call;
    int to = p;
    if (p < n_used) {
      if (moved) to = -1;  // a hole that is filled now: nobody held it
    } else {
      to = moved ? (int)(uint32_t)s : -1;
      if (moved) {
        st.ref[to] = st.ref[p];
        st.ref[p] = 0;
      }
    }
    if (page_map) page_map[p] = to;
  }
  const int words = (num_pages + 31) / 32;
  for (int w = t0; w < words; w += step) {
    const int below = n_used - w * 32, valid = num_pages - w * 32;
    const uint32_t lo = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1u;
    st.free_map[w] = ~lo & (valid >= 32 ? 0xffffffffu : (1u << valid) - 1u);
  }
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    const int len = seq_lens[b];
    if (len < 0 || len > max_pages * page_size) {
      if (threadIdx.x == 0) flag_error(st.hdr, kErrLen);
      continue;
    }
    const int n = pages_of(len, page_size);
    for (int e = threadIdx.x; e < n; e += kMoveThreads) {
      int32_t* at = block_table + (int64_t)b * max_pages + e;
      const int page = *at;
      if ((unsigned)page >= (unsigned)num_pages) {
        flag_error(st.hdr, kErrPage);
      } else if (page >= n_used) {
        const uint64_t s = st.stamp[page];
        if ((uint32_t)(s >> 32) == call) *at = (int)(uint32_t)s;
        else flag_error(st.hdr, kErrState);
      }
    }
  }
  move_units<V>(st, pools, page_size, true, jobs_per_pool);
}

// widest unit that every pool's rows and base allow
int move_width(const pks_pages_args& a) {
  uintptr_t all = 0;
  for (int i = 0; i < a.n_pools; ++i)
    all |= reinterpret_cast<uintptr_t>(a.pools[i].data) | (uintptr_t)a.pools[i].token_bytes;
  return (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
}

MovePools move_pools(const pks_pages_args& a) {
  MovePools m{};
  m.n = a.n_pools;
  for (int i = 0; i < a.n_pools; ++i) {
    m.data[i] = static_cast<uint8_t*>(a.pools[i].data);
    m.token_bytes[i] = a.pools[i].token_bytes;
  }
  return m;
}

int64_t move_jobs_per_pool(const pks_pages_args& a, int width) {
  int64_t most = 0;
  for (int i = 0; i < a.n_pools; ++i)
    most = a.pools[i].token_bytes > most ? a.pools[i].token_bytes : most;
  const int64_t job = (int64_t)kMoveThreads * kMoveUnroll * width;
  const int64_t n = (most * a.page_size + job - 1) / job;
  return n < 1 ? 1 : n;
}

}  // namespace

PagesLayout pages_layout(int32_t num_pages) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t n = (size_t)num_pages;
  PagesLayout L{};
  size_t off = 256;  // header
  L.ref = off;
  off = up(off + 4 * n);
  L.free_map = off;
  off = up(off + 4 * ((n + 31) / 32));
  L.cnt = off;
  off = up(off + 4 * n);
  L.last = off;
  off = up(off + 4 * n);
  L.stamp = off;
  off = up(off + 8 * n);
  L.zeroed = off;  // everything before starts as zeros
  L.moves = off;
  off = up(off + 16 * n);
  L.taken = off;
  off = up(off + 4 * n);
  L.total = off;
  return L;
}

cudaError_t launch_pages_init(const pks_pages_args& a, const PagesLayout& L, cudaStream_t s) {
  const PageState st = page_state(a.state, L);
  cudaError_t e = cudaMemsetAsync(a.state, 0, L.zeroed, s);
  if (e != cudaSuccess) return e;
  if (a.B > 0)
    k_pages_count<<<a.B, kRowThreads, 0, s>>>(st, a.seq_lens, a.block_table, a.num_pages,
                                              a.page_size, a.max_pages);
  k_pages_map<<<(a.num_pages + 255) / 256, 256, 0, s>>>(st, a.num_pages, a.page_size);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const pks_pages_args& a, const PagesLayout& L, int n,
                              const int32_t* src, const int32_t* dst, const int32_t* tokens,
                              cudaStream_t s) {
  return launch_ex(k_pages_fork, dim3(n), dim3(kRowThreads), 0, s, /*pdl=*/true, /*coop=*/false,
                   page_state(a.state, L), a.seq_lens, a.block_table, a.num_pages, a.page_size, a.B,
                   a.max_pages, n, src, dst, tokens);
}

cudaError_t launch_pages_free(const pks_pages_args& a, const PagesLayout& L, int n,
                              const int32_t* rows, const int32_t* keep, cudaStream_t s) {
  return launch_ex(k_pages_free, dim3(n), dim3(kRowThreads), 0, s, /*pdl=*/true, /*coop=*/false,
                   page_state(a.state, L), a.seq_lens, a.block_table, a.num_pages, a.page_size, a.B,
                   a.max_pages, n, rows, keep);
}

cudaError_t launch_pages_extend(const pks_pages_args& a, const PagesLayout& L, const int32_t* add,
                                cudaStream_t s) {
  const PageState st = page_state(a.state, L);
  cudaError_t e = launch_ex(k_pages_extend, dim3(1), dim3(kPlanThreads), 0, s, /*pdl=*/true,
                            /*coop=*/false, st, a.seq_lens, a.block_table, a.num_pages, a.page_size,
                            a.B, a.max_pages, add);
  if (e != cudaSuccess || a.n_pools == 0) return e;
  const int w = move_width(a);
  const int64_t jobs = move_jobs_per_pool(a, w);
  const dim3 grid(device_sm_count() * kMoveBlocks);
  const MovePools pools = move_pools(a);
  auto kern = w == 16 ? k_pages_copy_tails<int4>
                      : w == 4 ? k_pages_copy_tails<int32_t> : k_pages_copy_tails<uint8_t>;
  return launch_ex(kern, grid, dim3(kMoveThreads), 0, s, /*pdl=*/true, /*coop=*/false, st, pools,
                   a.num_pages, a.page_size, jobs);
}

cudaError_t launch_pages_compact(const pks_pages_args& a, const PagesLayout& L, int32_t* page_map,
                                 cudaStream_t s) {
  const PageState st = page_state(a.state, L);
  cudaError_t e = launch_ex(k_pages_pair, dim3(1), dim3(kPlanThreads), 0, s, /*pdl=*/true,
                            /*coop=*/false, st, a.num_pages, a.page_size);
  if (e != cudaSuccess) return e;
  const int w = move_width(a);
  const int64_t jobs = move_jobs_per_pool(a, w);
  const dim3 grid(device_sm_count() * kMoveBlocks);
  const MovePools pools = move_pools(a);
  auto kern = w == 16 ? k_pages_move<int4> : w == 4 ? k_pages_move<int32_t> : k_pages_move<uint8_t>;
  return launch_ex(kern, grid, dim3(kMoveThreads), 0, s, /*pdl=*/true, /*coop=*/false, st, pools,
                   (const int32_t*)a.seq_lens, a.block_table, page_map, a.num_pages, a.page_size,
                   a.B, a.max_pages, jobs);
}

}  // namespace pks
