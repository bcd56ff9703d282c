// Dense decode attention of a batch whose requests alias the pages of a shared
// prefix: the prefix takes part once for all of them.
//
// "Paged KV cache, or why reserving for the maximum length is wasteful",
// "Page sharing": requests with an identical prefix point at the same pages.
// Attention splits over any partition of the tokens,
//   out = sum_i w_i o_i / sum_i w_i l_i,  w_i = 2^(m_i - max m),
// with (m_i, l_i, o_i) the maximum, sum and unnormalised output of part i, so
// a request's attention is the shared prefix's part and its own tokens' part.
// The prefix part of all members of a group is one dense product per KV head,
// with (members x query tokens x heads of the group) rows: its K/V rows are
// read once instead of once a member, and with enough rows it belongs on the
// tensor cores with tensor-memory accumulators.
//
//   k_prefix_plan   which leading table entries each request shares with its
//                   group's longest member, the groups' common prefix, and the
//                   lists of work ("items") below
//   k_prefix_wide   items of up to 256 query rows against a token range (the
//                   prefixes; with more than 16 rows a request and KV head
//                   also the requests' own tokens), tcgen05
//   k_prefix_narrow own tokens of requests with up to 16 rows, streamed like
//                   the sparse attention's rows
//   k_prefix_merge  the parts' combination
//
// Both attention kernels are persistent; each has part of the SMs, as their
// estimated times are, and cuts its work into equal ranges (tiles of all items,
// or own tokens, head after head); a CTA writes a partial (m, l, o) for each
// item or request that its range touches, in slots that the merge derives from
// the plan again.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pks_internal.h"
#include "tcgen05.cuh"

namespace pks {
namespace {

constexpr int kTile = 128;        // tokens of a wide tile (MMA N of S, K of P.V)
constexpr int kRows = 128;        // query rows of one MMA
constexpr int kItemRows = 256;    // query rows of an item: two MMAs
// Most rows (Nq * G) of the narrow kernel.  With 16 rows, four drafts, us a pass:
// 64 requests 126, by the wide kernel (16 of its 128 rows in use) 136; 32 requests
// 83 and 82, 16 requests 60 and 57.
constexpr int kNarrowRows = 16;
constexpr int kNarrowTile = 16;
constexpr int kMaxB = 4096;

struct Item {
  int row0;     // prefix item: first row in group order; own item: first row of the request
  int nrows;    // 1..256
  int bt_row;   // block-table row its tokens are found through
  int own;      // rows of request bt_row against its own tokens: its length; else 0
  int t0, t1;   // token range
  int unit0;    // tiles of the items before it (one head)
  int slot0;    // partial rows of the items before it (one head)
};
// Where a wide CTA starts.
struct Start {
  Item it;
  int head, item;
  int tile;       // of the item
  int pad;
};
// What the merge needs of a request.
struct Request {
  int gunit, gslot, grows, gtiles;  // its group's prefix items: tiles 0 when it has none
  int row;                          // its first row in the group
  int ounit, oslot;                 // its own items (wide)
  int own;                          // own tokens
};

// plan header words
constexpr int kErrWord = 0, kTicket = 1, kItems = 2, kUnits = 3, kSlots = 4, kTiles = 5,
              kShare = 6, kWideCtas = 7, kBig = 8, kPieces = 9, kSmall = 10, kClaim = 11,
              kBigTiles = 12 /* 64 bits */, kDealtTiles = 14, kTag = 15;

struct PlanPtrs {
  int32_t* hdr;
  int32_t *lens, *eq, *first, *lead;   // per request
  int32_t *start;                      // first own token
  int32_t *order;                      // members in group order
  int32_t *npre;                       // [B + 1] narrow tiles before each request
  Request* req;
  Start* starts;                       // per wide CTA
  Item* items;
};

struct PrefixShape {
  int B, Hq, Hkv, G, Nq, R, D;
  int page_size, max_pages, num_pages;
  int causal;
  int narrow;      // own tokens by the narrow kernel
  int wide_grid, narrow_grid;
  int box;         // rows of a TMA box (0: the page size has none)
  int hg;          // KV heads of a narrow CTA
  int min_shared;  // the caller's, or 0
  int tag;         // of the shapes: a plan serves calls of the same shapes only
};

// Unless the caller says from how many shared tokens on (min_shared): shared tokens
// below which a group is not worth a prefix item, one wide tile; and, where the
// narrow kernel would read them as own tokens, the bytes of K and V that all groups
// have to save together, for the wide kernel beside it, its partials and the split
// of the SMs cost as much as reading those, the more the more requests there are.
// Rows that come one by one cost three times as much.  Measured (us a pass, shared /
// each its own, and the megabytes saved): 32 requests in groups of eight with 600
// tokens 67 / 57, 69; with 1000 73 / 64, 115; with 1500 69 / 67, 172; 64 in one with
// 500 90 / 80, 129; 8 in one with 3000 43.5 / 42, 86, with 6000 38 / 50, 172; 4 with
// 6000 35 / 38, 74; pages of 17, 4 in pairs 76 / 84, 61, 40 in groups of 25 33 / 39,
// 78.
constexpr int kMinShared = kTile;
__device__ __forceinline__ int64_t least_saved(const PrefixShape& sh) {
  const int64_t boxes = min(200000000, 40000000 + 3500000 * min(sh.B, 100));
  return sh.box ? boxes : boxes / 3;
}

// 2^x with the hardware's approximate exponential (a few ulp in fp32)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// quotient of two non-negative numbers that nearly always fit in 32 bits, where
// the division takes a fraction of the time
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
  return (int64_t)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ void flag_error(int32_t* err, int code) { atomicCAS(err, 0, code); }

constexpr int kWideLeast = 2;                  // tiles a wide CTA takes at least
constexpr int kNarrowLeast = 2;                // tiles a narrow CTA takes at least
// Tiles of a small narrow piece at least, when there are as many for every CTA
// (2,000 tiles on 152 CTAs: 83.4 us a pass, with pieces of their share of the rest
// 85.6; 100 tiles in pieces of 12 39 us, of 2 29 us).
constexpr int kSmallLeast = 12;
constexpr int kSmallPerSm = 8;                 // small pieces an SM at most
// Beside the wide kernel, a narrow CTA is dealt this share (in 1/16) of what it
// could stream in the time estimated for all; the rest goes to whichever SM is
// free.
constexpr int kDealt = 13;
// Estimated nanoseconds an SM spends with D = 128 (half with D = 64): on a wide
// tile with two row blocks (its products), on one with a single block (its bytes,
// while the narrow kernel loads the memory too), and on a kilobyte streamed by the
// narrow kernel.
constexpr int kPairNs = 1950, kSingleNs = 2000, kStreamNsPerKb = 24;

// The narrow kernel's pieces: `big` equal ones that cover the first big_tiles of
// the T tiles (all heads), one for each CTA that starts at once, and small ones
// for whichever CTA is free.  A piece has its place among the partials whoever
// computes it, so that results do not depend on who does.
struct Pieces {
  int64_t T, big_tiles;
  int big, n, small, share, tag;
  __device__ __forceinline__ Pieces(const int32_t* hdr, int ngroups) {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(hdr + kTiles - 1));
    const int4 b = __ldcg(reinterpret_cast<const int4*>(hdr + kBig));
    const int4 c = __ldcg(reinterpret_cast<const int4*>(hdr + kBigTiles));
    T = (int64_t)a.y * ngroups;
    big = b.x;
    n = b.y;
    small = b.z;
    big_tiles = (int64_t)(uint32_t)c.x | (int64_t)c.y << 32;
    share = c.z;  // (kDealtTiles)
    tag = c.w;    // (kTag)
  }
  __device__ __forceinline__ int64_t lo(int p) const {
    if (p < big) return (int64_t)p * share;
    const int64_t x = big_tiles + (int64_t)(p - big) * small;
    return x < T ? x : T;
  }
  // the piece that holds tile f
  __device__ __forceinline__ int of(int64_t f) const {
    if (f < big_tiles) return (int)quot(f, share);
    return big + (int)quot(f - big_tiles, small);
  }
};

// ------------------------------------------------------------------ plan ---

constexpr int kPlanThreads = 512;
constexpr int kPlanArrays = 14;
constexpr int kPlanWarps = 4;      // warps a request otherwise
// Requests up to which one block does it all (a pass of 5: 18.6 us by one block,
// 20.0 by several; of 107: 64.7 and 55.4; of 128 with long tables 460 and 418).
constexpr int kPlanOneBlock = 32;

// tokens every query of the request sees
__device__ __forceinline__ int seen_by_all(int len, int causal, int Nq) {
  if (!causal) return len;
  const int v = len - Nq + 1;
  return v < 0 ? 0 : v;
}

// Warps find what each request shares with its group's longest member; then one
// block, the only one or the last to finish, makes the plan.
__global__ void __launch_bounds__(kPlanThreads)
k_prefix_plan(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ block_table,
              const int32_t* __restrict__ prefix_group, PlanPtrs pl, PrefixShape sh) {
  extern __shared__ int s_dyn[];  // [kPlanArrays][B]
  __shared__ int s_total[3 + 8];  // tiles, those with one row block, narrow tiles; the scans'
  __shared__ int s_last, s_saved, s_equal[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, B = sh.B;
  const int max_len = sh.max_pages * sh.page_size;
  const bool alone = gridDim.x == 1;
  int* s_first = s_dyn;           // by request
  int* s_lead = s_first + B;
  int* s_eq = s_lead + B;
  int* s_len = s_eq + B;
  int* s_group = s_dyn + (kPlanArrays - 1) * B;  // (the last of the quantities, later)
  pdl_launch_dependents();
  pdl_wait(seq_lens, block_table, prefix_group);
  for (int b = tid; b < B; b += kPlanThreads) {
    int n = seq_lens[b];
    const int g = prefix_group ? prefix_group[b] : -1;
    if (n < 0 || n > max_len) {
      flag_error(pl.hdr + kErrWord, kErrLen);
      n = 0;
    }
    s_len[b] = n;
    s_group[b] = g < 0 ? -1 : g;
    if (blockIdx.x == 0) pl.lens[b] = n;
  }
  __syncthreads();
  // (four warps a request when there are more blocks than one)
  const int wpr = alone ? 1 : kPlanWarps, at_once = kPlanThreads / 32 / wpr;
  const int slot = (tid >> 5) / wpr, sub = (tid >> 5) % wpr;
  for (int b0 = blockIdx.x * at_once; b0 < B; b0 += gridDim.x * at_once) {
    const int b = b0 + slot;
    const int len = b < B ? s_len[b] : 0, g = b < B ? s_group[b] : -1;
    const int np = (len + sh.page_size - 1) / sh.page_size;
    int first = b, lead = b;
    if (tid < at_once) s_equal[tid] = 0x7fffffff;
    __syncthreads();
    if (g >= 0) {
      // longest member (the first of the longest) and first member of the group
      long long best = -1;
      int low = B;
      for (int c = lane; c < B; c += 32)
        if (s_group[c] == g) {
          const long long key = ((long long)s_len[c] << 12) | (kMaxB - 1 - c);
          best = key > best ? key : best;
          low = c < low ? c : low;
        }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        const long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
      }
      first = __reduce_min_sync(0xffffffffu, low);
      lead = kMaxB - 1 - (int)(best & (kMaxB - 1));
      // leading entries equal to the longest member's
      const int32_t* mine = block_table + (int64_t)b * sh.max_pages;
      const int32_t* its = block_table + (int64_t)lead * sh.max_pages;
      constexpr int kStep = 16;
      for (int p0 = sub * 32 * kStep; lead != b && p0 < np; p0 += wpr * 32 * kStep) {
        int differs = 0x7fffffff, x[kStep], y[kStep];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const int p = p0 + u * 32 + lane;
          x[u] = p < np ? mine[p] : 0;
          y[u] = p < np ? its[p] : 0;
        }
#pragma unroll
        for (int u = kStep - 1; u >= 0; --u)
          if (x[u] != y[u]) differs = p0 + u * 32 + lane;
        differs = __reduce_min_sync(0xffffffffu, differs);
        if (differs != 0x7fffffff) {
          if (lane == 0) atomicMin(&s_equal[slot], differs);
          break;
        }
      }
    }
    __syncthreads();
    if (lane == 0 && sub == 0 && b < B) {
      const int seen = seen_by_all(len, sh.causal, sh.Nq);
      const int64_t tok = (int64_t)min(np, s_equal[slot]) * sh.page_size;
      (alone ? s_eq : pl.eq)[b] = g < 0 ? 0 : tok < seen ? (int)tok : seen;
      (alone ? s_first : pl.first)[b] = first;
      (alone ? s_lead : pl.lead)[b] = lead;
    }
    __syncthreads();
  }
  if (!alone) {
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(pl.hdr + kTicket, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (tid == 0) pl.hdr[kTicket] = 0;
    for (int b = tid; b < B; b += kPlanThreads) {
      s_first[b] = __ldcg(pl.first + b);
      s_lead[b] = __ldcg(pl.lead + b);
      s_eq[b] = __ldcg(pl.eq + b);
    }
  }

  // eight quantities by request (those of a group by its first member), summed up
  // over the requests before: members; prefix items, tiles and partial rows; narrow
  // tiles; own items, tiles and partial rows
  int* s_pre = s_len + B;    // by first member: the group's prefix
  int* s_cnt = s_pre + B;    // ... members that take part
  int* s_at = s_cnt + B;
  int* s_item = s_at + B;
  int* s_unit = s_item + B;
  int* s_slot = s_unit + B;
  int* s_otile = s_slot + B;
  int* s_oitem = s_otile + B;
  int* s_ounit = s_oitem + B;
  int* s_oslot = s_ounit + B;
  int* s_most = s_at;        // first: the most shared, the longest member aside
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) {
    s_pre[b] = 0x7fffffff;
    s_cnt[b] = s_most[b] = 0;
  }
  if (tid < 3) s_total[tid] = 0;
  if (tid == 0) s_saved = 0;
  __syncthreads();
  // The groups' common prefixes: the least shared length among the members that
  // share at least half of what the second longest shares; members with less
  // stay on their own.
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads)
    if (s_lead[b] != b) atomicMax(&s_most[s_first[b]], s_eq[b]);
  __syncthreads();
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) {
    const int f = s_first[b], e = s_eq[b], most = s_most[f];
    if (most >= (sh.min_shared ? sh.min_shared : kMinShared) && e >= (most + 1) / 2) {
      atomicMin(&s_pre[f], e);
      atomicAdd(&s_cnt[f], 1);
    }
  }
  __syncthreads();
  auto tiles = [](int n) { return (n + kTile - 1) / kTile; };
  auto blocks = [](int rows) { return (rows + kItemRows - 1) / kItemRows; };
  auto single = [](int rows) { return (rows - 1) % kItemRows < kRows ? 1 : 0; };
  bool share = true;
  if (sh.narrow && !sh.min_shared) {
#pragma unroll 1
    for (int b = tid; b < B; b += kPlanThreads)  // (in tiles: 2^27 at most)
      if (s_cnt[b] >= 2) atomicAdd(&s_saved, (s_cnt[b] - 1) * tiles(s_pre[b]));
    __syncthreads();
    share = (int64_t)s_saved * sh.Hkv * (kTile * 4 * sh.D) >= least_saved(sh);
  }
  // the group (by its first member) that request b takes part in, or -1
  auto joined = [&](int b) {
    const int f = s_first[b];
    return share && s_cnt[f] >= 2 && s_eq[b] >= s_pre[f] ? f : -1;
  };
  const int own_blocks = sh.narrow ? 0 : blocks(sh.R);
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) {
    const bool has = share && s_cnt[b] >= 2;
    const int rows = s_cnt[b] * sh.R, nt = has ? tiles(s_pre[b]) : 0;
    const int f = joined(b), begin = f >= 0 ? s_pre[f] : 0, own = s_len[b] - begin;
    s_at[b] = has ? s_cnt[b] : 0;
    s_unit[b] = has ? blocks(rows) * nt : 0;
    s_otile[b] = sh.narrow ? (own + kNarrowTile - 1) / kNarrowTile : 0;
    s_ounit[b] = own_blocks * tiles(own);
    pl.start[b] = begin;
    const int u = s_unit[b] + s_ounit[b];
    if (u) atomicAdd(&s_total[0], u);
    const int ones = (has ? single(rows) * nt : 0) + (own_blocks ? single(sh.R) * tiles(own) : 0);
    if (ones) atomicAdd(&s_total[1], ones);
    if (s_otile[b]) atomicAdd(&s_total[2], s_otile[b]);
  }
  __syncthreads();
  const int U = s_total[0], own_tiles = s_total[2];
  // SMs for either kernel by the time they will need, and the tiles a wide CTA
  // takes (all of the same number, so that items cut at multiples of it run in
  // step; see the wide kernel)
  const int64_t total = (int64_t)U * sh.Hkv, singles = (int64_t)s_total[1] * sh.Hkv;
  const float pairs_ns = (float)(total - singles) * kPairNs * sh.D / 128;
  const float wide_ns = pairs_ns + (float)singles * kSingleNs * sh.D / 128;
  const float stage_kb = (float)kNarrowTile * sh.D * 4 / 1024;  // K and V of a tile, one head
  const float narrow_ns = (float)own_tiles * sh.Hkv * stage_kb * kStreamNsPerKb;
  int W = sh.wide_grid;
  // side by side only when the wide kernel needs three quarters of the narrow
  // one's time at least: its CTAs get less than their share of a memory that the
  // narrow kernel loads (with 2% of the bytes wide, 64 requests of up to 32k
  // tokens: 588 us side by side on 9 SMs, 950 on 3, 578 one after the other; with
  // half of them, 32 requests with four drafts: 88 against 97)
  const bool beside = own_tiles > 0 && total > 0 && 4 * wide_ns >= 3 * narrow_ns;
  if (beside) {
    W = (int)(wide_ns / (wide_ns + narrow_ns) * sh.wide_grid + 0.5f);
    W = max(1, min(sh.wide_grid - 1, W));
  }
  const int sms_left = beside ? sh.wide_grid - W : sh.wide_grid;
  W = (int)min((int64_t)W, (total + kWideLeast - 1) / kWideLeast);
  const int S = total > 0 ? (int)quot(total + W - 1, W) : 1;
  // items: a token range in cuts of S tiles, every row block of a cut in turn
  auto cuts = [&](int nt) { return (int)((unsigned)(nt + S - 1) / (unsigned)S); };
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) {
    const bool has = share && s_cnt[b] >= 2;
    const int rows = s_cnt[b] * sh.R, c = has ? cuts(tiles(s_pre[b])) : 0;
    const int f = joined(b), oc = own_blocks ? cuts(tiles(s_len[b] - (f >= 0 ? s_pre[f] : 0))) : 0;
    s_item[b] = c * blocks(rows);
    s_slot[b] = c * rows;
    s_oitem[b] = oc * own_blocks;
    s_oslot[b] = oc * sh.R;
  }
  __syncthreads();
  const int warp = tid >> 5;
  if (warp < 8) {  // a warp a quantity
    int* v = s_at + warp * B;
    int sum = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane, mine = b < B ? v[b] : 0;
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < B) v[b] = sum + x - mine;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_total[3 + warp] = sum;
  } else if (tid == 8 * 32) {  // the narrow kernel's pieces
    const int64_t T = (int64_t)own_tiles * (sh.Hkv / sh.hg);
    const int per_sm = sh.narrow_grid / sh.wide_grid;
    int64_t big = (int64_t)sms_left * per_sm, big_tiles = T;
    if (beside) {
      const float all_ns = pairs_ns + narrow_ns +
                           (float)singles * (stage_kb * kTile / kNarrowTile) * kStreamNsPerKb;
      const float tile_ns = sh.hg * stage_kb * kStreamNsPerKb * per_sm;
      big_tiles = min(T, big * (int64_t)(all_ns / sh.wide_grid * (kDealt / 16.f) / tile_ns));
    }
    big = min(big, (big_tiles + kNarrowLeast - 1) / kNarrowLeast);
    const int64_t share = big_tiles > 0 ? quot(big_tiles + big - 1, big) : 1;
    big = quot(big_tiles + share - 1, share);
    big_tiles = min(T, big * share);
    const int64_t rest = T - big_tiles, most = (int64_t)kSmallPerSm * sh.wide_grid;
    const int64_t even = quot(T + sh.narrow_grid - 1, sh.narrow_grid);
    const int64_t least = min((int64_t)kSmallLeast, max((int64_t)kNarrowLeast, even));
    const int64_t small = max(least, quot(rest + most - 1, most));
    pl.hdr[kTiles] = own_tiles;
    pl.hdr[kDealtTiles] = (int)share;
    pl.hdr[kBig] = (int)big;
    *reinterpret_cast<int64_t*>(pl.hdr + kBigTiles) = big_tiles;
    pl.hdr[kSmall] = (int)small;
    pl.hdr[kPieces] = (int)(big + quot(rest + small - 1, small));
    pl.hdr[kClaim] = 0;
  } else if (tid == 9 * 32) {
    pl.hdr[kUnits] = U;
    pl.hdr[kShare] = S;
    pl.hdr[kWideCtas] = (int)quot(total + S - 1, S);
  }
  __syncthreads();
  // (own items, tiles and partial rows come behind the prefixes')
  const int p_items = s_total[4], p_units = s_total[5], p_slots = s_total[6];
  const int n_items = p_items + s_total[8];
  if (tid == 0) {
    pl.hdr[kItems] = n_items;
    pl.hdr[kSlots] = p_slots + s_total[10];
    pl.npre[B] = own_tiles;
    pl.hdr[kTag] = sh.tag;
  }
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) pl.npre[b] = s_otile[b];
  // the items, and the CTAs that start in them
#pragma unroll 1
  for (int i = tid; i < n_items; i += kPlanThreads) {
    const bool own = i >= p_items;
    const int at = own ? i - p_items : i;
    const int* first_item = own ? s_oitem : s_item;
    int lo = 0, hi = B - 1;  // the last request whose first item is at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_item[mid] <= at) lo = mid; else hi = mid - 1;
    }
    const int j = at - first_item[lo];
    const int rows = own ? sh.R : s_cnt[lo] * sh.R, k = blocks(rows);
    const int f = joined(lo), begin = own && f >= 0 ? s_pre[f] : 0;
    const int end = own ? s_len[lo] : s_pre[lo];
    const int cut = (int)((unsigned)j / (unsigned)k), blk = j - cut * k;
    const int left = tiles(end - begin) - cut * S, nt = min(S, left);
    Item it;
    it.row0 = (own ? 0 : s_at[lo] * sh.R) + blk * kItemRows;
    it.nrows = min(kItemRows, rows - blk * kItemRows);
    it.bt_row = own ? lo : s_lead[lo];
    it.own = own ? s_len[lo] : 0;
    it.t0 = begin + cut * S * kTile;
    it.t1 = left > S ? it.t0 + S * kTile : end;
    it.unit0 = (own ? p_units + s_ounit[lo] : s_unit[lo]) + cut * S * k + blk * nt;
    it.slot0 = (own ? p_slots + s_oslot[lo] : s_slot[lo]) + cut * rows + blk * kItemRows;
    pl.items[i] = it;
#pragma unroll 1
    for (int h = 0; h < sh.Hkv; ++h) {
      const int64_t u0 = (int64_t)h * U + it.unit0, c = quot(u0 + S - 1, S);
      if (c * S < u0 + nt) {
        Start st = {};
        st.it = it;
        st.head = h;
        st.item = i;
        st.tile = (int)(c * S - u0);
        pl.starts[c] = st;
      }
    }
  }
  __syncthreads();  // s_at counts members from here on
  // members in group order, ascending within a group: one warp, 32 requests at
  // a time; and what the merge needs of each request
  if (tid < 32) {
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + tid;
      const int f = b < B ? joined(b) : -1;
      const uint32_t peers = __match_any_sync(0xffffffffu, f);
      int at = 0;
      if (f >= 0) at = s_at[f] + __popc(peers & ((1u << tid) - 1));
      __syncwarp();
      if (f >= 0 && (peers >> tid) == 1u) s_at[f] = at + 1;  // the last of its group here
      __syncwarp();
      if (f >= 0) {
        pl.order[at] = b;
        s_lead[b] = at;
      }
    }
  }
  __syncthreads();
  // (s_at now ends each group: its first member stands s_cnt places before)
#pragma unroll 1
  for (int b = tid; b < B; b += kPlanThreads) {
    const int f = joined(b);
    Request q = {};
    if (f >= 0) {
      q.gunit = s_unit[f];
      q.gslot = s_slot[f];
      q.grows = s_cnt[f] * sh.R;
      q.gtiles = tiles(s_pre[f]);
      q.row = (s_lead[b] - (s_at[f] - s_cnt[f])) * sh.R;
    }
    q.ounit = p_units + s_ounit[b];
    q.oslot = p_slots + s_oslot[b];
    q.own = s_len[b] - (f >= 0 ? s_pre[f] : 0);
    pl.req[b] = q;
  }
}

// ------------------------------------------------------------------ wide ---
// One CTA an SM, 512 threads:
//   warps 0-3, 4-7   softmax groups 0 and 1: a thread a query row
//   warps 8, 9       issue the MMAs of groups 0 and 1
//   warps 10-13      load the K/V tiles (TMA_WARPS of them those that come by TMA)
//   warps 14, 15     load Q, a piece ahead where it fits, and tell the others
// An item with more than 128 rows gives each group a row block of its own and
// every tile goes to both; with 128 or fewer both groups hold the same rows and
// take the tiles in turn, through all pieces (6 requests over prefixes of 7,000
// tokens: 33 us, 37 when group 0 began every piece), so that one group's softmax
// always runs beside the other's products.  Per job (a tile of a group):
//   S[128 x 128] = Q K^T        tcgen05.mma, fp32 in tensor memory
//   P            = 2^(S c - m)  a thread a row, bf16 into S's columns
//   O[128 x D]  += P V          tcgen05.mma, P from tensor memory, in two halves
//                               as the softmax delivers them
// An issuing thread's products run in its order, so the next S may overwrite the
// P before it, and the completion of S implies that of the P.V before it.  (One
// thread for both groups left the tensor pipe idle through its waits: 40% active;
// an issuer a group hides them behind the other's products.)
// K and V tiles share a ring of slots (K, V, K, V, ...) of 128-byte swizzled
// rows.  A tile of whole boxes (sh.box: the largest power of two up to 128 that
// divides the page size, from 8, the swizzle's period) comes by TMA, the last
// tile of a range and tiles of odd pages row by row with cp.async, which fills
// what lies beyond the range with zeros.  All CTAs take the same number of tiles
// and a prefix is cut into items of just as many, row blocks within a cut next to
// each other: CTAs that read the same tiles for different rows then do so in
// step, from L2 (1024 rows on 131,072 tokens: 0.64 GB read from memory instead of
// 2.15).  The running maximum moves only when a tile exceeds it by more than 8
// (log2 units).
//
// Measured on that product (K/V of 8 heads, 550 GFLOP): 1.45 PFLOP/s, the tensor
// pipe 72% active on the SMs it has.  Softmax arithmetic is not what bounds it
// (without the exponentials it takes as long); the pipe takes about 76 cycles for
// a product of 64 when one issuer feeds it, both operands coming from shared
// memory, and idles where the turns change.  With D = 64 half the products take
// 325 of 379 us: a group's next S waits for its P.V.  With a single row block and
// 64 KB a tile it is bound by memory.

constexpr int kWideThreads = 512;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kLoadWarps = 4, kQWarp = 14;
constexpr int kNotes = 4;  // pieces announced at a time, at most
constexpr long long kWaitCycles = 4000000000LL;  // about 2 s at 2 GHz, unless wait_limit is set

template <int D>
struct Wide {
  static constexpr int kBlk = D / 64;                          // 64-value column blocks
  static constexpr uint32_t kGroupBytes = kBlk * 1024;         // eight rows, block by block
  static constexpr uint32_t kTileBytes = kTile / 8 * kGroupBytes;  // K, V or Q tile
  static constexpr int kSlotsN = D == 128 ? 5 : 10;            // ring of K / V tiles
  static constexpr uint32_t kSmem = (2 + kSlotsN) * kTileBytes + 1024;
  // loads in flight beyond the newest; a piece has at least these (K and V of a tile)
  static constexpr int kLag = 2;
};
constexpr uint32_t kTmemS = 256;  // columns: O of the groups at 0 and 128, S at 256 and 384

// One CTA's share of one item.
struct Piece {
  Item it;
  int head, t_lo, nt;   // first tile and tiles
  bool pair;            // two row blocks
  int jobs0, jobs1;     // jobs of the softmax groups
  int turn;             // the group that begins
  int64_t slot;         // its first partial row
};
// What the issuers and the softmax need of a piece.
struct Note {
  int nt, by_tma, jobs0, jobs1;
  int nrows, row0, own;  // of its item
  int tok0, tok1;        // its first token, the item's last + 1
  int q_block;           // ring block of Q (of group 0 when there are two)
  int pair, turn, last;
  int64_t slot;
};
// What a loading warp has put into the ring's slots: the number of its half tiles
// (K or V; slot by slot in turn), and by slot whether the last came by TMA, whether
// any did, and the number of those modulo two.
struct Fills {
  uint32_t n, by_tma, used, count;
};
// A CTA's walk over its tiles, by the loads' warps.
struct Walk {
  const Item* items;
  int left;             // tiles to come
  int head, item, tile; // the next one
  int turn;             // the group whose job comes next
  const int* sizes;     // items and partial rows of a head (shared memory)
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ Piece next() {
    Piece p;
    p.it = items[item];
    p.head = head;
    p.t_lo = tile;
    p.nt = min(left, (p.it.t1 - p.it.t0 + kTile - 1) / kTile - tile);
    p.pair = p.it.nrows > kRows;
    p.turn = turn;
    p.jobs0 = p.pair ? p.nt : (p.nt + 1 - turn) / 2;
    p.jobs1 = p.pair ? p.nt : (p.nt + turn) / 2;
    if (!p.pair) turn ^= p.nt & 1;
    p.slot = (int64_t)head * sizes[1] + p.it.slot0 + (int64_t)kItemRows * blockIdx.x;
    left -= p.nt;
    tile = 0;
    if (++item == sizes[0]) {
      item = 0;
      ++head;
    }
    return p;
  }
};

// eight fp32 values, 32 bytes aligned: a whole sector a thread
__device__ __forceinline__ void store8(float* dst, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// registers of the softmax warpgroups and of the others: the launch's 512 x 128
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(kSoftmaxRegs + kOtherRegs == 2 * 128, "the launch's registers");

template <int D, int TMA_WARPS>
__global__ void __launch_bounds__(kWideThreads, 1)
k_prefix_wide(const int32_t* __restrict__ block_table, const __nv_bfloat16* __restrict__ q,
              const __nv_bfloat16* __restrict__ kv_k, const __nv_bfloat16* __restrict__ kv_v,
              PlanPtrs pl, float2* __restrict__ part_ml, float* __restrict__ part_o,
              PrefixShape sh, float scale_log2, long long wait_cycles,
              const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v) {
  using W = Wide<D>;
  extern __shared__ uint8_t smem_raw[];
  // bar_tma / bar_cp: a ring slot has landed, by either way of loading; bar_go: it
  // may be filled by the second; bar_free: its products are done (both issuers');
  // bar_note[i]: piece note i and its Q are there; bar_noted: they have been read;
  // bar_qfree[i]: the last product with Q block i is done (both issuers');
  // bar_s[g]: S of group g's job; bar_p[g][h]: half h of its P is written;
  // bar_turn[g]: the other issuer has issued its job's P.V and next S; bar_o[g]:
  // every product of the group's piece; bar_x[g] / bar_y[g]: the group's maxima
  // are posted / it has read the other's O; bar_drain[g]: every product of the
  // group, when a warp has given up
  __shared__ __align__(8) uint64_t bar_tma[W::kSlotsN], bar_cp[W::kSlotsN], bar_go[W::kSlotsN],
      bar_free[W::kSlotsN], bar_note[kNotes], bar_noted[kNotes], bar_qfree[2], bar_s[2],
      bar_p[2][2], bar_turn[2], bar_o[2], bar_x[2], bar_y[2], bar_drain[2];
  __shared__ float2 s_ml[kRows];  // a row's maximum and sum, group 1's and then group 0's
  __shared__ Fills s_fills[TMA_WARPS];
  __shared__ Note s_note[kNotes];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_sizes[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + 2 * W::kTileBytes;
  const float kNegInf = __int_as_float(0xff800000);

  if (warp == 0) tc::tmem_alloc(&s_tmem, 512);
  if (tid == kMmaWarp * 32) {
    for (int i = 0; i < W::kSlotsN; ++i) {
      tc::mbar_init(&bar_tma[i], TMA_WARPS);
      tc::mbar_init(&bar_cp[i], kQWarp - kLoadWarp);
      tc::mbar_init(&bar_go[i], 1);
      tc::mbar_init(&bar_free[i], 2);
    }
    for (int i = 0; i < kNotes; ++i) {
      tc::mbar_init(&bar_note[i], 2);
      tc::mbar_init(&bar_noted[i], kLoadWarp);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar_qfree[i], 2);
      tc::mbar_init(&bar_s[i], 1);
      tc::mbar_init(&bar_p[i][0], 4);
      tc::mbar_init(&bar_p[i][1], 4);
      tc::mbar_init(&bar_turn[i], 1);
      tc::mbar_init(&bar_o[i], 1);
      tc::mbar_init(&bar_x[i], 4);
      tc::mbar_init(&bar_y[i], 4);
      tc::mbar_init(&bar_drain[i], 1);
    }
    tc::mbar_init_fence();
    s_abort = 0;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait(pl.hdr, pl.starts);  // the plan
  pdl_launch_dependents();

  const int cta = blockIdx.x;
  Walk walk;
  {
    const Start st = pl.starts[cta];  // (one round trip with the header)
    const int S = pl.hdr[kShare], W = pl.hdr[kWideCtas], tag = pl.hdr[kTag];
    const int64_t total = (int64_t)pl.hdr[kUnits] * sh.Hkv - (int64_t)cta * S;
    if (lane == 0) {  // (all warps write the same)
      s_sizes[0] = pl.hdr[kItems];
      s_sizes[1] = pl.hdr[kSlots];
    }
    __syncwarp();
    walk.items = pl.items;
    walk.sizes = s_sizes;
    walk.head = st.head;
    walk.item = st.item;
    walk.tile = st.tile;
    walk.turn = 0;
    walk.left = cta >= W || tag != sh.tag ? 0 : (int)min((int64_t)S, total);
  }
  bool ok = true;
  // a wait of the whole warp
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, &s_abort, wait_cycles)) != 0;
  };
  // tiles of a piece that come by TMA: those before the range's end, in pages of
  // whole boxes, from a start that keeps every box in one page
  auto tma_tiles = [&](const Piece& pc) -> int {
    if (sh.box == 0 || pc.it.t0 % sh.box != 0) return 0;
    const int full = (pc.it.t1 - pc.it.t0) / kTile - pc.t_lo;
    return full < pc.nt ? full : pc.nt;
  };

  // the next piece's note, read and released
  auto read_note = [&](uint32_t n, Note& note) -> bool {
    if (!wait(&bar_note[n % kNotes], (n / kNotes) & 1)) return false;
    note = s_note[n % kNotes];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bar_noted[n % kNotes]);
    return true;
  };

  // The end of a warp's role: whether any warp has given up.  In the normal course
  // every copy and product has been waited for by then; else those that a warp has
  // left in flight end before the memory that they write is given up.
  auto gave_up = [&]() -> bool {
    __syncwarp();
    asm volatile("bar.sync 1, %0;\n" ::"n"(kWideThreads) : "memory");
    return s_abort != 0;
  };
  auto land = [&](uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity) && clock64() - t0 < kWaitCycles) {
    }
  };

  // Every role keeps its own count of the phases.
  if (warp < kMmaWarp) {
    // ================= softmax: a thread a query row =================
    tc::setmaxnreg_inc<kSoftmaxRegs>();
    const int g = warp >> 2;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + kTmemS + g * kTile, tO = tmem + lane_off + g * 128;
    const uint64_t scale2 = tc::pack2(__float_as_uint(scale_log2), __float_as_uint(scale_log2));
    uint32_t n_job = 0, n_note = 0, n_piece = 0, n_split = 0;
    for (bool more = walk.more(); more;) {
      Note pc;
      if (!(ok = read_note(n_note++, pc))) break;
      more = !pc.last;
      const int x = (pc.pair ? g * kRows : 0) + (tid & (kRows - 1));  // row of the item
      const int64_t row = pc.slot + x;
      const bool mine = x < pc.nrows;
      const int my_jobs = g ? pc.jobs1 : pc.jobs0;
      const bool idle = !__any_sync(0xffffffffu, mine);  // no row of this warp counts
      // tokens this row sees
      int limit = pc.tok1;
      if (pc.own && sh.causal && mine) limit = pc.own - sh.Nq + (pc.row0 + x) / sh.G + 1;
      limit -= pc.tok0;
      float m_run = kNegInf, l_run = 0.f;
      for (int i = 0; i < my_jobs; ++i) {
        if (!(ok = wait(&bar_s[g], n_job & 1))) break;
        ++n_job;
        tc::fence_after();
        if (!idle) {
          const int nv = limit - (pc.pair ? i : 2 * i + (g ^ pc.turn)) * kTile;  // valid columns
          uint32_t s0[32], s1[32], s2[32], s3[32];
          tc::tmem_ld32(tS, s0);
          tc::tmem_ld32(tS + 32, s1);
          tc::tmem_ld32(tS + 64, s2);
          tc::tmem_ld32(tS + 96, s3);
          tc::tmem_ld_wait(s0);
          tc::tmem_ld_pin(s1);
          tc::tmem_ld_pin(s2);
          tc::tmem_ld_pin(s3);
          if (__any_sync(0xffffffffu, nv < kTile)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (k >= nv) s0[k] = 0xff800000u;
              if (32 + k >= nv) s1[k] = 0xff800000u;
              if (64 + k >= nv) s2[k] = 0xff800000u;
              if (96 + k >= nv) s3[k] = 0xff800000u;
            }
          }
          float mx0 = kNegInf, mx1 = kNegInf, mx2 = kNegInf, mx3 = kNegInf;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            mx0 = tc::max3(mx0, __uint_as_float(s0[k]), __uint_as_float(s0[k + 1]));
            mx1 = tc::max3(mx1, __uint_as_float(s1[k]), __uint_as_float(s1[k + 1]));
            mx2 = tc::max3(mx2, __uint_as_float(s2[k]), __uint_as_float(s2[k + 1]));
            mx3 = tc::max3(mx3, __uint_as_float(s3[k]), __uint_as_float(s3[k + 1]));
          }
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scale_log2;
          const bool move = mx > m_run + 8.f;  // also true on the first valid tile
          const float m_new = move ? mx : m_run;
          const float alpha = move ? exp2f(m_run - m_new) : 1.f;
          m_run = m_new;
          // the weights; P is rounded to bf16 for the second product (each by
          // half a step, 2^-8 of itself, at most) while the sum keeps the fp32
          // values, so that lse carries no such rounding
          const float neg = m_new == kNegInf ? 0.f : -m_new;
          const uint64_t neg2 = tc::pack2(__float_as_uint(neg), __float_as_uint(neg));
          uint64_t sum_a = 0, sum_b = 0;
          auto weights = [&](uint32_t (&sv)[32], uint32_t* pk) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              float a0, a1, b0, b1;
              tc::unpack2(tc::fma2(tc::pack2(sv[k], sv[k + 1]), scale2, neg2), a0, a1);
              tc::unpack2(tc::fma2(tc::pack2(sv[k + 2], sv[k + 3]), scale2, neg2), b0, b1);
              a0 = ex2(a0);
              a1 = ex2(a1);
              b0 = ex2(b0);
              b1 = ex2(b1);
              sum_a = tc::add2(sum_a, tc::pack2(__float_as_uint(a0), __float_as_uint(a1)));
              sum_b = tc::add2(sum_b, tc::pack2(__float_as_uint(b0), __float_as_uint(b1)));
              const __nv_bfloat162 pa = __floats2bfloat162_rn(a0, a1);
              const __nv_bfloat162 pb = __floats2bfloat162_rn(b0, b1);
              pk[k / 2] = *reinterpret_cast<const uint32_t*>(&pa);
              pk[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&pb);
            }
          };
          // O of the jobs before is complete: S of this job was issued after it
          if (__any_sync(0xffffffffu, move && i > 0)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t ov[16];
              tc::tmem_ld16(tO + c, ov);
#pragma unroll
              for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
              tc::tmem_st16(tO + c, ov);
            }
          }
          // P takes the place of S columns, all of which are in registers
          uint32_t pk[16];
          weights(s0, pk);
          tc::tmem_st16(tS, pk);
          weights(s1, pk);
          tc::tmem_st16(tS + 16, pk);
          tc::tmem_st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar_p[g][0]);
          weights(s2, pk);
          tc::tmem_st16(tS + 32, pk);
          weights(s3, pk);
          tc::tmem_st16(tS + 48, pk);
          float la, lb, lc, ld;
          tc::unpack2(sum_a, la, lb);
          tc::unpack2(sum_b, lc, ld);
          l_run = l_run * alpha + ((la + lb) + (lc + ld));
          tc::tmem_st_wait();
        } else {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar_p[g][0]);
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar_p[g][1]);
      }
      // ---- the piece's partial
      if (!ok) break;
      if (my_jobs == 0) continue;  // (one tile: it was the other group's)
      if (!(ok = wait(&bar_o[g], n_piece & 1))) break;
      ++n_piece;
      tc::fence_after();
      float* dst = part_o + row * D;
      if (pc.pair || pc.nt == 1) {
        if (mine) part_ml[row] = make_float2(m_run, l_run);
        if (!idle) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tc::tmem_ld32(tO + c, ov);
            tc::tmem_ld_wait(ov);
            if (mine) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(ov[k + e]);
                store8(dst + c + k, v);
              }
            }
          }
        }
        tc::fence_before();  // the reads of O come before the P that lets it be overwritten
        continue;
      }
      // both groups hold the same rows: they exchange maxima and sums, and each
      // combines half of the columns (its warps read the other group's O, which
      // lies in the same lanes of the tensor memory)
      const int xr = tid & (kRows - 1);
      float2 e0 = make_float2(m_run, l_run), e1 = e0;
      if (g == 0) {
        if (!(ok = wait(&bar_x[1], n_split & 1))) break;
        e1 = s_ml[xr];
        s_ml[xr] = e0;
      } else {
        s_ml[xr] = e1;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_x[g]);
      if (g == 1) {
        if (!(ok = wait(&bar_x[0], n_split & 1))) break;
        e0 = s_ml[xr];
      }
      tc::fence_after();
      if (!idle) {
        const float M = e0.y == 0.f ? e1.x : e1.y == 0.f ? e0.x : fmaxf(e0.x, e1.x);
        const float w0 = e0.y == 0.f ? 0.f : exp2f(e0.x - M);
        const float w1 = e1.y == 0.f ? 0.f : exp2f(e1.x - M);
        if (mine && g == 0) part_ml[row] = make_float2(M, e0.y * w0 + e1.y * w1);
        const uint32_t tA = tmem + lane_off, tB = tA + 128;
#pragma unroll 1
        for (int c = g * (D / 2); c < (g + 1) * (D / 2); c += 32) {
          uint32_t a[32], b[32];
          tc::tmem_ld32(tA + c, a);
          tc::tmem_ld32(tB + c, b);
          tc::tmem_ld_wait(a);
          tc::tmem_ld_pin(b);
          if (mine) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                // (a part without tokens may hold 0 times infinity)
                const float va = w0 == 0.f ? 0.f : w0 * __uint_as_float(a[k + e]);
                const float vb = w1 == 0.f ? 0.f : w1 * __uint_as_float(b[k + e]);
                v[e] = va + vb;
              }
              store8(dst + c + k, v);
            }
          }
        }
      }
      // neither group goes on before the other has read its O and maxima
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_y[g]);
      if (!(ok = wait(&bar_y[1 - g], n_split & 1))) break;
      ++n_split;
    }
    if (!ok && lane == 0) {
      flag_error(pl.hdr + kErrWord, kErrTimeout);
      s_abort = 1;
    }
    gave_up();
  } else {
    tc::setmaxnreg_dec<kOtherRegs>();
    if (warp < kLoadWarp) {
      // ================= MMA issue of one group =================
      const int g = warp - kMmaWarp;
      const uint32_t tS = tmem + kTmemS + g * kTile, tO = tmem + g * 128;
      uint32_t n_slot = 0, n_job = 0, n_note = 0, n_turn = 0, ph_tma = 0, ph_cp = 0;
      bool issued = false;  // any product (every one comes behind an S)
      for (bool more_pieces = walk.more(); more_pieces && ok;) {
        Note pc;
        if (!(ok = read_note(n_note++, pc))) break;
        more_pieces = !pc.last;
        const int by_tma = pc.by_tma;
        const int my_jobs = g ? pc.jobs1 : pc.jobs0;
        const int q_block = pc.pair ? (pc.q_block + g) & 1 : pc.q_block;
        // a Q block that this issuer has no product with
        if ((pc.pair || my_jobs == 0) && tc::elect_one())
          tc::mbar_arrive(&bar_qfree[pc.pair ? q_block ^ 1 : q_block]);
        __syncwarp();
        // K of tile t has landed already (no wait, no phase taken)
        auto ready = [&](int t, int tma) -> bool {
          const uint32_t sl = (n_slot + 2 * t) % W::kSlotsN;
          const bool r = t < tma ? tc::mbar_test_wait(&bar_tma[sl], (ph_tma >> sl) & 1)
                                 : tc::mbar_test_wait(&bar_cp[sl], (ph_cp >> sl) & 1);
          return __all_sync(0xffffffffu, r) != 0;
        };
        // a tile's K (v = 0) or V has landed
        auto landed = [&](int t, int v) -> bool {
          const uint32_t sl = (n_slot + 2 * t + v) % W::kSlotsN;
          const bool tma = t < by_tma;
          const bool r = wait(tma ? &bar_tma[sl] : &bar_cp[sl],
                              ((tma ? ph_tma : ph_cp) >> sl) & 1);
          ph_tma ^= (uint32_t)tma << sl;
          ph_cp ^= (uint32_t)!tma << sl;
          return r;
        };
        // (the turn passes with four of S's steps to go: the other issuer's first
        // product then queues behind them without a gap)
        auto issue_s = [&](int t, bool last, uint64_t* pass) {
          issued = true;
          tc::fence_after();
          if (tc::elect_one()) {
            const uint32_t sl = (n_slot + 2 * t) % W::kSlotsN;
            const uint64_t dq = tc::desc_sw128(sQ + q_block * W::kTileBytes, 16, W::kGroupBytes);
            const uint64_t dk = tc::desc_sw128(sKV + sl * W::kTileBytes, 16, W::kGroupBytes);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
              tc::mma_ss(tS, dq + off, dk + off, tc::idesc_bf16(kRows, kTile, false),
                         kk > 0 ? 1u : 0u);
              if (kk == D / 16 - 4 && pass) tc::mbar_arrive(pass);
            }
            tc::mma_commit(&bar_s[g]);
            tc::mma_commit(&bar_free[sl]);
            if (last) tc::mma_commit(&bar_qfree[q_block]);
          }
          __syncwarp();
        };
        // the other group's tile: waited for and released like an own one, so that
        // no barrier completes two phases between two waits of a warp
        auto skip = [&](int t) -> bool {
          for (int v = 0; v < 2; ++v) {
            if (!landed(t, v)) return false;
            if (tc::elect_one()) tc::mbar_arrive(&bar_free[(n_slot + 2 * t + v) % W::kSlotsN]);
            __syncwarp();
          }
          return true;
        };
        const int step = pc.pair ? 1 : 2, t0 = pc.pair ? 0 : g ^ pc.turn;
        if (my_jobs > 0) {
          if (t0 == 1) ok = skip(0);
          if (ok && (ok = landed(t0, 0))) issue_s(t0, my_jobs == 1, nullptr);
        } else {  // the one tile is the other group's
          ok = skip(0);
        }
        for (int i = 0; i < my_jobs && ok; ++i, ++n_job) {
          const int t = t0 + i * step;
          if (!(ok = landed(t, 1))) break;
          const uint32_t sl = (n_slot + 2 * t + 1) % W::kSlotsN;
          const uint64_t dv = tc::desc_sw128(sKV + sl * W::kTileBytes, 1024, W::kGroupBytes);
          // K of the next tile, if it is there: S then follows P.V without a wait
          const bool more = i + 1 < my_jobs;
          const int tn = t + step;
          const bool early = more && step == 1 && ready(tn, by_tma);
          if (early && !(ok = landed(tn, 0))) break;
          // after the other group's products of the job before: the groups take
          // turns through all pieces, group 0 begins
          if (g == 1 || n_job > 0) {
            if (!(ok = wait(&bar_turn[g], n_turn & 1))) break;
            ++n_turn;
          }
          if (!(ok = wait(&bar_p[g][0], n_job & 1))) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !(ok = wait(&bar_p[g][1], n_job & 1))) break;
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                tc::mma_ts(tO, tS + kk * 8, dv + (uint64_t)((kk * 2 * W::kGroupBytes) >> 4),
                           tc::idesc_bf16(kRows, D, true), (i > 0 || kk > 0) ? 1u : 0u);
              if (h == 1) {
                tc::mma_commit(&bar_free[sl]);
                if (i == my_jobs - 1) tc::mma_commit(&bar_o[g]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          // then the next S, and the turn: before S when that has to wait for K
          if (early) {
            issue_s(tn, i + 2 == my_jobs, &bar_turn[1 - g]);
          } else {
            if (tc::elect_one()) tc::mbar_arrive(&bar_turn[1 - g]);
            __syncwarp();
            if (more) {
              if (step == 2) ok = skip(t + 1);
              if (!ok || !(ok = landed(tn, 0))) break;
              issue_s(tn, i + 2 == my_jobs, nullptr);
            }
          }
        }
        // tiles behind the group's last one
        if (ok && my_jobs > 0 && t0 + my_jobs * step - step + 1 < pc.nt)
          ok = skip(pc.nt - 1);
        n_slot += 2 * pc.nt;
      }
      if (!ok && tc::elect_one()) {
        flag_error(pl.hdr + kErrWord, kErrTimeout);
        s_abort = 1;
      }
      if (gave_up() && issued && tc::elect_one()) {
        tc::mma_commit(&bar_drain[g]);
        land(&bar_drain[g], 0);
      }
      __syncwarp();
    } else {
      // ================= loads =================
      const int lw = warp - kLoadWarp;
      constexpr int kChunks = D / 8;          // 16-byte chunks of a row
      constexpr int kRowsPer = 32 / kChunks;  // rows a warp instruction covers
      const int sub = lane / kChunks, cc = lane % kChunks;
      // warp lw fills rows 32 lw .. 32 lw + 31, this lane rows r + sub; chunk c of
      // row r of a 64-value block goes to chunk c ^ (r & 7)
      auto dst_of = [&](uint32_t tile, int r) {
        const int r8 = (r & 7) + sub;
        return tile + (r >> 3) * W::kGroupBytes + (cc >> 3) * 1024 + r8 * 128 +
               (((cc & 7) ^ r8) << 4);
      };
      auto publish = [&](uint64_t* bar) {
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
      };
      if (warp >= kQWarp) {
        // ---- Q blocks, 32 rows of a block and the next 32 by turns, and the notes
        const int qw = warp - kQWarp;
        uint32_t n_note = 0, n_block = 0, uses0 = 0, uses1 = 0;
        while (walk.more() && ok) {
          const Piece pc = walk.next();
          const uint32_t nn = n_note % kNotes;
          if (n_note >= (uint32_t)kNotes &&
              !(ok = wait(&bar_noted[nn], (n_note / kNotes - 1) & 1)))
            break;
          const int q_block = n_block & 1;
          // room: the blocks' products before are done
          if ((pc.pair || q_block == 0) && uses0 > 0 &&
              !(ok = wait(&bar_qfree[0], (uses0 - 1) & 1)))
            break;
          if ((pc.pair || q_block == 1) && uses1 > 0 &&
              !(ok = wait(&bar_qfree[1], (uses1 - 1) & 1)))
            break;
          uses0 += pc.pair || q_block == 0;
          uses1 += pc.pair || q_block == 1;
          n_block += pc.pair ? 2 : 1;
#pragma unroll 1
          for (int c = qw; c < (pc.pair ? 8 : 4); c += 2) {
            // query row of this lane: request, query token and head
            const int x = c * 32 + lane;
            int64_t off = -1;
            if (x < pc.it.nrows) {
              const int gr = pc.it.row0 + x;
              const int b = pc.it.own ? pc.it.bt_row : pl.order[gr / sh.R];
              const int r = pc.it.own ? gr : gr % sh.R;
              off = (((int64_t)b * sh.Nq + r / sh.G) * sh.Hq + pc.head * sh.G + r % sh.G) * D;
            }
            const uint32_t tile = sQ + ((q_block + (c >> 2)) & 1) * W::kTileBytes;
#pragma unroll 4
            for (int i = 0; i < 32; i += kRowsPer) {
              const int64_t o = __shfl_sync(0xffffffffu, off, i + sub);
              tc::cp_async16(dst_of(tile, (c & 3) * 32 + i), q + (o >= 0 ? o + cc * 8 : 0),
                             o >= 0 ? 16 : 0);
            }
          }
          tc::cp_async_commit();
          if (qw == 0 && lane == 0) {
            Note note;
            note.nt = pc.nt;
            note.by_tma = tma_tiles(pc);
            note.jobs0 = pc.jobs0;
            note.jobs1 = pc.jobs1;
            note.nrows = pc.it.nrows;
            note.row0 = pc.it.row0;
            note.own = pc.it.own;
            note.tok0 = pc.it.t0 + pc.t_lo * kTile;
            note.tok1 = pc.it.t1;
            note.q_block = q_block;
            note.pair = pc.pair;
            note.turn = pc.turn;
            note.last = !walk.more();
            note.slot = pc.slot;
            s_note[nn] = note;
          }
          tc::cp_async_wait<0>();
          publish(&bar_note[nn]);
          ++n_note;
        }
        if (!ok && lane == 0) {
          flag_error(pl.hdr + kErrWord, kErrTimeout);
          s_abort = 1;
        }
        tc::cp_async_wait<0>();
        gave_up();
      } else {
        // first row of this lane's box of an item's tile, when it comes by TMA (a bad
        // page gives zeros, from beyond the pool)
        const int n_box = sh.box && lw < TMA_WARPS ? kTile / sh.box / TMA_WARPS : 0;
        const int my_box = lw * n_box + lane;
        auto box_row = [&](const Item& it, int tile) -> int {
          if (lane >= n_box || it.t0 % sh.box != 0 || it.t0 + (tile + 1) * kTile > it.t1) return 0;
          const int tok = it.t0 + tile * kTile + my_box * sh.box;
          const int page = block_table[(int64_t)it.bt_row * sh.max_pages + tok / sh.page_size];
          if ((unsigned)page >= (unsigned)sh.num_pages) {
            flag_error(pl.hdr + kErrWord, kErrPage);
            return sh.num_pages * sh.page_size;
          }
          return page * sh.page_size + tok % sh.page_size;
        };
        uint32_t n_slot = 0;
        uint32_t ph_go = 0;
        Fills fills = {};  // (its number of half tiles: n_slot, until the end)
        int row = 0;
        if (walk.more()) {
          const Item first = pl.starts[cta].it;
          row = box_row(first, walk.tile);
        }
        while (walk.more() && ok) {
          const Piece pc = walk.next();
          Item then = {};  // the next piece's item, for its first row
          if (walk.more()) then = walk.items[walk.item];
          const int32_t* bt = block_table + (int64_t)pc.it.bt_row * sh.max_pages;
          // physical row of this lane's token of tile t (-1: none)
          auto token_row = [&](int t) -> int {
            const int tok = pc.it.t0 + (pc.t_lo + t) * kTile + lw * 32 + lane;
            if (tok >= pc.it.t1) return -1;
            const int page = bt[tok / sh.page_size];
            if ((unsigned)page >= (unsigned)sh.num_pages) {
              flag_error(pl.hdr + kErrWord, kErrPage);
              return -1;
            }
            return page * sh.page_size + tok % sh.page_size;
          };
          const int by_tma = tma_tiles(pc);
          int waiting = 0;  // tiles copied by cp.async and not published yet
          int done = 0;
          for (int t = 0; t < pc.nt && ok; ++t) {
            if (t >= by_tma) row = token_row(t);
            // the row of the tile after this one, in the next piece if need be
            int next_row = 0;
            if (t + 1 < pc.nt || walk.more())
              next_row = t + 1 < pc.nt ? box_row(pc.it, pc.t_lo + t + 1) : box_row(then, 0);
#pragma unroll
            for (int v = 0; v < 2; ++v, ++done) {
              const uint32_t n = n_slot + done, s = n % W::kSlotsN;
              // a warp that takes part in every fill waits for room; the others copy
              // only where warp 0 has let them
              if (lw < TMA_WARPS) {
                if (n >= (uint32_t)W::kSlotsN &&
                    !(ok = wait(&bar_free[s], (n / W::kSlotsN - 1) & 1)))
                  break;
                if (TMA_WARPS < kLoadWarps && t >= by_tma && lane == 0) tc::mbar_arrive(&bar_go[s]);
              } else if (t >= by_tma) {
                if (!(ok = wait(&bar_go[s], (ph_go >> s) & 1))) break;
                ph_go ^= 1u << s;
              }
              const uint32_t tile = sKV + s * W::kTileBytes;
              if (t < by_tma) {
                if (lw >= TMA_WARPS) continue;
                fills.by_tma |= 1u << s;
                fills.used |= 1u << s;
                fills.count ^= 1u << s;
                if (lane == 0) tc::mbar_arrive_expect(&bar_tma[s], W::kTileBytes / TMA_WARPS);
                __syncwarp();
                if (lane < n_box)
                  tc::tma_load_5d(tile + my_box * (sh.box / 8) * W::kGroupBytes,
                                  v ? &map_v : &map_k, 0, 0, 0, row / 8, pc.head, &bar_tma[s]);
              } else {
                fills.by_tma &= ~(1u << s);
                const __nv_bfloat16* pool = (v ? kv_v : kv_k) + pc.head * D + cc * 8;
#pragma unroll 8
                for (int r = 0; r < 32; r += kRowsPer) {
                  const int pr = __shfl_sync(0xffffffffu, row, r + sub);
                  tc::cp_async16(dst_of(tile, lw * 32 + r),
                                 pool + (pr >= 0 ? (int64_t)pr * sh.Hkv * D : 0), pr >= 0 ? 16 : 0);
                }
                tc::cp_async_commit();
                ++waiting;
              }
              if (waiting > W::kLag) {
                tc::cp_async_wait<W::kLag>();
                publish(&bar_cp[(n - W::kLag) % W::kSlotsN]);
                --waiting;
              }
            }
            row = next_row;
          }
          tc::cp_async_wait<0>();
          for (; waiting; --waiting) publish(&bar_cp[(n_slot + done - waiting) % W::kSlotsN]);
          n_slot += done;
        }
        if (!ok && lane == 0) {
          flag_error(pl.hdr + kErrWord, kErrTimeout);
          s_abort = 1;
        }
        if (gave_up() && lw < TMA_WARPS) {
          // A slot's barrier counts an arrival of every warp: what the furthest has
          // filled and this one has not (once around the ring at most, as a slot is
          // filled again only behind products with its last contents) gets this
          // warp's arrival without any copy.
          fills.n = n_slot;
          if (lane == 0) s_fills[lw] = fills;
          asm volatile("bar.sync 2, %0;\n" ::"n"(TMA_WARPS * 32) : "memory");
#pragma unroll
          for (int w = 0; w < TMA_WARPS; ++w)
            if (s_fills[w].n > fills.n) fills = s_fills[w];
          for (uint32_t n = n_slot; n < fills.n; ++n)
            if (lane == 0 && ((fills.by_tma >> (n % W::kSlotsN)) & 1))
              tc::mbar_arrive(&bar_tma[n % W::kSlotsN]);
          for (int i = 0; i < W::kSlotsN; ++i)
            if ((fills.used >> i) & 1) land(&bar_tma[i], (~fills.count >> i) & 1);
        }
        __syncwarp();
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- narrow ---
// Own tokens of requests with at most 16 rows a KV head, streamed: a CTA takes
// 16-token tiles of K and V rows of its HG heads through a ring in shared memory.
// A warp has one KV head and up to eight rows (two warps a head for more, on the
// same tiles); both products run transposed on mma.sync (tokens, then head
// dimension, as M; the rows as N), so no MMA carries padding rows.  The work is a
// few FLOP a byte and memory is what bounds it, as long as the work between a
// tile's arrival and its release is short: so a warp of its own finds the tiles'
// rows and fills the ring, by TMA where 16 tokens lie in whole 8-row boxes of
// pages, else row by row with cp.async, which fills what is missing with zeros.
// A ring stage holds K, then V, each as [64-value block][8 tokens of 16][head]
// [token][128 bytes, swizzled].

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int D, int HG>
struct Narrow {
  static constexpr int kBlk = D / 64;
  static constexpr uint32_t kBoxBytes = HG * 8 * 128;          // 64 values of 8 tokens, all heads
  static constexpr uint32_t kHalfBytes = kBlk * 2 * kBoxBytes;  // K or V of a tile
  static constexpr uint32_t kTileBytes = 2 * kHalfBytes;
  static constexpr int kPerSm = HG >= 8 ? 1 : HG == 4 ? 2 : 4;  // CTAs an SM
  static constexpr int kFit = (int)(192 * 1024 / kPerSm / kTileBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr size_t smem(int B) {
    return kStages * (size_t)kTileBytes + 1024 + sizeof(int32_t) * (size_t)(B + 1);
  }
};
constexpr int kTileRing = 8;  // descriptions of tiles, more than stages

template <int D, int HG, int WPH>
__global__ void __launch_bounds__((HG * WPH + 1) * 32, Narrow<D, HG>::kPerSm)
k_prefix_narrow(const int32_t* __restrict__ block_table, const __nv_bfloat16* __restrict__ q,
                const __nv_bfloat16* __restrict__ kv_k, const __nv_bfloat16* __restrict__ kv_v,
                PlanPtrs pl, float2* __restrict__ part_ml, float* __restrict__ part_o,
                PrefixShape sh, float scale_log2, int wait_first, long long wait_cycles,
                const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  using N = Narrow<D, HG>;
  constexpr int NT = (HG * WPH + 1) * 32, KS = D / 16, MT = D / 16, TILE = kNarrowTile;
  static_assert(N::kStages < kTileRing, "a description outlives its stage");
  const float kNegInf = __int_as_float(0xff800000);
  extern __shared__ uint8_t smem_raw[];
  // a tile: tokens from own position p0 of request b (own: all of them) for the
  // heads of group g, in a piece; mask: its tokens; kFirst / kLast of its request
  // in the piece, kEnd: no more tiles
  struct Tile {
    int b, g, p0, own, piece, flags;
    uint32_t mask;
    int pad;
  };
  constexpr int kFirst = 1, kLast = 2, kEnd = 4;
  __shared__ Tile s_tile[kTileRing];
  // bar_full: the producer's 32 lanes and its one announcement; bar_empty: the
  // consumer warps
  __shared__ __align__(8) uint64_t bar_full[N::kStages], bar_empty[N::kStages];
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  // [B + 1] narrow tiles before each request
  int32_t* s_pre = reinterpret_cast<int32_t*>(smem_raw + (base - tc::smem_u32(smem_raw)) +
                                              N::kStages * (size_t)N::kTileBytes);
  const int B = sh.B, ngroups = sh.Hkv / HG;
  if (tid == 0) {
    for (int i = 0; i < N::kStages; ++i) {
      tc::mbar_init(&bar_full[i], 33);
      tc::mbar_init(&bar_empty[i], HG * WPH);
    }
    tc::mbar_init_fence();
    s_abort = 0;
  }
  // Behind the wide kernel this grid runs beside that one and waits for it only at
  // its end.  In place of a wait it relies on what it reads having been complete
  // before it could start: every CTA of the wide kernel waited for the plan, and so
  // for everything before the plan, before it let this grid start.  What the SM's L1
  // may hold from before goes with a fence; the plan's numbers are read from L2, and
  // table and queries through pointers that are named here (no non-coherent loads).
  if (wait_first) pdl_wait();
  else if (warp == HG * WPH) __threadfence();  // (for all, by the barrier below)
  behind(block_table, q, pl.hdr, pl.npre);
  pdl_launch_dependents();
  const Pieces pieces(pl.hdr, ngroups);
  const int Treq = __ldcg(pl.hdr + kTiles);
  const int cta = blockIdx.x;
  for (int i = tid; i <= B; i += NT) s_pre[i] = __ldcg(pl.npre + i);
  if (pieces.tag != sh.tag || (cta >= pieces.big && pieces.n == pieces.big)) {
    if (!wait_first) pdl_wait();
    return;
  }
  __syncthreads();
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, &s_abort, wait_cycles)) != 0;
  };

  uint32_t n_fills = 0;  // the producer's
  if (warp == HG * WPH) {
    // ================= producer: the tiles in order =================
    int piece = -1, claimed = 0;
    int64_t f = 0, f_end = 0, seg_end = 0;  // next tile, end of the piece and of the request
    int cb = 0, cg = 0, cstart = 0, clen = 0;
    bool opened = false;
    auto request = [&]() {
      seg_end = (int64_t)cg * Treq + s_pre[cb + 1];
      cstart = pl.start[cb];
      clen = pl.lens[cb] - cstart;
    };
    auto claim = [&]() {  // (used a piece later, so that its latency is hidden)
      if (lane == 0) claimed = pieces.big + atomicAdd(pl.hdr + kClaim, 1);
    };
    auto open_piece = [&](int p) {
      piece = p;
      if (p >= pieces.n) return;
      f = pieces.lo(p);
      f_end = pieces.lo(p + 1);
      cg = 0;
      int64_t rest = f;
      while (rest >= Treq) {
        rest -= Treq;
        ++cg;
      }
      const int fb = (int)rest;
      int l = 0, h = B - 1;
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (s_pre[mid] <= fb) l = mid; else h = mid - 1;
      }
      cb = l;
      request();
      opened = true;
      claim();
    };
    // the next tile: its description, and its lane's (token's) page, still to
    // come, with the row in it (-1: no token)
    auto describe = [&](Tile& t, int& page, int& in_page) {
      t = Tile{};
      t.flags = kEnd;
      page = in_page = -1;
      if (piece < pieces.n && f == f_end) open_piece(__shfl_sync(0xffffffffu, claimed, 0));
      if (piece >= pieces.n) return;
      while (f == seg_end) {  // the next request with tiles
        if (++cb == B) {
          cb = 0;
          ++cg;
        }
        request();
        opened = true;
      }
      t.b = cb;
      t.g = cg;
      t.p0 = (int)(f - ((int64_t)cg * Treq + s_pre[cb])) * TILE;
      t.own = clen;
      t.piece = piece;
      t.flags = (opened ? kFirst : 0) | (f + 1 == seg_end || f + 1 == f_end ? kLast : 0);
      opened = false;
      const int n = clen - t.p0;
      if (lane < n && lane < TILE) {
        const int tok = cstart + t.p0 + lane;
        page = block_table[(int64_t)cb * sh.max_pages + tok / sh.page_size];
        in_page = tok % sh.page_size;
      }
      ++f;
    };
    if (cta < pieces.big) {
      open_piece(cta);
    } else {
      claim();
      open_piece(__shfl_sync(0xffffffffu, claimed, 0));
    }
    // two tiles described ahead: their table entries are on the way
    Tile t0, t1, t2;
    int pg0, pg1, pg2, ip0, ip1, ip2;
    describe(t0, pg0, ip0);
    describe(t1, pg1, ip1);
    uint32_t k = 0;
    for (;; ++k) {
      describe(t2, pg2, ip2);
      const uint32_t s = k % N::kStages;
      if (k >= (uint32_t)N::kStages && !(ok = wait(&bar_empty[s], (k / N::kStages - 1) & 1))) break;
      int row = -1;
      if (ip0 >= 0) {
        if ((unsigned)pg0 < (unsigned)sh.num_pages) row = pg0 * sh.page_size + ip0;
        else flag_error(pl.hdr + kErrWord, kErrPage);
      }
      t0.mask = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) s_tile[k % kTileRing] = t0;
      const uint32_t tile = base + s * N::kTileBytes;
      if (t0.flags & kEnd) {
        tc::mbar_arrive(&bar_full[s]);
        if (lane == 0) tc::mbar_arrive(&bar_full[s]);
        ++k;
        break;
      }
      // whole boxes: all 16 tokens, in steps of eight from a box's first row
      const bool whole = sh.box > 0 && t0.mask == 0xffffu &&
                         __shfl_sync(0xffffffffu, ip0, 0) % 8 == 0;
      if (whole) {
        if (lane == 0) tc::mbar_arrive_expect(&bar_full[s], N::kTileBytes);
        __syncwarp();
        // lane 4 v + 2 j + h: K or V, block j, half h of the tokens
        const int v = lane >> 2, j = (lane >> 1) & 1, h = lane & 1;
        const int pr = __shfl_sync(0xffffffffu, row, (h * 8) & 31);
        if (v < 2 && j < N::kBlk)
          tc::tma_load_3d(tile + v * N::kHalfBytes + (j * 2 + h) * N::kBoxBytes,
                          v ? &map_v : &map_k, j * 64, pr, t0.g * HG, &bar_full[s]);
        tc::mbar_arrive(&bar_full[s]);
      } else {
        // a lane's 16-byte chunk c of the rows of every kStep-th head, from h0, of
        // every kTok-th token, from r0
        constexpr int kChunks = D / 8, kPer = HG * kChunks;
        constexpr int kTok = kPer < 32 ? 32 / kPer : 1, kStep = 32 / kChunks;
        const int c = lane % kChunks, h0 = lane / kChunks % HG, r0 = kPer < 32 ? lane / kPer : 0;
        const uint32_t dst0 = tile + (c >> 3) * 2 * N::kBoxBytes + h0 * 1024;
        const int64_t src0 = (t0.g * HG + h0) * D + c * 8, row_step = (int64_t)sh.Hkv * D;
#pragma unroll 8
        for (int i = 0; i < TILE; i += kTok) {
          const int r = i + r0, pr = __shfl_sync(0xffffffffu, row, r);
          const uint32_t dst = dst0 + (r >> 3) * N::kBoxBytes + (r & 7) * 128 +
                               (((c & 7) ^ (r & 7)) << 4);
          const int64_t src = src0 + (pr >= 0 ? pr * row_step : 0);
#pragma unroll
          for (int h = 0; h < HG; h += kStep) {
            tc::cp_async16(dst + h * 1024, kv_k + src + h * D, pr >= 0 ? 16 : 0);
            tc::cp_async16(dst + h * 1024 + N::kHalfBytes, kv_v + src + h * D, pr >= 0 ? 16 : 0);
          }
        }
        tc::cp_async_arrive(&bar_full[s]);
        if (lane == 0) tc::mbar_arrive(&bar_full[s]);
      }
      t0 = t1;
      pg0 = pg1;
      ip0 = ip1;
      t1 = t2;
      pg1 = pg2;
      ip1 = ip2;
    }
    if (!ok && lane == 0) {
      flag_error(pl.hdr + kErrWord, kErrTimeout);
      s_abort = 1;
    }
    tc::cp_async_wait<0>();
    n_fills = k;
    __syncwarp();
  } else {
    // ================= consumers =================
    const int hh = warp % HG, c0 = (warp / HG) * 8;  // KV head of the group, first row
    const int g8 = lane >> 2, t4 = lane & 3;
    uint32_t qb[KS][2];
    float o[MT][4], m_h[2] = {kNegInf, kNegInf}, l_h[2] = {0.f, 0.f};
    int lim[2] = {0, 0};  // own tokens that the thread's two rows see
    for (uint32_t k = 0;; ++k) {
      const uint32_t s = k % N::kStages;
      if (!(ok = wait(&bar_full[s], (k / N::kStages) & 1))) break;
      const Tile t = s_tile[k % kTileRing];
      if (t.flags & kEnd) break;
      if (t.flags & kFirst) {
        const int head = t.g * HG + hh, j = c0 + g8;
        const __nv_bfloat16* src =
            q + (((int64_t)t.b * sh.Nq + j / sh.G) * sh.Hq + (int64_t)head * sh.G + j % sh.G) * D +
            t4 * 2;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qb[ks][0] = j < sh.R ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
          qb[ks][1] = j < sh.R ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m_h[e] = kNegInf;
          l_h[e] = 0.f;
          lim[e] = sh.causal ? t.own - sh.Nq + (c0 + 2 * t4 + e) / sh.G + 1 : t.own;
        }
      }
      const uint32_t sk = base + s * N::kTileBytes + hh * 1024, sv = sk + N::kHalfBytes;
      float sacc[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c) sacc[c][0] = sacc[c][1] = sacc[c][2] = sacc[c][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int r = lane & 7, h = (lane >> 3) & 1, c = 2 * ks + (lane >> 4);
        uint32_t a[4];
        ldsm_x4(sk + ((c >> 3) * 2 + h) * N::kBoxBytes + r * 128 + (((c & 7) ^ r) << 4), a);
        mma_16816(sacc[ks & 1], a, qb[ks][0], qb[ks][1]);
      }
      const bool v0 = (t.mask >> g8) & 1, v1 = (t.mask >> (g8 + 8)) & 1;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool v = (i < 2 ? v0 : v1) && t.p0 + g8 + (i < 2 ? 0 : 8) < lim[i & 1];
        x[i] = v ? (sacc[0][i] + sacc[1][i]) * scale_log2 : kNegInf;
      }
      float al[2], p[4];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(x[e], x[e + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        // the running maximum moves when the tile exceeds it by more than 8
        const bool mv = mx > m_h[e] + 8.f;
        const float mn = mv ? mx : m_h[e];
        al[e] = mv ? exp2f(m_h[e] - mn) : 1.f;
        moved |= mv;
        p[e] = x[e] == kNegInf ? 0.f : ex2(x[e] - mn);
        p[e + 2] = x[e + 2] == kNegInf ? 0.f : ex2(x[e + 2] - mn);
        l_h[e] = l_h[e] * al[e] + (p[e] + p[e + 2]);
        m_h[e] = mn;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          o[mt][0] *= al[0];
          o[mt][1] *= al[1];
          o[mt][2] *= al[0];
          o[mt][3] *= al[1];
        }
      }
      // rounded to bf16 for the second product only
      const uint32_t pb0 = movmatrix_t(pack_bf16(p[0], p[1]));
      const uint32_t pb1 = movmatrix_t(pack_bf16(p[2], p[3]));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = lane & 7, h = lane >> 4, c = 2 * mt + ((lane >> 3) & 1);
        uint32_t a[4];
        ldsm_x4_t(sv + ((c >> 3) * 2 + h) * N::kBoxBytes + r * 128 + (((c & 7) ^ r) << 4), a);
        mma_16816(o[mt], a, pb0, pb1);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_empty[s]);
      if (t.flags & kLast) {
        const int64_t at = (((int64_t)t.piece + (int64_t)t.g * B + t.b) * HG + hh) * sh.R;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = l_h[e];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int j = c0 + 2 * t4 + e;
          if (j >= sh.R) continue;
          float* po = part_o + (at + j) * D;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            po[mt * 16 + g8] = o[mt][e];
            po[mt * 16 + g8 + 8] = o[mt][e + 2];
          }
          if (g8 == 0) part_ml[at + j] = make_float2(m_h[e], l);
        }
      }
    }
    if (!ok && lane == 0) {
      flag_error(pl.hdr + kErrWord, kErrTimeout);
      s_abort = 1;
    }
  }
  __syncthreads();
  // In the normal course every copy has been waited for by now.  When a consumer gave
  // up, the last fill of any stage may still be on its way: it lands before the
  // shared memory is given up.
  if (s_abort && warp == HG * WPH) {
    const long long t0 = clock64();
    for (uint32_t n = n_fills > (uint32_t)N::kStages ? n_fills - N::kStages : 0; n < n_fills; ++n)
      while (!tc::mbar_try_wait(&bar_full[n % N::kStages], (n / N::kStages) & 1) &&
             clock64() - t0 < kWaitCycles) {
      }
  }
  if (!wait_first) pdl_wait();
}

// ----------------------------------------------------------------- merge ---
// LPR lanes a (request, query token, head).  The parts: the group's prefix items
// and the request's own (each cut of a token range lies in the ranges of one or
// two CTAs), or the narrow CTAs that its own tokens are spread over.  A few loads
// that wait for one another and little else, so few rows take a warp each, which
// has all parts in flight at once, and many take eight lanes, where finding the
// parts is shared by four rows.  Very few rows, which may have hundreds of parts
// each, take a block each.  Measured (a whole pass, us, by a warp / by eight
// lanes): 88,320 rows of one or two parts 98 / 57, 15,360 34.9 / 26.7, 7,680
// 31.0 / 26.7; of about ten parts 16,384 rows 224 / 221, 6,144 equal, 4,096
// 86 / 89, 512 35 / 39; by a warp / by a block of four: 42 rows of up to 400 parts
// 51 / 33, 256 of 150 41 / 31, 380 to 1,000 of ten or fewer between 8% less and 7%
// more, 2,560 50 / 55.
constexpr int kManyRowsPerSm = 40, kFewRowsPerSm = 7, kFewWarps = 4;
template <int D, int LPR, int WPR>
__global__ void __launch_bounds__(WPR > 1 ? WPR * 32 : 128)
k_prefix_merge(PlanPtrs pl, const float2* __restrict__ wml, const float* __restrict__ wo,
               const float2* __restrict__ nml, const float* __restrict__ no,
               __nv_bfloat16* __restrict__ out, float* __restrict__ lse, PrefixShape sh) {
  constexpr int V = D / LPR;               // output values a lane
  constexpr int C = V < 4 ? V : 4;         // of them next to each other
  constexpr int kBatch = V > 8 ? 4 : 8;  // partial rows in flight
  const float kNegInf = __int_as_float(0xff800000);
  const int lane = threadIdx.x & (LPR - 1), first = threadIdx.x & 31 & ~(LPR - 1);
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / (LPR * WPR);
  const int warp = WPR > 1 ? threadIdx.x >> 5 : 0;  // of the row
  pdl_launch_dependents();
  const int64_t rows = (int64_t)sh.B * sh.Nq * sh.Hq;
  const int at_row = (int)min(row, rows - 1);  // (a warp's lanes stay together)
  const int h = at_row % sh.Hq, bq = at_row / sh.Hq, b = bq / sh.Nq, qi = bq % sh.Nq;
  const int head = h / sh.G, r = qi * sh.G + h % sh.G;  // row of the request for this KV head
  pdl_wait(pl.req, pl.npre, pl.hdr);
  const Request rq = pl.req[b];
  const int pre = pl.npre[b];
  const int U = pl.hdr[kUnits], S = pl.hdr[kShare], slots_head = pl.hdr[kSlots];
  const int Treq = pl.hdr[kTiles];
  const Pieces pieces(pl.hdr, sh.Hkv / sh.hg);
  const bool planned = pieces.tag == sh.tag;
  if (row == 0 && lane == 0 && warp == 0) {
    pl.hdr[kClaim] = 0;  // for the next call by this plan
    if (!planned) flag_error(pl.hdr + kErrWord, kErrState);
  }

  // candidate j of a run of wide items: CTA j % 2 of cut j / 2 (-1: there is none)
  auto wide_at = [&](int j, int unit, int slot, int rows, int nt, int x) -> int64_t {
    const int cut = j >> 1, len = min(S, nt - cut * S), k = (rows + kItemRows - 1) / kItemRows;
    const int blk = x / kItemRows;
    const int64_t u0 = (int64_t)head * U + unit + (int64_t)cut * S * k + blk * len;
    const int64_t c0 = quot(u0, S), c = c0 + (j & 1);
    if (u0 + len <= c * S) return -1;  // (the item ends before CTA c begins)
    return (int64_t)head * slots_head + slot + (int64_t)cut * rows + x + kItemRows * c;
  };
  const int n0 = 2 * ((rq.gtiles + S - 1) / S);
  int n1 = 0, c0 = 0;
  const int g = sh.narrow ? head / sh.hg : 0;
  if (rq.own > 0) {
    if (sh.narrow) {
      const int64_t f0 = (int64_t)g * Treq + pre;
      c0 = pieces.of(f0);
      n1 = pieces.of(f0 + (rq.own + kNarrowTile - 1) / kNarrowTile - 1) - c0 + 1;
    } else {
      n1 = 2 * (((rq.own + kTile - 1) / kTile + S - 1) / S);
    }
  }
  const int n = planned ? n0 + n1 : 0;  // (a return above would hold the loads back)
  auto at = [&](int j) -> int64_t {
    if (j < n0) return wide_at(j, rq.gunit, rq.gslot, rq.grows, rq.gtiles, rq.row + r);
    j -= n0;
    if (!sh.narrow) return wide_at(j, rq.ounit, rq.oslot, sh.R, (rq.own + kTile - 1) / kTile, r);
    return (((int64_t)c0 + j + (int64_t)g * sh.B + b) * sh.hg + head % sh.hg) * sh.R + r;
  };
  const float2* ml1 = sh.narrow ? nml : wml;
  const float* o1 = sh.narrow ? no : wo;
  // (up to LPR parts at a time; nearly always all of them: the running maximum
  // rescales what came before)
  float M = kNegInf, L = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  const int n_warp = LPR == 32 ? n : __reduce_max_sync(0xffffffffu, n);
  for (int j0 = 0; j0 < n_warp; j0 += LPR * WPR) {
    const int j = j0 + lane * WPR + warp;
    const int64_t my = j < n ? at(j) : -1;
    float2 e = make_float2(kNegInf, 0.f);
    if (my >= 0) e = __ldcg((j < n0 ? wml : ml1) + my);
    const float* src = (j < n0 ? wo : o1) + (my >= 0 ? my : 0) * D;
    float m = e.y == 0.f ? kNegInf : e.x;
#pragma unroll
    for (int s = LPR / 2; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float m_new = fmaxf(M, m);
    const float keep = L == 0.f ? 0.f : exp2f(M - m_new);
    const float wgt = e.y == 0.f ? 0.f : exp2f(e.x - m_new);
    float l = wgt * e.y;
#pragma unroll
    for (int s = LPR / 2; s >= 1; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    if (j0 > 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= keep;
    }
    L = (L == 0.f ? 0.f : L * keep) + l;
    M = m_new;
    // the rows that count, kBatch loads in flight
    uint32_t left = __ballot_sync(0xffffffffu, wgt != 0.f);
    if (LPR < 32) left = (left >> first) & ((1u << (LPR & 31)) - 1);
    while (LPR == 32 ? left : __any_sync(0xffffffffu, left)) {
      float x[kBatch][V], f[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        f[u] = 0.f;
        const int k = left ? __ffs(left) - 1 : 0;
        const float fk = __shfl_sync(0xffffffffu, wgt, k, LPR);
        const float* p = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(src), k, LPR));
        if (left) {
          f[u] = fk;
#pragma unroll
          for (int v = 0; v < V; v += C) {
            const float* at = p + v * LPR + lane * C;
            if (C == 4) {
              const float4 t = __ldcg(reinterpret_cast<const float4*>(at));
              x[u][v] = t.x;
              x[u][v + 1] = t.y;
              x[u][v + C - 2] = t.z;
              x[u][v + C - 1] = t.w;
            } else {
              const float2 t = __ldcg(reinterpret_cast<const float2*>(at));
              x[u][v] = t.x;
              x[u][v + 1] = t.y;
            }
          }
          left &= left - 1;
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += f[u] * x[u][v];
    }
  }
  if (WPR > 1) {  // the warps' sums
    __shared__ float s_m[WPR], s_l[WPR], s_o[WPR][D];
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[warp][(v / C * LPR + lane) * C + v % C] = acc[v];
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
    __syncthreads();
    if (warp > 0) return;
    const float l = lane < WPR ? s_l[lane & (WPR - 1)] : 0.f;
    const float m = l == 0.f ? kNegInf : s_m[lane & (WPR - 1)];
    M = m;
#pragma unroll
    for (int s = WPR / 2; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    const float f = l == 0.f ? 0.f : exp2f(m - M);
    L = f * l;
#pragma unroll
    for (int s = WPR / 2; s >= 1; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
    L = __shfl_sync(0xffffffffu, L, 0);
    M = __shfl_sync(0xffffffffu, M, 0);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
    for (int k = 0; k < WPR; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      if (fk == 0.f) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += fk * s_o[k][(v / C * LPR + lane) * C + v % C];
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  if (row >= rows || !planned) return;
  __nv_bfloat16* dst = out + row * D + lane * C;
#pragma unroll
  for (int v = 0; v < V; v += C) {
    uint32_t w[C / 2];
#pragma unroll
    for (int e = 0; e < C; e += 2) w[e / 2] = pack_bf16(acc[v + e] * inv, acc[v + e + 1] * inv);
    if (C == 4)
      *reinterpret_cast<uint2*>(dst + v * LPR) = make_uint2(w[0], w[C / 2 - 1]);
    else
      *reinterpret_cast<uint32_t*>(dst + v * LPR) = w[0];
  }
  if (lse && lane == 0)
    lse[row] = L == 0.f ? kNegInf : (M + log2f(L)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host ---

PrefixShape prefix_shape(const pks_prefix_args& a) {
  PrefixShape sh{};
  sh.B = a.B;
  sh.Hq = a.Hq;
  sh.Hkv = a.Hkv;
  sh.G = a.Hq / a.Hkv;
  sh.Nq = a.n_queries > 1 ? a.n_queries : 1;
  sh.R = sh.Nq * sh.G;
  sh.D = a.D;
  sh.page_size = a.page_size;
  sh.max_pages = a.max_pages;
  sh.num_pages = a.num_pages;
  sh.causal = a.causal;
  sh.min_shared = a.min_shared;
  sh.narrow = sh.R <= kNarrowRows;
  sh.hg = attn_heads_per_cta(a.Hkv);
  sh.wide_grid = device_sm_count();
  sh.box = a.page_size & -a.page_size;
  if (sh.box > kTile) sh.box = kTile;
  if (sh.box < 8) sh.box = 0;
  sh.narrow_grid = device_sm_count() * (sh.hg >= 8 ? 1 : sh.hg == 4 ? 2 : 4);
  uint32_t tag = 2166136261u;  // (FNV-1a, a word at a time)
  for (int x : {sh.B, sh.Hq, sh.Hkv, sh.Nq, sh.D, sh.page_size, sh.max_pages, sh.num_pages,
                sh.causal, a.prefix_group != nullptr ? 1 : 0})
    tag = (tag ^ (uint32_t)x) * 16777619u;
  sh.tag = (int)(tag | 1u);  // (never the zeroed workspace's)
  return sh;
}

PlanPtrs plan_ptrs(void* ws, const PrefixLayout& L) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(p + off); };
  PlanPtrs pl;
  pl.hdr = i32(L.hdr);
  pl.lens = i32(L.per_request);
  const size_t step = L.per_request_step / sizeof(int32_t);
  pl.eq = pl.lens + step;
  pl.first = pl.eq + step;
  pl.lead = pl.first + step;
  pl.start = pl.lead + step;
  pl.order = pl.start + step;
  pl.npre = pl.order + step;
  pl.req = reinterpret_cast<Request*>(p + L.requests);
  pl.starts = reinterpret_cast<Start*>(p + L.starts);
  pl.items = reinterpret_cast<Item*>(p + L.items);
  return pl;
}

// Dynamic shared memory limit of one kernel on the current device: raised once
// to `bytes` (the same for every call), outside any stream.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

cudaError_t encode_map(CUtensorMap* map, const void* pool, int rank, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                            const_cast<void*>(pool), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tensor map of a K or V pool as heads x rows x D for the narrow kernel, a box
// being eight tokens of `heads` heads and 64 of their values, 128-byte swizzled.
cudaError_t narrow_map(CUtensorMap* map, const void* pool, const pks_prefix_args& a, int heads) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.num_pages * (cuuint64_t)a.page_size,
                              (cuuint64_t)a.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)a.Hkv * a.D * 2, (cuuint64_t)a.D * 2};
  const cuuint32_t box[3] = {64, 8, (cuuint32_t)heads};
  return encode_map(map, pool, 3, dims, strides, box);
}

// The wide kernel's: heads x groups of eight rows x 64-value blocks x rows x
// values, a box being all blocks of `rows` tokens of a head, in the tile's layout.
cudaError_t wide_map(CUtensorMap* map, const void* pool, const pks_prefix_args& a, int rows) {
  const cuuint64_t row = (cuuint64_t)a.Hkv * a.D * 2;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)a.D / 64,
                              (cuuint64_t)a.num_pages * (cuuint64_t)a.page_size / 8,
                              (cuuint64_t)a.Hkv};
  const cuuint64_t strides[4] = {row, 128, 8 * row, (cuuint64_t)a.D * 2};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)a.D / 64, (cuuint32_t)rows / 8, 1};
  return encode_map(map, pool, 5, dims, strides, box);
}

template <int D>
cudaError_t launch_wide(const pks_prefix_args& a, const PrefixLayout& L, const PrefixShape& sh,
                        float scale_log2, cudaStream_t s) {
  static bool done[2][64] = {};
  // Boxes of 64 rows or more are issued by one warp; smaller ones, which would take
  // it too long, by four, and so are the other pages' rows (1024 rows on 131,072
  // tokens, us, by one / four: D = 128, pages of 8 568 / 383, of 16 453 / 383, of 64
  // with the narrow kernel beside it 415 / 425; D = 64, pages of 16 449 / 329).
  const bool spread = sh.box <= kTile / kLoadWarps;
  auto kern = spread ? k_prefix_wide<D, kLoadWarps> : k_prefix_wide<D, 1>;
  cudaError_t e = allow_smem(kern, Wide<D>::kSmem, done[spread]);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  CUtensorMap map_k{}, map_v{};
  if (sh.box > 0) {
    if ((e = wide_map(&map_k, a.kv_k, a, sh.box)) != cudaSuccess) return e;
    if ((e = wide_map(&map_v, a.kv_v, a, sh.box)) != cudaSuccess) return e;
  }
  return launch_ex(kern, dim3(sh.wide_grid), dim3(kWideThreads), Wide<D>::kSmem, s,
                   /*pdl=*/true, /*coop=*/false, a.block_table,
                   static_cast<const __nv_bfloat16*>(a.q),
                   static_cast<const __nv_bfloat16*>(a.kv_k),
                   static_cast<const __nv_bfloat16*>(a.kv_v), plan_ptrs(ws, L),
                   reinterpret_cast<float2*>(ws + L.wide_ml),
                   reinterpret_cast<float*>(ws + L.wide_o), sh, scale_log2,
                   a.wait_limit > 0 ? (long long)a.wait_limit : kWaitCycles, map_k, map_v);
}

template <int D, int HG, int WPH>
cudaError_t launch_narrow(const pks_prefix_args& a, const PrefixLayout& L, const PrefixShape& sh,
                          float scale_log2, bool wait_first, cudaStream_t s) {
  static bool done[64] = {false};
  using N = Narrow<D, HG>;
  auto kern = k_prefix_narrow<D, HG, WPH>;
  cudaError_t e = allow_smem(kern, N::smem(kMaxB), done);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  CUtensorMap map_k{}, map_v{};
  if (sh.box > 0) {
    if ((e = narrow_map(&map_k, a.kv_k, a, HG)) != cudaSuccess) return e;
    if ((e = narrow_map(&map_v, a.kv_v, a, HG)) != cudaSuccess) return e;
  }
  return launch_ex(kern, dim3(sh.narrow_grid), dim3((HG * WPH + 1) * 32), N::smem(a.B), s,
                   /*pdl=*/true, /*coop=*/false, a.block_table,
                   static_cast<const __nv_bfloat16*>(a.q),
                   static_cast<const __nv_bfloat16*>(a.kv_k),
                   static_cast<const __nv_bfloat16*>(a.kv_v), plan_ptrs(ws, L),
                   reinterpret_cast<float2*>(ws + L.narrow_ml),
                   reinterpret_cast<float*>(ws + L.narrow_o), sh, scale_log2, wait_first ? 1 : 0,
                   a.wait_limit > 0 ? (long long)a.wait_limit : kWaitCycles, map_k, map_v);
}

template <int D>
cudaError_t launch_parts(const pks_prefix_args& a, const PrefixLayout& L, const PrefixShape& sh,
                         cudaStream_t s) {
  const float scale = a.sm_scale > 0.f ? a.sm_scale : 1.f / sqrtf((float)D);
  const float scale_log2 = scale * 1.4426950408889634f;
  const bool wide = a.prefix_group || !sh.narrow;
  cudaError_t e = cudaSuccess;
  if (wide) e = launch_wide<D>(a, L, sh, scale_log2, s);
  if (e != cudaSuccess) return e;
  if (sh.narrow) {
#define PKS_NARROW(HG_)                                                                    \
  if (sh.hg == HG_)                                                                        \
    e = sh.R <= 8 ? launch_narrow<D, HG_, 1>(a, L, sh, scale_log2, !wide, s)               \
                  : launch_narrow<D, HG_, 2>(a, L, sh, scale_log2, !wide, s);
    PKS_NARROW(1)
    PKS_NARROW(2)
    PKS_NARROW(4)
    PKS_NARROW(8)
#undef PKS_NARROW
    if (e != cudaSuccess) return e;
  }
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int64_t rows = (int64_t)sh.B * sh.Nq * sh.Hq;
  const bool many = rows >= (int64_t)kManyRowsPerSm * sh.wide_grid;
  const bool few = rows <= (int64_t)kFewRowsPerSm * sh.wide_grid;
  const int per_block = many ? 16 : few ? 1 : 4;
  return launch_ex(many  ? k_prefix_merge<D, 8, 1>
                   : few ? k_prefix_merge<D, 32, kFewWarps>
                         : k_prefix_merge<D, 32, 1>,
                   dim3((unsigned)((rows + per_block - 1) / per_block)),
                   dim3(few ? 32 * kFewWarps : 128), 0, s,
                   /*pdl=*/true, /*coop=*/false, plan_ptrs(ws, L),
                   reinterpret_cast<const float2*>(ws + L.wide_ml),
                   reinterpret_cast<const float*>(ws + L.wide_o),
                   reinterpret_cast<const float2*>(ws + L.narrow_ml),
                   reinterpret_cast<const float*>(ws + L.narrow_o),
                   static_cast<__nv_bfloat16*>(a.out), a.lse, sh);
}

}  // namespace

PrefixLayout prefix_layout(const pks_prefix_args& a) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const PrefixShape sh = prefix_shape(a);
  const int64_t B = sh.B, R = sh.R;
  PrefixLayout L{};
  size_t off = 0;
  L.hdr = off;
  off += 256;
  L.per_request = off;
  L.per_request_step = up(sizeof(int32_t) * (size_t)(B + 1));
  off += 7 * L.per_request_step;
  L.requests = off;
  off = up(off + sizeof(Request) * (size_t)B);
  L.starts = off;
  off = up(off + sizeof(Start) * (size_t)sh.wide_grid);
  // items of one head: prefix rows in blocks of 256, each group with a remainder
  // (a group has two members at least), own rows likewise when the narrow kernel
  // leaves them, and the cuts (at most the CTAs' number)
  const bool groups = a.prefix_group != nullptr;
  const int64_t own_items = sh.narrow ? 0 : B * ((R + kItemRows - 1) / kItemRows);
  L.items = off;
  off = up(off + sizeof(Item) * (size_t)((groups ? B * R / kItemRows + B / 2 : 0) + own_items +
                                         sh.wide_grid + 1));
  // partial rows: each row once a head for its first cut; the further cuts, at
  // most one a CTA over all heads; and the places of the CTAs apart
  const int64_t once = (groups ? B * R : 0) + (sh.narrow ? 0 : B * R);
  const size_t wide = once ? (size_t)(sh.Hkv * once + 2 * (int64_t)kItemRows * sh.wide_grid) : 0;
  L.wide_ml = off;
  off = up(off + sizeof(float2) * wide);
  L.wide_o = off;
  off = up(off + sizeof(float) * wide * (size_t)a.D);
  const int64_t small = groups ? (int64_t)kSmallPerSm * sh.wide_grid : 0;
  const size_t narrow = sh.narrow ? (size_t)((sh.narrow_grid + small +
                                              (int64_t)(sh.Hkv / sh.hg) * B) * sh.hg * R) : 0;
  L.narrow_ml = off;
  off = up(off + sizeof(float2) * narrow);
  L.narrow_o = off;
  off = up(off + sizeof(float) * narrow * (size_t)a.D);
  L.total = off;
  return L;
}

cudaError_t launch_prefix_plan(const pks_prefix_args& a, const PrefixLayout& L, cudaStream_t s) {
  static bool done[64] = {false};
  cudaError_t e = allow_smem(k_prefix_plan, kPlanArrays * sizeof(int32_t) * kMaxB, done);
  if (e != cudaSuccess) return e;
  const PrefixShape sh = prefix_shape(a);
  const int at_once = kPlanThreads / 32 / kPlanWarps, most = 2 * sh.wide_grid;
  const int blocks = (a.B + at_once - 1) / at_once;
  const int grid = !a.prefix_group || a.B <= kPlanOneBlock ? 1 : blocks < most ? blocks : most;
  return launch_ex(k_prefix_plan, dim3(grid), dim3(kPlanThreads),
                   kPlanArrays * sizeof(int32_t) * (size_t)a.B, s, /*pdl=*/true,
                   /*coop=*/false, a.seq_lens,
                   a.block_table, a.prefix_group, plan_ptrs(a.workspace, L), sh);
}

cudaError_t launch_prefix_attention(const pks_prefix_args& a, const PrefixLayout& L,
                                    cudaStream_t s) {
  const PrefixShape sh = prefix_shape(a);
  return a.D == 64 ? launch_parts<64>(a, L, sh, s) : launch_parts<128>(a, L, sh, s);
}

}  // namespace pks
