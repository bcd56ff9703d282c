// Writing a 4-bit cache and reading it back.
//
// A block takes some rows, finds their places in the pool once, and then all their K and V
// records, a warp (or several, when rows are few) a row.
//  - Writing, a lane has a whole group of 32 values: what is worked out once a group
//    (minimum, scale, reciprocal) is most of the work when four lanes share one (131,072
//    rows written and read back 492 -> 309 us).  The rest is two values at once where
//    fp32 pairs allow it (a fifth fewer instructions, the same 253 -> 246 us).
//  - Reading, a lane has a quarter of every group: one 16-byte load of codes, one of scales,
//    and a store of 16 bytes (of a two-byte type) a group, four lanes 64 bytes side by side.
//    Two records at once; one or four: 265 and 261 us for the same 253.
//
// Bound by memory: a bf16 row of D = 128 is 256 bytes in and 80 out, and four instructions in
// five still are arithmetic.  Rows of eight heads of 128 in bf16: 131,072 written and read
// back 239 us (6.0 TB/s), 154,000 read 138 us (6.0 TB/s).  More blocks an SM by fewer registers
// are slower (48 registers: by 1%, 40: by 8%).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pks_internal.h"
#include "q4.cuh"

namespace pks {
namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kRowsEach = 8;  // of a warp, at most, whose places a block finds at once
// what eight magic numbers (1.5 2^23 as bits, shifted by 4 i) add up to beside the codes
constexpr uint32_t kMagicSum = 0x4b400000u * 0x11111111u;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// two fp32 values in one register pair
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2_down(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// 1 from the border on, else 0
__device__ __forceinline__ float from_on(float x, float border) {
  float r;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(border));
  return r;
}

// eight values of a lane, as they lie in memory
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
};
__device__ __forceinline__ void unpack(const Eight<__nv_bfloat16>& e, float (&x)[8]) {
  const uint32_t w[4] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Eight<__half>& e, float (&x)[8]) {
  const uint32_t w[4] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const Eight<float>& e, float (&x)[8]) {
  const uint32_t w[8] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w,
                         e.w[1].x, e.w[1].y, e.w[1].z, e.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Eight<__nv_bfloat16>& e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  e.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Eight<__half>& e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  e.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Eight<float>& e) {
  e.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  e.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                      __float_as_uint(x[7]));
}

// Smallest and largest of a lane's 32 values (NaN when one is).  Two-byte types two at once.
template <typename T>
__device__ __forceinline__ void extent(const Eight<T> (&in)[4], float& lo, float& hi) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      unpack(in[i], x);
      if (i == 0) lo = hi = x[0];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo = min_nan(lo, x[e]);
        hi = max_nan(hi, x[e]);
      }
    }
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    T2 a{}, b{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {in[i].w[0].x, in[i].w[0].y, in[i].w[0].z, in[i].w[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const T2 x = *reinterpret_cast<const T2*>(&w[e]);
        a = i + e == 0 ? x : __hmin2_nan(a, x);
        b = i + e == 0 ? x : __hmax2_nan(b, x);
      }
    }
    lo = min_nan((float)a.x, (float)a.y);
    hi = max_nan((float)b.x, (float)b.y);
  }
}

// (s in the low half, m in the high half) of a group, and what its codes are found with.
// The numbers are those of the definition in exact arithmetic, for any fp32 values:
//  - s: rounded up from the quotient, one step more where 15 s still falls short of
//    max - m (whose own rounding error, err, is counted).
//  - n: guessed from the reciprocal, at most one too low (the guess leans down by
//    2^-9, more than its error of 2^-17), then compared with the border above it,
//    (n + 1/2) s, which is at most 16 bits long.  x - m may need more than fp32 has (a
//    small m below a large s), so it is rounded down: then it is at or above a number
//    of fp32 exactly when x - m is.
struct Scale {
  uint32_t pair;
  float s, inv, m;
  bool flat;  // all codes are 0
};
__device__ __forceinline__ Scale scale_of(float lo, float hi) {
  Scale g;
  const __half mh = __float2half_rd(lo);
  const float m = __half2float(mh);
  const float t = hi - m;
  const float back = t - hi;
  const float err = (hi - (t - back)) + (-m - back);
  __half sh = __float2half_ru(__fdiv_rn(t, 15.f));
  if (__fmaf_rn(-15.f, __half2float(sh), t) + err > 0.f)
    sh = __ushort_as_half(__half_as_ushort(sh) + 1);  // (s >= 0)
  g.s = __half2float(sh);
  const bool bad = !(fabsf(m) <= 65504.f && g.s <= 65504.f);
  g.pair = bad ? 0x7e00u : (uint32_t)__half_as_ushort(mh) << 16 | __half_as_ushort(sh);
  g.flat = bad || g.s == 0.f;
  g.inv = g.flat ? 0.f : __frcp_rn(g.s);
  g.m = m;
  return g;
}
// codes of eight values, the first in the lowest bits
__device__ __forceinline__ uint32_t codes(const float (&x)[8], const Scale& g) {
  const uint64_t least = two(-g.m, -g.m), inv = two(g.inv, g.inv),
                 lean = two(-0.001953125f, -0.001953125f), scale = two(g.s, g.s),
                 half = two(0.5f * g.s, 0.5f * g.s), magic = two(12582912.f, 12582912.f),
                 back = two(-12582912.f, -12582912.f);
  uint32_t w = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    const uint64_t xa = add2_down(two(x[i], x[i + 1]), least);
    const uint64_t r = add2(fma2(xa, inv, lean), magic);  // to the nearest whole number
    const uint64_t border = fma2(add2(r, back), scale, half);
    const uint64_t n = add2(r, two(from_on(first(xa), first(border)),
                                   from_on(second(xa), second(border))));
    w = (w * 16 + __float_as_uint(second(n))) * 16 + __float_as_uint(first(n));
  }
  return g.flat ? 0 : w - kMagicSum;
}

// The place in the pool of row i of a call (page * page_size + slot), -1 for none.
__device__ __forceinline__ int place_of(int i, const int32_t* starts, int B,
                                          const int32_t* seq_lens, const int32_t* block_table,
                                          int page_size, int max_pages, int num_pages,
                                          int32_t* error) {
  if (i < starts[0] || i >= starts[B]) return -1;
  int lo = 0, hi = B;  // starts[lo] <= i < starts[hi], whatever lies between
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int64_t len = seq_lens[lo];
  int bad = 0;
  int at = -1;
  if (len < 0 || len > (int64_t)max_pages * page_size) {
    bad = kErrLen;
  } else {
    const int64_t pos = len - (int64_t)starts[lo + 1] + i;
    if (pos < 0 || pos >= len) {
      bad = kErrToken;
    } else {
      const int p = (int)pos / page_size, slot = (int)pos - p * page_size;
      const int page = block_table[(int64_t)lo * max_pages + p];
      if (page < 0 || page >= num_pages) bad = kErrPage;
      else at = page * page_size + slot;
    }
  }
  if (bad && error) *error = bad;
  return at;
}

// d = a b + c, a and b halves, rounded once
__device__ __forceinline__ float fma_mixed(uint16_t a, uint16_t b, float c) {
  float d;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
  return d;
}
// a word a group
__device__ __forceinline__ void group_words(const uint8_t* at, bool on, uint32_t (&w)[4]) {
  const uint4 x = on ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
  w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
}
__device__ __forceinline__ void group_words(const uint8_t* at, bool on, uint32_t (&w)[2]) {
  const uint2 x = on ? *reinterpret_cast<const uint2*>(at) : make_uint2(0, 0);
  w[0] = x.x, w[1] = x.y;
}

// Lanes of a record, and records of a lane at once
template <int D, bool WRITE>
constexpr int kLanes = WRITE ? D / q4::kGroup : 4;
template <bool WRITE>
constexpr int kAtOnce = WRITE ? 1 : 2;

struct RowShape {
  int B, n_rows, Hkv, page_size, max_pages, num_pages;
  int warps;          // a row: 1 to 8, a power of two
  int each;           // rows that a block finds the places of at once, a warp's share of them
  int row_bytes;      // of a token in the pool
  int64_t k_row, k_head, v_row, v_head;
};

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kRowThreads)
k_q4_rows(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ block_table,
          const int32_t* __restrict__ starts, T* __restrict__ k, T* __restrict__ v,
          uint8_t* __restrict__ pool_k, uint8_t* __restrict__ pool_v, int32_t* error,
          RowShape sh) {
  constexpr int NB = D / q4::kGroup, REC = q4::record_bytes(D);
  constexpr int LANES = kLanes<D, WRITE>, AT_ONCE = 32 / LANES;  // records of a warp
  constexpr int U = kAtOnce<WRITE>;                                  // of a lane
  extern __shared__ int32_t s_starts[];
  __shared__ int s_place[kRowWarps * kRowsEach];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = warp & (sh.warps - 1), mine = warp / sh.warps, side = kRowWarps / sh.warps;
  const int rows = side * sh.each;
  pdl_wait(seq_lens, block_table, starts, k, v, pool_k, pool_v);
  pdl_launch_dependents();
  for (int i = tid; i <= sh.B; i += kRowThreads) s_starts[i] = starts[i];
  for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < sh.n_rows; r0 += (int64_t)gridDim.x * rows) {
    __syncthreads();
    if (tid < rows)
      s_place[tid] = r0 + tid < sh.n_rows
                         ? place_of((int)r0 + tid, s_starts, sh.B, seq_lens, block_table,
                                    sh.page_size, sh.max_pages, sh.num_pages, error)
                         : -1;
    __syncthreads();
    for (int r = mine; r < rows; r += side) {
      const int place = s_place[r];
      if (place < 0) continue;  // (a whole warp)
      const int64_t row = r0 + r, at = (int64_t)place * sh.row_bytes;
      T* k_row = k + row * sh.k_row;
      T* v_row = v + row * sh.v_row;
      // K's records, then V's; the shuffles need all lanes: those without a record go along
      for (int j0 = part * AT_ONCE * U; j0 < 2 * sh.Hkv; j0 += sh.warps * AT_ONCE * U) {
        T* values[U];
        uint8_t* rec[U];
        bool is_v[U], on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * AT_ONCE + lane / LANES;
          on[u] = j < 2 * sh.Hkv;
          is_v[u] = j >= sh.Hkv;
          const int h = is_v[u] ? j - sh.Hkv : j;
          values[u] = is_v[u] ? v_row + h * sh.v_head : k_row + h * sh.k_head;
          rec[u] = (is_v[u] ? pool_v : pool_k) + at + h * REC;
        }
        if constexpr (WRITE) {
          const int b = lane & (NB - 1);
          Eight<T> in[4];
          const uint4* from = reinterpret_cast<const uint4*>(values[0] + 32 * b);
          constexpr int W = sizeof(T) / 2;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < W; ++i)
              in[t].w[i] = on[0] ? from[t * W + i] : make_uint4(0, 0, 0, 0);
          float lo, hi;
          extent(in, lo, hi);
          const Scale g = scale_of(lo, hi);
          uint32_t w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float x[8];
            unpack(in[t], x);
            w[t] = codes(x, g);
          }
          // V: the halves of groups b & ~1 and b | 1 stand in one word, those of chunks 0 to 3
          // (values 0 to 15) with the even one's lane
          const bool odd = b & 1;
          const uint32_t got0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[2], 1);
          const uint32_t got1 = __shfl_xor_sync(0xffffffffu, odd ? w[1] : w[3], 1);
          uint32_t* to = reinterpret_cast<uint32_t*>(rec[0]);
          if (on[0]) {
            if (is_v[0]) {
              const uint32_t low0 = odd ? got0 : w[0], low1 = odd ? got1 : w[1];
              const uint32_t high0 = odd ? w[2] : got0, high1 = odd ? w[3] : got1;
              to += (odd ? 4 : 0) * (NB / 2) + (b >> 1);
              to[0] = __byte_perm(low0, high0, 0x5410);
              to[NB / 2] = __byte_perm(low0, high0, 0x7632);
              to[NB] = __byte_perm(low1, high1, 0x5410);
              to[NB / 2 * 3] = __byte_perm(low1, high1, 0x7632);
            } else {
#pragma unroll
              for (int t = 0; t < 4; ++t) to[t * NB + b] = w[t];
            }
            reinterpret_cast<uint32_t*>(rec[0] + D / 2)[b] = g.pair;
          }
        } else {
          const int t = lane & 3;
          uint32_t code[U][NB], sm[U][NB];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            group_words(rec[u] + 4 * NB * t, on[u], code[u]);
            group_words(rec[u] + D / 2, on[u], sm[u]);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              // K: word t NB + b; V: 16-bit words (2 t) NB + b and (2 t + 1) NB + b
              uint32_t w = code[u][b];
              if (is_v[u])
                w = __byte_perm(code[u][b / 2], code[u][(NB + b) / 2], b & 1 ? 0x7632 : 0x5410);
              const uint16_t scale = (uint16_t)sm[u][b];
              const float least = __half2float(__ushort_as_half((uint16_t)(sm[u][b] >> 16)));
              // codes i and i + 4 as halves: 1024 + n or 1024 + 16 n, whose bits a mask gives
              float x[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t y = ((i & 2 ? w >> 8 : w) & (i & 1 ? 0x00f000f0u : 0x000f000fu)) |
                                   0x64006400u;
                const __half2 h = *reinterpret_cast<const __half2*>(&y);
                const __half2 n = i & 1 ? __hfma2(h, __float2half2_rn(0.0625f),
                                                  __float2half2_rn(-64.f))
                                        : __hadd2(h, __float2half2_rn(-1024.f));
                x[i] = fma_mixed(__half_as_ushort(__low2half(n)), scale, least);
                x[i + 4] = fma_mixed(__half_as_ushort(__high2half(n)), scale, least);
              }
              Eight<T> o;
              pack(x, o);
              if (on[u])
#pragma unroll
                for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
                  reinterpret_cast<uint4*>(values[u] + 32 * b + 8 * t)[i] = o.w[i];
            }
          }
        }
      }
    }
  }
}

template <typename T, int D, bool WRITE>
cudaError_t launch(const pks_q4_rows_args& a, cudaStream_t s) {
  RowShape sh{};
  sh.B = a.B;
  sh.n_rows = a.n_rows;
  sh.Hkv = a.Hkv;
  sh.page_size = a.page_size;
  sh.max_pages = a.max_pages;
  sh.num_pages = a.num_pages;
  sh.row_bytes = q4::token_bytes(a.Hkv, D);
  sh.k_row = a.k_row;
  sh.k_head = a.k_head;
  sh.v_row = a.v_row;
  sh.v_head = a.v_head;
  // few rows: as many warps a row as have work, so that they run side by side
  const int most = device_sm_count() * (2048 / kRowThreads);
  const int each = 32 / kLanes<D, WRITE> * kAtOnce<WRITE>;
  sh.warps = 1;
  while (sh.warps < kRowWarps && sh.warps * each < 2 * a.Hkv &&
         (int64_t)a.n_rows * sh.warps < (int64_t)most * kRowWarps / 2)
    sh.warps *= 2;
  sh.each = 1;
  while (sh.each < kRowsEach &&
         (int64_t)a.n_rows * sh.warps >= (int64_t)most * kRowWarps * 2 * sh.each)
    sh.each *= 2;
  const int rows = kRowWarps / sh.warps * sh.each;
  const int blocks = (int)(((int64_t)a.n_rows + rows - 1) / rows);
  return launch_ex(k_q4_rows<T, D, WRITE>, dim3(blocks < most ? blocks : most), dim3(kRowThreads),
                   sizeof(int32_t) * (size_t)(a.B + 1), s, /*pdl=*/true, /*coop=*/false,
                   a.seq_lens, a.block_table, a.starts, static_cast<T*>(a.k),
                   static_cast<T*>(a.v), static_cast<uint8_t*>(a.pool_k),
                   static_cast<uint8_t*>(a.pool_v), a.error, sh);
}

template <bool WRITE>
cudaError_t launch_type(const pks_q4_rows_args& a, cudaStream_t s) {
  const bool wide = a.D == 128;
  if (a.dtype == PKS_Q4_BF16)
    return wide ? launch<__nv_bfloat16, 128, WRITE>(a, s) : launch<__nv_bfloat16, 64, WRITE>(a, s);
  if (a.dtype == PKS_Q4_FP16)
    return wide ? launch<__half, 128, WRITE>(a, s) : launch<__half, 64, WRITE>(a, s);
  return wide ? launch<float, 128, WRITE>(a, s) : launch<float, 64, WRITE>(a, s);
}

}  // namespace

cudaError_t launch_q4_rows(const pks_q4_rows_args& a, bool write, cudaStream_t s) {
  return write ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace pks
