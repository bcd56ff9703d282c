// Writing a 4-bit cache and reading it back.
//
// A row's head record is D/8 lanes' work, eight values a lane: lane 4 b + t has
// values 32 b + 8 t .. + 7, so that the four lanes of a group find its minimum and
// maximum with two shuffles and each lane's codes are one 32-bit word.  A block
// takes some rows, finds their places in the pool once, and then all their K and V
// records.
//
// Bound by memory: a bf16 row of D = 128 is 256 bytes in and 80 out.

#include <cuda_fp16.h>

#include "pks_internal.h"
#include "q4.cuh"

namespace pks {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowsMax = 8;  // rows of a block at a time

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

// Codes of eight values and (s in the low half, m in the high half) of their group,
// whose other values are on the three lanes beside.  The numbers are those of the
// definition in exact arithmetic, for any fp32 values:
//  - s: rounded up from the quotient, one step more where 15 s still falls short of
//    max - m (whose own rounding error, err, is counted).
//  - n: guessed from the reciprocal, at most one too low (the guess leans down by
//    2^-9, more than its error of 2^-11), then compared with the border above it.
//    Both sides of the comparison are exact: near m (15 s below 2^-7 |m|) as
//    x - m >= (n + 1/2) s, else as x >= m + (n + 1/2) s, at most 24 bits long.
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& sm) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, d));
  }
  const __half mh = __float2half_rd(lo);
  const float m = __half2float(mh);
  const float t = hi - m;
  const float back = t - hi;
  const float err = (hi - (t - back)) + (-m - back);
  __half sh = __float2half_ru(__fdiv_rn(t, 15.f));
  if (__fmaf_rn(-15.f, __half2float(sh), t) + err > 0.f)
    sh = __ushort_as_half(__half_as_ushort(sh) + 1);  // (s >= 0)
  const float s = __half2float(sh);
  const bool bad = !(fabsf(m) <= 65504.f && s <= 65504.f);
  sm = bad ? 0x7e00u : (uint32_t)__half_as_ushort(mh) << 16 | __half_as_ushort(sh);
  if (bad || s == 0.f) return 0;
  const float inv = __frcp_rn(s);
  const bool near = fabsf(m) > 2048.f * s;
  const float from = near ? m : 0.f, base = near ? 0.f : m;
  const float c = __fmaf_rn(-base, inv, -0.001953125f);
  const float first = __fmaf_rn(0.5f, s, base);  // the border between 0 and 1
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float xa = x[i] - from;
    const float r = __fmaf_rn(xa, inv, c) + 12582912.f;  // to the nearest whole number
    const float border = __fmaf_rn(r - 12582912.f, s, first);
    const uint32_t n = (__float_as_uint(r) & 15u) + (xa >= border ? 1u : 0u);
    w |= n << (4 * i);
  }
  return w;
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

struct RowShape {
  int B, n_rows, Hkv, page_size, max_pages, num_pages;
  int rows;           // of a block at a time
  int row_bytes;      // of a token in the pool
  uint32_t magic;     // ceil(2^32 / (2 Hkv)): divides record numbers
  int64_t k_row, k_head, v_row, v_head;
};

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kRowThreads)
k_q4_rows(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ block_table,
          const int32_t* __restrict__ starts, T* __restrict__ k, T* __restrict__ v,
          uint8_t* __restrict__ pool_k, uint8_t* __restrict__ pool_v, int32_t* error,
          RowShape sh) {
  constexpr int NB = D / q4::kGroup, LANES = D / 8, AT_ONCE = kRowThreads / LANES;
  constexpr int REC = q4::record_bytes(D), UNROLL = 4;
  extern __shared__ int32_t s_starts[];
  __shared__ int s_place[kRowsMax];
  const int tid = threadIdx.x, lane = tid % LANES, b = lane >> 2, t = lane & 3;
  pdl_wait(seq_lens, block_table, starts, k, v, pool_k, pool_v);
  pdl_launch_dependents();
  for (int i = tid; i <= sh.B; i += kRowThreads) s_starts[i] = starts[i];
  const int records = sh.rows * 2 * sh.Hkv;
  for (int64_t r0 = (int64_t)blockIdx.x * sh.rows; r0 < sh.n_rows;
       r0 += (int64_t)gridDim.x * sh.rows) {
    __syncthreads();
    if (tid < sh.rows)
      s_place[tid] = r0 + tid < sh.n_rows
                         ? place_of((int)r0 + tid, s_starts, sh.B, seq_lens, block_table,
                                    sh.page_size, sh.max_pages, sh.num_pages, error)
                         : -1;
    __syncthreads();
    // (the shuffles need all lanes: lanes without a record go along)
    for (int it0 = tid / LANES; it0 < records + tid / LANES; it0 += AT_ONCE * UNROLL) {
      T* at[UNROLL];          // the lane's values
      uint8_t* rec[UNROLL];   // the token's row in the pool; nullptr: no place
      uint32_t off[UNROLL];
      bool is_v[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int it = it0 + u * AT_ONCE;
        const int r = (int)__umulhi((uint32_t)it, sh.magic);
        const int kv = it - r * 2 * sh.Hkv;
        is_v[u] = kv >= sh.Hkv;
        const int h = is_v[u] ? kv - sh.Hkv : kv;
        const int place = it < records ? s_place[r] : -1;
        const int64_t row = r0 + r;
        at[u] = is_v[u] ? v + row * sh.v_row + h * sh.v_head : k + row * sh.k_row + h * sh.k_head;
        at[u] += 8 * lane;
        rec[u] = place < 0 ? nullptr
                           : (is_v[u] ? pool_v : pool_k) + (int64_t)place * sh.row_bytes;
        off[u] = h * REC;
      }
      // the lane's word: K, word t NB + b; V, of chunk g = 2 t (even b) or 2 t + 1
      // (odd b) the halves of groups b & ~1 and b | 1
      auto code_at = [&](int u) {
        const int w = is_v[u] ? (2 * t + (b & 1)) * (NB / 2) + (b >> 1) : t * NB + b;
        return reinterpret_cast<uint32_t*>(rec[u] + off[u] + 4 * w);
      };
      auto pair_at = [&](int u) {
        return reinterpret_cast<uint32_t*>(rec[u] + off[u] + D / 2 + 4 * b);
      };
      if constexpr (WRITE) {
        Eight<T> in[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
          for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
            in[u].w[i] = rec[u] ? reinterpret_cast<const uint4*>(at[u])[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          float x[8];
          unpack(in[u], x);
          uint32_t sm;
          uint32_t w = quantise(x, sm);
          const uint32_t got = __shfl_xor_sync(0xffffffffu, b & 1 ? w & 0xffffu : w >> 16, 4);
          if (is_v[u]) w = b & 1 ? got | (w & 0xffff0000u) : (w & 0xffffu) | got << 16;
          if (rec[u]) {
            *code_at(u) = w;
            if (t == 0) *pair_at(u) = sm;
          }
        }
      } else {
        uint32_t w[UNROLL], sm[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          w[u] = rec[u] ? *code_at(u) : 0;
          sm[u] = rec[u] ? *pair_at(u) : 0;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const uint32_t got =
              __shfl_xor_sync(0xffffffffu, b & 1 ? w[u] & 0xffffu : w[u] >> 16, 4);
          if (is_v[u]) w[u] = b & 1 ? got | (w[u] & 0xffff0000u) : (w[u] & 0xffffu) | got << 16;
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&sm[u]));
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float n = __uint_as_float((w[u] >> (4 * i) & 15u) | 0x4b000000u) - 8388608.f;
            x[i] = __fmaf_rn(n, f.x, f.y);
          }
          Eight<T> o;
          pack(x, o);
          if (rec[u])
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
              reinterpret_cast<uint4*>(at[u])[i] = o.w[i];
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
  sh.magic = (uint32_t)(((uint64_t(1) << 32) + 2 * a.Hkv - 1) / (2 * a.Hkv));
  sh.k_row = a.k_row;
  sh.k_head = a.k_head;
  sh.v_row = a.v_row;
  sh.v_head = a.v_head;
  // few rows: a block each, so that they run side by side
  const int per_sm = 8, most = device_sm_count() * per_sm;
  sh.rows = 1;
  while (sh.rows < kRowsMax && (int64_t)sh.rows * most < a.n_rows) sh.rows *= 2;
  const int blocks = (int)(((int64_t)a.n_rows + sh.rows - 1) / sh.rows);
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
