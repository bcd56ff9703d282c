// Attention over a paged KV cache held in 4 bits, dense or over selected tokens.
//
// A cached value is m + s n (group of 32 values: s, m fp16; n 0..15), so with the
// query's sums Q_b over the values of group b
//   q . K = sum_b ( s_b sum_{d in b} q_d n_d  +  m_b Q_b )
//   sum_t p_t V_t[d] = sum_t (p_t s_tb) n_td  +  sum_t p_t m_tb        (d in group b)
// and both products run on the codes themselves (mma.sync, tokens or values as M,
// the query rows of a KV head as N):
//  - The bit pattern of n in a 16-bit word is the subnormal bf16 n 2^-133 (and fp16
//    n 2^-24), one step up 16 n of it: eight codes become four operand registers
//    with four ANDs and a shift, and no conversion.  Powers of two are put right in
//    the queries (those at the odd places are a sixteenth) and at the end.  Of V two
//    registers in four even go without the AND: a byte of two codes is n + 16 n' of
//    them, and n's sum is taken off at the end (integer pipe: 16 x 131072 tokens 433 -> 420 us).
//  - K: bf16, the queries scaled by a power of two, so that all products are exact.
//    Each group's sum is scaled by s_b on its own (fp32); the m_b Q_b of two groups are
//    one more MMA, with the (s, m) pairs as they lie against 0 and Q_b, which is cut into
//    fp16 pieces, one a lane: two of them to 2^-24 of what 32 queries of the largest size
//    sum up to, the third what is left of large sums (m taken out of the pairs: 420 us for 413).
//  - V: fp16.  p is rounded to fp16, and p s once a group (by 2^-11 of it at most while
//    they are normal numbers: kTop and what follows there).  sum p m is one more MMA.
// Maxima, sums, scores and accumulators are fp32.
//
// One persistent CTA an SM.  All (request, head group, row chunk) segments are cut into
// stages of 16 or 32 tokens a consumer warp; the CTAs take equal runs of stages (or, where
// segments are few and short, one segment each).  Producer
// warps find the tokens' rows and fill a ring of stages, each in its turn; a consumer
// warp owns one head and some tokens of every stage and keeps the head's sums in registers.
// Segments that several CTAs hold parts of are joined by k_q4_merge.
//
// Bound by memory where the tokens are many (16 x 131072 tokens of eight heads of 128, eight
// queries a head: 388 us, 6.9 TB/s of codes), else by what the consumers issue: a head's 32
// tokens take 1750 cycles from L2 (2640 with sixteen queries a head), of which the tensor
// pipe is busy for a third and the integer pipe, which takes the codes apart, for half.
// Measured against it:
//  - sixteen consumer warps of half the registers, queries in shared memory: 468 us for 434;
//  - one warp a head for scores and one for values: 569 for 456;
//  - one tile of 16 tokens at a time: 593 for 468;
//  - consumers of 200 registers: 462 for 450.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "pks_internal.h"
#include "q4.cuh"
#include "tcgen05.cuh"

namespace pks {
namespace {

constexpr long long kWaitCycles = 4000000000LL;  // about 2 s at 2 GHz, unless wait_limit is set
constexpr long long kLandCycles = 1LL << 26;  // for copies in flight to land, 30 ms
constexpr int kConsumers = 8;  // warps, two a scheduler
// Producer warps (PW): four, each filling every fourth stage; with kTokens teams of two, one
// for K and one for V, of four warps or eight.  Eight keep up with long lists, four start
// sooner.  Selected tokens, four warps and eight: 7 stages a CTA 30 and 32 us, 13 40 and
// 42, 20 50 both, 27 67 and 65, 54 95 and 89, 108 163 and 144.
constexpr int kLongRun = 24;  // stages a CTA above which there are eight
// Stages up to which a CTA has a segment to itself, without a plan and parts to join: four, and
// one more for every sixteen segments.  5 requests of 2 stages 6.9 us and 8.6 split, of 4 8.9
// and 8.8, of 5 10.4 and 8.9; 16 of 5 10.6 and 11.7, of 8 13.7 and 12.2; 64 lists of 8 13.9 and
// 19.1.
constexpr int kWholeStages = 4, kWholeMore = 16;
constexpr int kMaxTokens = 256;  // of a stage
constexpr int kMaxStages = 12;
constexpr int kLeastStages = 4;  // with fewer a producer could pass a barrier a round behind
constexpr int kSmemMax = 227 * 1024 - 6144;  // dynamic; the rest is the static part
// Rows from here on may go by kTokens.  64 lists of 1024 tokens, by kTokens and by kLanes:
// rows of 160 bytes 32 and 32 us, 240 38 and 36, 320 40 and 44, 480 42 and 46.
constexpr int kTokenBytesLeast = 320;
// Output rows up to which a block of k_q4_merge joins one, else a warp: 64 rows 61 us and
// 112, 1024 85 and 89, 2048 58.5 both, 4096 65 and 57, 8192 75 and 56.
constexpr int kFewRows = 2048;
constexpr float kNone = -3e38f;  // reference of a row that has seen no token
// Weights p are kept at 2^(kTop - 3) to 2^kTop at the largest score, 2^11 to 2^14, so that those of
// 2^-25 of the largest are normal numbers of fp16 still, and those above 2^-36 are not 0.  The
// same has to hold for p s, whatever V's size.  So the sums of a group are in a unit 2^sx, by
// which its scales are divided:
//  - 1 while they have their usual size, the largest of a stage below 2 and not below 2^-kSmall
//    (2^-kSmallShort in segments of up to kShortSegment tokens).  That none is 2 is seen to at
//    every stage, that some are large enough at one stage in two rounds of the ring (at every
//    stage, in a few operations: 16 x 131072 tokens 407 us for 389);
//  - else what brings the largest of such a stage into [1, 2), or, so that it seldom changes,
//    within 2^-kKeep below, 2^-15 at the least; a larger one than 2 units moves it at once.
// 16 x 131072 tokens with a unit other than 1 take 485 us for 388; worked out anew at every stage
// 632 us; by a branch that scales before the scores 504.
// What is lost of a token is so 15 2^-36 units at most, 2^-9 of 15 s over as many tokens as the
// limits say; segments of more than kLongSegment tokens always have a unit of their own.
constexpr float kTop = 14.f;
constexpr int kSmall = 7, kSmallShort = 11, kKeep = 3;
constexpr int kShortSegment = 1 << 16, kLongSegment = 1 << 20;
// What a warp keeps of it in shared memory: 32 + sx a byte, kLong for such a segment, kAgain where
// the next stage is looked at too
constexpr uint32_t kUsual = 0x20202020u, kLong = 0x80000000u, kAgain = 0x40000000u;

// Tokens of a warp's 16 as the rows of its MMA tiles, four bits each (lowest: row 0).
// Lanes of one shared-memory access hold tokens whose records lie in different
// banks: rows 2 i and 2 i + 1 must stand 64 bytes apart (mod 128), the rows 0, 2, 4, 6
// and 1, 3, 5, 7 32 bytes.  By the distance between tokens: odd multiples of 16 bytes,
// odd multiples of 32, of 64 (V's accesses in two).
constexpr uint64_t kOrderOdd = 0xbf9d7351ae8c6240ull;
constexpr uint64_t kOrderTwo = 0xdfceb9a857463120ull;
constexpr uint64_t kOrderFour = 0xefdcab9867542310ull;

// How a stage gets its tokens:
//  kRuns   - dense, all heads: the tokens of one page by one bulk copy.  For any page that
//            leaves a stage no more than 32 of them: 16 x 16384 tokens of 80 bytes 34 us, 42
//            by kLanes, whatever the page; of 400 bytes 79 us, 87 by kTokens, and 81 and
//            87 on pages of two
//  kTokens - rows of 320 bytes or more: a bulk copy a token, at a distance in shared
//            memory that suits the banks; two warps a stage, one for K and one for V
//            (four warps: 7.3 TB/s of rows of 640 bytes, 6.3 of 320, 1.7 of 80)
//  kBoxes  - dense, rows of 128-byte lines (D = 128 and Hkv a multiple of 8): TMA boxes of 16
//            or 32 tokens, whose swizzle suits the banks; what fills no box as kLanes
//  kLanes  - other small rows: 16 or 8 bytes a lane (cp.async)
enum Copies { kRuns, kTokens, kBoxes, kLanes };

struct Q4Shape {
  int Bv;            // requests; with selected tokens, requests times queries
  int Hq, G, page_size, max_pages, num_pages;
  int k, trim;       // entries a list, 0: dense
  int lists;         // lists a request (1 when dense)
  int Nq;            // query tokens a segment works on (1 with selected tokens)
  int causal;
  int R;             // query rows of a KV head: Nq * G
  int HG, NHG, NRC;  // heads of a CTA, groups of them, chunks of rows
  int WPH, TS, ts_log2;  // warps a head, tokens a stage (a power of two)
  int cap;           // tokens a request can have
  uint32_t page_magic;   // ceil(2^32 / page_size), 0 for 1
  int row_bytes;     // of a token in the pool
  int taken;         // of it what a head group takes, copied in units of 8 or 16 bytes
  int unit;
  int slice;         // distance between tokens in shared memory
  int copies;        // see above
  int box;           // kBoxes: tokens of one
  int lanes;         // kLanes: that copy a token, a unit or two each
  uint64_t order;
  int stages, q_at, scratch_at, nv_at;  // of the ring; where what lies behind it begins
  int whole;  // a CTA has a segment to itself (no parts to join)
  int grid;
};

// d = a b, and d += a b
#define PKS_MMA(NAME, TYPE)                                                                      \
  __device__ __forceinline__ void NAME(float(&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,      \
                                       uint32_t a3, uint32_t b0, uint32_t b1) {                  \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                   \
        ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"              \
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));                       \
  }                                                                                              \
  __device__ __forceinline__ void NAME##_add(float(&d)[4], uint32_t a0, uint32_t a1,             \
                                             uint32_t a2, uint32_t a3, uint32_t b0,              \
                                             uint32_t b1) {                                      \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                   \
        ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"                  \
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));                                 \
  }
PKS_MMA(mma_bf16, "bf16")
PKS_MMA(mma_f16, "f16")
#undef PKS_MMA
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 bits_half2(uint32_t u) {
  return *reinterpret_cast<const __half2*>(&u);
}
__device__ __forceinline__ int unit_of(uint32_t units, int b) {  // sx of group b
  return (int)(units >> 8 * b & 63) - 32;
}
// all ones where a half is NaN or infinite
__device__ __forceinline__ uint32_t infinite(uint32_t u) {
  return __vcmpgeu2(u & 0x7fff7fffu, 0x7c007c00u);
}
// the halves' sizes, 0 for those that are not finite
__device__ __forceinline__ uint32_t finite(uint32_t u) {
  return u & 0x7fff7fffu & ~infinite(u);
}
__device__ __forceinline__ float low_half(uint32_t u) {
  return __half2float(__low2half(bits_half2(u)));
}

// N words from shared memory (8- or 16-byte aligned)
template <int N>
__device__ __forceinline__ void lds(const uint8_t* at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}
__device__ __forceinline__ void sts_zero8(uint32_t addr) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %1};\n" ::"r"(addr), "r"(0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

// What a stage holds, from its producer to the consumers.  mask: the tokens present,
// of each 16, and the flags above them.
struct alignas(16) StageNote {
  int v, c, p0, nv;  // segment (request or list, chunk), first position, positions in all
  uint32_t mask[16];
};
// kLast: the CTA's last stage of the segment; kWhole: it has all of them; kSecond: not
// the CTA's first segment; kEdge: some token lies beyond some query's limit; kEnd: the
// CTA's last stage (counted by the producers: by the consumers, 1860 cycles a stage for 1750)
constexpr uint32_t kLast = 1u << 16, kWhole = 2u << 16, kSecond = 4u << 16, kEdge = 8u << 16,
                   kEnd = 16u << 16;
// Registers a thread of this warpgroup has from here on.  All of a CTA's together no
// more than it was launched with.  Consumers have 216 where 208 are too few (sixteen rows of eight
// heads of 128 by boxes 2636 cycles a stage for 2784) and the producers can do with 72; eight
// rows by boxes are slower with them (1845 for 1750).
template <int NT, int PW, int SLICE>
constexpr bool kMoreRegisters = PW == 4 && (SLICE == 0 || (NT == 2 && SLICE == 640));
template <int NT, int PW, int SLICE>
constexpr int kConsumerRegisters = kMoreRegisters<NT, PW, SLICE> ? 216 : 208;
template <int NT, int PW, int SLICE>
constexpr int kProducerRegisters = kMoreRegisters<NT, PW, SLICE> ? 72 : PW == 8 ? 48 : 88;
template <int N, bool MORE>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// a += b, two at once
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
// d = a b + c, two at once
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// W stages over n CTAs: the first W % n of them take one more than the rest
struct Shares {
  int each, more;
  __device__ __forceinline__ Shares(int W, int n) : each(W / n), more(W - W / n * n) {}
  __device__ __forceinline__ int first(int cta) const { return each * cta + min(cta, more); }
  __device__ __forceinline__ int holder(int stage) const {
    const int big = more * (each + 1);
    return stage < big ? stage / (each + 1) : more + (stage - big) / each;
  }
};

// SLICE: 640 or 656 where a stage's rows are the records of eight heads of 128 values, by
// boxes or by tokens: distances that the compiler knows save an address computation for
// most loads from shared memory (16 x 131072 tokens 450 -> 441 us); 0: any others.
template <int D, int NT, int TT, int PW, int SLICE>
__global__ void __launch_bounds__((kConsumers + PW) * 32, 1)
k_q4_attention(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ block_table,
               const int32_t* __restrict__ lists, const __nv_bfloat16* __restrict__ q,
               const uint8_t* __restrict__ pool_k, const uint8_t* __restrict__ pool_v,
               __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
               int32_t* __restrict__ prefix, float2* __restrict__ part_ml,
               float* __restrict__ part_o, int32_t* __restrict__ err, const Q4Shape sh,
               float scale_log2, long long wait_cycles, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v) {
  constexpr int NW = kConsumers, NWARPS = NW + PW, NTHREADS = NWARPS * 32;
  constexpr int NB = D / q4::kGroup, REC = q4::record_bytes(D);
  constexpr int RC = 8 * NT;  // query rows a chunk
  const float kNegInf = __int_as_float(0xff800000), kAlways = __int_as_float(0x7fc00000);
  extern __shared__ uint8_t smem_raw[];
  // bar_full: the producer's announcement (and its lanes' copies); bar_empty and
  // bar_join: the consumer warps
  __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_join;
  __shared__ StageNote s_note[kMaxStages];
  __shared__ int s_row_all[4][kMaxTokens];  // tokens' rows in the pool (-1: none)
  __shared__ __align__(16) uint32_t s_by_unit[NW][NB];
  __shared__ uint32_t s_units[NW];
  __shared__ int s_warp[NWARPS], s_first, s_rest, s_lo, s_count, s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (ring - tc::smem_u32(smem_raw));
  constexpr bool FIXED = SLICE > 0;
  const int slice = FIXED ? SLICE : sh.slice, TS = FIXED ? 16 * TT : sh.TS;
  const int ts_log2 = FIXED ? (TT == 2 ? 5 : 4) : sh.ts_log2;
  const int HG = FIXED ? 8 : sh.HG, WPH = FIXED ? 1 : sh.WPH;
  const int copies = SLICE == 640 ? kBoxes : SLICE == 656 ? kTokens : sh.copies;
  const int half = TS * slice;
  auto place = [&](uint32_t o) {  // of byte o of a stage's K or V: boxes come swizzled
    return copies == kBoxes ? o ^ (o >> 7 & 7) << 4 : o;
  };
  int* s_nv = reinterpret_cast<int*>(smem + sh.nv_at);
  const int consumers = HG * WPH;
  if (tid == 0) {
    for (int i = 0; i < sh.stages; ++i) {
      tc::mbar_init(&bar_full[i], copies == kTokens ? 2 : copies == kLanes ? 33 : 1);
      tc::mbar_init(&bar_empty[i], consumers);
    }
    tc::mbar_init(&bar_join, consumers);
    tc::mbar_init_fence();
    s_abort = 0;
  }
  // (table, lists and queries are renewed where they are read: kept in registers from
  // here on, their addresses cost the consumers spills)
  pdl_wait(seq_lens);
  pdl_launch_dependents();

  // ---- the stages of every segment, and this CTA's run of them ----
  const int chunks = sh.NHG * sh.NRC, cta = blockIdx.x;
  auto stages_of = [&](int n) { return (n + TS - 1) >> ts_log2; };
  auto tokens_of = [&](int v) {
    int n = seq_lens[sh.lists == 1 ? v : v / sh.lists];
    if (n < 0 || n > sh.cap) {
      *err = kErrLen;
      n = 0;
    }
    if (sh.k) n = n == 0 ? 0 : sh.trim ? min(n, sh.k) : sh.k;
    s_nv[v] = n;
    return n;
  };
  if (sh.whole) {  // a CTA a segment
    const int v = cta / chunks, c = cta - v * chunks;
    if (tid == 0) {
      s_first = v;
      s_count = stages_of(tokens_of(v));
      s_rest = c * s_count;
      s_lo = 0;
    }
    __syncthreads();
    if (s_count == 0) {
      const int hg = c / sh.NRC, r0 = (c - hg * sh.NRC) * RC, rows = min(RC, sh.R - r0);
      for (int i = tid; i < HG * rows * (D / 8); i += NTHREADS) {
        const int x = i / (D / 8), h = x / rows, r = r0 + x - h * rows, qi = r / sh.G;
        const int64_t row =
            ((int64_t)v * sh.Nq + qi) * sh.Hq + (hg * HG + h) * sh.G + r - qi * sh.G;
        const int at = i - x * (D / 8);
        *reinterpret_cast<uint4*>(out + row * D + 8 * at) = make_uint4(0, 0, 0, 0);
        if (lse && at == 0) lse[row] = kNegInf;
      }
      return;
    }
  } else {
    const int per = (sh.Bv + NTHREADS - 1) / NTHREADS, v_lo = min(tid * per, sh.Bv),
              v_hi = min(v_lo + per, sh.Bv);
    int mine = 0;
    for (int v = v_lo; v < v_hi; ++v) mine += stages_of(tokens_of(v)) * chunks;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int W = 0, before = upto - mine;  // (stages before this thread's first segment)
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      const int x = s_warp[w];
      if (w < warp) before += x;
      W += x;
    }
    if (cta == 0) {
      int at = before;
      for (int v = v_lo; v < v_hi; ++v) {
        prefix[v] = at;
        at += stages_of(s_nv[v]) * chunks;
      }
      if (tid == 0) prefix[sh.Bv] = W;
    }
    const int n_ctas = min(sh.grid, W);
    if (cta >= n_ctas) return;
    const Shares shares(W, n_ctas);
    const int lo = shares.first(cta);
    if (lo >= before && lo < before + mine) {
      int rest = lo - before, v = v_lo;
      for (;; ++v) {
        const int units = stages_of(s_nv[v]) * chunks;
        if (rest < units) break;
        rest -= units;
      }
      s_first = v;
      s_rest = rest;
      s_lo = lo;
      s_count = shares.first(cta + 1) - lo;
    }
    __syncthreads();
  }
  // Waits of a warp.  Looks at the clock and at the other warps once in many polls (each of
  // which the hardware holds back): polling takes issue slots from the warps that work.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const long long t0 = clock64();  // (before the first look: a tiny limit is over behind it)
    bool there = tc::mbar_test_wait(bar, parity);
    if (!there) {
      while (!there && !*(volatile int*)&s_abort && clock64() - t0 <= wait_cycles) {
#pragma unroll 1
        for (int i = 0; i < 32 && !there; ++i) there = tc::mbar_try_wait(bar, parity);
      }
    }
    return __all_sync(0xffffffffu, there) != 0;
  };
  auto give_up = [&]() {
    if (lane == 0) {
      s_abort = 1;
      *err = kErrTimeout;
    }
  };

  if (warp >= NW) {
    // =========================== producers ===========================
    set_registers<kProducerRegisters<NT, PW, SLICE>, false>();
    behind(seq_lens, block_table, lists);
    const int me = warp - NW, count = s_count, lo = s_lo, hi = lo + count;
    int* s_row = s_row_all[me & 3];
    int v = s_first, n = s_nv[v], T = stages_of(n), c = 0, tile = s_rest;
    if (chunks > 1) {
      c = tile / T;
      tile -= c * T;
    }
    int seg_at = lo - tile;  // first stage of the segment at hand
    int request = sh.lists == 1 ? v : v / sh.lists;
    int next = 0;            // of the CTA's run, the stage that these stand at
    auto forward = [&](int step) {  // (not beyond the run's last stage)
      next += step;
      while (step >= T - tile) {
        step -= T - tile;
        tile = 0;
        seg_at += T;
        if (++c == chunks) {
          c = 0;
          do n = s_nv[++v];
          while (n == 0);
          T = stages_of(n);
          request = sh.lists == 1 ? v : v / sh.lists;
        }
      }
      tile += step;
    };
    // t / page_size by a rounded-up reciprocal, which is at most one too large
    auto page_of = [&](int t, int& slot) {
      int p = sh.page_magic ? (int)__umulhi((uint32_t)t, sh.page_magic) : t;
      slot = t - p * sh.page_size;
      if (slot < 0) {
        --p;
        slot += sh.page_size;
      }
      return p;
    };
    auto flags_of = [&](int i) -> uint32_t {
      uint32_t f = 0;
      if (tile == T - 1 || i == count - 1) f |= kLast;
      if (i == count - 1) f |= kEnd;
      if (seg_at >= lo && seg_at + T <= hi) f |= kWhole;
      if (seg_at > lo) f |= kSecond;
      if (sh.causal && ((tile + 1) << ts_log2) > n - (sh.Nq - 1 - c % sh.NRC * RC / sh.G))
        f |= kEdge;
      return f;
    };
    // a token that is not there: no weight, but what its place holds takes part in a product
    auto absent = [&](uint32_t dst_v, int at) {
      for (int h = 0; h < HG; ++h)
#pragma unroll
        for (int o = 0; o < 4 * NB; o += 8)
          sts_zero8(dst_v + place(at * slice + h * REC + D / 2 + o));
    };
    // (the stages that one warp fills are never further apart than the ring is long)
    const int stride = copies == kTokens ? PW / 2 : 4;
    const int mine_from = copies == kTokens ? me >> 1 : me;
    if (mine_from >= stride) return;
    int stage = mine_from, round = 0, i = mine_from;
    bool ok = true;
    if (i < count) forward(i);
    if (copies == kTokens) {
      // ---- a token a lane (or two), K or V ----
      constexpr int PER = 2;
      const bool is_v = me & 1;
      const uint8_t* pool = is_v ? pool_v : pool_k;
      int t[PER], page[PER], slot[PER], row[PER];
      auto tokens = [&]() {  // of the stage at hand, as positions
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int at = 32 * u + lane, p = (tile << ts_log2) + at;
          t[u] = -1;
          if (at < TS && p < n) t[u] = sh.k ? lists[(int64_t)v * sh.k + p] : p;
        }
      };
      auto pages = [&]() {
        const int* table = block_table + (int64_t)request * sh.max_pages;
        const int len = sh.k ? seq_lens[request] : 0;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          if (sh.k && t[u] != -1 && (t[u] < 0 || t[u] >= len)) {
            *err = kErrToken;
            t[u] = -1;
          }
          page[u] = t[u] < 0 ? -1 : table[page_of(t[u], slot[u])];
        }
      };
      auto rows = [&]() {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          row[u] = -1;
          if (t[u] < 0) continue;
          if (page[u] < 0 || page[u] >= sh.num_pages) *err = kErrPage;
          else row[u] = page[u] * sh.page_size + slot[u];
        }
      };
      if (i < count) {
        tokens();
        pages();
        rows();
      }
      for (; i < count; i += stride) {
        const int4 seg = make_int4(v, c, tile << ts_log2, n);
        const uint32_t f = flags_of(i);
        const bool more = i + stride < count;
        // the next stage's places are looked up while this one waits and is filled
        if (more) {
          forward(stride);
          tokens();
        }
        if (round > 0) ok = wait(&bar_empty[stage], (round & 1) ^ 1);
        if (!ok) break;
        if (more) pages();
        const uint32_t dst = ring + (uint32_t)(2 * stage + is_v) * half;
        StageNote* note = &s_note[stage];
        uint32_t here[PER];
        int present = 0;
        bool gone = false;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          here[u] = __ballot_sync(0xffffffffu, row[u] >= 0);
          present += __popc(here[u]);
          if (!is_v && lane < 2) note->mask[2 * u + lane] = (here[u] >> 16 * lane & 0xffffu) | f;
          if (is_v && row[u] < 0 && 32 * u + lane < TS) {
            absent(dst, 32 * u + lane);
            gone = true;
          }
        }
        if (gone) tc::fence_async_smem();
        if (!is_v && lane == 0) *reinterpret_cast<int4*>(note) = seg;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect(&bar_full[stage], (uint32_t)present * sh.taken);
        __syncwarp();
        const int off = seg.y / sh.NRC * HG * REC;
#pragma unroll
        for (int u = 0; u < PER; ++u)
          if (row[u] >= 0)
            bulk_load(dst + (32 * u + lane) * slice,
                      pool + (int64_t)row[u] * sh.row_bytes + off, sh.taken, &bar_full[stage]);
        if (more) rows();
        stage += stride;
        if (stage >= sh.stages) {
          stage -= sh.stages;
          ++round;
        }
      }
    } else {
      for (; i < count; i += stride) {
        if (i != next) forward(i - next);
        const int p0 = tile << ts_log2, here = min(n - p0, TS);  // tokens in reach
        const int* table = block_table + (int64_t)request * sh.max_pages;
        // ---- where the stage's tokens lie
        int run_at = 0, run = 0, run_row = -1;  // a run of tokens in one page, a lane each
        bool whole = true;                      // all in reach are there
        uint32_t full = 0;                      // boxes, and tokens in them
        auto lone = [&](bool mine, int tokens) {  // tokens of a lane's page that go one by one
          for (int at = lane; at < TS; at += 32) s_row[at] = -1;
          __syncwarp();
          if (mine)
            for (int r = 0; r < tokens; ++r) s_row[run_at + r] = run_row + r;
          __syncwarp();
        };
        if (copies == kBoxes) {
          run_at = lane * sh.box;
          const bool some = run_at < here;
          if (some) {
            int slot;
            const int page = table[page_of(p0 + run_at, slot)];
            if (page < 0 || page >= sh.num_pages) *err = kErrPage;
            else run_row = page * sh.page_size + slot;
          }
          const bool boxed = run_row >= 0 && run_at + sh.box <= here;
          full = __ballot_sync(0xffffffffu, boxed);
          whole = __all_sync(0xffffffffu, boxed || run_at >= TS);
          if (!whole) lone(run_row >= 0 && !boxed, here - run_at);
        } else if (copies == kRuns) {
          int slot;
          const int page0 = page_of(p0, slot);
          run_at = lane == 0 ? 0 : lane * sh.page_size - slot;
          if (run_at < here) {
            const int page = table[page0 + lane];
            if (page < 0 || page >= sh.num_pages) {
              *err = kErrPage;
            } else {
              run = min((lane + 1) * sh.page_size - slot, here) - run_at;
              run_row = page * sh.page_size + (lane == 0 ? slot : 0);
            }
          }
          whole = __all_sync(0xffffffffu, run_at >= here || run_row >= 0);
          if (!whole) lone(true, run);  // (told apart below)
        } else {
          const int len = sh.k ? seq_lens[request] : 0;
          for (int at0 = 0; at0 < TS; at0 += 128) {  // (four tokens a lane at once)
            int t[4], page[4], slot[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int at = at0 + 32 * u + lane;
              t[u] = at >= here ? -1 : sh.k ? lists[(int64_t)v * sh.k + p0 + at] : p0 + at;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (sh.k && t[u] != -1 && (t[u] < 0 || t[u] >= len)) {
                *err = kErrToken;
                t[u] = -1;
              }
              page[u] = t[u] < 0 ? -1 : table[page_of(t[u], slot[u])];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int at = at0 + 32 * u + lane;
              int row = -1;
              if (t[u] >= 0) {
                if (page[u] < 0 || page[u] >= sh.num_pages) *err = kErrPage;
                else row = page[u] * sh.page_size + slot[u];
              }
              if (at < TS) s_row[at] = row;
            }
          }
          __syncwarp();
          whole = false;
        }
        // ---- fill it
        if (round > 0) ok = wait(&bar_empty[stage], (round & 1) ^ 1);
        if (!ok) break;
        const uint32_t dst_k = ring + (uint32_t)stage * 2 * half, dst_v = dst_k + half;
        StageNote* note = &s_note[stage];
        const uint32_t f = flags_of(i);
        int present = here;
        bool gone = false;
        if (whole) {
          if (lane < 16) note->mask[lane] = ((1u << min(max(here - 16 * lane, 0), 16)) - 1) | f;
          for (int at = here + lane; at < TS; at += 32) {
            absent(dst_v, at);
            gone = true;
          }
        } else {
          present = 0;
          for (int at0 = 0; at0 < TS; at0 += 32) {
            const int at = at0 + lane;
            const bool there =
                at < TS && (s_row[at] >= 0 || (copies == kBoxes && full >> at / sh.box & 1));
            const uint32_t m = __ballot_sync(0xffffffffu, there);
            if (lane < 2) note->mask[at0 / 16 + lane] = (m >> 16 * lane & 0xffffu) | f;
            present += __popc(m);
            if (at < TS && !there) {
              absent(dst_v, at);
              gone = true;
            }
          }
        }
        if (gone) tc::fence_async_smem();
        if (lane == 0) *reinterpret_cast<int4*>(note) = make_int4(v, c, p0, n);
        __syncwarp();
        if (copies == kRuns) {
          if (lane == 0) tc::mbar_arrive_expect(&bar_full[stage], 2u * present * slice);
          __syncwarp();
          if (run > 0) {
            const int64_t src = (int64_t)run_row * sh.row_bytes;
            const uint32_t o = run_at * slice;
            bulk_load(dst_k + o, pool_k + src, run * slice, &bar_full[stage]);
            bulk_load(dst_v + o, pool_v + src, run * slice, &bar_full[stage]);
          }
        } else if (copies == kLanes || !whole) {
          // `lanes` lanes a token, each with a unit or two of it; some tokens at once
          constexpr int U = 4;
          const int ln = sh.lanes, tok = lane / ln, unit = lane & (ln - 1), step = 32 / ln;
          const int cpt = sh.taken / sh.unit;
          const uint32_t o0 = unit * sh.unit, o1 = (unit + ln) * sh.unit;
          const bool on0 = unit < cpt, on1 = unit + ln < cpt;
          const int64_t to_v = pool_v - pool_k;
          const uint8_t* part = pool_k + c / sh.NRC * HG * REC;
#pragma unroll 1
          for (int at0 = tok; at0 < TS; at0 += step * U) {
            int row[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int at = at0 + u * step;
              row[u] = at < TS ? s_row[at] : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (row[u] < 0) continue;
              const uint8_t* src = part + (int64_t)row[u] * sh.row_bytes;
              auto copy = [&](uint32_t o) {
                const uint32_t to = dst_k + place((at0 + u * step) * slice + o);
                if (sh.unit == 16) {
                  tc::cp_async16(to, src + o, 16);
                  tc::cp_async16(to + half, src + to_v + o, 16);
                } else {
                  cp_async8(to, src + o);
                  cp_async8(to + half, src + to_v + o);
                }
              };
              if (on0) copy(o0);
              if (on1) copy(o1);
            }
          }
          if (copies == kLanes) {
            __syncwarp();  // (all lanes have read the rows that the next stage overwrites)
            tc::cp_async_arrive(&bar_full[stage]);
            if (lane == 0) tc::mbar_arrive(&bar_full[stage]);
          } else {  // (the end of a request: these copies land before the boxes are announced)
            tc::cp_async_commit();
            tc::cp_async_wait<0>();
            __syncwarp();
          }
        }
        if (copies == kBoxes) {
          if (lane == 0)
            tc::mbar_arrive_expect(&bar_full[stage], 2u * __popc(full) * sh.box * slice);
          __syncwarp();
          if (full >> lane & 1) {
            const uint32_t o = run_at * slice;
            const int line = c / sh.NRC * (slice / 128);
            tc::tma_load_3d(dst_k + o, &map_k, 0, line, run_row, &bar_full[stage]);
            tc::tma_load_3d(dst_v + o, &map_v, 0, line, run_row, &bar_full[stage]);
          }
        }
        stage += stride;
        if (stage >= sh.stages) {
          stage -= sh.stages;
          ++round;
        }
      }
    }
    if (!ok) give_up();
    // this warp's copies in flight land before the CTA gives its memory up, whoever gave up
    for (int j = i - stride; j >= 0 && j >= i - sh.stages; j -= stride) {
      const int r = j / sh.stages;
      const long long t0 = clock64();
      while (!tc::mbar_try_wait(&bar_full[j - r * sh.stages], r & 1) &&
             clock64() - t0 < kLandCycles) {
      }
    }
    return;
  }

  // =========================== consumers ===========================
  set_registers<kConsumerRegisters<NT, PW, SLICE>, true>();
  if (warp >= consumers) return;
  const int h = warp / WPH, sub = warp - h * WPH;
  const int g = lane >> 2, t = lane & 3;
  auto token = [&](int r) { return (int)(sh.order >> (4 * r) & 15); };
  auto at = [&](int tok, int off) -> uint32_t {  // (16 tokens on, a box is swizzled alike)
    return sub * TT * 16 * slice + place(tok * slice + h * REC + off);
  };
  // rows g and g + 8 of the tokens' tiles; K codes and pairs
  const int tok0 = token(g), tok1 = token(g + 8);
  uint32_t k_code0 = at(tok0, 4 * NB * t), k_code1 = at(tok1, 4 * NB * t);
  uint32_t k_pair0 = at(tok0, D / 2), k_pair1 = at(tok1, D / 2);
  // tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the tile's order; V codes and pairs
  uint32_t v_code[4], v_pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = token(2 * t + (i & 1) + 8 * (i >> 1));
    v_code[i] = half + at(tok, 2 * NB * g);
    v_pair[i] = half + at(tok, D / 2);
  }
  // (kept, not worked out again for every tile)
  asm volatile("" : "+r"(k_code0), "+r"(k_code1), "+r"(k_pair0), "+r"(k_pair1), "+r"(v_code[0]),
               "+r"(v_code[1]), "+r"(v_code[2]), "+r"(v_code[3]));
  asm volatile("" : "+r"(v_pair[0]), "+r"(v_pair[1]), "+r"(v_pair[2]), "+r"(v_pair[3]));
  const int m_word = 4 * (g & (NB - 1));

  // queries as B operands, in shared memory where registers are short; the pieces of their sums
  constexpr bool QSHARED = NT * TT == 4, TWICE = FIXED && !QSHARED;
  uint32_t qf[QSHARED ? 1 : NT][NB][4], qs[NT][NB];
  uint4* q_shared = reinterpret_cast<uint4*>(smem + sh.q_at) + warp * NT * NB * 32 + lane;
  // of columns 2t, 2t + 1: scale of the scores, minus the reference, sum of weights
  float cs[NT][2], nref[NT][2], sum[NT][2];
  float o[NT][NB][2][4], om[NT][2];
  float limit = kAlways;  // of the scores, above which a stage is looked at more closely
  int stage = 0;
  uint32_t phase = 0, join_phase = 0;
  bool ok = true;
  auto join = [&]() {  // of the consumer warps
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bar_join);
    ok = ok && wait(&bar_join, join_phase);
    join_phase ^= 1;
  };

  bool ready = false;  // the stage at hand has landed
  int q_v = s_first, q_c = 0;  // the segment whose queries are to be read next
  if (chunks > 1) q_c = s_rest / stages_of(s_nv[q_v]);
  bool fresh = true;
  uint32_t flags = 0;
  do {
    if (__builtin_expect(fresh, 0)) {
      // ---------------- the segment's queries (while its tokens are on their way) ------
      fresh = false;
      limit = kAlways;
      __syncwarp();
      if (lane == 0) s_units[warp] = kUsual | (s_nv[q_v] > kLongSegment ? kLong | kAgain : 0);
      __syncwarp();
      const int hg = q_c / sh.NRC, rc = q_c - hg * sh.NRC;
      const int head = hg * HG + h;
      const __nv_bfloat16* from = q;
      behind(from);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = rc * RC + nt * 8 + g;
        float x[NB][8];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[b][e] = 0.f;
        if (r < sh.R) {
          const int qi = r / sh.G;
          const int64_t row =
              ((int64_t)q_v * sh.Nq + qi) * sh.Hq + head * sh.G + r - qi * sh.G;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 y = *reinterpret_cast<const uint4*>(from + row * D + 32 * b + 8 * t);
            const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[b][2 * e] = __uint_as_float(u[e] << 16);
              x[b][2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
          }
        }
        float big = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[b][e]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // the row times 2^p, here its largest value in [2^120, 2^121) (or below, from 2^-126 on)
        const int e2 = max((int)(__float_as_uint(big) >> 23) - 127, -126);
        const int p = 120 - e2;
        const float f1 = __int_as_float((127 + (p >> 1)) << 23);
        const float f2 = __int_as_float((127 + p - (p >> 1)) << 23);
        uint32_t piece[NB];  // of the sums: a lane's, by t
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[b][e] = x[b][e] * f1 * f2;
            s += x[b][e];
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          // values i and i + 4 of a word stand in one register; the odd ones come out of it
          // 16 times too large.  Up to [2^127, 2^128)
          auto two = [&](int i, float f) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[b][i] * f, x[b][i + 4] * f);
            return *reinterpret_cast<const uint32_t*>(&y);
          };
          const uint4 qb = make_uint4(two(0, 128.f), two(1, 8.f), two(2, 128.f), two(3, 8.f));
          if constexpr (QSHARED) {
            q_shared[(nt * NB + b) * 32] = qb;
          } else {
            qf[nt][b][0] = qb.x, qf[nt][b][1] = qb.y, qf[nt][b][2] = qb.z, qf[nt][b][3] = qb.w;
          }
          // the sum in the unit of the codes' products, 2^(p + 7 - 133): at most 1, in
          // pieces of 11 bits
          const float y = s * __int_as_float(1 << 23);  // 2^-126
          const __half h0 = __float2half_rn(y);
          const float r1 = y - __half2float(h0);
          const __half h1 = __float2half_rn(r1);
          const __half h2 = __float2half_rn(r1 - __half2float(h1));
          piece[b] = t == 3 ? 0 : __half_as_ushort(t == 0 ? h0 : t == 1 ? h1 : h2);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) qs[nt][b] = piece[b] << 16;
        // scores in powers of two; never 0 or infinite, so that a product with it is a number
        // where a score is 0 and minus infinity where a token does not count (a score times
        // 2^-126 is nothing beside the others)
        const int c2 = 6 + e2;
        const float c = scale_log2 * __int_as_float((127 + (c2 >> 1)) << 23) *
                        __int_as_float((127 + c2 - (c2 >> 1)) << 23);
        const float mine_c = fminf(fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          cs[nt][j] = __shfl_sync(0xffffffffu, mine_c, (2 * t + j) * 4);
          nref[nt][j] = -kNone;
          sum[nt][j] = om[nt][j] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[nt][b][e >> 2][e & 3] = 0.f;
      }
    }
    if (!ready) ok = wait(&bar_full[stage], phase);
    if (!ok) break;
    // ---------------- all of the stage that this warp needs, and on with the ring ----------
    const StageNote* note = &s_note[stage];
    uint32_t mask[TT];
#pragma unroll
    for (int u = 0; u < TT; ++u) mask[u] = note->mask[sub * TT + u];
    flags = mask[0];
    const int4 seg = *reinterpret_cast<const int4*>(note);  // v, c, p0, nv
    uint32_t k0[TT][NB], k1[TT][NB], kp0[TT][NB], kp1[TT][NB];
    uint32_t w[TT][4][NB / 2], s01[TT][NB], s23[TT][NB], ma0[TT], ma2[TT];
    const uint8_t* base = smem + (uint32_t)stage * 2 * half;
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const uint8_t* from = base + u * 16 * slice;
      lds(from + k_code0, k0[u]);
      lds(from + k_code1, k1[u]);
      lds(from + k_pair0, kp0[u]);
      lds(from + k_pair1, kp1[u]);
    }
    auto load_v = [&]() {
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const uint8_t* from = base + u * 16 * slice;
        uint32_t x[4][NB], m[4][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lds(from + v_pair[i], x[i]);
          lds(from + v_pair[i] + m_word, m[i]);
          lds(from + v_code[i], w[u][i]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          s01[u][b] = __byte_perm(x[0][b], x[1][b], 0x5410);
          s23[u][b] = __byte_perm(x[2][b], x[3][b], 0x5410);
        }
        ma0[u] = __byte_perm(m[0][0], m[1][0], 0x7632);
        ma2[u] = __byte_perm(m[2][0], m[3][0], 0x7632);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_empty[stage]);
      if (++stage == sh.stages) {
        stage = 0;
        phase ^= 1;
        if (phase) limit = kAlways;
      }
    };
    if constexpr (!QSHARED) load_v();  // (early, but where registers are short)
    // ---------------- scores ----------------
    float tot[TT][NT][4];
#pragma unroll
    for (int u = 0; u < TT; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16(tot[u][nt], kp0[u][0], kp1[u][0], kp0[u][1], kp1[u][1], qs[nt][0], qs[nt][1]);
        if constexpr (NB == 4)
          mma_f16_add(tot[u][nt], kp0[u][2], kp1[u][2], kp0[u][3], kp1[u][3], qs[nt][2], qs[nt][3]);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint4 qb[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (QSHARED) qb[nt] = q_shared[(nt * NB + b) * 32];
        else qb[nt] = make_uint4(qf[nt][b][0], qf[nt][b][1], qf[nt][b][2], qf[nt][b][3]);
      }
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const uint32_t x0 = k0[u][b], x1 = k1[u][b], y0 = x0 >> 8, y1 = x1 >> 8;
        const float s0 = low_half(kp0[u][b]), s1 = low_half(kp1[u][b]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4];
          mma_bf16(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u,
                   qb[nt].x, qb[nt].y);
          mma_bf16_add(acc, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u,
                       y1 & 0x00f000f0u, qb[nt].z, qb[nt].w);
          tot[u][nt][0] = fmaf(acc[0], s0, tot[u][nt][0]);
          tot[u][nt][1] = fmaf(acc[1], s0, tot[u][nt][1]);
          tot[u][nt][2] = fmaf(acc[2], s1, tot[u][nt][2]);
          tot[u][nt][3] = fmaf(acc[3], s1, tot[u][nt][3]);
        }
      }
    }
    if constexpr (QSHARED) load_v();
    // ---------------- weights ----------------
    // As if all tokens counted, no reference had to move and all scales had their usual size,
    // unless a closer look says otherwise, which is rare.
    float x[TT][NT][4], p[TT][NT][4];
    uint32_t pt0[TT][NT], pt1[TT][NT];
    auto exponents = [&]() {
#pragma unroll
      for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          fma2(x[u][nt][0], x[u][nt][1], tot[u][nt][0], tot[u][nt][1], cs[nt][0], cs[nt][1],
               nref[nt][0], nref[nt][1]);
          fma2(x[u][nt][2], x[u][nt][3], tot[u][nt][2], tot[u][nt][3], cs[nt][0], cs[nt][1],
               nref[nt][0], nref[nt][1]);
        }
    };
    auto weights = [&]() {
#pragma unroll
      for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) p[u][nt][e] = ex2(x[u][nt][e]);
          pt0[u][nt] = movmatrix_t(half2_bits(__floats2half2_rn(p[u][nt][0], p[u][nt][1])));
          pt1[u][nt] = movmatrix_t(half2_bits(__floats2half2_rn(p[u][nt][2], p[u][nt][3])));
        }
    };
    exponents();
    float x_top = kNegInf;
    uint32_t any = 0, all = 0xffffu;
#pragma unroll
    for (int u = 0; u < TT; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        x_top = fmaxf(fmaxf(x_top, fmaxf(x[u][nt][0], x[u][nt][1])),
                      fmaxf(x[u][nt][2], x[u][nt][3]));
      all &= mask[u];
    }
#pragma unroll
    for (int u = 0; u < TT; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) any |= s01[u][b] | s23[u][b];
    const bool look = __any_sync(0xffffffffu, !(x_top <= limit) || (any & 0x40004000u)) ||
                      all != 0xffffu || (flags & kEdge);
    if (__builtin_expect(look, 0)) {
      bool rescale;
      const bool redo = __any_sync(0xffffffffu, x_top > kTop) || all != 0xffffu || (flags & kEdge);
      const uint32_t units = s_units[warp];
      limit = kTop;
      if (units == kUsual || (units & kAgain) || (stage == 0 && phase)) {
        // (one of these bits is set from 2^-kSmall on, or 2^-kSmallShort)
        const uint32_t least = seg.w > kShortSegment ? 0x60006000u : 0x70007000u;
        bool unusual = any & 0x40004000u;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t y = 0;
#pragma unroll
          for (int u = 0; u < TT; ++u) y |= s01[u][b] | s23[u][b];
          unusual |= !(y & least) && (y || all == 0xffffu);  // (0: of tokens that are not there)
        }
        rescale = __any_sync(0xffffffffu, unusual) || units != kUsual;
        if (all != 0xffffu) limit = kAlways;  // (few tokens say little about those to come)
      } else {  // in the units at hand, if nothing is too large for them
        uint32_t f[NB];
        lds(reinterpret_cast<const uint8_t*>(s_by_unit[warp]), f);
        bool over = false;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t top = 0;
#pragma unroll
          for (int u = 0; u < TT; ++u) top = __vmaxu2(top, __vmaxu2(s01[u][b], s23[u][b]));
          over |= __vcmpgeu2(top, 0x7c007c00u - f[b]) != 0;
        }
        rescale = __any_sync(0xffffffffu, over);
        if (!rescale) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < TT; ++u) {
              s01[u][b] = half2_bits(__hmul2(bits_half2(s01[u][b]), bits_half2(f[b])));
              s23[u][b] = half2_bits(__hmul2(bits_half2(s23[u][b]), bits_half2(f[b])));
            }
          limit = kAlways;
        }
      }
      if (rescale) {
        const uint32_t units = s_units[warp];
        const int least = seg.w > kShortSegment ? -kSmall : -kSmallShort;
        uint32_t now = units & kLong;
        if constexpr (NB == 2) now |= kUsual & 0xffff0000u;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t top = 0;
#pragma unroll
          for (int u = 0; u < TT; ++u)
            top = __vmaxu2(top, __vmaxu2(finite(s01[u][b]), finite(s23[u][b])));
          top = max(top >> 16, top & 0xffffu);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int was = unit_of(units, b);
          const int e = max((int)(__float_as_uint(low_half(top)) >> 23) - 127, -15);
          int sx = e;
          if (e <= was && e >= was - kKeep) sx = was;
          else if (e <= 0 && e >= least && !(units & kLong)) sx = 0;
          now |= (uint32_t)(32 + sx) << 8 * b;
          if (sx != was) {
            const float f = __int_as_float((127 + was - sx) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 8; ++i) o[nt][b][i >> 2][i & 3] *= f;
            if (sx > was) now |= kAgain;  // (a single large one does not set the unit for long)
          }
          const uint32_t f = sx == 15 ? 0x02000200u : (uint32_t)(15 - sx) * 0x04000400u;
          if (lane == 0) s_by_unit[warp][b] = f;
#pragma unroll
          for (int u = 0; u < TT; ++u) {
            s01[u][b] = half2_bits(__hmul2(bits_half2(s01[u][b]), bits_half2(f)));
            s23[u][b] = half2_bits(__hmul2(bits_half2(s23[u][b]), bits_half2(f)));
          }
        }
        __syncwarp();
        if (lane == 0) s_units[warp] = now;
        __syncwarp();
        if (now != kUsual) limit = kAlways;
      }
      if (redo) {
        // tokens that are not there, or beyond a query's limit
        const int left = seg.w - sh.Nq + 1 - seg.z - sub * TT * 16;  // of the first query's
        const int first = seg.y % sh.NRC * RC + 2 * t;
#pragma unroll
        for (int u = 0; u < TT; ++u) {
          const bool on0 = mask[u] >> tok0 & 1, on1 = mask[u] >> tok1 & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int lim =
                  (flags & kEdge ? left + min((first + nt * 8 + j) / sh.G, sh.Nq - 1) : 16 * TT) -
                  16 * u;
              if (!on0 || tok0 >= lim) tot[u][nt][j] = kNegInf;
              if (!on1 || tok1 >= lim) tot[u][nt][2 + j] = kNegInf;
            }
        }
        // at an edge, an s or m that is not finite must not reach the queries that do not see its
        // token: it goes straight to the sums of those that do
        uint32_t bad_m = 0;
#pragma unroll
        for (int u = 0; u < TT; ++u) bad_m |= infinite(ma0[u]) | infinite(ma2[u]);
        if (flags & kEdge && __any_sync(0xffffffffu, (any & 0x40004000u) | bad_m)) {
          uint32_t hit[NT] = {};  // by groups, for column g
#pragma unroll
          for (int u = 0; u < TT; ++u) {
            uint32_t seen0[NT], seen1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              auto seen = [&](int e) {
                return movmatrix_t((tot[u][nt][e] == kNegInf ? 0u : 0xffffu) |
                                   (tot[u][nt][e + 1] == kNegInf ? 0u : 0xffff0000u));
              };
              seen0[nt] = seen(0);
              seen1[nt] = seen(2);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {  // (the lanes of row b have its m)
              const uint32_t bad0 = infinite(s01[u][b]) |
                                    infinite(__shfl_sync(0xffffffffu, ma0[u], 4 * b + t));
              const uint32_t bad1 = infinite(s23[u][b]) |
                                    infinite(__shfl_sync(0xffffffffu, ma2[u], 4 * b + t));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if ((seen0[nt] & bad0) | (seen1[nt] & bad1)) hit[nt] |= 1u << b;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            hit[nt] |= __shfl_xor_sync(0xffffffffu, hit[nt], 1);
            hit[nt] |= __shfl_xor_sync(0xffffffffu, hit[nt], 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t mine = __shfl_sync(0xffffffffu, hit[nt], (2 * t + j) * 4);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                if (mine >> b & 1)
#pragma unroll
                  for (int m = 0; m < 2; ++m)
                    o[nt][b][m][j] = o[nt][b][m][2 + j] = __int_as_float(0x7fc00000);
            }
          }
#pragma unroll
          for (int u = 0; u < TT; ++u) {
            ma0[u] &= ~infinite(ma0[u]);
            ma2[u] &= ~infinite(ma2[u]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              s01[u][b] &= ~infinite(s01[u][b]);
              s23[u][b] &= ~infinite(s23[u][b]);
            }
          }
        }
        // the references, in reach of the largest score
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = kNegInf;
#pragma unroll
            for (int u = 0; u < TT; ++u) top = fmaxf(top, fmaxf(tot[u][nt][j], tot[u][nt][2 + j]));
            top *= cs[nt][j];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float was = nref[nt][j];
            if (top + nref[nt][j] > kTop) nref[nt][j] = kTop - 3.f - top;
            const float f = ex2(nref[nt][j] - was);
            sum[nt][j] *= f;
            om[nt][j] *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                o[nt][b][m][j] *= f;
                o[nt][b][m][2 + j] *= f;
              }
          }
        exponents();
      }
      if constexpr (TWICE) weights();
    } else {
      // (a second copy: one for both 1860 cycles a stage instead of 1750; with sixteen rows, and
      // with distances that are not known, two cost more, 2900 for 2780)
      if constexpr (TWICE) weights();
    }
    if constexpr (!TWICE) weights();
    ready = __all_sync(0xffffffffu, tc::mbar_test_wait(&bar_full[stage], phase)) != 0;
    // ---------------- values ----------------
    // The products start from zero every time and are added on their own: the tensor
    // core cuts off what lies below the accumulator's last place, and both sums grow
    // to many times their difference (131,072 tokens: 0.017 of the result's norm
    // instead of 0.0018).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float acc[4];
      mma_f16(acc, ma0[0], 0u, ma2[0], 0u, pt0[0][nt], pt1[0][nt]);
#pragma unroll
      for (int u = 1; u < TT; ++u)
        mma_f16_add(acc, ma0[u], 0u, ma2[u], 0u, pt0[u][nt], pt1[u][nt]);
      add2(om[nt][0], om[nt][1], acc[0], acc[1]);
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        add2(sum[nt][0], sum[nt][1], p[u][nt][0], p[u][nt][1]);
        add2(sum[nt][0], sum[nt][1], p[u][nt][2], p[u][nt][3]);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float acc[NT][2][4];
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const uint32_t sel = b & 1 ? 0x7632 : 0x5410;
        const uint32_t x01 = __byte_perm(w[u][0][b / 2], w[u][1][b / 2], sel);
        const uint32_t x23 = __byte_perm(w[u][2][b / 2], w[u][3][b / 2], sel);
        const uint32_t y01 = __byte_perm(x01, 0, 0x4341), y23 = __byte_perm(x23, 0, 0x4341);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = half2_bits(__hmul2(bits_half2(pt0[u][nt]), bits_half2(s01[u][b])));
          const uint32_t b1 = half2_bits(__hmul2(bits_half2(pt1[u][nt]), bits_half2(s23[u][b])));
          if (u == 0) {
            mma_f16(acc[nt][0], x01 & 0x000f000fu, x01 & 0x00f000f0u, x23 & 0x000f000fu,
                    x23 & 0x00f000f0u, b0, b1);
            mma_f16(acc[nt][1], y01 & 0x000f000fu, y01, y23 & 0x000f000fu, y23, b0, b1);
          } else {
            mma_f16_add(acc[nt][0], x01 & 0x000f000fu, x01 & 0x00f000f0u, x23 & 0x000f000fu,
                        x23 & 0x00f000f0u, b0, b1);
            mma_f16_add(acc[nt][1], y01 & 0x000f000fu, y01, y23 & 0x000f000fu, y23, b0, b1);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          add2(o[nt][b][m][0], o[nt][b][m][1], acc[nt][m][0], acc[nt][m][1]);
          add2(o[nt][b][m][2], o[nt][b][m][3], acc[nt][m][2], acc[nt][m][3]);
        }
    }
    if (__builtin_expect(!(flags & kLast), 1)) continue;

    fresh = !(flags & kEnd);
    if (fresh) {
      q_v = seg.x;
      q_c = seg.y + 1;
      if (q_c == chunks) {
        q_c = 0;
        do ++q_v;
        while (s_nv[q_v] == 0);
      }
    }

    // ---------------- end of the segment, or of the CTA's part of it ----------------
    const int hg = seg.y / sh.NRC, rc = seg.y - hg * sh.NRC, head = hg * HG + h;
    const uint32_t units = s_units[warp];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          sum[nt][j] += __shfl_xor_sync(0xffffffffu, sum[nt][j], d);
      }
      // the codes' units, 2^-24 and (values 1 and 3 of four) 2^-20, value 3 without value 2,
      // which its byte held too; plus sum p m
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float unit = __int_as_float((127 + 24 + unit_of(units, b)) << 23);
        const float m0 = __shfl_sync(0xffffffffu, om[nt][0], 4 * b + t);
        const float m1 = __shfl_sync(0xffffffffu, om[nt][1], 4 * b + t);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m) {
            o[nt][b][m][2] -= o[nt][b][m][0];
            o[nt][b][m][3] -= o[nt][b][m][1];
          }
          o[nt][b][m][0] = fmaf(o[nt][b][m][0], unit, m0);
          o[nt][b][m][1] = fmaf(o[nt][b][m][1], unit, m1);
          o[nt][b][m][2] = fmaf(o[nt][b][m][2], 0.0625f * unit, m0);
          o[nt][b][m][3] = fmaf(o[nt][b][m][3], 0.0625f * unit, m1);
        }
      }
    }
    // the head's warps, pairwise through shared memory
    constexpr int PER = NT * (8 * NB + 4);  // floats a lane: accumulators, sums, references
    for (int d = 1; d < WPH && ok; d <<= 1) {
      const int pairs = WPH / 2;
      float* slot = reinterpret_cast<float*>(smem + sh.scratch_at) +
                    (size_t)(h * pairs + sub / (2 * d)) * PER * 32 + lane;
      if (sub % (2 * d) == d) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float* p = slot + nt * (8 * NB + 4) * 32;
#pragma unroll
          for (int i = 0; i < 8 * NB; ++i) p[i * 32] = o[nt][i >> 3][i >> 2 & 1][i & 3];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[(8 * NB + j) * 32] = sum[nt][j];
            p[(8 * NB + 2 + j) * 32] = nref[nt][j];
          }
        }
      }
      join();
      if (ok && sub % (2 * d) == 0 && sub + d < WPH) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float* p = slot + nt * (8 * NB + 4) * 32;
          float fa[2], fb[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float other = p[(8 * NB + 2 + j) * 32], low = fminf(nref[nt][j], other);
            fa[j] = ex2(low - nref[nt][j]);
            fb[j] = ex2(low - other);
            nref[nt][j] = low;
            sum[nt][j] = sum[nt][j] * fa[j] + p[(8 * NB + j) * 32] * fb[j];
          }
#pragma unroll
          for (int i = 0; i < 8 * NB; ++i) {
            float& a = o[nt][i >> 3][i >> 2 & 1][i & 3];
            a = a * fa[i & 1] + p[i * 32] * fb[i & 1];
          }
        }
      }
      join();
    }
    if (!ok) break;
    if (sub != 0) continue;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = nt * 8 + 2 * t + j, r = rc * RC + col;
        if (r >= sh.R) continue;
        if (flags & kWhole) {
          const int i = r / sh.G;
          const int64_t row = ((int64_t)seg.x * sh.Nq + i) * sh.Hq + head * sh.G + r - i * sh.G;
          const float l = sum[nt][j];
          const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const __nv_bfloat162 a =
                __floats2bfloat162_rn(o[nt][b][0][j] * f, o[nt][b][0][2 + j] * f);
            const __nv_bfloat162 c =
                __floats2bfloat162_rn(o[nt][b][1][j] * f, o[nt][b][1][2 + j] * f);
            *reinterpret_cast<uint2*>(out + row * D + 32 * b + 4 * g) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                           *reinterpret_cast<const uint32_t*>(&c));
          }
          if (lse && g == 0)
            lse[row] = l == 0.f ? kNegInf : (log2f(l) - nref[nt][j]) * 0.6931471805599453f;
        } else {
          const int64_t slot = ((int64_t)2 * cta + (flags & kSecond ? 1 : 0)) * HG * RC +
                               h * RC + col;
          if (g == 0) part_ml[slot] = make_float2(-nref[nt][j], sum[nt][j]);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            *reinterpret_cast<float4*>(part_o + slot * D + 32 * b + 4 * g) =
                make_float4(o[nt][b][0][j], o[nt][b][0][2 + j], o[nt][b][1][j],
                            o[nt][b][1][2 + j]);
        }
      }
  } while (!(flags & kEnd));
  if (!ok) give_up();
}

// Rows whose segment several CTAs hold: sum the parts by the definition of the
// softmax over a partition, w = 2^(reference - largest).  WARPS warps a row, each
// taking every WARPS-th part.  Rows without tokens get zeros.
template <int D, int WARPS>
__global__ void __launch_bounds__(256)
k_q4_merge(const int32_t* __restrict__ prefix, const float2* __restrict__ part_ml,
           const float* __restrict__ part_o, __nv_bfloat16* __restrict__ out,
           float* __restrict__ lse, const Q4Shape sh, int RC) {
  constexpr int PL = D / 32;  // values a lane
  __shared__ float s_o[WARPS > 1 ? 8 : 1][D];
  __shared__ float2 s_ml[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = WARPS > 1 ? warp : 0;
  pdl_wait(prefix, part_ml, part_o, out, lse);
  pdl_launch_dependents();
  const int64_t row = WARPS > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
  if (row >= (int64_t)sh.Bv * sh.Nq * sh.Hq) return;  // (whole blocks where WARPS > 1)
  const int64_t v = row / ((int64_t)sh.Nq * sh.Hq);
  const int in = (int)(row - v * sh.Nq * sh.Hq), i = in / sh.Hq, hq = in - i * sh.Hq;
  const int head = hq / sh.G, r = i * sh.G + hq - head * sh.G;
  const int hg = head / sh.HG, h = head - hg * sh.HG, rc = r / RC, col = r - rc * RC;
  const int W = prefix[sh.Bv], p0 = prefix[v], units = prefix[v + 1] - p0;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float ref = kNone, l = 0.f;
  bool write = units == 0;
  if (units > 0) {
    const int T = units / (sh.NHG * sh.NRC), s0 = p0 + (hg * sh.NRC + rc) * T, s1 = s0 + T;
    const Shares shares(W, min(sh.grid, W));
    const int first = shares.holder(s0), last = shares.holder(s1 - 1);
    write = first != last;
    if (write) {
      for (int c = first + w; c <= last; c += WARPS) {
        const int second = c == first && shares.first(c) < s0 ? 1 : 0;
        const int64_t slot = ((int64_t)2 * c + second) * sh.HG * RC + h * RC + col;
        const float2 ml = part_ml[slot];
        float4 x;
        if constexpr (PL == 4) {
          x = *reinterpret_cast<const float4*>(part_o + slot * D + 4 * lane);
        } else {
          const float2 y = *reinterpret_cast<const float2*>(part_o + slot * D + 2 * lane);
          x = make_float4(y.x, y.y, 0.f, 0.f);
        }
        const float top = fmaxf(ref, ml.x), fa = ex2(ref - top), fb = ex2(ml.x - top);
        ref = top;
        l = l * fa + ml.y * fb;
        acc.x = acc.x * fa + x.x * fb;
        acc.y = acc.y * fa + x.y * fb;
        acc.z = acc.z * fa + x.z * fb;
        acc.w = acc.w * fa + x.w * fb;
      }
    }
  }
  if (!write) return;
  if constexpr (WARPS > 1) {
    if (lane == 0) s_ml[warp] = make_float2(ref, l);
    if constexpr (PL == 4) *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
    else *reinterpret_cast<float2*>(&s_o[warp][2 * lane]) = make_float2(acc.x, acc.y);
    __syncthreads();
    if (warp != 0) return;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    ref = kNone;
    l = 0.f;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) ref = fmaxf(ref, s_ml[u].x);
#pragma unroll
    for (int u = 0; u < WARPS; ++u) {
      const float f = ex2(s_ml[u].x - ref);
      l += s_ml[u].y * f;
      acc.x += s_o[u][PL * lane] * f;
      acc.y += s_o[u][PL * lane + 1] * f;
      if constexpr (PL == 4) {
        acc.z += s_o[u][PL * lane + 2] * f;
        acc.w += s_o[u][PL * lane + 3] * f;
      }
    }
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * f, acc.y * f);
  __nv_bfloat16* to = out + row * D + PL * lane;
  if constexpr (PL == 4) {
    const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                               *reinterpret_cast<const uint32_t*>(&c));
  } else {
    *reinterpret_cast<__nv_bfloat162*>(to) = a;
  }
  if (lse && lane == 0)
    lse[row] = l == 0.f ? __int_as_float(0xff800000) : (ref + log2f(l)) * 0.6931471805599453f;
}

// Heads of a CTA: all of them, or the largest divisor that the warps can take
int heads_of(int hkv) {
  if (hkv <= kConsumers) return hkv;
  int d = kConsumers;
  while (hkv % d) --d;
  return d;
}

struct Config {
  Q4Shape sh;
  int NT, PW;
  bool fixed;  // SLICE is slice
  size_t smem;
};

Config configure(const pks_q4_attention_args& a) {
  Config cf{};
  Q4Shape& sh = cf.sh;
  const int nq = a.n_queries > 1 ? a.n_queries : 1;
  sh.lists = a.k ? nq : 1;
  sh.Bv = a.B * sh.lists;
  sh.Nq = a.k ? 1 : nq;
  sh.Hq = a.Hq;
  sh.G = a.Hq / a.Hkv;
  sh.page_size = a.page_size;
  sh.max_pages = a.max_pages;
  sh.num_pages = a.num_pages;
  sh.k = a.k;
  sh.trim = a.trim;
  sh.causal = a.k ? 0 : a.causal;
  sh.R = sh.Nq * sh.G;
  // eight query rows at a time, or sixteen
  cf.NT = sh.R > 8 ? 2 : 1;
  const int hg = heads_of(a.Hkv);
  const bool fixed = a.D == 128 && hg == 8;
  // tokens 32 at a time, or 16 where sixteen rows and unknown distances leave no registers
  // (32 with queries in shared memory: four drafted tokens 124 -> 113 us)
  const int tiles = cf.NT == 2 && !fixed ? 1 : 2;
  sh.HG = hg;
  sh.NHG = a.Hkv / hg;
  sh.NRC = (sh.R + 8 * cf.NT - 1) / (8 * cf.NT);
  sh.WPH = kConsumers / hg;
  sh.TS = 16 * tiles * sh.WPH;
  sh.ts_log2 = 31 - __builtin_clz(sh.TS);
  sh.cap = (int)((int64_t)a.max_pages * a.page_size);
  sh.page_magic =
      a.page_size > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.page_size - 1) / a.page_size) : 0;
  sh.row_bytes = q4::token_bytes(a.Hkv, a.D);
  sh.taken = sh.NHG == 1 ? sh.row_bytes : hg * q4::record_bytes(a.D);
  sh.unit = sh.taken % 16 ? 8 : 16;
  // (kRuns: a lane a page of the stage, which begins in the middle of one unless it is
  // whole pages long)
  const int pages = sh.TS % a.page_size == 0 ? sh.TS / a.page_size
                                             : (sh.TS - 2) / a.page_size + 2;
  const bool runs = !a.k && sh.NHG == 1 && sh.row_bytes % 128 != 0 && pages <= 32;
  for (sh.box = 32 < sh.TS ? 32 : sh.TS; a.page_size % sh.box;) sh.box /= 2;
  const bool boxes = !a.k && sh.row_bytes % 128 == 0 && sh.taken % 128 == 0 && sh.box >= 16;
  // (kTokens: two tokens a lane at most)
  sh.copies = boxes                                                           ? kBoxes
              : runs                                                          ? kRuns
              : sh.unit == 16 && sh.taken >= kTokenBytesLeast && sh.TS <= 64 ? kTokens
                                                                              : kLanes;
  sh.slice = (sh.taken + 15) / 16 * 16;
  if ((sh.copies == kTokens || sh.copies == kLanes) && sh.slice % 32 == 0) sh.slice += 16;
  const int units = sh.taken / sh.unit, chunks = sh.slice / 16;
  for (sh.lanes = 1; sh.lanes < units && sh.lanes < 32;) sh.lanes *= 2;
  sh.order = chunks % 2 || sh.copies == kBoxes ? kOrderOdd
             : chunks % 4 == 2                 ? kOrderTwo
                                               : kOrderFour;
  const int scratch = hg * (sh.WPH / 2) * cf.NT * (a.D / 4 + 4) * 32 * 4;
  const int nv = (4 * sh.Bv + 15) / 16 * 16, stage = 2 * sh.TS * sh.slice;
  const int queries = cf.NT * tiles == 4 ? kConsumers * cf.NT * (a.D / 32) * 512 : 0;
  const int n = (kSmemMax - 1024 - scratch - queries - nv) / stage;
  sh.stages = n > kMaxStages ? kMaxStages : n;
  // (kLeastStages fit for every shape: a stage is 44 KiB at most)
  sh.q_at = sh.stages * stage;
  sh.scratch_at = sh.q_at + queries;
  sh.nv_at = sh.scratch_at + scratch;
  cf.smem = (size_t)sh.nv_at + nv + 1024;
  // a CTA a segment where they are few and short, else no more than a full batch has stages
  const int64_t each = ((sh.k ? sh.k : sh.cap) + sh.TS - 1) / sh.TS;
  const int64_t segments = (int64_t)sh.Bv * sh.NHG * sh.NRC, most = segments * each;
  sh.grid = device_sm_count();
  sh.whole = each <= kWholeStages + segments / kWholeMore && segments <= sh.grid;
  const int64_t needed = sh.whole ? segments : most;
  if (needed < sh.grid) sh.grid = needed > 0 ? (int)needed : 1;
  cf.PW = fixed && sh.copies == kTokens && most > (int64_t)kLongRun * sh.grid ? 8 : 4;
  cf.fixed = fixed;
  return cf;
}

// Tensor map of a pool for kBoxes: 128-byte lines, a token row's lines, tokens; a box being
// the lines of one head group of some tokens.
cudaError_t pool_map(CUtensorMap* map, const void* pool, const Q4Shape& sh) {
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
  const cuuint64_t dims[3] = {128, (cuuint64_t)sh.row_bytes / 128,
                              (cuuint64_t)sh.num_pages * (cuuint64_t)sh.page_size};
  const cuuint64_t strides[2] = {128, (cuuint64_t)sh.row_bytes};
  const cuuint32_t box[3] = {128, (cuuint32_t)sh.slice / 128, (cuuint32_t)sh.box};
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NT, int TT, int PW, int SLICE>
cudaError_t launch_main(const pks_q4_attention_args& a, const Q4Layout& L, const Config& cf,
                        cudaStream_t s) {
  static bool done[64] = {false};
  auto kern = k_q4_attention<D, NT, TT, PW, SLICE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    // consumers wait for registers that the launch does not have
    cudaFuncAttributes built;
    if ((e = cudaFuncGetAttributes(&built, kern)) != cudaSuccess) return e;
    if (kConsumers * kConsumerRegisters<NT, PW, SLICE> + PW * kProducerRegisters<NT, PW, SLICE> >
        (kConsumers + PW) * built.numRegs)
      return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const float scale = a.sm_scale > 0.f ? a.sm_scale : 1.f / sqrtf((float)a.D);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  int32_t* prefix = reinterpret_cast<int32_t*>(ws + L.prefix);
  float2* ml = reinterpret_cast<float2*>(ws + L.part_ml);
  float* po = reinterpret_cast<float*>(ws + L.part_o);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const Q4Shape& sh = cf.sh;
  CUtensorMap map_k{}, map_v{};
  if (sh.copies == kBoxes) {
    if ((e = pool_map(&map_k, a.pool_k, sh)) != cudaSuccess) return e;
    if ((e = pool_map(&map_v, a.pool_v, sh)) != cudaSuccess) return e;
  }
  e = launch_ex(kern, dim3(sh.grid), dim3((kConsumers + PW) * 32), cf.smem, s, /*pdl=*/true,
                /*coop=*/false, a.seq_lens, a.block_table, a.topk_idx,
                static_cast<const __nv_bfloat16*>(a.q), static_cast<const uint8_t*>(a.pool_k),
                static_cast<const uint8_t*>(a.pool_v), out, a.lse, prefix, ml, po,
                reinterpret_cast<int32_t*>(ws), sh, scale * 1.4426950408889634f,
                a.wait_limit > 0 ? (long long)a.wait_limit : kWaitCycles, map_k, map_v);
  if (e != cudaSuccess || sh.whole) return e;
  const int64_t rows = (int64_t)sh.Bv * sh.Nq * sh.Hq;
  const bool few = rows <= kFewRows;
  return launch_ex(few ? k_q4_merge<D, 8> : k_q4_merge<D, 1>,
                   dim3((unsigned)(few ? rows : (rows + 7) / 8)), dim3(256), 0, s, /*pdl=*/true,
                   /*coop=*/false, (const int32_t*)prefix, (const float2*)ml, (const float*)po,
                   out, a.lse, sh, 8 * NT);
}

template <int NT>
cudaError_t launch_rows(const pks_q4_attention_args& a, const Q4Layout& L, const Config& cf,
                        cudaStream_t s) {
  constexpr int TT = NT == 2 ? 1 : 2;
  if (cf.fixed) {
    if (cf.sh.copies == kBoxes) return launch_main<128, NT, 2, 4, 640>(a, L, cf, s);
    return cf.PW == 8 ? launch_main<128, NT, 2, 8, 656>(a, L, cf, s)
                      : launch_main<128, NT, 2, 4, 656>(a, L, cf, s);
  }
  return a.D == 64 ? launch_main<64, NT, TT, 4, 0>(a, L, cf, s)
                   : launch_main<128, NT, TT, 4, 0>(a, L, cf, s);
}

}  // namespace

bool q4_supported(const pks_q4_attention_args& a) {
  const Q4Shape sh = configure(a).sh;  // the stages of a full batch are counted in 32 bits
  const int64_t each = ((sh.k ? sh.k : sh.cap) + sh.TS - 1) / sh.TS;
  return each * sh.NHG * sh.NRC * sh.Bv <= INT32_MAX && sh.stages >= kLeastStages;
}

Q4Layout q4_layout(const pks_q4_attention_args& a) {
  const Config cf = configure(a);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Q4Layout L{};
  L.prefix = 256;
  L.part_ml = up(L.prefix + sizeof(int32_t) * (size_t)(cf.sh.Bv + 1));
  // a CTA's first segment and its last
  const size_t rows = (size_t)2 * cf.sh.grid * cf.sh.HG * 8 * cf.NT;
  L.part_o = up(L.part_ml + sizeof(float2) * rows);
  L.total = up(L.part_o + sizeof(float) * rows * (size_t)a.D);
  return L;
}

cudaError_t launch_q4_attention(const pks_q4_attention_args& a, const Q4Layout& L,
                                cudaStream_t s) {
  const Config cf = configure(a);
  return cf.NT == 2 ? launch_rows<2>(a, L, cf, s) : launch_rows<1>(a, L, cf, s);
}

}  // namespace pks
