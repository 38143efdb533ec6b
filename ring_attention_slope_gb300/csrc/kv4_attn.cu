// Attention of each sequence's newest tokens over its pages of the 4-bit cache
// (a decode step).
//
// For a query row with scaled scores x_j (log2 units) over the visible keys j:
//   out = sum_j 2^(x_j - m) v_j / l,  l = sum_j 2^(x_j - m),  lse = (m + log2 l) ln 2,
// where a cached channel is scale * code + min with one scale and min (bf16) for
// each group G of 32 channels of a token's head.  The codes go to the tensor
// cores as they are and the scales stay outside:
//   q . k_j  = sum_G ( scale_jG * (sum_c q_c code_jc) + min_jG * (sum_c q_c) )
//   sum_j w_j v_jc = sum_j r_jG code_jc + sum_j ( w_j (min_jG + 8 scale_jG) - 8 r_jG ),  r_jG = w_j scale_jG
// so a code costs a mask and half a shift, not a conversion.  r is rounded to bf16 for the tensor cores, and its
// error meets code - 8 rather than code: most values lie near the middle of their group's range.
//
// Codes as matrix operands.  A float whose exponent field is 0 or 1 is linear in its bits, so the low 8
// bits of a 16-bit float, alone, are an exact multiple of its smallest subnormal: a 4-bit code in bits 0-3 is
// code * 2^-24 in fp16 and code * 2^-133 in bf16, one in bits 4-7 sixteen times that, and the tensor cores
// multiply both exactly.  One shift by 8 serves the other eight bits, so eight codes take a shift and
// four masks.  Keys use fp16: a query row is scaled by a power of two to a largest value near 2^14, and its
// channels that meet bits 4-7 by 1/16, both exact.  Values use bf16, because the other operand, weight *
// scale, needs bf16's range (fp16's would flush it): the weight carries a factor 2^64 so that products with
// 2^-133 stay normal fp32 numbers.  Its rounding to bf16 (2^-8 relative) is the one the attention kernel of
// the prefill also makes on its weights.
//
// Keys are the M rows of S^T = K Q^T (16 keys x 8 query rows), values those of
// O^T = V^T P^T (16 channels x 8 query rows): with the few query rows of a decode
// step on the narrow side no multiply is wasted on padding at 8 heads per KV head.
// The block layout in memory is the operand layout, so a lane's codes of 16 keys
// are its own 16-byte words; P^T needs one 8x8 transpose (movmatrix) a group.
//
// Measured at 64/8 heads of 64: 8 sequences of 102400 tokens 103 us = 5.1 TB/s of cache (75% of the copy rate); 32
// ragged ones up to 32768 29.0 us; one of 65536 19 us; one of 1000 7.0 us; 8 of 16384 26 us with one query each, 35
// with two and 80 with five (40 rows, three tiles, each of which reads the pages again).  (Around the groups' minimums
// instead of their middles 3 to 4% less, with 2.4 times the error.)  At the first the ALU pipe is over half busy,
// the issue slots over 60%, DRAM two thirds: a warp's step of 64 tokens is about as long in instructions as its codes
// are on the way.  (The copies alone, without the arithmetic, took 84 us.)  The short ones are latency: the
// lengths, the page table, one copy, the steps, the join of the warps and that of the CTAs, one after another.
//
// Work split: every sequence's visible steps of 64 or 32 tokens, for each KV head (and each tile of 8 NT query
// rows), laid end to end and cut into ranges for the CTAs of a grid that fills the GPU once: equal ones, or, where
// the CTAs suffice for that, ranges that end with their pairs, one piece to a CTA (see cta_range).  The cut knows the
// lengths only on the device, so ragged batches and captured graphs balance alike.  Pieces that are not whole
// (sequence, head) pairs leave partials (m, l, unnormalised out) in the workspace, and a second launch, queued as
// a programmatic dependent, joins them in a fixed order.  Inside a CTA four warps take every fourth step, each with
// its own ring of bulk copies, and join once at the end of a piece.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "host.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "sm103_ptx.cuh"
#include "waits.cuh"

namespace slope {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 640;          // of the attention launch: the workspace has two partials for each
constexpr int kMinSteps = kWarps;      // a range is at least this many steps
constexpr int kPieceTokens = 800;      // what a piece's start and end cost, in tokens of steps, at most (see cta_range)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescale = 8.f;        // the running maximum moves when a score passes it by this (log2)
constexpr float kNoMax = -1e30f;       // running maximum before any key

struct Kv4AttnParams {
  const __nv_bfloat16* q;
  int64_t q_srow, q_shead;
  const uint8_t* data;
  int64_t n_pages;
  const int32_t* table;
  int64_t table_stride;
  int64_t max_tokens;  // max_pages * page_size
  const int32_t* kv_lens;
  int32_t B, q_len, Hkv, group;
  int32_t page_shift;  // log2 of the page size
  int32_t row_tiles;   // tiles of 8 NT of the q_len * group rows of a KV head
  int32_t window;
  float scale_log2;
  void* out;
  int64_t out_srow, out_shead;
  int32_t out_bf16;
  float* lse;  // may be null
  int64_t lse_srow, lse_shead;
  int4* heads;      // workspace: {sequence, pair, first CTA, last CTA} of the pairs that several CTAs share, or {-1}
  int32_t by_pair;  // an entry of `heads` for each pair (where there are fewer than CTAs), else for each first CTA
  float* partials;  // workspace: two for each CTA, {m[R], l[R], out[R][DV]}
  int* status;
  uint64_t wait_limit_ns;
};

template <int DQK, int DV, int NT>
struct Kv4Cfg {
  static constexpr int R = 8 * NT;  // query rows of a tile
  static constexpr int NG = DQK / 32, NV = DV / 32, NC = DV / 64, NW = NG + NV;
  static constexpr int kKeyBytes = kv4_key_bytes(DQK), kValueBytes = kv4_value_bytes(DV);
  static constexpr int kBlockBytes = kv4_block_bytes(DQK, DV);
  // CTAs on an SM, by registers: 128 a thread at four, 168 at three, 255 at two
  static constexpr int kCtas = NT == 1 ? (DQK == 64 && DV == 64 ? 4 : 3) : (DQK == 64 && DV == 64 ? 3 : 2);
  // tokens of a step, which costs about a hundred instructions whatever its size: four blocks, or two wide ones
  static constexpr int kStep = kBlockBytes <= 1280 ? 64 : 32, kStepLog = kStep == 64 ? 6 : 5;
  static constexpr int kStageBytes = kStep / kKv4Block * kBlockBytes;
  static constexpr int kStages = kCtas == 2 ? 3 : 2;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kRedFloats = kWarps * R * DV + 2 * kWarps * R;
  static constexpr int kSmemBytes = kRingBytes + kRedFloats * 4 + kWarps * kStages * 8 + 64;
  static constexpr int kPartialFloats = 2 * R + R * DV;
  static_assert(kCtas * (kSmemBytes + 1024) <= 232448 + 1024, "shared memory of the resident CTAs");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The products and the transpose below are functions of their operands: not volatile, so that the compiler
// may interleave independent ones.  Every warp runs them as a whole.
// d = a b (no accumulator in)
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8x8 matrix of 16-bit elements held two to a lane (row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The keys of a sequence that some of its queries see, in steps of 64 or 32 tokens.
struct SeqSteps {
  int len;    // tokens in the cache
  int first;  // first step
  int count;  // steps, at least 1 (a sequence without keys still has rows to write)
};
template <int kStep>
__device__ __forceinline__ SeqSteps seq_steps(const Kv4AttnParams& p, int b) {
  SeqSteps s;
  const int64_t n = p.kv_lens[b];
  s.len = static_cast<int>(n < 0 ? 0 : n > p.max_tokens ? p.max_tokens : n);
  s.first = p.window > 0 ? max(0, s.len - p.q_len - p.window + 1) / kStep : 0;
  s.count = max(1, (s.len + kStep - 1) / kStep - s.first);
  return s;
}

// A CTA's range of units and the pair it starts in.  A pair is a (sequence, KV head, row tile); its
// units are its steps, after `cost` for starting and finishing it, or (cost < 0) its steps rounded up to
// whole ranges.
struct CtaRange {
  int64_t begin, end, per;
  int64_t pair_begin;  // first unit of the pair
  int b, pair;         // the one that holds unit `begin`
  int cost;
};
// Lengths of ranges that are tried for one piece to a CTA: 4, 8, 16 and 32 steps.
constexpr int kTries = 4;
__device__ constexpr int try_steps(int i) { return kMinSteps << i; }
struct CutScratch {
  int64_t sums[kWarps], pair_begin;
  int ranges[kWarps][kTries], b, pair;
};
__device__ __forceinline__ int pair_units(int steps, int cost, int64_t per) {
  if (cost >= 0) return steps + cost;
  const unsigned n = static_cast<unsigned>(per);
  return static_cast<int>((steps + n - 1) / n * n);
}

// The second half of cta_range: U holds every unit (64-bit divisions and scans cost a small call 0.8 us).
template <int kStep, typename U>
__device__ __forceinline__ CtaRange cut(const Kv4AttnParams& p, CutScratch& scratch, U steps, int count0) {
  constexpr U kPiece = kPieceTokens / kStep;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = p.Hkv * p.row_tiles;
  const U grid = gridDim.x;
  bool fits[kTries];
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    int64_t n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n += scratch.ranges[w][i];
    fits[i] = n * pairs <= gridDim.x;
  }
  U per = 0, total;
  int cost = -1;
#pragma unroll
  for (int i = kTries - 1; i >= 0; --i)
    if (fits[i] && try_steps(i) <= kPiece) per = try_steps(i);
  if (per == 0) {
    const U even = (steps + grid - 1) / grid, c = min(kPiece, even / 2);
    total = steps + static_cast<U>(p.B) * pairs * c;
    const U evenly = max(static_cast<U>(kMinSteps), (total + grid - 1) / grid);
#pragma unroll
    for (int i = kTries - 1; i >= 0; --i)
      if (fits[i] && try_steps(i) <= evenly) per = try_steps(i);
    if (per == 0) {
      per = evenly;
      cost = static_cast<int>(c);
    }
  }
  if (cost < 0) total = grid * per;  // or less: the search below finds no sequence then
  const U begin = min(total, static_cast<U>(blockIdx.x) * per), end = min(total, begin + per);
  CtaRange r;
  r.per = per;
  r.cost = cost;
  r.begin = r.end = begin;
  r.pair_begin = 0;
  r.b = r.pair = 0;
  if (begin >= end) return r;
  // the sequence that holds unit `begin`
  U carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int count = b >= p.B ? 0 : b0 == 0 ? count0 : seq_steps<kStep>(p, b).count;
    const U mine = b < p.B ? static_cast<U>(pair_units(count, cost, per)) * pairs : 0;
    U incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const U o = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += o;
    }
    __syncthreads();
    if (lane == 31) scratch.sums[warp] = incl;
    __syncthreads();
    U before = carry;
    for (int w = 0; w < warp; ++w) before += static_cast<U>(scratch.sums[w]);
    for (int w = 0; w < kWarps; ++w) carry += static_cast<U>(scratch.sums[w]);
    incl += before;
    if (mine > 0 && incl - mine <= begin && begin < incl) {
      const U units = mine / pairs, pair = (begin - (incl - mine)) / units;
      scratch.b = b;
      scratch.pair = static_cast<int>(pair);
      scratch.pair_begin = incl - mine + pair * units;
    }
    if (carry > begin) break;  // the same for every thread
  }
  if (carry <= begin) return r;  // past the last pair
  __syncthreads();
  r.end = end;
  r.b = scratch.b;
  r.pair = scratch.pair;
  r.pair_begin = scratch.pair_begin;
  return r;
}

// Every thread of the CTA calls it.
//
// A pair's fixed cost (its queries, its first copies' latency, the join of the warps) is worth about 800
// tokens.  Without it in the cut, a batch with many short sequences gave one CTA the tail of all of them:
// 32 sequences of 8 .. 32768 tokens took 148 us.  Where a range has few steps in all, the cost is
// taken as half of them, so that a small call still spreads over the CTAs.
//
// Where ranges no longer than that would be (or than the fixed cost), cut at the pairs' ends too, are no more
// than the CTAs, each CTA gets one: a CTA that straddles pairs would pay the cost again.  (10 sequences of 39
// tokens, 5 queries of 16 heads: 21.4 -> 8.7 us; 60 of 200 tokens, 64 heads: 14.1 -> 9.7 us; 64 of 1024:
// 19.1 -> 15.7 us.)
template <int kStep>
__device__ CtaRange cta_range(const Kv4AttnParams& p, CutScratch& scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = p.Hkv * p.row_tiles;
  int64_t steps = 0;
  int ranges[kTries];  // of try_steps(i) steps, kept from overflowing
  int count0 = 0;      // steps of sequence threadIdx.x
#pragma unroll
  for (int i = 0; i < kTries; ++i) ranges[i] = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int count = seq_steps<kStep>(p, b).count;
    if (b < kThreads) count0 = count;
    steps += count;
#pragma unroll
    for (int i = 0; i < kTries; ++i) ranges[i] = min(ranges[i] + (count + try_steps(i) - 1) / try_steps(i), 1 << 16);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, m);
#pragma unroll
  for (int i = 0; i < kTries; ++i) ranges[i] = __reduce_add_sync(0xffffffffu, ranges[i]);
  if (lane == 0) {
    scratch.sums[warp] = steps;
#pragma unroll
    for (int i = 0; i < kTries; ++i) scratch.ranges[warp][i] = ranges[i];
  }
  __syncthreads();
  steps = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) steps += scratch.sums[w];
  steps *= pairs;
  if (steps + static_cast<int64_t>(p.B) * pairs * (kPieceTokens / kStep) < (1u << 31))
    return cut<kStep, uint32_t>(p, scratch, static_cast<uint32_t>(steps), count0);
  return cut<kStep, uint64_t>(p, scratch, static_cast<uint64_t>(steps), count0);
}

template <int DV, int R>
__device__ __forceinline__ void store_row(const Kv4AttnParams& p, int b, int pair, int row, int ch, float4 o, float m,
                                          float l) {
  const int h = pair / p.row_tiles, r = (pair - h * p.row_tiles) * R + row;
  if (r >= p.q_len * p.group) return;
  const int64_t tok = static_cast<int64_t>(b) * p.q_len + r / p.group;
  const int head = h * p.group + r % p.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = tok * p.out_srow + head * p.out_shead + ch;
  if (p.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (ch == 0 && p.lse != nullptr)
    p.lse[tok * p.lse_srow + head * p.lse_shead] = l == 0.f ? -INFINITY : (m + lg2_approx(l)) * kLn2;
}

template <int DQK, int DV, int NT>
__global__ void __launch_bounds__(kThreads, Kv4Cfg<DQK, DV, NT>::kCtas)
    kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  using C = Kv4Cfg<DQK, DV, NT>;
  constexpr int kStep = C::kStep;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ CutScratch s_scratch;
  __shared__ int s_abort;
  float* const red = reinterpret_cast<float*>(smem + C::kRingBytes);  // [warp][row][channel]
  float* const red_m = red + kWarps * C::R * DV;                      // [warp][row]
  float* const red_l = red_m + kWarps * C::R;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(red_l + kWarps * C::R);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;
  uint8_t* const ring = smem + warp * C::kStages * C::kStageBytes;
  uint64_t* const full = bars + warp * C::kStages;

  pdl_launch_dependents();
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  const CtaRange range = cta_range<kStep>(p, s_scratch);
  if (threadIdx.x == 0 && !p.by_pair) p.heads[blockIdx.x] = make_int4(-1, 0, 0, 0);

  // the warp's ring: the stages that the next copy fills and the next step reads, and that one's parity
  int put = 0, get = 0;
  uint32_t parity = 0;
  int b = range.b, pair = range.pair;
  int64_t pair_begin = range.pair_begin;
  bool ok = true;
  for (int64_t u = range.begin; u < range.end;) {
    // ---- the piece: steps [st0, st1) of one pair
    const SeqSteps sb = seq_steps<kStep>(p, b);
    const int cost = max(0, range.cost);
    const int64_t pair_end = pair_begin + pair_units(sb.count, range.cost, range.per);
    const int64_t u_end = min(range.end, pair_end);
    const int st0 = sb.first + max(0, static_cast<int>(u - pair_begin) - cost);
    const int st1 = sb.first + min(sb.count, max(0, static_cast<int>(u_end - pair_begin) - cost));
    const int kvh = pair / p.row_tiles, rt = pair - kvh * p.row_tiles;
    const int n_it = max(0, (st1 - st0 - warp + kWarps - 1) / kWarps);

    // ---- the queries' loads, ahead of the pages' and the copies'
    const int n_rows = p.q_len * p.group;
    uint4 qraw[NT][C::NG];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = rt * C::R + t * 8 + g;
      const __nv_bfloat16* const qrow = p.q + (static_cast<int64_t>(b) * p.q_len + r / p.group) * p.q_srow +
                                        (kvh * p.group + r % p.group) * p.q_shead + 8 * q4;
#pragma unroll
      for (int G = 0; G < C::NG; ++G)
        qraw[t][G] = r < n_rows ? *reinterpret_cast<const uint4*>(qrow + 32 * G) : make_uint4(0u, 0u, 0u, 0u);
    }

    // ---- bulk copies: iteration i takes step st0 + warp + 4 i, in one copy or, where a page is smaller than a
    // step, in two or four.  Each lane looks one copy's page up, 32 at a time and the next 32 ahead, and starts it.
    const int32_t* const row = p.table + b * p.table_stride;
    const int cs = max(0, C::kStepLog - p.page_shift);                   // log2 of an iteration's copies
    const int low_hi = sb.len - p.q_len;                       // smallest last position of any row
    const int high_lo = p.window > 0 ? sb.len - p.window : 0;  // largest first position
    auto pos_of = [&](int copy) { return (st0 + warp + kWarps * (copy >> cs)) * kStep + ((copy & ((1 << cs) - 1)) << (C::kStepLog - cs)); };
    auto page_of = [&](int copy) -> int {  // -1: no such step or token, or a page outside the cache
      const int pos = pos_of(copy);
      if ((copy >> cs) >= n_it || pos >= sb.len) return -1;
      const int pg = row[pos >> p.page_shift];
      return pg >= 0 && pg < p.n_pages ? pg : -1;
    };
    const uint8_t* src = nullptr;                               // of the lane's copy
    const uint32_t copy_bytes = C::kStageBytes >> cs;
    uint32_t there = 0;  // bit: the copy has a page
    uint32_t plain = 0;  // bit of an iteration's first copy: every row sees all of its step's tokens
    int next_page;
    auto refill = [&](int first) {  // the pages of copies first .. first + 31 are in next_page
      const int pos = pos_of(first + lane);
      const int in_page = (pos / kKv4Block) & ((1 << (p.page_shift - 4)) - 1);
      src = p.data + (((static_cast<int64_t>(next_page) * p.Hkv + kvh) << (p.page_shift - 4)) + in_page) * C::kBlockBytes;
      there = __ballot_sync(0xffffffffu, next_page >= 0);
      plain = __ballot_sync(0xffffffffu, next_page >= 0 && pos + (kStep >> cs) - 1 <= low_hi && pos >= high_lo);
      if (cs > 0) plain &= plain >> 1;
      if (cs > 1) plain &= plain >> 2;
      next_page = page_of(first + 32 + lane);
    };
    next_page = page_of(lane);
    refill(0);
    int sent = 0;  // iterations
    auto send = [&]() {
      if (sent >= n_it || !ok) return;
      const int at = (sent << cs) & 31;
      if (at == 0 && sent > 0) refill(sent << cs);
      uint64_t* const bar = &full[put];
      const bool mine = lane >> cs == at >> cs;
      if (lane == at) mbar_arrive_expect_tx(bar, __popc(there >> at & ((2u << ((1 << cs) - 1)) - 1u)) * copy_bytes);
      __syncwarp();
      if (mine && (there >> lane & 1u))
        bulk_load(ring + put * C::kStageBytes + (lane - at) * copy_bytes, src, copy_bytes, bar);
      put = put == C::kStages - 1 ? 0 : put + 1;
      ++sent;
    };
    for (int i = 0; i < C::kStages - 1; ++i) send();

    // ---- queries as matrix operands
    uint32_t qb[NT][C::NG][4];
    float qsum[NT][C::NG][2];  // of rows 2 q4 and 2 q4 + 1, in the units of the products
    float sl2[NT][2];
    int hi[NT][2];             // last position those rows see
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4(&w)[C::NG] = qraw[t];
      float top = 0.f;
#pragma unroll
      for (int G = 0; G < C::NG; ++G) {
        const uint32_t x[4] = {w[G].x, w[G].y, w[G].z, w[G].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^k brings the row's largest value to [2^13, 2^14); a row of zeros, or one that is not finite, stays
      const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      const int k = (top > 0.f && e < 128) ? min(13 - e, 120) : 0;
      const float up = __uint_as_float(static_cast<uint32_t>(max(k + 127, 1)) << 23);
      float sums[C::NG];
#pragma unroll
      for (int G = 0; G < C::NG; ++G) {
        const uint32_t x[4] = {w[G].x, w[G].y, w[G].z, w[G].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(x[i] << 16) * up;
          v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u) * up;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // codes i and i + 4 share a word's 16-bit halves; odd i sit at bits 4-7
          const float f = (i & 1) ? 0.0625f : 1.f;
          qb[t][G][i] = pack_f16x2(v[i] * f, v[i + 4] * f);
        }
        float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        sums[G] = s * 0x1p-24f;
      }
      // a largest value of 2^117 or more would need a unit past fp32's range: such a row becomes NaN
      const float unit = k < -103 ? __uint_as_float(0x7fc00000u) : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(24 - k + 127) << 23);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int from = (2 * q4 + j) * 4;
#pragma unroll
        for (int G = 0; G < C::NG; ++G) qsum[t][G][j] = __shfl_sync(0xffffffffu, sums[G], from);
        sl2[t][j] = __shfl_sync(0xffffffffu, unit, from);
        const int rj = rt * C::R + t * 8 + 2 * q4 + j;
        hi[t][j] = sb.len - p.q_len + min(rj / p.group, p.q_len - 1);
      }
    }

    // ---- the steps
    float nm[NT][2], l[NT][2], o[C::NC][2][2][NT][4];  // nm: 64 - running maximum
    uint64_t bias[NT][C::NV];                           // of both rows
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        nm[t][j] = 64.f - kNoMax;
        l[t][j] = 0.f;
      }
#pragma unroll
      for (int G = 0; G < C::NV; ++G) bias[t][G] = 0;
#pragma unroll
      for (int c = 0; c < C::NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][i >> 1][i & 1][t][e] = 0.f;
    }
    // Half a step in three phases.  kEdge: some row does not see some of its keys.
    // Scores of 32 tokens, a half of a step, from position pos0 on, whose two blocks lie in `mem` (bit j of
    // `none`: block j is not there at all).
    auto scores = [&](auto edge_c, const uint8_t* const mem, const int pos0, const int none, float(&x)[2][NT][4]) {
      constexpr bool kEdge = decltype(edge_c)::value;
      // scores of keys g (elements 0, 1) and g + 8 (2, 3) of both blocks for rows 2 q4 and 2 q4 + 1
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* const blk_mem = mem + j * C::kBlockBytes;
        uint32_t kw[2 * C::NG];  // [token g, g + 8][group]
#pragma unroll
        for (int i = 0; i < C::NG / 2; ++i) {
          const uint4 r = *reinterpret_cast<const uint4*>(blk_mem + (i * 32 + lane) * 16);
          kw[4 * i] = r.x, kw[4 * i + 1] = r.y, kw[4 * i + 2] = r.z, kw[4 * i + 3] = r.w;
        }
        uint32_t word[2][C::NG];  // scale and min of tokens g and g + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* const wp = blk_mem + C::kKeyBytes + C::kValueBytes + (g + 8 * i) * 4 * C::NW;
#pragma unroll
          for (int h = 0; h < C::NG / 2; ++h) {
            const uint2 r = *reinterpret_cast<const uint2*>(wp + 8 * h);
            word[i][2 * h] = r.x, word[i][2 * h + 1] = r.y;
          }
        }
#pragma unroll
        for (int G = 0; G < C::NG; ++G) {
          const uint32_t w0 = kw[G], w1 = kw[C::NG + G], v0 = w0 >> 8, v1 = w1 >> 8;
          const float s0 = __uint_as_float(word[0][G] & 0xffff0000u), s1 = __uint_as_float(word[1][G] & 0xffff0000u);
          const float n0 = __uint_as_float(word[0][G] << 16), n1 = __uint_as_float(word[1][G] << 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float acc[4];
            mma_f16_first(acc, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, qb[t][G][0],
                          qb[t][G][1]);
            mma_f16(acc, v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u, qb[t][G][2],
                    qb[t][G][3]);
            float(&xx)[4] = x[j][t];
            if (G == 0) {
              xx[0] = fmaf(s0, acc[0], n0 * qsum[t][G][0]);
              xx[1] = fmaf(s0, acc[1], n0 * qsum[t][G][1]);
              xx[2] = fmaf(s1, acc[2], n1 * qsum[t][G][0]);
              xx[3] = fmaf(s1, acc[3], n1 * qsum[t][G][1]);
            } else {
              xx[0] = fmaf(s0, acc[0], fmaf(n0, qsum[t][G][0], xx[0]));
              xx[1] = fmaf(s0, acc[1], fmaf(n0, qsum[t][G][1], xx[1]));
              xx[2] = fmaf(s1, acc[2], fmaf(n1, qsum[t][G][0], xx[2]));
              xx[3] = fmaf(s1, acc[3], fmaf(n1, qsum[t][G][1], xx[3]));
            }
          }
        }
      }
      if constexpr (kEdge) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int pos = pos0 + j * kKv4Block + g + 8 * (e >> 1), last = hi[t][e & 1];
              if ((none >> j & 1) || pos > last || (p.window > 0 && last - pos >= p.window)) x[j][t][e] = -INFINITY;
            }
      }
    };
    // Their weights times 2^64, and the running maximum and sum.
    auto weights = [&](const float(&x)[2][NT][4], float(&w)[2][NT][4]) {
      // y: log2 of the weight times 2^64.  A row whose score passes the running maximum by 2^8 moves it
      // (any other weight stays below 2^8).
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j][t][e] = fmaf(x[j][t][e], sl2[t][e & 1], nm[t][e & 1]);
          top = fmax3(top, fmaxf(w[j][t][0], w[j][t][1]), fmaxf(w[j][t][2], w[j][t][3]));
        }
      if (__any_sync(0xffffffffu, top > 64.f + kRescale)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float m = 64.f - nm[t][j];
            float hi_x = fmaxf(fmaxf(x[0][t][j], x[0][t][2 + j]), fmaxf(x[1][t][j], x[1][t][2 + j])) * sl2[t][j];
            hi_x = fmaxf(hi_x, __shfl_xor_sync(0xffffffffu, hi_x, 4));
            hi_x = fmaxf(hi_x, __shfl_xor_sync(0xffffffffu, hi_x, 8));
            hi_x = fmaxf(hi_x, __shfl_xor_sync(0xffffffffu, hi_x, 16));
            nm[t][j] = 64.f - fmaxf(m, hi_x);
            const float alpha = ex2_approx(m - (64.f - nm[t][j]));
            l[t][j] *= alpha;
#pragma unroll
            for (int G = 0; G < C::NV; ++G)
              bias[t][G] = mul_f32x2(bias[t][G], j == 0 ? pack_f32x2(alpha, 1.f) : pack_f32x2(1.f, alpha));
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[c][i >> 1][i & 1][t][j] *= alpha;
                o[c][i >> 1][i & 1][t][2 + j] *= alpha;
              }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              w[i][t][j] = fmaf(x[i][t][j], sl2[t][j], nm[t][j]);
              w[i][t][2 + j] = fmaf(x[i][t][2 + j], sl2[t][j], nm[t][j]);
            }
          }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j][t][e] = ex2_approx(w[j][t][e]);
          l[t][0] += w[j][t][0] + w[j][t][2];
          l[t][1] += w[j][t][1] + w[j][t][3];
        }
    };
    // The weighted values.
    auto accumulate = [&](auto edge_c, const uint8_t* const mem, const float(&w)[2][NT][4]) {
      constexpr bool kEdge = decltype(edge_c)::value;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* const blk_mem = mem + j * C::kBlockBytes;
        uint32_t word[2][C::NV];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* const wp = blk_mem + C::kKeyBytes + C::kValueBytes + (g + 8 * i) * 4 * C::NW + 4 * C::NG;
#pragma unroll
          for (int h = 0; h < C::NV / 2; ++h) {
            const uint2 r = *reinterpret_cast<const uint2*>(wp + 8 * h);
            word[i][2 * h] = r.x, word[i][2 * h + 1] = r.y;
          }
        }
        // the weights' operands for each group of values, and what the products leave out (see the top)
        const uint64_t minus8 = pack_f32x2(-8.f, -8.f);
        uint32_t pb[NT][C::NV][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float(&ww)[4] = w[j][t];
#pragma unroll
          for (int G = 0; G < C::NV; ++G) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // tokens g and g + 8
              const uint64_t w2 = pack_f32x2(ww[2 * i], ww[2 * i + 1]);
              uint64_t s2 = pack_f32x2(__uint_as_float(word[i][G] & 0xffff0000u), __uint_as_float(word[i][G] & 0xffff0000u));
              float mid = fmaf(__uint_as_float(word[i][G] & 0xffff0000u), 8.f, __uint_as_float(word[i][G] << 16));
              uint64_t m2 = pack_f32x2(mid, mid);
              if constexpr (kEdge) {  // a hidden key's scale and min may be anything, NaN too
                const float2 sf = unpack_f32x2(s2);
                s2 = pack_f32x2(ww[2 * i] == 0.f ? 0.f : sf.x, ww[2 * i + 1] == 0.f ? 0.f : sf.y);
                m2 = pack_f32x2(ww[2 * i] == 0.f ? 0.f : mid, ww[2 * i + 1] == 0.f ? 0.f : mid);
              }
              const float2 ws = unpack_f32x2(mul_f32x2(w2, s2));
              const uint32_t r = pack_bf16x2(ws.x, ws.y);
              const uint64_t r2 = pack_f32x2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
              bias[t][G] = fma_f32x2(w2, m2, fma_f32x2(r2, minus8, bias[t][G]));
              pb[t][G][i] = transpose8x8(r);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
          const uint4 r = *reinterpret_cast<const uint4*>(blk_mem + C::kKeyBytes + (c * 32 + lane) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the chunk's two groups
            const uint32_t z0 = __byte_perm(r.x, r.y, h ? 0x7632 : 0x5410), z1 = __byte_perm(r.z, r.w, h ? 0x7632 : 0x5410);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // channels 2 i in rows g, and 2 i + 1, sixteen times as large, in rows g + 8
              const uint32_t a0 = (z0 >> (8 * i)) & 0x000f000fu, a1 = (z0 >> (8 * i)) & 0x00f000f0u;
              const uint32_t a2 = (z1 >> (8 * i)) & 0x000f000fu, a3 = (z1 >> (8 * i)) & 0x00f000f0u;
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_bf16(o[c][h][i][t], a0, a1, a2, a3, pb[t][2 * c + h][0], pb[t][2 * c + h][1]);
            }
          }
        }
      }
    };

    uint32_t mask = 0;  // `plain` from this iteration on
    float x[2][NT][4], w[2][NT][4];
    for (int it = 0; it < n_it; ++it) {
      if (((it << cs) & 31) == 0) mask = plain;  // sending is at most a few iterations ahead
      // refill first: the stage it takes was read in the last iteration
      __syncwarp();
      send();
      if (!__all_sync(0xffffffffu, mbar_try_wait(&full[get], parity))) {
        ok = wait_bounded(&full[get], parity, &s_abort, p.status, p.wait_limit_ns, 20);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          sent -= it;  // copies that no step has taken
          break;
        }
      }
      const uint8_t* const mem = ring + get * C::kStageBytes;
      get = get == C::kStages - 1 ? 0 : get + 1;
      parity ^= get == 0 ? 1u : 0u;
      if (mask & 1u) {
#pragma unroll 1
        for (int half = 0; half < kStep / 32; ++half) {
          const uint8_t* const m = mem + half * 2 * C::kBlockBytes;
          scores(std::false_type{}, m, 0, 0, x);
          weights(x, w);
          accumulate(std::false_type{}, m, w);
        }
      } else {
#pragma unroll 1
        for (int half = 0; half < kStep / 32; ++half) {
          const uint8_t* const m = mem + half * 2 * C::kBlockBytes;
          const int pos = (st0 + warp + kWarps * it) * kStep + half * 32;
          auto none = [&](int at) { return page_of((it << cs) + ((at & (kStep - 1)) >> (C::kStepLog - cs))) < 0 ? 1 : 0; };
          scores(std::true_type{}, m, pos, none(pos) | none(pos + kKv4Block) << 1, x);
          weights(x, w);
          accumulate(std::true_type{}, m, w);
        }
      }
      mask >>= 1 << cs;
    }
    if (!ok) {
      // the copies still in flight land before anything else uses the CTA's shared memory
      for (; sent > 0; --sent) {
        wait_final(&full[get], parity, p.wait_limit_ns);
        get = get == C::kStages - 1 ? 0 : get + 1;
        parity ^= get == 0 ? 1u : 0u;
      }
    }

    // ---- join the warps: l and bias over the lanes that hold other keys, then everything over the warps
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float both[C::NV];
#pragma unroll
        for (int G = 0; G < C::NV; ++G) both[G] = j == 0 ? unpack_f32x2(bias[t][G]).x : unpack_f32x2(bias[t][G]).y;
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
          l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], s);
#pragma unroll
          for (int G = 0; G < C::NV; ++G) both[G] += __shfl_xor_sync(0xffffffffu, both[G], s);
        }
        const int rr = t * 8 + 2 * q4 + j;
        if (g == 0) {
          red_m[warp * C::R + rr] = 64.f - nm[t][j];
          red_l[warp * C::R + rr] = l[t][j] * 0x1p-64f;
        }
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float bs = both[2 * c + h] * 0x1p-64f;
            *reinterpret_cast<float4*>(red + (warp * C::R + rr) * DV + 64 * c + 32 * h + 4 * g) =
                make_float4(fmaf(o[c][h][0][t][j], 0x1p69f, bs), fmaf(o[c][h][0][t][2 + j], 0x1p65f, bs),
                            fmaf(o[c][h][1][t][j], 0x1p69f, bs), fmaf(o[c][h][1][t][2 + j], 0x1p65f, bs));
          }
      }
    __syncthreads();
    const bool whole = u == pair_begin && u_end == pair_end;
    float* const part =
        p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (u == pair_begin ? 1 : 0)) * C::kPartialFloats;
    for (int i = threadIdx.x; i < C::R * DV / 4; i += kThreads) {
      const int rr = i / (DV / 4), ch = (i % (DV / 4)) * 4;
      float mm = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, red_m[w * C::R + rr]);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(red_m[w * C::R + rr] - mm);
        const float4 v = *reinterpret_cast<const float4*>(red + (w * C::R + rr) * DV + ch);
        ll = fmaf(f, red_l[w * C::R + rr], ll);
        sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
        sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
      }
      if (whole) {
        store_row<DV, C::R>(p, b, pair, rr, ch, sum, mm, ll);
      } else {
        *reinterpret_cast<float4*>(part + 2 * C::R + rr * DV + ch) = sum;
        if (ch == 0) {
          part[rr] = mm;
          part[C::R + rr] = ll;
        }
      }
    }
    if (threadIdx.x == 0 && u == pair_begin && (!whole || p.by_pair))  // begun here: finished here or in a later CTA's range
      p.heads[p.by_pair ? b * p.Hkv * p.row_tiles + pair : blockIdx.x] =
          make_int4(whole ? -1 : b, pair, blockIdx.x, static_cast<int>((pair_end - 1) / range.per));
    __syncthreads();
    u = u_end;
    pair_begin = pair_end;  // (where the range ends inside the pair, none of this is used)
    if (++pair == p.Hkv * p.row_tiles) {
      pair = 0;
      ++b;
    }
  }
}

// Joins the partials of a pair that several CTAs share.  CTA (c, y) takes the pair of entry c, 32 lanes times
// four of its channels, and its warps every kJoinWarps-th partial, which they join at the end: all in a fixed
// order, so the same result every time.  Latency is all that this launch costs, so each lane has four
// partials' loads in flight and as many warps share a pair as the launch has room for (see launch_nt).
template <int DV, int R, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) kv4_join_kernel(const __grid_constant__ Kv4AttnParams p) {
  __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
  __shared__ float4 s_v[kJoinWarps][32];
  pdl_wait();
  const int4 head = p.heads[blockIdx.x];
  if (head.x < 0) return;
  constexpr int kFloats = 2 * R + R * DV, kAhead = 4;
  static_assert(R * DV % 128 == 0, "whole CTAs of 32 times four channels");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = blockIdx.y * 32 + lane;
  const int rr = i / (DV / 4), ch = (i % (DV / 4)) * 4;
  const int first = head.z, n = head.w - first + 1;
  float mm = kNoMax, ll = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m, float l, float4 v, float to) {
    const float f = ex2_approx(m - to);
    ll = fmaf(f, l, ll);
    sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
    sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
  };
  auto move = [&](float to) {
    const float alpha = ex2_approx(mm - to);
    mm = to;
    ll *= alpha;
    sum.x *= alpha, sum.y *= alpha, sum.z *= alpha, sum.w *= alpha;
  };
  for (int c0 = warp; c0 < n; c0 += kAhead * kJoinWarps) {
    float m[kAhead], l[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = min(c0 + k * kJoinWarps, n - 1);
      // the first CTA's partial is its second, the others' their first
      const float* const part = p.partials + (static_cast<int64_t>(first + c) * 2 + (c == 0 ? 1 : 0)) * kFloats;
      m[k] = part[rr];
      l[k] = part[R + rr];
      v[k] = *reinterpret_cast<const float4*>(part + 2 * R + rr * DV + ch);
    }
    float now = mm;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) now = fmaxf(now, m[k]);
    move(now);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k * kJoinWarps < n) add(m[k], l[k], v[k], now);
  }
  s_m[warp][lane] = mm, s_l[warp][lane] = ll, s_v[warp][lane] = sum;
  __syncthreads();
  if (warp != 0) return;
  float now = mm;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) now = fmaxf(now, s_m[w][lane]);
  move(now);
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) add(s_m[w][lane], s_l[w][lane], s_v[w][lane], now);
  store_row<DV, R>(p, head.x, head.y, rr, ch, sum, mm, ll);
}

constexpr int kMaxDevices = 64;

// SMs of the current device, and its number (both looked up once a device).
int sm_count(int* device) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  *device = dev;
  if ((sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 0;
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

template <int DQK, int DV, int NT>
cudaError_t launch_nt(Kv4AttnParams p, cudaStream_t stream) {
  using C = Kv4Cfg<DQK, DV, NT>;
  p.row_tiles = (p.q_len * p.group + C::R - 1) / C::R;
  int dev = 0;
  const int sms = sm_count(&dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  cudaError_t e;
  static std::atomic<bool> ready[kMaxDevices];  // the kernel's attributes are set on the device
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv4_attn_kernel<DQK, DV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv4_attn_kernel<DQK, DV, NT>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  const int grid = std::min(kMaxCtas, sms * C::kCtas);
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv * p.row_tiles;
  p.by_pair = pairs <= grid ? 1 : 0;
  kv4_attn_kernel<DQK, DV, NT><<<grid, kThreads, C::kSmemBytes, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.by_pair ? pairs : grid), C::R * DV / 128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Few pairs: each may be shared by many CTAs, and the launch is small.
  if (p.by_pair && pairs * cfg.gridDim.y <= 2 * sms) {
    cfg.blockDim = dim3(32 * 16);
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<DV, C::R, 16>, p);
  }
  cfg.blockDim = dim3(32 * 4);
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<DV, C::R, 4>, p);
}

// One tile of 8 rows while they suffice, else 16: a block's codes are unpacked once for all of them.
template <int DQK, int DV>
cudaError_t launch_d(const Kv4AttnParams& p, cudaStream_t stream) {
  if (p.q_len * p.group <= 8) return launch_nt<DQK, DV, 1>(p, stream);
  return launch_nt<DQK, DV, 2>(p, stream);
}

cudaError_t launch_kv4_attn(const Kv4AttnParams& p, int dqk, int dv, cudaStream_t stream) {
  if (dqk == 64 && dv == 64) return launch_d<64, 64>(p, stream);
  if (dqk == 64 && dv == 128) return launch_d<64, 128>(p, stream);
  if (dqk == 128 && dv == 64) return launch_d<128, 64>(p, stream);
  if (dqk == 128 && dv == 128) return launch_d<128, 128>(p, stream);
  if (dqk == 192 && dv == 64) return launch_d<192, 64>(p, stream);
  if (dqk == 192 && dv == 128) return launch_d<192, 128>(p, stream);
  return cudaErrorInvalidValue;
}

constexpr size_t kHeadBytes = (kMaxCtas * sizeof(int4) + 255) / 256 * 256;

size_t workspace_bytes_for(int64_t rows, int dv) {
  const int64_t R = rows <= 8 ? 8 : 16;
  return kHeadBytes + static_cast<size_t>(kMaxCtas) * 2 * (2 * R + R * dv) * sizeof(float);
}

}  // namespace
}  // namespace slope

using namespace slope;

extern "C" {

size_t slope_kv4_attn_workspace_size(int64_t B, int64_t Hq, const slope_kv4_cache* cache, int32_t q_len) {
  if (cache == nullptr || !kv4_supported(cache->dqk, cache->dv)) return 0;
  if (B < 0 || B > 65535 || cache->Hkv < 1 || Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0) return 0;
  if (q_len < 1 || q_len > SLOPE_KV4_MAX_Q_LEN) return 0;
  return workspace_bytes_for(Hq / cache->Hkv * q_len, cache->dv);
}

slope_status slope_kv4_attn(const slope_tensor* q, const slope_kv4_cache* cache, const int32_t* block_table,
                            int64_t table_stride, int64_t max_pages, const int32_t* kv_lens, int32_t q_len,
                            int64_t window, float scale, slope_tensor* out, slope_tensor* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const CallRange range("slope_kv4_attn");
  slope_status st;
  if ((st = check_kv4_cache(cache)) != SLOPE_OK) return st;
  if (q == nullptr) return SLOPE_ERR_NULL;
  if (q->dtype != SLOPE_BF16) return SLOPE_ERR_DTYPE;
  if (q->ndim != 3) return SLOPE_ERR_SHAPE;
  if (q_len < 1) return SLOPE_ERR_SHAPE;
  if (q_len > SLOPE_KV4_MAX_Q_LEN) return SLOPE_ERR_UNSUPPORTED;
  const int64_t T = q->shape[0], Hq = q->shape[1];
  if (T < 0 || T % q_len != 0 || T / q_len > 65535) return SLOPE_ERR_SHAPE;
  if (Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0 || q->shape[2] != cache->dqk) return SLOPE_ERR_SHAPE;
  if (window < 0 || window > (int64_t(1) << 30)) return SLOPE_ERR_SHAPE;
  if (max_pages < 0 || max_pages > ((int64_t(1) << 28) - 1) / cache->page_size || table_stride < max_pages)
    return SLOPE_ERR_SHAPE;
  if ((st = check_out(out, T, Hq, cache->dv, true)) != SLOPE_OK) return st;
  if (lse != nullptr && (st = check_lse(lse, Hq, T)) != SLOPE_OK) return st;
  if (T == 0) return SLOPE_OK;
  if (q->data == nullptr || kv_lens == nullptr || (max_pages > 0 && block_table == nullptr)) return SLOPE_ERR_NULL;
  if (q->stride[2] != 1 || q->stride[0] <= 0 || q->stride[1] <= 0 || q->stride[0] % 8 || q->stride[1] % 8 ||
      !aligned(q->data, 16))
    return SLOPE_ERR_STRIDE;
  if (!aligned(kv_lens, 4) || !aligned(block_table, 4)) return SLOPE_ERR_STRIDE;
  const int64_t rows = Hq / cache->Hkv * q_len;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_for(rows, cache->dv))
    return SLOPE_ERR_WORKSPACE;

  Kv4AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.q_srow = q->stride[0];
  p.q_shead = q->stride[1];
  p.data = static_cast<const uint8_t*>(cache->data);
  p.n_pages = cache->n_pages;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_tokens = max_pages * cache->page_size;
  p.kv_lens = kv_lens;
  p.B = static_cast<int32_t>(T / q_len);
  p.q_len = q_len;
  p.Hkv = cache->Hkv;
  p.group = static_cast<int32_t>(Hq / cache->Hkv);
  p.page_shift = 4;
  while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
  p.window = static_cast<int32_t>(window);
  p.scale_log2 = resolve_scale(scale, cache->dqk) * 1.44269504088896340736f;
  p.out = out->data;
  p.out_srow = out->stride[0];
  p.out_shead = out->stride[1];
  p.out_bf16 = out->dtype == SLOPE_BF16 ? 1 : 0;
  if (lse != nullptr) {
    p.lse = static_cast<float*>(lse->data);
    p.lse_srow = lse->stride[1];
    p.lse_shead = lse->stride[0];
  }
  p.heads = static_cast<int4*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeadBytes);
  p.status = device_status_ptr();
  if (p.status == nullptr) return cuda_fail("device status word (cudaGetSymbolAddress)");
  p.wait_limit_ns = wait_limit_ns();
  const cudaError_t e = launch_kv4_attn(p, cache->dqk, cache->dv, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache attention kernel launch", e);
}

}  // extern "C"
