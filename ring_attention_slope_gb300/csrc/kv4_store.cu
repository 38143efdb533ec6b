// Writing keys and values into the 4-bit paged cache and reading them back.
//
// Both are passes over memory (2 bytes of a bf16 channel against 0.625 of a
// cached one).  Eight lanes share 64 channels of one token's head: a lane loads
// 8 channels (16 bytes of bf16), four lanes find their group's minimum and
// maximum by shuffles, and each lane ends with 8 codes, one 32-bit word.  A warp
// takes the same 64 channels of four consecutive tokens, and a CTA those of 16:
// where a run of tokens fills a block, the words of a block's sector come from
// one warp and those of its neighbours from the same CTA.
//
// Measured, bf16: writing 5001 tokens, 32 heads of 192/128, 37 us = 3.7 TB/s, and reading them back 29 us = 4.6 TB/s
// (54% and 67% of the copy rate); 12288 tokens, 8 heads of 64/64, 12.6 and 8.2 us (fp32 13.0 and 16.2); 32 tokens 2.8
// and 2.2 us, two dependent loads and the launch.  What bounds the write is instructions as much as memory: at 32768
// tokens (27 us) the issue slots are 71% busy, the ALU pipe 61%, DRAM 32%.  So it is for the read: at 32768 tokens
// (15 us) the ALU pipe is 68% busy, the issue slots 59%, DRAM 24% (most of what it wrote was still in L2).  (A lane
// with sixteen channels instead of eight was no faster, one CTA for all heads of 16 tokens 13% slower.)
//
// Rounding a quotient: with inv the scale's reciprocal to 2^-22 and q = d inv, the remainder d - q scale is
// exact and q + remainder inv differs from d / scale by 2^-44 before its own rounding.  Where d = x - min is
// exact and has at most 22 bits, as for bf16 values within 2^14 of each other, that decides every code: a
// quotient that is a half comes out as that half (and halves, common among bf16 values, round to even), and
// one that is not differs from it by a place of d at least, more than rounding to 24 bits can bridge.
// Otherwise (fp32 values, bf16 ones further apart, scales whose remainders may be subnormal) a code next to a
// half is decided again from error-free differences: d's own rounding moves the quotient by at most 2^-24 of 16,
// so 1e-5 is near enough.  (Not in fp64, of which an SM does two operations a clock: with that path the
// 12K-token store took 39 us.)
#include <cuda_bf16.h>

#include <cfloat>

#include "host.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace slope {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 16;                        // tokens of a CTA
constexpr int kHeadsPerPass = kThreads / 8 / kTokens;  // heads a CTA takes at a time

struct Kv4StoreParams {
  uint8_t* data;
  int64_t n_slots;
  int64_t T;
  const int32_t* slots;
  void* k;
  void* v;
  int64_t k_srow, k_shead, v_srow, v_shead;
  int32_t page_shift, Hkv;
  int32_t per_cta;  // heads of a CTA
};

// A token's block of head 0, and where it lies in it.
struct Place {
  uint8_t* block;
  int64_t head_bytes;  // from a head's block to the next one's
  int t;               // token in the block
};

template <int DQK, int DV>
__device__ __forceinline__ Place place_of(const Kv4StoreParams& p, int64_t slot) {
  Place at;
  const int in_page = static_cast<int>(slot) & ((1 << p.page_shift) - 1);
  at.head_bytes = static_cast<int64_t>(kv4_block_bytes(DQK, DV)) << (p.page_shift - 4);
  at.block = p.data + (slot >> p.page_shift) * p.Hkv * at.head_bytes + in_page / kKv4Block * kv4_block_bytes(DQK, DV);
  at.t = in_page % kKv4Block;
  return at;
}

template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  // channels 2 i and 2 i + 1
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t u = (&r[0].x)[i];
      return pack_f32x2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
      return pack_f32x2(__uint_as_float((&r[i / 2].x)[i % 2 * 2]), __uint_as_float((&r[i / 2].x)[i % 2 * 2 + 1]));
    }
  }
};

// Smaller of two numbers, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Of a lane's 8 channels: smallest (NaN if any is), largest, smallest magnitude.
struct Extremes {
  float lo, hi, small;
};
__device__ __forceinline__ Extremes extremes(const Raw8<__nv_bfloat16>& x) {
  __nv_bfloat162 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const __nv_bfloat162*>(&x.r[0])[i];
  const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3]));
  const __nv_bfloat162 hi = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __habs2(v[i]);
  const __nv_bfloat162 small = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
  return {min_nan(__low2float(lo), __high2float(lo)), fmaxf(__low2float(hi), __high2float(hi)),
          fminf(__low2float(small), __high2float(small))};
}
__device__ __forceinline__ Extremes extremes(const Raw8<float>& x) {
  Extremes e{INFINITY, -INFINITY, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __uint_as_float((&x.r[i / 4].x)[i % 4]);
    e.lo = min_nan(e.lo, f);
    e.hi = fmaxf(e.hi, f);
  }
  return e;
}

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, halves to even

// The code of one value, from error-free steps: with d + e = x - mn exactly, n the integer below the quotient
// (or, next to an integer, the one on its other side), d - (n + 1/2) scale has the sign of the exact difference
// and is exact where it is small, and e decides a tie.  (An e below 2^-52 of d is one that fp64 does not see.)
__device__ __noinline__ float code_of(float x, float mn, float scale, float inv) {
  const float d = __fsub_rn(x, mn);
  const float back = __fsub_rn(d, x);
  float e = __fadd_rn(__fsub_rn(x, __fsub_rn(d, back)), __fsub_rn(-mn, back));
  if (fabsf(e) <= fabsf(d) * 0x1p-52f) e = 0.f;
  const float q = __fmul_rn(d, inv), t = fmaf(fmaf(-q, scale, d), inv, q);
  const float n = rintf(fminf(fmaxf(t, 0.f), 15.f) - 0.5f);
  const float over = __fadd_rn(fmaf(-(n + 0.5f), scale, d), e);
  const bool odd = static_cast<int>(n) & 1;
  return fminf(fmaxf(over > 0.f || (over == 0.f && odd) ? n + 1.f : n, 0.f), 15.f);
}

// Eight lanes' 64 channels of one token's head: the lane's eight codes, and its group's word.
// Every lane of the warp calls it.
struct Quantised {
  uint32_t codes, word;
};
template <typename T>
__device__ __forceinline__ Quantised quantise(const Raw8<T>& x) {
  const Extremes ex = extremes(x);
  float lo = ex.lo, hi = ex.hi;
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const __nv_bfloat16 min_b = __float2bfloat16_rn(lo);
  const float mn = __bfloat162float(min_b);
  const float span = __fsub_rn(hi, mn);
  const bool nan_group = !(span <= FLT_MAX);  // a NaN or an infinity among them, or too wide a range
  float scale = __bfloat162float(__float2bfloat16_rn(__fmul_rn(span, 1.f / 15.f)));
  if (!(scale >= FLT_MIN) || nan_group) scale = 0.f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  if (scale == 0.f) inv = 0.f;
  // The quotients; scale 0 makes them 0.  bf16: none is below 0 (the minimum is exact) or above
  // 15 / (1 - 2^-8), so none rounds to a number past 0 .. 15.
  uint64_t t[4], r[4];
  const uint64_t mn2 = pack_f32x2(-mn, -mn), inv2 = pack_f32x2(inv, inv), ns2 = pack_f32x2(-scale, -scale);
  const uint64_t round2 = pack_f32x2(kRound, kRound);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t d = add_f32x2(x.pair(i), mn2), q = mul_f32x2(d, inv2);
    t[i] = fma_f32x2(fma_f32x2(q, ns2, d), inv2, q);
    if constexpr (sizeof(T) == 4) {
      const float2 f = unpack_f32x2(t[i]);
      t[i] = pack_f32x2(fminf(fmaxf(f.x, 0.f), 15.f), fminf(fmaxf(f.y, 0.f), 15.f));
    }
    r[i] = add_f32x2(t[i], round2);
  }
  bool again;
  if constexpr (sizeof(T) == 2) {
    again = ex.small * 16384.f < fabsf(mn) || fmaxf(fabsf(lo), fabsf(hi)) > 16384.f * fabsf(mn) || scale < 0x1p-100f;
  } else {
    float off = 0.f;  // largest distance from the nearest integer
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack_f32x2(t[i]), b = unpack_f32x2(r[i]);
      off = fmaxf(off, fmaxf(fabsf(a.x - (b.x - kRound)), fabsf(a.y - (b.y - kRound))));
    }
    again = off > 0.5f - 1e-5f || scale < 0x1p-100f;
  }
  if (again && scale > 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_f32x2(x.pair(i));
      r[i] = pack_f32x2(code_of(f.x, mn, scale, inv) + kRound, code_of(f.y, mn, scale, inv) + kRound);
    }
  }
  // 1.5 * 2^23 + n has n in its low bits: shifted and added, the eight patterns leave the codes and a constant
  uint32_t codes = 0u - 0x4b400000u * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_f32x2(r[i]);
    codes += (__float_as_uint(f.x) << (8 * i)) + (__float_as_uint(f.y) << (8 * i + 4));
  }
  if (nan_group) codes = 0;
  const uint32_t word = nan_group ? 0x00007fc0u
                                  : (__float_as_uint(scale) & 0xffff0000u) | static_cast<uint32_t>(__bfloat16_as_ushort(min_b));
  return {codes, word};
}

template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4StoreParams p) {
  constexpr int kKc = DQK / 64, kVc = DV / 64, kChunks = kKc + kVc;
  constexpr int kNk = kv4_key_bytes(DQK), kNv = kv4_value_bytes(DV), kWords = kv4_words(DQK, DV);
  const int lane8 = threadIdx.x % 8;
  const bool high = lane8 >= 4;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  int64_t slot = -1;
  if (tok < p.T) {
    slot = p.slots[tok];
    if (slot >= p.n_slots) slot = -1;
  }
  // lanes without a slot go along for the shuffles
  const bool live = slot >= 0;
  const Place at = place_of<DQK, DV>(p, live ? slot : 0);
  const int h_end = min(p.Hkv, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  int h = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens);  // the same for a whole warp
  const T* k = static_cast<const T*>(p.k) + tok * p.k_srow + h * p.k_shead + lane8 * 8;
  const T* v = static_cast<const T*>(p.v) + tok * p.v_srow + h * p.v_shead + lane8 * 8;
  // the lane's places in a block: key words of its groups, value words, scale words
  uint8_t* block = at.block + h * at.head_bytes;
  const int k_at = (at.t % 8 * 4 + (lane8 & 3)) * 16, k_word = at.t / 8 * (DQK / kKv4Group) + (high ? 1 : 0);
  const int v_at = kNk + kv4_value_offset(at.t, 0, 2 * (lane8 & 3) + (high ? 1 : 0));
  const int w_at = kNk + kNv + 4 * (at.t * kWords + (high ? 1 : 0));
  Raw8<T> x[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    x[c] = Raw8<T>{};
    if (live && h < h_end) x[c].load(c < kKc ? k + c * 64 : v + (c - kKc) * 64);
  }
  for (; h < h_end; h += kHeadsPerPass) {
    k += kHeadsPerPass * p.k_shead;
    v += kHeadsPerPass * p.v_shead;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const Quantised z = quantise(x[c]);
      // the next head's channels are in flight while this one's other chunks are worked on
      if (live && h + kHeadsPerPass < h_end) x[c].load(c < kKc ? k + c * 64 : v + (c - kKc) * 64);
      // a value's lanes l and l + 4 hold the codes of the same operand lanes g = 2 l, 2 l + 1 for the chunk's
      // two groups: the lower keeps its first four and gets the other's first four, the upper the second ones
      const uint32_t other = c < kKc ? 0 : __shfl_xor_sync(0xffffffffu, high ? z.codes : z.codes >> 16, 4);
      if (!live) continue;
      if (c < kKc) {
        const int w = k_word + 2 * c;
        *reinterpret_cast<uint32_t*>(block + k_at + (w >> 2) * 512 + (w & 3) * 4) = z.codes;
      } else {
        *reinterpret_cast<uint32_t*>(block + v_at + (c - kKc) * 512) =
            high ? __byte_perm(other, z.codes, 0x7610) : __byte_perm(z.codes, other, 0x5410);
      }
      if ((lane8 & 3) == 0) *reinterpret_cast<uint32_t*>(block + w_at + 8 * c) = z.word;
    }
    block += kHeadsPerPass * at.head_bytes;
  }
}

template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4StoreParams p) {
  constexpr int kKc = DQK / 64, kVc = DV / 64, kChunks = kKc + kVc;
  constexpr int kNk = kv4_key_bytes(DQK), kNv = kv4_value_bytes(DV), kWords = kv4_words(DQK, DV);
  constexpr int kWide = kChunks == 2 ? 2 : 1;  // heads whose loads are in flight together
  const int lane8 = threadIdx.x % 8, high = lane8 / 4;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  if (tok >= p.T) return;
  const int64_t slot = p.slots[tok];
  if (slot < 0 || slot >= p.n_slots) return;
  const Place at = place_of<DQK, DV>(p, slot);
  const int h_end = min(p.Hkv, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  int h = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens);
  T* k = static_cast<T*>(p.k) + tok * p.k_srow + h * p.k_shead + lane8 * 8;
  T* v = static_cast<T*>(p.v) + tok * p.v_srow + h * p.v_shead + lane8 * 8;
  const uint8_t* block = at.block + h * at.head_bytes;
  const int k_at = (at.t % 8 * 4 + (lane8 & 3)) * 16, k_word = at.t / 8 * (DQK / kKv4Group) + high;
  const int v_at = kNk + kv4_value_offset(at.t, 0, 2 * (lane8 & 3)) + 2 * high;
  constexpr int kNextG = kv4_value_offset(0, 0, 1) - kv4_value_offset(0, 0, 0);
  const int w_at = kNk + kNv + 4 * (at.t * kWords + high);
  for (; h < h_end; h += kWide * kHeadsPerPass) {
    uint32_t codes[kWide][kChunks], word[kWide][kChunks];
#pragma unroll
    for (int a = 0; a < kWide; ++a) {
      if (h + a * kHeadsPerPass >= h_end) break;
      const uint8_t* const b = block + a * kHeadsPerPass * at.head_bytes;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c < kKc) {
          const int w = k_word + 2 * c;
          codes[a][c] = __ldg(reinterpret_cast<const uint32_t*>(b + k_at + (w >> 2) * 512 + (w & 3) * 4));
        } else {
          const uint8_t* const vb = b + v_at + (c - kKc) * 512;
          codes[a][c] = __ldg(reinterpret_cast<const uint16_t*>(vb)) |
                        static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(vb + kNextG))) << 16;
        }
        word[a][c] = __ldg(reinterpret_cast<const uint32_t*>(b + w_at + 8 * c));
      }
    }
#pragma unroll
    for (int a = 0; a < kWide; ++a) {
      if (h + a * kHeadsPerPass >= h_end) break;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float scale = __uint_as_float(word[a][c] & 0xffff0000u), mn = __uint_as_float(word[a][c] << 16);
        const uint64_t s2 = pack_f32x2(scale, scale), m2 = pack_f32x2(mn, mn), base2 = pack_f32x2(-8388608.f, -8388608.f);
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 2^23 + code as a float, less 2^23
          const uint64_t n = pack_f32x2(__uint_as_float(((codes[a][c] >> (8 * i)) & 15u) | 0x4b000000u),
                                        __uint_as_float(((codes[a][c] >> (8 * i + 4)) & 15u) | 0x4b000000u));
          x[i] = unpack_f32x2(fma_f32x2(s2, add_f32x2(n, base2), m2));
        }
        T* const dst = c < kKc ? k + a * kHeadsPerPass * p.k_shead + c * 64 : v + a * kHeadsPerPass * p.v_shead + (c - kKc) * 64;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                                                      pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
        } else {
          *reinterpret_cast<float4*>(dst) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
        }
      }
    }
    k += kWide * kHeadsPerPass * p.k_shead;
    v += kWide * kHeadsPerPass * p.v_shead;
    block += kWide * kHeadsPerPass * at.head_bytes;
  }
}

template <typename T, int DQK, int DV>
cudaError_t launch_store_d(const Kv4StoreParams& p, bool write, dim3 grid, cudaStream_t stream) {
  if (write)
    kv4_write_kernel<T, DQK, DV><<<grid, kThreads, 0, stream>>>(p);
  else
    kv4_read_kernel<T, DQK, DV><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_store(const Kv4StoreParams& p, int dqk, int dv, bool write, dim3 grid, cudaStream_t stream) {
  if (dqk == 64 && dv == 64) return launch_store_d<T, 64, 64>(p, write, grid, stream);
  if (dqk == 64 && dv == 128) return launch_store_d<T, 64, 128>(p, write, grid, stream);
  if (dqk == 128 && dv == 64) return launch_store_d<T, 128, 64>(p, write, grid, stream);
  if (dqk == 128 && dv == 128) return launch_store_d<T, 128, 128>(p, write, grid, stream);
  if (dqk == 192 && dv == 64) return launch_store_d<T, 192, 64>(p, write, grid, stream);
  if (dqk == 192 && dv == 128) return launch_store_d<T, 192, 128>(p, write, grid, stream);
  return cudaErrorInvalidValue;
}

// k and v of one token count and type, rows readable 8 channels at a time; fills the parameters.
slope_status prepare_store(const slope_kv4_cache* cache, const slope_tensor* k, const slope_tensor* v,
                           const int32_t* slots, Kv4StoreParams& p) {
  slope_status st;
  if ((st = check_kv4_cache(cache)) != SLOPE_OK) return st;
  if (k == nullptr || v == nullptr) return SLOPE_ERR_NULL;
  const int64_t d[2] = {cache->dqk, cache->dv};
  const slope_tensor* t[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    if (t[i]->dtype != SLOPE_BF16 && t[i]->dtype != SLOPE_F32) return SLOPE_ERR_DTYPE;
    if (t[i]->dtype != k->dtype) return SLOPE_ERR_DTYPE;
    if (t[i]->ndim != 3 || t[i]->shape[0] != k->shape[0] || t[i]->shape[1] != cache->Hkv || t[i]->shape[2] != d[i])
      return SLOPE_ERR_SHAPE;
    if (t[i]->shape[0] < 0 || t[i]->shape[0] > (int64_t(1) << 30)) return SLOPE_ERR_SHAPE;
    if (t[i]->shape[0] == 0) continue;
    if (t[i]->data == nullptr) return SLOPE_ERR_NULL;
    if (t[i]->stride[2] != 1 || t[i]->stride[0] <= 0 || t[i]->stride[1] <= 0 || t[i]->stride[0] % 8 ||
        t[i]->stride[1] % 8 || !aligned(t[i]->data, 16))
      return SLOPE_ERR_STRIDE;
  }
  p.T = k->shape[0];
  if (p.T > 0 && slots == nullptr) return SLOPE_ERR_NULL;
  if (p.T > 0 && !aligned(slots, 4)) return SLOPE_ERR_STRIDE;
  p.data = static_cast<uint8_t*>(cache->data);
  p.n_slots = cache->n_pages * cache->page_size;
  p.slots = slots;
  p.k = k->data;
  p.v = v->data;
  p.k_srow = k->stride[0], p.k_shead = k->stride[1];
  p.v_srow = v->stride[0], p.v_shead = v->stride[1];
  p.page_shift = 4;
  while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
  p.Hkv = cache->Hkv;
  return SLOPE_OK;
}

dim3 store_grid(Kv4StoreParams& p) {
  const int64_t tx = (p.T + kTokens - 1) / kTokens;
  // a CTA takes one head at a time, and more in turn while more than about 32 CTAs are left for
  // each of the 152 SMs
  p.per_cta = kHeadsPerPass;
  while (p.per_cta < p.Hkv && tx * ((p.Hkv + p.per_cta - 1) / p.per_cta) > 4864) p.per_cta *= 2;
  return dim3(static_cast<unsigned>(tx), static_cast<unsigned>((p.Hkv + p.per_cta - 1) / p.per_cta));
}

}  // namespace

slope_status check_kv4_cache(const slope_kv4_cache* c) {
  if (c == nullptr) return SLOPE_ERR_NULL;
  if (!kv4_supported(c->dqk, c->dv)) return SLOPE_ERR_UNSUPPORTED;
  if (c->n_pages < 0 || c->Hkv < 1 || c->Hkv > 65535) return SLOPE_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return SLOPE_ERR_SHAPE;
  if (c->n_pages > ((int64_t(1) << 31) - 1) / c->page_size) return SLOPE_ERR_SHAPE;
  if (c->n_pages > 0 && c->data == nullptr) return SLOPE_ERR_NULL;
  if (!aligned(c->data, 16)) return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

}  // namespace slope

using namespace slope;

extern "C" {

size_t slope_kv4_block_bytes(int32_t dqk, int32_t dv) {
  return kv4_supported(dqk, dv) ? static_cast<size_t>(kv4_block_bytes(dqk, dv)) : 0;
}

size_t slope_kv4_cache_bytes(int64_t n_pages, int32_t page_size, int32_t Hkv, int32_t dqk, int32_t dv) {
  const slope_kv4_cache c{reinterpret_cast<void*>(16), n_pages, page_size, Hkv, dqk, dv};
  if (check_kv4_cache(&c) != SLOPE_OK) return 0;
  return static_cast<size_t>(n_pages) * static_cast<size_t>(page_size / kKv4Block) * static_cast<size_t>(Hkv) *
         slope_kv4_block_bytes(dqk, dv);
}

slope_status slope_kv4_write(const slope_kv4_cache* cache, const slope_tensor* k, const slope_tensor* v,
                             const int32_t* slots, void* stream) {
  const CallRange range("slope_kv4_write");
  Kv4StoreParams p{};
  const slope_status st = prepare_store(cache, k, v, slots, p);
  if (st != SLOPE_OK) return st;
  if (p.T == 0) return SLOPE_OK;
  const dim3 grid = store_grid(p);
  auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = k->dtype == SLOPE_BF16
                            ? launch_store<__nv_bfloat16>(p, cache->dqk, cache->dv, true, grid, s)
                            : launch_store<float>(p, cache->dqk, cache->dv, true, grid, s);
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache write kernel launch", e);
}

slope_status slope_kv4_read(const slope_kv4_cache* cache, const int32_t* slots, slope_tensor* k, slope_tensor* v,
                            void* stream) {
  const CallRange range("slope_kv4_read");
  Kv4StoreParams p{};
  const slope_status st = prepare_store(cache, k, v, slots, p);
  if (st != SLOPE_OK) return st;
  if (p.T == 0) return SLOPE_OK;
  const dim3 grid = store_grid(p);
  auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = k->dtype == SLOPE_BF16
                            ? launch_store<__nv_bfloat16>(p, cache->dqk, cache->dv, false, grid, s)
                            : launch_store<float>(p, cache->dqk, cache->dv, false, grid, s);
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache read kernel launch", e);
}

}  // extern "C"
