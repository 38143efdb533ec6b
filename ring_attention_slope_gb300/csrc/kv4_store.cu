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
// Rounding a quotient: with inv the correctly rounded reciprocal of the scale and q = d inv,
// fma(fma(-q, scale, d), inv, q) is the correctly rounded d / scale (Markstein, 1990).  Where
// d = x - min is exact, as it is for bf16 values within 2^16 of each other, a quotient that rounds to a
// half is one (d - (n + 1/2) scale is a multiple of d's last place, so a quotient next to a half is further
// off than half a place), and rounding halves to even decides it rightly: halves are common among bf16 values.
// Otherwise d's own rounding moves the quotient by at most 2^-24 of 16: one closer than 1e-5 to a
// half, which is rare then, is divided again in fp64.
#include <cuda_bf16.h>

#include <cfloat>

#include "host.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace slope {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;                        // tokens of a CTA
constexpr int kUnitsPerPass = kThreads / 8 / kTokens;  // (head, 64-channel chunk) pairs a CTA takes at a time

struct Kv4StoreParams {
  uint8_t* data;
  int64_t n_slots;
  int64_t T;
  const int32_t* slots;
  void* k;
  void* v;
  int64_t k_srow, k_shead, v_srow, v_shead;
  int32_t page_shift, Hkv;
  int32_t units;     // Hkv * (dqk + dv) / 64
  int32_t per_cta;   // units of a CTA
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

// Of a lane's 8 channels: smallest, largest, smallest magnitude, and whether one is not finite.
struct Extremes {
  float lo, hi, small;
  bool bad;
};
__device__ __forceinline__ Extremes extremes(const Raw8<__nv_bfloat16>& x) {
  __nv_bfloat162 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const __nv_bfloat162*>(&x.r[0])[i];
  const __nv_bfloat162 lo = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
  const __nv_bfloat162 hi = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __habs2(v[i]);
  const __nv_bfloat162 small = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
  const __nv_bfloat162 large = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
  return {fminf(__low2float(lo), __high2float(lo)), fmaxf(__low2float(hi), __high2float(hi)),
          fminf(__low2float(small), __high2float(small)),
          !(__low2float(large) <= FLT_MAX && __high2float(large) <= FLT_MAX)};
}
__device__ __forceinline__ Extremes extremes(const Raw8<float>& x) {
  Extremes e{INFINITY, -INFINITY, 0.f, false};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __uint_as_float((&x.r[i / 4].x)[i % 4]);
    e.lo = fminf(e.lo, f);
    e.hi = fmaxf(e.hi, f);
    e.bad |= !(fabsf(f) <= FLT_MAX);
  }
  return e;
}

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, halves to even

template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4StoreParams p) {
  constexpr int kKc = DQK / 64, kPerHead = kKc + DV / 64;
  constexpr int kNk = kv4_key_bytes(DQK), kNv = kv4_value_bytes(DV), kWords = kv4_words(DQK, DV);
  const int lane8 = threadIdx.x % 8;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  int64_t slot = -1;
  if (tok < p.T) {
    slot = p.slots[tok];
    if (slot >= p.n_slots) slot = -1;
  }
  // lanes without a slot go along for the shuffles
  const bool live = slot >= 0;
  const Place at = place_of<DQK, DV>(p, live ? slot : 0);
  const T* const k = static_cast<const T*>(p.k) + tok * p.k_srow + lane8 * 8;
  const T* const v = static_cast<const T*>(p.v) + tok * p.v_srow + lane8 * 8;
  auto fetch = [&](int u, Raw8<T>& x) {
    const int head = u / kPerHead, c = u - head * kPerHead;
    x = Raw8<T>{};
    if (live) x.load(c < kKc ? k + static_cast<int64_t>(head) * p.k_shead + c * 64
                             : v + static_cast<int64_t>(head) * p.v_shead + (c - kKc) * 64);
  };
  const int u_end = min(p.units, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  int u = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens);  // the same for a whole warp
  Raw8<T> next;
  if (u < u_end) fetch(u, next);
  for (; u < u_end; u += kUnitsPerPass) {
    const Raw8<T> x = next;
    if (u + kUnitsPerPass < u_end) fetch(u + kUnitsPerPass, next);
    const Extremes ex = extremes(x);
    float lo = ex.lo, hi = ex.hi;
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const uint32_t bad_lanes = __ballot_sync(0xffffffffu, ex.bad) >> (threadIdx.x & 28);
    const __nv_bfloat16 min_b = __float2bfloat16_rn(lo);
    const float mn = __bfloat162float(min_b);
    const float span = __fsub_rn(hi, mn);
    float scale = __bfloat162float(__float2bfloat16_rn(__fmul_rn(span, 1.f / 15.f)));
    const bool nan_group = (bad_lanes & 15u) != 0 || !(fabsf(mn) <= FLT_MAX) || !(span <= FLT_MAX);
    if (!(scale >= FLT_MIN) || nan_group) scale = 0.f;
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    // The quotients; scale 0 makes them 0.  bf16: none is below 0 (the minimum is exact) or above
    // 15 / (1 - 2^-8), so none rounds to a number past 0 .. 15.
    uint64_t r[4];
    float off = 0.f;  // largest distance from the nearest integer
    const uint64_t mn2 = pack_f32x2(-mn, -mn), inv2 = pack_f32x2(inv, inv), ns2 = pack_f32x2(-scale, -scale);
    const uint64_t round2 = pack_f32x2(kRound, kRound), unround2 = pack_f32x2(-kRound, -kRound);
    const bool inexact = sizeof(T) == 4 || ex.small * 65536.f < fabsf(mn) ||
                         fmaxf(fabsf(lo), fabsf(hi)) > 65536.f * fabsf(mn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t d = add_f32x2(x.pair(i), mn2), q = mul_f32x2(d, inv2);
      uint64_t t = fma_f32x2(fma_f32x2(q, ns2, d), inv2, q);
      if constexpr (sizeof(T) == 4) {
        const float2 f = unpack_f32x2(t);
        t = pack_f32x2(fminf(fmaxf(f.x, 0.f), 15.f), fminf(fmaxf(f.y, 0.f), 15.f));
      }
      r[i] = add_f32x2(t, round2);
      if (inexact) {
        const float2 e = unpack_f32x2(add_f32x2(t, mul_f32x2(add_f32x2(r[i], unround2), pack_f32x2(-1.f, -1.f))));
        off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
      }
    }
    if (inexact && off > 0.5f - 1e-5f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_f32x2(x.pair(i));
        auto divide = [&](float v) {
          const double t = rint((static_cast<double>(v) - static_cast<double>(mn)) / static_cast<double>(scale));
          return static_cast<float>(fmin(fmax(t, 0.), 15.)) + kRound;
        };
        r[i] = pack_f32x2(divide(f.x), divide(f.y));
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
    const uint32_t c_lo = codes & 0xffffu, c_hi = codes >> 16;
    const uint32_t word = nan_group ? 0x00007fc0u
                                    : (__float_as_uint(scale) & 0xffff0000u) | static_cast<uint32_t>(__bfloat16_as_ushort(min_b));
    const int head = u / kPerHead, c = u - head * kPerHead;
    uint8_t* const block = at.block + head * at.head_bytes;
    const bool high = lane8 >= 4;
    if (c < kKc) {
      const int group = c * 2 + (high ? 1 : 0);
      if (live) {
        *reinterpret_cast<uint32_t*>(block + kv4_key_offset(DQK, at.t, group, lane8 & 3)) = codes;
        if ((lane8 & 3) == 0) *reinterpret_cast<uint32_t*>(block + kNk + kNv + 4 * (at.t * kWords + group)) = word;
      }
    } else {
      // lanes l and l + 4 hold the codes of the same lanes g = 2 l, 2 l + 1 for the chunk's two groups: the
      // lower keeps its first four and gets the other's first four, the upper the second ones
      const uint32_t other = __shfl_xor_sync(0xffffffffu, high ? c_lo : c_hi, 4);
      const int chunk = c - kKc, g = 2 * (lane8 & 3) + (high ? 1 : 0);
      if (live) {
        *reinterpret_cast<uint32_t*>(block + kNk + kv4_value_offset(at.t, chunk, g)) =
            high ? other | (c_hi << 16) : c_lo | (other << 16);
        if ((lane8 & 3) == 0)
          *reinterpret_cast<uint32_t*>(block + kNk + kNv + 4 * (at.t * kWords + DQK / kKv4Group + chunk * 2 + (high ? 1 : 0))) =
              word;
      }
    }
  }
}

template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4StoreParams p) {
  constexpr int kKc = DQK / 64, kPerHead = kKc + DV / 64;
  constexpr int kNk = kv4_key_bytes(DQK), kNv = kv4_value_bytes(DV), kWords = kv4_words(DQK, DV);
  const int lane8 = threadIdx.x % 8, high = lane8 / 4;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  if (tok >= p.T) return;
  const int64_t slot = p.slots[tok];
  if (slot < 0 || slot >= p.n_slots) return;
  const Place at = place_of<DQK, DV>(p, slot);
  T* const k = static_cast<T*>(p.k) + tok * p.k_srow + lane8 * 8;
  T* const v = static_cast<T*>(p.v) + tok * p.v_srow + lane8 * 8;
  const int u_end = min(p.units, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  constexpr int kAhead = 4;  // units whose loads are in flight together
  for (int u0 = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens); u0 < u_end; u0 += kAhead * kUnitsPerPass) {
    uint32_t codes[kAhead], word[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int u = min(u0 + a * kUnitsPerPass, u_end - 1);
      const int head = u / kPerHead, c = u - head * kPerHead;
      const uint8_t* const block = at.block + head * at.head_bytes;
      const uint8_t* const words = block + kNk + kNv + 4 * (at.t * kWords + high);
      if (c < kKc) {
        codes[a] = __ldg(reinterpret_cast<const uint32_t*>(block + kv4_key_offset(DQK, at.t, c * 2 + high, lane8 & 3)));
        word[a] = __ldg(reinterpret_cast<const uint32_t*>(words + 8 * c));
      } else {
        const int chunk = c - kKc;
        const uint8_t* const b = block + kNk + kv4_value_offset(at.t, chunk, 2 * (lane8 & 3)) + 2 * high;
        constexpr int kNextG = kv4_value_offset(0, 0, 1) - kv4_value_offset(0, 0, 0);
        codes[a] = __ldg(reinterpret_cast<const uint16_t*>(b)) |
                   static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(b + kNextG))) << 16;
        word[a] = __ldg(reinterpret_cast<const uint32_t*>(words + 4 * (DQK / kKv4Group) + 8 * chunk));
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int u = u0 + a * kUnitsPerPass;
      if (u >= u_end) break;
      const int head = u / kPerHead, c = u - head * kPerHead;
      const float scale = __uint_as_float(word[a] & 0xffff0000u), mn = __uint_as_float(word[a] << 16);
      const uint64_t s2 = pack_f32x2(scale, scale), m2 = pack_f32x2(mn, mn), base2 = pack_f32x2(-8388608.f, -8388608.f);
      float2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 2^23 + code as a float, less 2^23
        const uint64_t n = pack_f32x2(__uint_as_float(((codes[a] >> (8 * i)) & 15u) | 0x4b000000u),
                                      __uint_as_float(((codes[a] >> (8 * i + 4)) & 15u) | 0x4b000000u));
        x[i] = unpack_f32x2(fma_f32x2(s2, add_f32x2(n, base2), m2));
      }
      T* const dst = c < kKc ? k + static_cast<int64_t>(head) * p.k_shead + c * 64
                             : v + static_cast<int64_t>(head) * p.v_shead + (c - kKc) * 64;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                                                    pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
      } else {
        *reinterpret_cast<float4*>(dst) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
      }
    }
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
  p.units = cache->Hkv * ((cache->dqk + cache->dv) / 64);
  return SLOPE_OK;
}

dim3 store_grid(Kv4StoreParams& p) {
  const int64_t tx = (p.T + kTokens - 1) / kTokens;
  // a few passes to a CTA once there are enough CTAs without them
  p.per_cta = kUnitsPerPass;
  while (p.per_cta < p.units && (tx * ((p.units + p.per_cta - 1) / p.per_cta) > 4864 ||
                                 (p.units + p.per_cta - 1) / p.per_cta > 65535))
    p.per_cta *= 2;
  return dim3(static_cast<unsigned>(tx), static_cast<unsigned>((p.units + p.per_cta - 1) / p.per_cta));
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
