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
// Rounding a quotient: the fast path multiplies by the scale's reciprocal, which
// is off by at most 3 * 2^-24 * 16 < 3e-6 code steps (three fp32 roundings of a
// quotient below 16).  A quotient closer than 1e-5 to a half is divided again in
// fp64, so that every code is the one the definition names.
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
  int32_t page_size, Hkv, dqk, dv;
  int32_t units;     // Hkv * (dqk + dv) / 64
  int32_t per_cta;   // units of a CTA
};

// Where a (token, unit) lies: the block's address, the token's number in it, and the unit's part.
struct Place {
  uint8_t* block;
  int t;       // token in the block
  int head;
  int chunk;   // 64-channel chunk of the keys, or of the values
  bool value;
};

__device__ __forceinline__ Place place_of(const Kv4StoreParams& p, int64_t slot, int unit) {
  const int kc = p.dqk / 64, per_head = kc + p.dv / 64;
  Place at;
  at.head = unit / per_head;
  const int c = unit - at.head * per_head;
  at.value = c >= kc;
  at.chunk = at.value ? c - kc : c;
  const int64_t page = slot / p.page_size;
  const int in_page = static_cast<int>(slot - page * p.page_size);
  const int64_t block = (page * p.Hkv + at.head) * (p.page_size / kKv4Block) + in_page / kKv4Block;
  at.block = p.data + block * kv4_block_bytes(p.dqk, p.dv);
  at.t = in_page % kKv4Block;
  return at;
}

template <typename T>
__device__ __forceinline__ void load8(const T* x, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(x));
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 r = __ldcs(reinterpret_cast<const float4*>(x + 4 * i));
      v[4 * i] = r.x, v[4 * i + 1] = r.y, v[4 * i + 2] = r.z, v[4 * i + 3] = r.w;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4StoreParams p) {
  const int lane8 = threadIdx.x % 8;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  int64_t slot = -1;
  if (tok < p.T) {
    slot = p.slots[tok];
    if (slot >= p.n_slots) slot = -1;
  }
  const int u_end = min(p.units, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  for (int u = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens); u < u_end; u += kUnitsPerPass) {
    // lanes of one warp have the same unit; those without a slot go along for the shuffles
    const bool live = slot >= 0;
    const Place at = place_of(p, live ? slot : 0, u);
    const int ch = at.chunk * 64 + lane8 * 8;
    float x[8];
    if (live) {
      const T* src = at.value ? static_cast<const T*>(p.v) + tok * p.v_srow + at.head * p.v_shead + ch
                              : static_cast<const T*>(p.k) + tok * p.k_srow + at.head * p.k_shead + ch;
      load8(src, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    float lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      bad |= !(fabsf(x[i]) <= FLT_MAX);
    }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const uint32_t bad_lanes = __ballot_sync(0xffffffffu, bad) >> (threadIdx.x & 28);
    __nv_bfloat16 min_b = __float2bfloat16_rn(lo);
    const float mn = __bfloat162float(min_b);
    const float span = __fsub_rn(hi, mn);
    __nv_bfloat16 scale_b = __float2bfloat16_rn(__fmul_rn(span, 1.f / 15.f));
    float scale = __bfloat162float(scale_b);
    if (!(scale >= FLT_MIN)) scale = 0.f;
    const bool nan_group = (bad_lanes & 15u) != 0 || !(fabsf(mn) <= FLT_MAX) || !(span <= FLT_MAX);
    if (nan_group) scale = 0.f;
    uint32_t codes = 0;
    if (scale > 0.f) {
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = (x[i] - mn) * inv;
        float r = rintf(t);
        if (fabsf(t - r) > 0.5f - 1e-5f)
          r = static_cast<float>(rint((static_cast<double>(x[i]) - static_cast<double>(mn)) / static_cast<double>(scale)));
        codes |= static_cast<uint32_t>(fminf(fmaxf(r, 0.f), 15.f)) << (4 * i);
      }
    }
    const uint32_t word = nan_group ? 0x00007fc0u
                                    : (__float_as_uint(scale) & 0xffff0000u) | static_cast<uint32_t>(__bfloat16_as_ushort(min_b));
    // values: lanes l and l + 4 hold the same lanes' codes of the chunk's two groups and swap halves
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 4);
    if (!live) continue;
    const int group = at.chunk * 2 + lane8 / 4;
    const int nk = kv4_key_bytes(p.dqk), nv = kv4_value_bytes(p.dv);
    if (!at.value) {
      *reinterpret_cast<uint32_t*>(at.block + kv4_key_offset(p.dqk, at.t, group, lane8 & 3)) = codes;
    } else {
      const bool high = lane8 >= 4;
      const int g = 2 * (lane8 & 3) + (high ? 1 : 0);
      const uint32_t w = high ? (other >> 16) | (codes & 0xffff0000u) : (codes & 0xffffu) | (other << 16);
      *reinterpret_cast<uint32_t*>(at.block + nk + kv4_value_offset(at.t, at.chunk, g)) = w;
    }
    if ((lane8 & 3) == 0) {
      const int wi = at.t * kv4_words(p.dqk, p.dv) + (at.value ? p.dqk / kKv4Group : 0) + group;
      *reinterpret_cast<uint32_t*>(at.block + nk + nv + 4 * wi) = word;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4StoreParams p) {
  const int lane8 = threadIdx.x % 8;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / 8 % kTokens;
  if (tok >= p.T) return;
  const int64_t slot = p.slots[tok];
  if (slot < 0 || slot >= p.n_slots) return;
  const int u_end = min(p.units, static_cast<int>(blockIdx.y + 1) * p.per_cta);
  for (int u = blockIdx.y * p.per_cta + threadIdx.x / (8 * kTokens); u < u_end; u += kUnitsPerPass) {
    const Place at = place_of(p, slot, u);
    const int group = at.chunk * 2 + lane8 / 4;
    const int nk = kv4_key_bytes(p.dqk), nv = kv4_value_bytes(p.dv);
    uint32_t codes;
    if (!at.value) {
      codes = *reinterpret_cast<const uint32_t*>(at.block + kv4_key_offset(p.dqk, at.t, group, lane8 & 3));
    } else {
      const uint8_t* b = at.block + nk + (lane8 >= 4 ? 2 : 0);
      const int g = 2 * (lane8 & 3);
      codes = *reinterpret_cast<const uint16_t*>(b + kv4_value_offset(at.t, at.chunk, g)) |
              static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(b + kv4_value_offset(at.t, at.chunk, g + 1))) << 16;
    }
    const int wi = at.t * kv4_words(p.dqk, p.dv) + (at.value ? p.dqk / kKv4Group : 0) + group;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(at.block + nk + nv + 4 * wi);
    const float scale = __uint_as_float(word & 0xffff0000u), mn = __uint_as_float(word << 16);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(scale, static_cast<float>((codes >> (4 * i)) & 15u), mn);
    const int ch = at.chunk * 64 + lane8 * 8;
    T* dst = at.value ? static_cast<T*>(p.v) + tok * p.v_srow + at.head * p.v_shead + ch
                      : static_cast<T*>(p.k) + tok * p.k_srow + at.head * p.k_shead + ch;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
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
  p.page_size = cache->page_size;
  p.Hkv = cache->Hkv;
  p.dqk = cache->dqk;
  p.dv = cache->dv;
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
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % kKv4Block) return SLOPE_ERR_SHAPE;
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
  if (k->dtype == SLOPE_BF16)
    kv4_write_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else
    kv4_write_kernel<float><<<grid, kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
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
  if (k->dtype == SLOPE_BF16)
    kv4_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else
    kv4_read_kernel<float><<<grid, kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache read kernel launch", e);
}

}  // extern "C"
