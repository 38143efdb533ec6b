// Keys and values of new tokens into the pages of the 16-bit cache, and what the calls on that cache check alike.
//
// The store is a scatter of rows: bf16 is copied, fp32 rounded to nearest even.  A thread takes the same 8 channels (16 bytes
// in the cache) of kTokens tokens, whose slots and then rows it loads together, so a call of a few tokens costs two loads'
// latency and a chunk of a prompt runs near the copy rate (8 heads of 64: 32 tokens 1.7 us, 12288 9.7 us, 5.3 TB/s, of which
// the start and the end take 1.5).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "kv_cache.cuh"
#include "sm103_ptx.cuh"

namespace slope {
namespace {

constexpr int kTokens = 4;  // of a thread

struct KvWriteParams {
  const void* k;
  const void* v;
  int64_t k_srow, k_shead, v_srow, v_shead;  // of the rows written
  __nv_bfloat16* ck;
  __nv_bfloat16* cv;
  int64_t k_stride[3], v_stride[3];  // of the cache
  float* weights;                    // may be null
  int64_t w_spage, w_shead;
  const int32_t* slots;
  int64_t T, n_slots;
  int32_t page_shift, Hkv, k_words, v_words;  // words of 8 channels of a head
};

template <typename X>
__device__ __forceinline__ uint4 load8(const X* x) {
  if constexpr (sizeof(X) == 2) {
    return *reinterpret_cast<const uint4*>(x);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
    return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
  }
}

template <typename X>
__global__ void __launch_bounds__(256) kv_write_kernel(const __grid_constant__ KvWriteParams p) {
  pdl_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int word = blockIdx.y * blockDim.x + threadIdx.x;
  int64_t slot[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    slot[i] = t0 + i < p.T ? p.slots[t0 + i] : -1;
    if (slot[i] >= p.n_slots) slot[i] = -1;
  }
  const int mask = (1 << p.page_shift) - 1;
  if (p.weights != nullptr && word < p.Hkv) {
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
      if (slot[i] >= 0) p.weights[(slot[i] >> p.page_shift) * p.w_spage + word * p.w_shead + (slot[i] & mask)] = 0.f;
  }
  const bool value = word >= p.Hkv * p.k_words;
  const int w = value ? word - p.Hkv * p.k_words : word, per = value ? p.v_words : p.k_words;
  if (w >= p.Hkv * per) return;
  const int h = w / per, ch = (w - h * per) * 8;
  const X* const src = static_cast<const X*>(value ? p.v : p.k) + h * (value ? p.v_shead : p.k_shead) + ch;
  const int64_t srow = value ? p.v_srow : p.k_srow;
  __nv_bfloat16* const dst = (value ? p.cv + h * p.v_stride[1] : p.ck + h * p.k_stride[1]) + ch;
  const int64_t spage = value ? p.v_stride[0] : p.k_stride[0], stoken = value ? p.v_stride[2] : p.k_stride[2];
  uint4 x[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
    if (slot[i] >= 0) x[i] = load8(src + (t0 + i) * srow);
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
    if (slot[i] >= 0)
      *reinterpret_cast<uint4*>(dst + (slot[i] >> p.page_shift) * spage + (slot[i] & mask) * stoken) = x[i];
}

template <typename X>
cudaError_t launch_write(const KvWriteParams& p, cudaStream_t stream) {
  const int64_t words = static_cast<int64_t>(p.Hkv) * (p.k_words + p.v_words);
  const int threads = static_cast<int>(std::min<int64_t>(256, (words + 31) / 32 * 32));
  const dim3 grid(static_cast<unsigned>((p.T + kTokens - 1) / kTokens), static_cast<unsigned>((words + threads - 1) / threads));
  return launch_early(kv_write_kernel<X>, grid, threads, 0, stream, p);
}

bool strides_ok(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] <= 0 || s[i] % 8 || s[i] >= (int64_t(1) << 39)) return false;
  return true;
}

// [T, Hkv, d] rows of bf16 or fp32 for the store.
slope_status check_rows(const slope_tensor* t, int64_t T, int64_t H, int64_t d, slope_dtype dtype) {
  if (t == nullptr) return SLOPE_ERR_NULL;
  if (t->dtype != SLOPE_BF16 && t->dtype != SLOPE_F32) return SLOPE_ERR_DTYPE;
  if (t->dtype != dtype) return SLOPE_ERR_DTYPE;
  if (t->ndim != 3 || t->shape[0] != T || t->shape[1] != H || t->shape[2] != d) return SLOPE_ERR_SHAPE;
  if (T == 0) return SLOPE_OK;
  if (t->data == nullptr) return SLOPE_ERR_NULL;
  if (t->stride[2] != 1 || t->stride[0] <= 0 || t->stride[1] <= 0 || t->stride[0] % 8 || t->stride[1] % 8 ||
      !aligned(t->data, 16))
    return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

}  // namespace

slope_status check_kv_cache(const slope_kv_cache* c) {
  if (c == nullptr) return SLOPE_ERR_NULL;
  if (!attn_partial_supported(c->dqk, c->dv)) return SLOPE_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return SLOPE_ERR_SHAPE;
  if (c->n_pages < 1 || c->n_pages > 0x7fffffffLL / c->page_size) return SLOPE_ERR_SHAPE;
  if (c->Hkv < 1 || c->Hkv > 65535) return SLOPE_ERR_SHAPE;
  if (c->k == nullptr || c->v == nullptr) return SLOPE_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !strides_ok(c->k_stride) || !strides_ok(c->v_stride)) return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

slope_status check_kv_q(const slope_tensor* q, const slope_kv_cache* c) {
  if (q == nullptr) return SLOPE_ERR_NULL;
  if (q->dtype != SLOPE_BF16) return SLOPE_ERR_DTYPE;
  if (q->ndim != 3) return SLOPE_ERR_SHAPE;
  if (q->shape[0] < 0 || q->shape[0] >= kKvMaxTokens) return SLOPE_ERR_SHAPE;
  if (q->shape[1] < 1 || q->shape[1] > 65535 || q->shape[1] % c->Hkv != 0 || q->shape[2] != c->dqk) return SLOPE_ERR_SHAPE;
  if (q->shape[0] == 0) return SLOPE_OK;
  if (q->data == nullptr) return SLOPE_ERR_NULL;
  if (q->stride[2] != 1 || q->stride[0] <= 0 || q->stride[1] <= 0 || q->stride[0] % 8 || q->stride[1] % 8 ||
      q->stride[0] >= (int64_t(1) << 39) || q->stride[1] >= (int64_t(1) << 39) || !aligned(q->data, 16))
    return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

slope_status check_kv_batch(const slope_kv_batch* b, const slope_kv_cache* c, int64_t T) {
  if (b == nullptr) return SLOPE_ERR_NULL;
  if (b->B < 0 || b->B > kKvMaxBatch) return SLOPE_ERR_SHAPE;
  if (b->cu_q == nullptr && (b->q_len < 0 || b->B * static_cast<int64_t>(b->q_len) != T)) return SLOPE_ERR_SHAPE;
  if (b->max_pages < 0 || b->max_pages > (kKvMaxTokens - 1) / c->page_size || b->table_stride < b->max_pages)
    return SLOPE_ERR_SHAPE;
  if (b->B == 0) return SLOPE_OK;
  if (b->kv_lens == nullptr || (b->max_pages > 0 && b->block_table == nullptr)) return SLOPE_ERR_NULL;
  if (!aligned(b->kv_lens, 4) || !aligned(b->block_table, 4) || !aligned(b->cu_q, 4)) return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

slope_status check_kv_weights(const slope_tensor* w, const slope_kv_cache* c) {
  if (w == nullptr) return SLOPE_ERR_NULL;
  if (w->dtype != SLOPE_F32) return SLOPE_ERR_DTYPE;
  if (w->ndim != 3 || w->shape[0] != c->n_pages || w->shape[1] != c->Hkv || w->shape[2] != c->page_size) return SLOPE_ERR_SHAPE;
  if (w->data == nullptr) return SLOPE_ERR_NULL;
  if (w->stride[2] != 1 || w->stride[0] <= 0 || w->stride[1] <= 0 || !aligned(w->data, 4)) return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

bool make_page_map(CUtensorMap* m, const void* base, const slope_kv_cache* c, int64_t d, const int64_t* stride) {
  const auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  std::memset(m, 0, sizeof(*m));
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->Hkv), static_cast<cuuint64_t>(c->n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride[2]) * 2, static_cast<cuuint64_t>(stride[1]) * 2,
                                 static_cast<cuuint64_t>(stride[0]) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min(c->page_size, kBlockN)), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_q_map(CUtensorMap* m, const slope_tensor* q, int heads, int tokens) {
  const auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  std::memset(m, 0, sizeof(*m));
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(q->shape[2]), static_cast<cuuint64_t>(q->shape[1]),
                              static_cast<cuuint64_t>(q->shape[0])};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(q->stride[1]) * 2, static_cast<cuuint64_t>(q->stride[0]) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int kv_sm_count() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 0;
  sms = std::min(sms, kKvMaxSms);
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

}  // namespace slope

using namespace slope;

extern "C" slope_status slope_kv_write(const slope_kv_cache* cache, const slope_tensor* k, const slope_tensor* v,
                                       const int32_t* slots, slope_tensor* weights, void* stream) {
  const CallRange range("slope_kv_write");
  slope_status st;
  if ((st = check_kv_cache(cache)) != SLOPE_OK) return st;
  if (k == nullptr || v == nullptr) return SLOPE_ERR_NULL;
  const int64_t T = k->ndim == 3 ? k->shape[0] : -1;
  if (T < 0 || T > 0x7fffffffLL) return SLOPE_ERR_SHAPE;
  if ((st = check_rows(k, T, cache->Hkv, cache->dqk, k->dtype)) != SLOPE_OK) return st;
  if ((st = check_rows(v, T, cache->Hkv, cache->dv, k->dtype)) != SLOPE_OK) return st;
  if (weights != nullptr && (st = check_kv_weights(weights, cache)) != SLOPE_OK) return st;
  if (T == 0) return SLOPE_OK;
  if (slots == nullptr) return SLOPE_ERR_NULL;
  if (!aligned(slots, 4)) return SLOPE_ERR_STRIDE;
  KvWriteParams p{};
  p.k = k->data;
  p.v = v->data;
  p.k_srow = k->stride[0];
  p.k_shead = k->stride[1];
  p.v_srow = v->stride[0];
  p.v_shead = v->stride[1];
  p.ck = static_cast<__nv_bfloat16*>(cache->k);
  p.cv = static_cast<__nv_bfloat16*>(cache->v);
  for (int i = 0; i < 3; ++i) {
    p.k_stride[i] = cache->k_stride[i];
    p.v_stride[i] = cache->v_stride[i];
  }
  if (weights != nullptr) {
    p.weights = static_cast<float*>(weights->data);
    p.w_spage = weights->stride[0];
    p.w_shead = weights->stride[1];
  }
  p.slots = slots;
  p.T = T;
  p.n_slots = cache->n_pages * cache->page_size;
  p.page_shift = log2_of(cache->page_size);
  p.Hkv = cache->Hkv;
  p.k_words = cache->dqk / 8;
  p.v_words = cache->dv / 8;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = k->dtype == SLOPE_BF16 ? launch_write<__nv_bfloat16>(p, s) : launch_write<float>(p, s);
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache store kernel launch", e);
}
