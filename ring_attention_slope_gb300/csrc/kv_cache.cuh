// What the calls on the 16-bit paged cache share: argument checks, TMA views of the pages, and the batch as the
// kernels see it.
#pragma once

#include <cuda.h>

#include <utility>

#include "host.cuh"
#include "kernels.cuh"
#include "slope_kv.h"

namespace slope {

constexpr int64_t kKvMaxTokens = int64_t(1) << 28;  // of q's rows, and of a sequence
constexpr int64_t kKvMaxBatch = 65535;              // sequences of a call
constexpr int kKvMaxSeqs = 512;                     // of a launch

// Argument checks of a cache, its pointers and strides among them.
slope_status check_kv_cache(const slope_kv_cache* c);
// Of what q, weights and the batch have in common in the two attention calls.
slope_status check_kv_q(const slope_tensor* q, const slope_kv_cache* c);
slope_status check_kv_batch(const slope_kv_batch* b, const slope_kv_cache* c, int64_t T);
slope_status check_kv_weights(const slope_tensor* w, const slope_kv_cache* c);

// {64 channels, rows of a page up to 128, 1 head, 1 page} boxes of keys or values, 128-byte swizzle; pages out of
// range read 0.
bool make_page_map(CUtensorMap* m, const void* base, const slope_kv_cache* c, int64_t d, const int64_t* stride);
// {64 channels, `heads` heads, `tokens` tokens} boxes of q, 128-byte swizzle.
bool make_q_map(CUtensorMap* m, const slope_tensor* q, int heads, int tokens);

// SMs of the current device that the calls make use of (0 on failure), and how many at most: workspaces are sized for those.
constexpr int kKvMaxSms = 160;
int kv_sm_count();

inline int log2_of(int64_t n) {
  int s = 0;
  while ((int64_t(1) << s) < n) ++s;
  return s;
}

// The batch on the device, of one launch.
struct KvSeqs {
  const int32_t* cu_q;  // or null
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride;
  int64_t max_tokens;  // max_pages * page_size
  int64_t n_pages;
  int32_t T;
  int32_t q_len;
  int32_t b0, B;  // sequences b0 .. b0 + B - 1
  int32_t page_shift;
};

// A sequence: its rows of q, and its tokens in the cache.
struct KvSeq {
  int32_t row0, n, len;
};

#ifdef __CUDACC__
// Launches a kernel that begins with what needs no memory and then waits for the kernel before it (pdl_wait): its start
// runs under that one's end.
template <typename... Args, typename... Given>
cudaError_t launch_early(void (*kernel)(Args...), dim3 grid, int threads, size_t bytes, cudaStream_t stream, Given&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Given>(args)...);
}

__device__ __forceinline__ KvSeq kv_seq(const KvSeqs& s, int b) {
  KvSeq r;
  const int at = s.b0 + b;
  if (s.cu_q != nullptr) {
    r.row0 = min(max(s.cu_q[at], 0), s.T);
    r.n = max(0, min(s.cu_q[at + 1], s.T) - r.row0);
  } else {
    r.row0 = at * s.q_len;
    r.n = s.q_len;
  }
  const int64_t len = s.kv_lens[at];
  r.len = static_cast<int32_t>(len < 0 ? 0 : len > s.max_tokens ? s.max_tokens : len);
  return r;
}
#endif

// The batch's fields that every launch of a call has alike.
inline KvSeqs kv_seqs(const slope_kv_batch* b, const slope_kv_cache* c, int64_t T) {
  KvSeqs s{};
  s.cu_q = b->cu_q;
  s.kv_lens = b->kv_lens;
  s.table = b->block_table;
  s.table_stride = b->table_stride;
  s.max_tokens = b->max_pages * c->page_size;
  s.n_pages = c->n_pages;
  s.T = static_cast<int32_t>(T);
  s.q_len = b->q_len;
  s.page_shift = log2_of(c->page_size);
  return s;
}

// How the rows of a key head's queries fill tiles of 128: `heads` heads (all of the group, or an even part of more
// than 128) of `tokens` tokens, token by token.
struct RowTile {
  int32_t parts, heads, tokens;
};
inline RowTile row_tile(int64_t group) {
  RowTile r;
  r.parts = static_cast<int32_t>((group + kBlockM - 1) / kBlockM);
  r.heads = static_cast<int32_t>((group + r.parts - 1) / r.parts);
  r.tokens = kBlockM / r.heads;
  return r;
}

}  // namespace slope
