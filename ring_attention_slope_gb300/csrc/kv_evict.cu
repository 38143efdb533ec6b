// Eviction from the 16-bit cache: of each sequence and key head the tokens with the largest accumulated weights stay and
// move together, in order.
//
// Selection.  A weight becomes a 32-bit key whose order is the weights' (a missing page 0, NaN 1, then -inf .. inf), and
// the smallest key that stays is found 11, 11 and 10 bits at a time from the top: a histogram of the keys that match
// the bits so far, and the bin that holds the wanted rank.  Then every key above it stays, and as many equal ones as are
// left, the first ones.  A cluster of CTAs shares a (sequence, head) pair: each has a run of tokens, whose keys it keeps
// in shared memory, and they read one another's histograms and counts there, so the weights are read once.
//
// Moving.  Token j of those kept comes from position old[j] >= j, so within its own pages a chunk of kept tokens may
// overwrite only what chunks before it read.  A CTA takes one chunk after another by ticket: it reads the rows into
// registers, says so in a flag, waits for the (at most two) chunks whose rows lie where its own go, and writes.  Each row is
// read and written once, by as many CTAs as the GPU holds.  A chunk waits only for chunks of lower tickets, which are running and
// read before they wait, so every wait ends; all the same it is bounded.
//
// On one GB300, 8 heads of 64, into other pages and in place: sequences of 65536, 3251, 161 and 9 tokens to 16384 38 us and as
// much (selection 23 and moving 21 by themselves: three passes after one another over the bins of a cluster; then chunk after chunk,
// two or three to a CTA, a chain of old positions, pages, rows and stores); 8 x 100K to 32768 244 us, 4.6 TB/s read and
// written, and 279, where chunks wait for others' reads too; 32 x 8K to 4096 113 and 136; one of 2000 tokens 11.7 us, latencies,
// and 2 more.  Keys loaded one at a time and a CTA for every chunk took 75 us for the first of these.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv_cache.cuh"
#include "sm103_ptx.cuh"
#include "waits.cuh"

namespace cg = cooperative_groups;

namespace slope {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kRun = 8192;          // keys of a CTA, as long as clusters allow it
constexpr int kHeldKeys = 40960;    // of them in shared memory at most; more are made again in every pass
constexpr int kMoveThreads = 128, kMoveWords = 8;  // of a thread, 16 bytes each
constexpr int kMoveCtas = 7;                       // on an SM, by registers

struct KvEvictParams {
  KvSeqs seqs;
  int32_t Hkv;
  const float* weights_in;
  float* weights;
  int64_t w_spage, w_shead;
  int32_t keep, first, recent;
  const int32_t* out_table;  // null: within the sequence's own pages
  int64_t out_stride;
  int32_t* kept;
  int32_t* out_lens;
  const uint4* k_in;
  uint4* k;
  const uint4* v_in;
  uint4* v;
  int64_t k_stride[3], v_stride[3];  // in words of 8 channels
  int32_t chunk, chunks;             // kept tokens of a chunk, chunks of a pair
  int32_t held;                      // keys of a CTA in shared memory
  uint32_t* tickets;                 // workspace: one for each launch that moves
  int32_t launches;
  uint32_t* flags;                   // workspace: [pair][chunk], the chunk's rows are read
  int32_t* bounds;                   // workspace: [pair][chunk + 1], kept tokens before position chunk * c
  int* status;
  uint64_t wait_limit_ns;
};

// Keys of weights: larger weight, larger key; equal weights, equal keys.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 is 0
  return (u >> 31) != 0 ? ~u : u | 0x80000000u;
}

// Exclusive sums over the CTA's threads, and the total.
__device__ __forceinline__ uint2 block_scan(uint2 v, uint2* scratch, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 incl = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, m), y = __shfl_up_sync(0xffffffffu, incl.y, m);
    if (lane >= m) incl.x += x, incl.y += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  static_assert(kSelectThreads <= 1024, "a warp's lanes for the warps");
  const uint2 mine = lane < kSelectThreads / 32 ? scratch[lane] : make_uint2(0, 0);
  uint2 before;
  before.x = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0u);
  before.y = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0u);
  total.x = __reduce_add_sync(0xffffffffu, mine.x);
  total.y = __reduce_add_sync(0xffffffffu, mine.y);
  return make_uint2(before.x + incl.x - v.x, before.y + incl.y - v.y);
}

__global__ void __launch_bounds__(kSelectThreads, 2) kv_select_kernel(const __grid_constant__ KvEvictParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) uint32_t s_hist[kBins];
  __shared__ uint32_t s_bin[3];             // the bin with the wanted rank, the rank within it, and the keys in it
  __shared__ uint32_t s_slice[kMaxCluster];  // keys in each CTA's slice of the bins
  __shared__ uint2 s_scan[kSelectThreads / 32], s_count;
  pdl_wait();
  pdl_launch_dependents();  // (not before: the move reads the lengths ahead of its own wait)
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int pair = blockIdx.x / ranks, b = pair / p.Hkv, h = pair - b * p.Hkv;
  const KvSeq seq = kv_seq(p.seqs, b);
  const int n = seq.len, keep = p.keep;
  int32_t* const kept = p.kept + static_cast<int64_t>(pair) * keep;
  uint32_t* const flags = p.flags + static_cast<int64_t>(pair) * p.chunks;
  int32_t* const bounds = p.bounds + static_cast<int64_t>(pair) * (p.chunks + 1);
  const int stride = ranks * kSelectThreads, me = rank * kSelectThreads + threadIdx.x;

  if (pair == 0)
    for (int i = me; i < p.launches; i += stride) p.tickets[i] = 0;
  for (int c = me; c < p.chunks; c += stride) flags[c] = 0;
  if (n <= keep) {
    for (int j = me; j < keep; j += stride) kept[j] = j < n ? j : -1;
    return;  // (the whole cluster does)
  }
  auto sync = [&]() {
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  // tokens before and after the ones to choose from
  for (int j = me; j < p.first; j += stride) kept[j] = j;
  for (int j = me; j < p.recent; j += stride) kept[keep - p.recent + j] = n - p.recent + j;
  const int mid = n - p.first - p.recent;  // > want
  const uint32_t want = static_cast<uint32_t>(keep - p.first - p.recent);
  const int each = (mid + ranks - 1) / ranks;
  const int t0 = p.first + min(mid, rank * each), t1 = p.first + min(mid, (rank + 1) * each);

  const int32_t* const row = p.seqs.table + static_cast<int64_t>(b) * p.seqs.table_stride;
  const int in_page = (1 << p.seqs.page_shift) - 1;
  const float* const weights = p.weights_in + h * p.w_shead;
  auto read_key = [&](int t) -> uint32_t {
    const int pg = row[t >> p.seqs.page_shift];
    return pg < 0 || pg >= p.seqs.n_pages ? 0u : weight_key(weights[pg * p.w_spage + (t & in_page)]);
  };
  // eight loads of pages, then of weights, in flight
  constexpr int kAhead = 8;
  const int held = min(t1 - t0, p.held);
  for (int i0 = threadIdx.x; i0 < held; i0 += kAhead * kSelectThreads) {
    int pg[kAhead];
    float w[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + e * kSelectThreads;
      pg[e] = i < held ? row[(t0 + i) >> p.seqs.page_shift] : -1;
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (pg[e] >= p.seqs.n_pages) pg[e] = -1;
      w[e] = pg[e] >= 0 ? weights[pg[e] * p.w_spage + ((t0 + i0 + e * kSelectThreads) & in_page)] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (i0 + e * kSelectThreads < held) s_keys[i0 + e * kSelectThreads] = pg[e] >= 0 ? weight_key(w[e]) : 0u;
  }
  auto key = [&](int t) -> uint32_t { return t - t0 < p.held ? s_keys[t - t0] : read_key(t); };
  // the thread's own run of tokens, an odd number of them (which spreads the runs over the banks)
  const int run = ((t1 - t0 + kSelectThreads - 1) / kSelectThreads) | 1;
  const int a0 = t0 + min(t1 - t0, static_cast<int>(threadIdx.x) * run), a1 = min(t1, a0 + run);

  // ---- the smallest key that stays, and how many equal to it
  uint32_t prefix = 0, left = want;  // of the keys that match the prefix, the left-th largest is looked for
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const uint32_t high = shift == 32 ? 0u : ~0u << shift;  // bits known so far
    shift -= bits;
    for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s_hist[i] = 0;
    __syncthreads();  // (and the keys are there)
    for (int t = t0 + threadIdx.x; t < t1; t += kSelectThreads) {
      const uint32_t k = key(t);
      if ((k & high) == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1)], 1u);
    }
    sync();
    // Each CTA adds its slice of the bins up, four to a thread from the top (slice 0 is the top one).
    const int slice = kBins / ranks, bin = kBins - rank * slice - 4 - 4 * static_cast<int>(threadIdx.x);
    uint32_t c[4] = {0, 0, 0, 0};  // of bin .. bin + 3
    if (4 * static_cast<int>(threadIdx.x) < slice) {
#pragma unroll 8
      for (int r = 0; r < ranks; ++r) {
        const uint4 x = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(s_hist, r) + bin);
        c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w;
      }
    }
    uint2 total;
    uint32_t above = block_scan(make_uint2(c[0] + c[1] + c[2] + c[3], 0), s_scan, total).x;
    if (ranks > 1) {
      if (static_cast<int>(threadIdx.x) < ranks) *cluster.map_shared_rank(&s_slice[rank], threadIdx.x) = total.x;
      cluster.sync();
      for (int r = 0; r < rank; ++r) above += s_slice[r];
    }
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      if (above < left && left <= above + c[i]) {
        for (int r = 0; r < ranks; ++r) {
          uint32_t* const to = cluster.map_shared_rank(s_bin, r);
          to[0] = bin + i, to[1] = left - above, to[2] = c[i];
        }
      }
      above += c[i];
    }
    sync();  // the bin is known
    if (want > 0) {
      prefix |= s_bin[0] << shift;
      left = s_bin[1];
      if (left == s_bin[2]) {  // all of the bin stay: every key above the ones below it
        prefix -= 1;           // (some key does not stay, so this is not the lowest bin)
        left = 0;
        break;
      }
    }
  }
  if (want == 0) prefix = ~0u, left = 0;  // no key is as large

  // ---- counts of larger and equal keys before the thread's run, in this CTA and in those before it
  uint2 mine = make_uint2(0, 0), total;
  for (int t = a0; t < a1; ++t) {
    const uint32_t k = key(t);
    mine.x += k > prefix ? 1u : 0u, mine.y += k == prefix ? 1u : 0u;
  }
  uint2 before = block_scan(mine, s_scan, total);
  if (threadIdx.x == 0) s_count = total;
  sync();
  if (threadIdx.x < 32) {
    uint2 c = make_uint2(0, 0);
    if (static_cast<int>(threadIdx.x) < rank) c = *cluster.map_shared_rank(&s_count, threadIdx.x);
    c.x = __reduce_add_sync(0xffffffffu, c.x);
    c.y = __reduce_add_sync(0xffffffffu, c.y);
    if (threadIdx.x == 0) s_scan[0] = c;
  }
  sync();  // (no CTA leaves before its counts are read)
  before.x += s_scan[0].x, before.y += s_scan[0].y;

  // ---- places
  int edge = (a0 + p.chunk - 1) / p.chunk;  // the next bound that lies in the run
  for (int t = a0; t < a1; ++t) {
    const uint32_t k = key(t);
    const int j = p.first + static_cast<int>(before.x + min(before.y, left));
    if (t == edge * p.chunk) {
      if (edge <= p.chunks) bounds[edge] = j;
      ++edge;
    }
    if (k > prefix || (k == prefix && before.y < left)) kept[j] = t;
    before.x += k > prefix ? 1u : 0u, before.y += k == prefix ? 1u : 0u;
  }
  // the bounds outside the chosen range
  for (int c = me; c <= p.chunks; c += stride) {
    const int64_t t = static_cast<int64_t>(c) * p.chunk;
    if (t < p.first)
      bounds[c] = static_cast<int>(t);
    else if (t >= n)
      bounds[c] = keep;
    else if (t >= n - p.recent)
      bounds[c] = keep - (n - static_cast<int>(t));
  }
}

// Words of a token's head: keys, then values.
template <int DQK, int DV>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) kv_move_kernel(const __grid_constant__ KvEvictParams p, int launch) {
  constexpr int kKey = DQK / 8, kAll = (DQK + DV) / 8;
  constexpr int kChunk = kMoveThreads * kMoveWords / kAll / 8 * 8;
  __shared__ uint32_t s_first[kKvMaxSeqs];  // chunks before a sequence's
  __shared__ uint32_t s_total, s_ticket;
  __shared__ int64_t s_src[kChunk], s_dst[kChunk];  // page << 32 | index in the page; -1: not moved
  __shared__ int s_give_up;
  const int B = p.seqs.B, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    uint32_t sum = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      uint32_t n = 0;
      if (b0 + lane < B) n = static_cast<uint32_t>((min(kv_seq(p.seqs, b0 + lane).len, p.keep) + kChunk - 1) / kChunk) * p.Hkv;
      uint32_t incl = n;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += o;
      }
      if (b0 + lane < B) s_first[b0 + lane] = sum + incl - n;
      sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      s_total = sum;
      s_give_up = 0;
    }
  }
  pdl_wait();
  // (the lengths may be their own output: a length that has changed gives the same chunks)
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < B; b += kMoveThreads) p.out_lens[p.seqs.b0 + b] = min(kv_seq(p.seqs, b).len, p.keep);
  if (threadIdx.x == 0) s_ticket = atomicAdd(&p.tickets[launch], 1u);
  __syncthreads();
  const uint32_t total = s_total;
  const int shift = p.seqs.page_shift, in_page = (1 << shift) - 1;
  for (uint32_t ticket = s_ticket; ticket < total;) {
    int seq = 0;
    for (int hi = B - 1; seq < hi;) {  // the last sequence whose first chunk is not after the ticket's
      const int mid = (seq + hi + 1) >> 1;
      if (s_first[mid] <= ticket)
        seq = mid;
      else
        hi = mid - 1;
    }
    // a sequence's chunks of all heads in turn, so that a chunk's forerunners are a round ahead
    const int b = p.seqs.b0 + seq, c = static_cast<int>((ticket - s_first[seq]) / static_cast<uint32_t>(p.Hkv));
    const int h = static_cast<int>(ticket - s_first[seq]) - c * p.Hkv;
    const int64_t pair = static_cast<int64_t>(b) * p.Hkv + h;
    uint32_t next = 0;
    if (threadIdx.x == 0) next = atomicAdd(&p.tickets[launch], 1u);  // on its way
    const int j0 = c * kChunk, count = min(kChunk, p.keep - j0);
    bool moves = false;
    for (int i = threadIdx.x; i < kChunk; i += kMoveThreads) {
      const int j = j0 + i, old = i < count ? p.kept[pair * p.keep + j] : -1;
      int64_t src = -1, dst = -1;
      if (old >= 0 && (p.out_table != nullptr || old != j)) {
        const int32_t* const row = p.seqs.table + static_cast<int64_t>(b) * p.seqs.table_stride;
        const int from = row[old >> shift];
        const int to = p.out_table != nullptr ? p.out_table[static_cast<int64_t>(b) * p.out_stride + (j >> shift)] : row[j >> shift];
        if (from >= 0 && from < p.seqs.n_pages && to >= 0 && to < p.seqs.n_pages) {
          src = static_cast<int64_t>(from) << 32 | (old & in_page);
          dst = static_cast<int64_t>(to) << 32 | (j & in_page);
          moves = true;
        }
      }
      s_src[i] = src, s_dst[i] = dst;
    }
    uint32_t* const flags = p.flags + pair * p.chunks;
    moves = __syncthreads_or(moves);
    if (!moves && threadIdx.x == 0) atomicExch(&flags[c], 1u);
    if (moves) {
      uint4 x[kMoveWords];
#pragma unroll
      for (int i = 0; i < kMoveWords; ++i) {
        const int word = threadIdx.x + i * kMoveThreads, e = word / kAll, w = word - e * kAll;
        if (e >= kChunk || s_src[e] < 0) continue;
        const int64_t pg = s_src[e] >> 32, t = s_src[e] & 0xffffffff;
        x[i] = w < kKey ? p.k_in[pg * p.k_stride[0] + h * p.k_stride[1] + t * p.k_stride[2] + w]
                        : p.v_in[pg * p.v_stride[0] + h * p.v_stride[1] + t * p.v_stride[2] + (w - kKey)];
      }
      float weight = 0.f;
      if (threadIdx.x < kChunk && s_src[threadIdx.x] >= 0)
        weight = p.weights_in[(s_src[threadIdx.x] >> 32) * p.w_spage + h * p.w_shead + (s_src[threadIdx.x] & 0xffffffff)];

      if (p.out_table == nullptr) {
        __threadfence();  // the reads come before the flag
        __syncthreads();
        if (threadIdx.x == 0) {
          atomicExch(&flags[c], 1u);
          // the kept tokens that lie where this chunk's go, and their chunks
          const int32_t* const bounds = p.bounds + pair * (p.chunks + 1) + c;
          const int lo = bounds[0], hi = bounds[1];
          const uint64_t start = globaltimer_ns();
          for (int o = lo / kChunk; hi > lo && o <= (hi - 1) / kChunk && o < c && !s_give_up; ++o) {
            while (atomicAdd(&flags[o], 0u) == 0u) {
              if (*reinterpret_cast<volatile int*>(p.status) != 0) {
                s_give_up = 1;
                break;
              }
              if (globaltimer_ns() - start > p.wait_limit_ns) {
                record_timeout(p.status, 81);
                s_give_up = 1;
                break;
              }
            }
          }
          __threadfence();
        }
        __syncthreads();
        if (s_give_up) return;
      }
#pragma unroll
      for (int i = 0; i < kMoveWords; ++i) {
        const int word = threadIdx.x + i * kMoveThreads, e = word / kAll, w = word - e * kAll;
        if (e >= kChunk || s_src[e] < 0) continue;
        const int64_t pg = s_dst[e] >> 32, t = s_dst[e] & 0xffffffff;
        if (w < kKey)
          p.k[pg * p.k_stride[0] + h * p.k_stride[1] + t * p.k_stride[2] + w] = x[i];
        else
          p.v[pg * p.v_stride[0] + h * p.v_stride[1] + t * p.v_stride[2] + (w - kKey)] = x[i];
      }
      if (threadIdx.x < kChunk && s_src[threadIdx.x] >= 0)
        p.weights[(s_dst[threadIdx.x] >> 32) * p.w_spage + h * p.w_shead + (s_dst[threadIdx.x] & 0xffffffff)] = weight;
    }
    if (threadIdx.x == 0) s_ticket = next;
    __syncthreads();
    ticket = s_ticket;
    __syncthreads();
  }
}

int chunk_of(int dqk, int dv) { return kMoveThreads * kMoveWords / ((dqk + dv) / 8) / 8 * 8; }

template <int DQK, int DV>
cudaError_t launch_move(KvEvictParams p, int64_t B, cudaStream_t stream) {
  static_assert(kMoveThreads * kMoveWords / ((DQK + DV) / 8) / 8 * 8 <= kMoveThreads, "a weight to a thread");
  for (int i = 0; i < p.launches; ++i) {
    p.seqs.b0 = i * kKvMaxSeqs;
    p.seqs.B = static_cast<int32_t>(std::min<int64_t>(kKvMaxSeqs, B - p.seqs.b0));
    const int64_t chunks = static_cast<int64_t>(p.seqs.B) * p.Hkv * p.chunks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(chunks, kMoveCtas * kv_sm_count())));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = i == 0 ? 1 : 0;  // the first starts as the selection ends
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_move_kernel<DQK, DV>, p, i);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_evict(const KvEvictParams& p, int64_t B, int dqk, int dv, cudaStream_t stream) {
  int ranks = 1;
  while (ranks < kMaxCluster && p.seqs.max_tokens > static_cast<int64_t>(ranks) * kRun) ranks *= 2;
  KvEvictParams s = p;
  s.held = static_cast<int32_t>(std::min<int64_t>(kHeldKeys, (p.seqs.max_tokens + ranks - 1) / ranks));
  const int bytes = s.held * 4;
  cudaError_t e = cudaFuncSetAttribute(kv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldKeys * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kv_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * p.Hkv * ranks));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, kv_select_kernel, s)) != cudaSuccess) return e;
  if (dqk == 64 && dv == 64) return launch_move<64, 64>(p, B, stream);
  if (dqk == 64 && dv == 128) return launch_move<64, 128>(p, B, stream);
  if (dqk == 128 && dv == 64) return launch_move<128, 64>(p, B, stream);
  if (dqk == 128 && dv == 128) return launch_move<128, 128>(p, B, stream);
  if (dqk == 192 && dv == 64) return launch_move<192, 64>(p, B, stream);
  if (dqk == 192 && dv == 128) return launch_move<192, 128>(p, B, stream);
  return cudaErrorInvalidValue;
}

constexpr int kMinChunk = 24;  // chunk_of's smallest
constexpr int64_t kMoveLaunches = (kKvMaxBatch + kKvMaxSeqs - 1) / kKvMaxSeqs;  // of a call, a ticket each

struct Workspace {
  size_t flags, bounds, total;
};
Workspace workspace_of(int64_t pairs, int64_t chunks) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  Workspace w;
  w.flags = up(kMoveLaunches * sizeof(uint32_t));  // the tickets are before them
  w.bounds = w.flags + up(pairs * chunks * sizeof(uint32_t));
  w.total = w.bounds + up(pairs * (chunks + 1) * sizeof(int32_t));
  return w;
}

}  // namespace
}  // namespace slope

using namespace slope;

extern "C" {

size_t slope_kv_evict_workspace_size(int64_t B, int64_t Hkv, int64_t keep) {
  if (B < 0 || B > kKvMaxBatch || Hkv < 1 || Hkv > 65535 || keep < 1 || keep >= kKvMaxTokens) return 0;
  return workspace_of(B * Hkv, (keep + kMinChunk - 1) / kMinChunk).total;
}

slope_status slope_kv_evict(const slope_kv_cache* cache, slope_tensor* weights, int64_t B, const int32_t* block_table,
                            int64_t table_stride, int64_t max_pages, const int32_t* kv_lens, int64_t keep, int64_t first,
                            int64_t recent, const int32_t* out_table, int64_t out_stride, int64_t out_pages,
                            int32_t* kept, int32_t* out_lens, void* workspace, size_t workspace_bytes, void* stream) {
  const CallRange range("slope_kv_evict");
  slope_status st;
  if ((st = check_kv_cache(cache)) != SLOPE_OK || (st = check_kv_weights(weights, cache)) != SLOPE_OK) return st;
  const slope_kv_batch batch{B, nullptr, 0, kv_lens, block_table, table_stride, max_pages};
  if ((st = check_kv_batch(&batch, cache, 0)) != SLOPE_OK) return st;
  if (keep < 1 || keep >= kKvMaxTokens || first < 0 || recent < 0 || first > keep || recent > keep - first) return SLOPE_ERR_SHAPE;
  const int64_t max_tokens = max_pages * cache->page_size;
  if (out_table != nullptr && (out_pages < 0 || out_stride < out_pages || out_pages > (kKvMaxTokens - 1) / cache->page_size ||
                               out_pages * cache->page_size < std::min(keep, max_tokens)))
    return SLOPE_ERR_SHAPE;
  if (B == 0) return SLOPE_OK;
  if (kept == nullptr || out_lens == nullptr) return SLOPE_ERR_NULL;
  if (!aligned(kept, 4) || !aligned(out_lens, 4) || !aligned(out_table, 4)) return SLOPE_ERR_STRIDE;
  const int64_t pairs = B * cache->Hkv, chunk = chunk_of(cache->dqk, cache->dv), chunks = (keep + chunk - 1) / chunk;
  if (pairs * chunks >= (int64_t(1) << 31) || pairs * kMaxCluster >= (int64_t(1) << 31)) return SLOPE_ERR_UNSUPPORTED;
  const Workspace w = workspace_of(pairs, chunks);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return SLOPE_ERR_WORKSPACE;

  KvEvictParams p{};
  p.seqs = kv_seqs(&batch, cache, 0);
  p.Hkv = cache->Hkv;
  p.weights_in = p.weights = static_cast<float*>(weights->data);
  p.w_spage = weights->stride[0];
  p.w_shead = weights->stride[1];
  p.keep = static_cast<int32_t>(keep);
  p.first = static_cast<int32_t>(first);
  p.recent = static_cast<int32_t>(recent);
  p.out_table = out_table;
  p.out_stride = out_stride;
  p.kept = kept;
  p.out_lens = out_lens;
  p.k_in = p.k = static_cast<uint4*>(cache->k);
  p.v_in = p.v = static_cast<uint4*>(cache->v);
  for (int i = 0; i < 3; ++i) {
    p.k_stride[i] = cache->k_stride[i] / 8;
    p.v_stride[i] = cache->v_stride[i] / 8;
  }
  p.chunk = static_cast<int32_t>(chunk);
  p.chunks = static_cast<int32_t>(chunks);
  char* const ws = static_cast<char*>(workspace);
  p.tickets = reinterpret_cast<uint32_t*>(ws);
  p.launches = static_cast<int32_t>((B + kKvMaxSeqs - 1) / kKvMaxSeqs);
  p.flags = reinterpret_cast<uint32_t*>(ws + w.flags);
  p.bounds = reinterpret_cast<int32_t*>(ws + w.bounds);
  p.status = device_status_ptr();
  if (p.status == nullptr) return cuda_fail("device status word (cudaGetSymbolAddress)");
  p.wait_limit_ns = wait_limit_ns();
  if (kv_sm_count() <= 0) return cuda_fail("device attributes");
  const cudaError_t e = launch_evict(p, B, cache->dqk, cache->dv, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("cache eviction kernel launch", e);
}

}  // extern "C"
