// How the kernels on the paged cache share their work out: every CTA reads the sequences' lengths, works out the same
// cut into pieces, and claims pieces from a counter until none is left.
//
// A sequence's work is `heads` times `blocks` pairs of up to `steps` steps each (what a step is, the kernel says).  A
// pair is cut into equal pieces of at most `per` steps.
#pragma once

#include "kv_cache.cuh"

namespace slope {

constexpr int kTries = 6;  // lengths of pieces that are tried

struct SeqCut {
  int blocks, steps;
};
__device__ __forceinline__ int pieces_of(int steps, int per) { return max(1, (steps + per - 1) / per); }

constexpr int kCutWarps = 12;  // of a CTA at most
struct CutScratch {
  unsigned long long sums[kCutWarps][kTries];
  int most[kCutWarps];
  uint32_t total, slots;  // pieces, and those of pairs with several
  int per;
};

// The sequences' records and first pieces, in shared memory.
struct CutLists {
  KvSeq seqs[kKvMaxSeqs];
  uint32_t units[kKvMaxSeqs + 1];  // pieces before the sequence's
  uint32_t slots[kKvMaxSeqs + 1];  // joined pieces before the sequence's
};

// Sums over the CTA's threads; every thread gets them.
template <int kN>
__device__ __forceinline__ void block_sums(CutScratch& s, unsigned long long (&v)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) s.sums[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    v[i] = 0;
    for (int w = 0; w < warps; ++w) v[i] += s.sums[w][i];
  }
}

// Every thread of the CTA calls it: reads the sequences, chooses the pieces' length and fills the lists.  cut_of(seq) gives a
// sequence's SeqCut; kPieceSteps is what a piece's start and end cost, in steps.
//
// Lengths from half to three times an even share of all steps are tried; the one whose rounds over the grid are
// shortest wins.  No length is below half a share, so fewer than 4 * grid pieces are joined (a pair of several pieces
// has fewer than twice as many as its steps divided by `per`).
template <int kPieceSteps, typename Cut>
__device__ __forceinline__ void make_cut(const KvSeqs& p, int heads, const Cut& cut_of, CutScratch& s, CutLists& lists) {
  const int B = p.B;
  unsigned long long all[1] = {0};
  int most = 1;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const KvSeq q = kv_seq(p, b);
    lists.seqs[b] = q;
    const SeqCut c = cut_of(q);
    all[0] += static_cast<unsigned long long>(c.blocks) * c.steps;
    if (c.blocks > 0) most = max(most, c.steps);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((threadIdx.x & 31) == 0) s.most[threadIdx.x >> 5] = most;
  block_sums(s, all);  // (its barriers order s.most too)
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) most = max(most, s.most[w]);
  const unsigned long long share = max(1ull, (all[0] * heads + gridDim.x - 1) / gridDim.x);
  constexpr int kQuarters[kTries] = {2, 3, 4, 5, 8, 12};  // of a share
  int per[kTries];
  unsigned long long count[kTries];
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    per[i] = static_cast<int>(min(static_cast<unsigned long long>(most), (share * kQuarters[i] + 3) / 4));
    count[i] = 0;
  }
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const SeqCut c = cut_of(lists.seqs[b]);
#pragma unroll
    for (int i = 0; i < kTries; ++i) count[i] += static_cast<unsigned long long>(c.blocks) * pieces_of(c.steps, per[i]);
  }
  block_sums(s, count);
  int best = per[0];
  unsigned long long best_cost = ~0ull;
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    const int pieces = pieces_of(most, per[i]);
    const unsigned long long rounds = (count[i] * heads + gridDim.x - 1) / gridDim.x;
    const unsigned long long cost = rounds * ((most + pieces - 1) / pieces + kPieceSteps);
    if (cost < best_cost) {
      best_cost = cost;
      best = per[i];
    }
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    uint32_t unit = 0, slot = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      uint32_t u = 0, sl = 0;
      if (b < B) {
        const SeqCut c = cut_of(lists.seqs[b]);
        const int n = pieces_of(c.steps, best);
        u = static_cast<uint32_t>(heads) * c.blocks * n;
        sl = n > 1 ? u : 0;
      }
      uint32_t iu = u, is = sl;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint32_t ou = __shfl_up_sync(0xffffffffu, iu, m), os = __shfl_up_sync(0xffffffffu, is, m);
        if (lane >= m) iu += ou, is += os;
      }
      if (b < B) lists.units[b] = unit + iu - u, lists.slots[b] = slot + is - sl;
      unit += __shfl_sync(0xffffffffu, iu, 31);
      slot += __shfl_sync(0xffffffffu, is, 31);
    }
    if (lane == 0) {
      s.total = unit;
      s.slots = slot;
      s.per = best;
    }
  }
  __syncthreads();
}

// The sequence (of the launch) that piece w belongs to.
__device__ __forceinline__ int seq_of(const CutLists& lists, int B, uint32_t w) {
  int b = 0;
  for (int hi = B - 1; b < hi;) {  // the last one whose first piece is not after w: one that has pieces
    const int mid = (b + hi + 1) >> 1;
    if (lists.units[mid] <= w)
      b = mid;
    else
      hi = mid - 1;
  }
  return b;
}

// For a CTA that takes no more pieces: claims until an index past the end comes back, so that every CTA takes exactly one
// of those, and the one that is handed the last puts the counter back to 0.
__device__ __forceinline__ void release_pieces(uint32_t* counter, uint32_t total, uint32_t w) {
  for (;; w = atomicAdd(counter, 1u)) {
    if (w >= total) {
      if (w == total + gridDim.x - 1) atomicExch(counter, 0u);
      return;
    }
  }
}

}  // namespace slope
