// How the kernels on the paged cache share their work out: every CTA's producer warp reads the sequences' lengths, works
// out the same cut into pieces, and claims pieces from a counter until none is left.
//
// A sequence's work is `heads` times `blocks` pairs of up to `steps` steps each (what a step is, the kernel says).  A
// pair is cut into equal pieces of at most `per` steps.
#pragma once

#include "kv_cache.cuh"

namespace slope {

struct SeqCut {
  int blocks, steps;
  bool join;  // the pieces of a pair are joined (else each writes results of its own)
};
__device__ __forceinline__ int pieces_of(int steps, int per) { return max(1, (steps + per - 1) / per); }

// The sequences' records and first pieces, in shared memory.
struct CutLists {
  KvSeq seqs[kKvMaxSeqs];
  uint32_t units[kKvMaxSeqs];  // pieces before the sequence's
  uint32_t slots[kKvMaxSeqs];  // joined pieces before the sequence's
};
struct Cut {
  uint32_t total, slots;  // pieces, and those of pairs with several
  int per;
};
// Joined pieces of a launch at most: no length of pieces is below 1 / (2 kFine) of a share of the steps (an even division
// of them by the grid), and a pair of several pieces has fewer than twice as many as its steps divided by their length.
template <int kFine>
int64_t max_joined(int64_t grid) {
  return kFine * (4 * grid + grid / 8) + 8;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One whole warp calls it: reads the sequences, chooses the pieces' length and fills the lists.  cut_of(seq) gives a
// sequence's SeqCut; kPieceSteps is what a piece's start and end cost, in steps.
//
// The longest pair is cut into pieces of about 1 / (2 kFine) to 4 / kFine of a share, and the length of those is tried as
// every pair's.  The length with the least time wins: that of one piece or of an even share of all of them, whichever is more,
// and half a piece for the uneven end where there are more pieces than CTAs.  (Estimates in fp32, the same in every CTA.)
template <int kPieceSteps, int kFine, typename CutOf>
__device__ __forceinline__ Cut make_cut(const KvSeqs& p, int heads, const CutOf& cut_of, CutLists& lists) {
  constexpr int kTries = 6;
  constexpr float kShares[kTries] = {0.5f, 0.75f, 1.f, 1.5f, 2.5f, 4.f};
  const int B = p.B, lane = threadIdx.x & 31;
  const float per_cta = static_cast<float>(heads) / static_cast<float>(gridDim.x);
  float all = 0.f;
  int most = 1;
  for (int b = lane; b < B; b += 32) {
    const KvSeq q = kv_seq(p, b);
    lists.seqs[b] = q;
    const SeqCut c = cut_of(q);
    all += static_cast<float>(c.blocks) * static_cast<float>(c.steps);
    if (c.blocks > 0) most = max(most, c.steps);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const float share = fmaxf(1.f, warp_sum(all) * per_cta);
  int per[kTries];
  float count[kTries], inv[kTries];
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    const float n = fmaxf(1.f, rintf(__fdividef(static_cast<float>(most), share * (kShares[i] / kFine))));  // pieces of the longest
    per[i] = static_cast<int>(ceilf(__fdividef(static_cast<float>(most), n)));
    if (2.f * kFine * static_cast<float>(per[i]) < share) per[i] = most;  // (see max_joined)
    inv[i] = __frcp_rn(static_cast<float>(per[i]));
    count[i] = 0.f;
  }
  __syncwarp();
  for (int b = lane; b < B; b += 32) {
    const SeqCut c = cut_of(lists.seqs[b]);
#pragma unroll
    for (int i = 0; i < kTries; ++i)
      count[i] += static_cast<float>(c.blocks) * fmaxf(1.f, ceilf(static_cast<float>(c.steps) * inv[i] - 1e-4f));
  }
  Cut r;
  r.per = most;
  float best = INFINITY;
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    const float rounds = warp_sum(count[i]) * per_cta, piece = static_cast<float>(per[i] + kPieceSteps);
    const float cost = fmaxf(piece, share + rounds * kPieceSteps) + (rounds > 1.f ? 0.5f * piece : 0.f);
    if (cost < best) {
      best = cost;
      r.per = per[i];
    }
  }
  r.total = r.slots = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    uint32_t u = 0, sl = 0;
    if (b < B) {
      const SeqCut c = cut_of(lists.seqs[b]);
      const int n = pieces_of(c.steps, r.per);
      u = static_cast<uint32_t>(heads) * c.blocks * n;
      sl = n > 1 && c.join ? u : 0;
    }
    uint32_t iu = u, is = sl;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t ou = __shfl_up_sync(0xffffffffu, iu, m), os = __shfl_up_sync(0xffffffffu, is, m);
      if (lane >= m) iu += ou, is += os;
    }
    if (b < B) lists.units[b] = r.total + iu - u, lists.slots[b] = r.slots + is - sl;
    r.total += __shfl_sync(0xffffffffu, iu, 31);
    r.slots += __shfl_sync(0xffffffffu, is, 31);
  }
  __syncwarp();
  return r;
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

// Steps [first, last) of piece c out of `pieces`.
__device__ __forceinline__ void piece_steps(int steps, int pieces, int c, int& first, int& last) {
  const int each = steps / pieces, more = steps - each * pieces;
  first = c * each + min(c, more);
  last = first + each + (c < more ? 1 : 0);
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
