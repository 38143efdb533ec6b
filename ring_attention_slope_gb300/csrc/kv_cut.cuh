// How the weights' kernel on the paged cache shares its work out: every CTA's producer warp reads the sequences' lengths, works
// out the same cut into pieces, and claims pieces from a counter until none is left.  (Attention: kv_share.cuh.  The weights'
// pieces mostly write results of their own, so cutting a pair costs them little.)
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
// a / b, without a division's forty instructions where a < 2^20: a quotient next to a whole number is at least 1 / (2 b) away
// from it with the half added, and off by at most 2^-22 of itself.
// (The rare other case is kept out of line: code that runs once, before a call's first load, is as slow as it is long.)
static __device__ __noinline__ uint32_t divide_any(uint32_t a, uint32_t b) { return a / b; }
__device__ __forceinline__ uint32_t divide(uint32_t a, uint32_t b) {
  if (__builtin_expect(a >= (1u << 20), 0)) return divide_any(a, b);
  return __float2uint_rz(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b)));
}
__device__ __forceinline__ int pieces_of(int steps, int per) {
  return max(1, static_cast<int>(divide(static_cast<uint32_t>(steps + per - 1), static_cast<uint32_t>(per))));
}

// The sequences' records and first pieces, in shared memory.
struct CutLists {
  KvSeq seqs[kKvMaxSeqs];
  uint32_t units[kKvMaxSeqs];  // pieces before the sequence's
  uint32_t slots[kKvMaxSeqs];  // joined pieces before the sequence's
  uint32_t joins[kKvMaxSeqs];  // pairs of several pieces before the sequence's
};
struct Cut {
  uint32_t total, joins;  // pieces, and pairs that have several
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
// The longest pair is cut so that no CTA has more than one piece, or into pieces of about 1 / (2 kFine) to 3 / kFine of
// a share, and the length of those is tried as every pair's.  The length with the least time wins: that of the rounds over
// the grid where the pieces are all alike, else that of one piece or of an even share of all of them, whichever is
// more, and half a piece for the uneven end.  Estimates are in fp32, the same in every CTA.  This runs before a call's
// first load: the six lengths are tried side by side, as one after another they took 1.3 us.
template <int kPieceSteps, int kFine, typename CutOf>
__device__ __forceinline__ Cut make_cut(const KvSeqs& p, int heads, const CutOf& cut_of, CutLists& lists) {
  const int B = p.B, lane = threadIdx.x & 31;
  const float per_cta = __fdividef(static_cast<float>(heads), static_cast<float>(gridDim.x));
  float all = 0.f;
  int most = 1;
  uint32_t pairs = 0;        // of a lane at most 2^24
  SeqCut mine{0, 0, false};  // of the lane's only sequence, where there are no more than 32
#pragma unroll 1
  for (int b = lane; b < B; b += 32) {
    const KvSeq q = kv_seq(p, b);
    lists.seqs[b] = q;
    mine = cut_of(q);
    all += static_cast<float>(mine.blocks) * static_cast<float>(mine.steps);
    pairs = min(pairs + static_cast<uint32_t>(mine.blocks), 1u << 24);
    if (mine.blocks > 0) most = max(most, mine.steps);
  }
  __syncwarp();
  most = __reduce_max_sync(0xffffffffu, most);
  const float sum = warp_sum(all) * per_cta, share = fmaxf(1.f, sum), longest = static_cast<float>(most);
  constexpr int kTries = 6;
  constexpr float kShares[kTries] = {0.f, 0.5f, 0.75f, 1.f, 1.6f, 3.f};
  // the shortest length with which the pieces are surely no more than the CTAs (a pair has less than one more than its
  // steps divided by it)
  const float spare = 1.f - static_cast<float>(__reduce_add_sync(0xffffffffu, pairs)) * per_cta;
  const float one_each = spare > 0.f ? fmaxf(1.f, ceilf(__fdividef(sum, spare))) : longest;
  int per[kTries];
  float inv[kTries];
  uint32_t count[kTries];  // of a lane at most 2^24
  auto add = [&](const SeqCut& c) {
#pragma unroll
    for (int i = 0; i < kTries; ++i)
      count[i] = static_cast<uint32_t>(fminf(
          static_cast<float>(count[i]) +
              static_cast<float>(c.blocks) * fmaxf(1.f, ceilf(static_cast<float>(c.steps) * inv[i] - 1e-4f)),
          16777216.f));
  };
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    // pieces of the longest
    const float n = fmaxf(1.f, i == 0 ? ceilf(__fdividef(longest, one_each) - 1e-4f)
                                      : rintf(__fdividef(longest, share * (kShares[i] / kFine))));
    per[i] = static_cast<int>(ceilf(__fdividef(longest, n)));
    if (2.f * kFine * static_cast<float>(per[i]) < share) per[i] = most;  // (see max_joined)
    inv[i] = __fdividef(1.f, static_cast<float>(per[i]));
    count[i] = 0;
  }
  if (B <= 32) {
    add(mine);
  } else {
#pragma unroll 1
    for (int b = lane; b < B; b += 32) add(cut_of(lists.seqs[b]));
  }
  Cut r;
  r.per = most;
  float best = INFINITY;
#pragma unroll
  for (int i = 0; i < kTries; ++i) {
    const float rounds = static_cast<float>(__reduce_add_sync(0xffffffffu, count[i])) * per_cta;
    const float piece = static_cast<float>(per[i] + kPieceSteps);
    const float even = share + rounds * kPieceSteps;
    // Alike: if full rounds of the longest pieces would be no more than a ninth longer than the even share (a 1K chunk at 16K,
    // 32/4 heads of 128: 116 us, and 17 queries each of 30 sequences of 2040, 64/8 heads of 64, 25.4; at 0.8 the same; with
    // none alike, 1.0, 108 and 31).  The half piece decides in no call measured: 0 and a whole one are as fast.
    const float cost = rounds <= 1.f                   ? fmaxf(piece, even)
                       : even > 0.9f * rounds * piece ? ceilf(rounds) * piece
                                                       : fmaxf(piece, even) + 0.5f * piece;
    if (cost < best) {
      best = cost;
      r.per = per[i];
    }
  }
  r.total = r.joins = 0;
  uint32_t slots = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    uint32_t u = 0, sl = 0, jn = 0;
    if (b < B) {
      const SeqCut c = cut_of(lists.seqs[b]);
      const int n = pieces_of(c.steps, r.per);
      u = static_cast<uint32_t>(heads) * c.blocks * n;
      if (n > 1 && c.join) sl = u, jn = static_cast<uint32_t>(heads) * c.blocks;
    }
    uint32_t iu = u, is = sl, ij = jn;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t ou = __shfl_up_sync(0xffffffffu, iu, m), os = __shfl_up_sync(0xffffffffu, is, m);
      const uint32_t oj = __shfl_up_sync(0xffffffffu, ij, m);
      if (lane >= m) iu += ou, is += os, ij += oj;
    }
    if (b < B) lists.units[b] = r.total + iu - u, lists.slots[b] = slots + is - sl, lists.joins[b] = r.joins + ij - jn;
    r.total += __shfl_sync(0xffffffffu, iu, 31);
    slots += __shfl_sync(0xffffffffu, is, 31);
    r.joins += __shfl_sync(0xffffffffu, ij, 31);
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
  const int each = static_cast<int>(divide(static_cast<uint32_t>(steps), static_cast<uint32_t>(pieces)));
  const int more = steps - each * pieces;
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
