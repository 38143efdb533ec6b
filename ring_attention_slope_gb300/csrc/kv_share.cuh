// How attention over the paged cache shares its work out: every CTA's producer warp reads the sequences' lengths, works out
// the same shares, and claims them from a counter until none is left.
//
// A pair is (sequence, part of a KV head, row block), its steps the key tiles that its rows see.  All pairs stand in one
// line: sequences with nearly the longest steps first, in a sequence head by head, a head's latest rows first.  Whole pairs
// are claimed in that order, so that neighbours share a head's keys through L2, for as many full rounds over the grid as
// the long sequences give; what is left of the line is cut into equal shares, one for each CTA.  A share begins and ends
// inside pairs, so a CTA has at most two pieces that are to be joined with others', and a pair's pieces are those of
// consecutive shares.  Where that is slower (few steps to a pair) every pair is claimed whole.
//
// Measured in kv_attn.cu.  Half, three quarters or seven eighths of the cost for a block whose second Q tile is empty, as it has half
// the work, was wrong (4 chunks of 777 tokens, 192/128: 198 -> 240, 201, 199 us): its steps, one chain of latencies after
// another, take as long.
#pragma once

#include "kv_cache.cuh"
#include "kv_cut.cuh"

namespace slope {

// The row blocks of a sequence and their steps.
struct RowCut {
  int block_tokens, window;
  __device__ __forceinline__ int blocks(const KvSeq& q) const { 
    if (q.n <= block_tokens) return min(q.n, 1);
    return static_cast<int>(divide(static_cast<uint32_t>(q.n + block_tokens - 1), static_cast<uint32_t>(block_tokens)));
  }
  // Key tiles [first, last) that some row of block `blk` sees.
  __device__ __forceinline__ void range(const KvSeq& q, int blk, int& first, int& last) const {
    const int pos0 = q.len - q.n + blk * block_tokens, tokens = min(block_tokens, q.n - blk * block_tokens);
    const int lo = window > 0 ? max(0, pos0 - window + 1) : 0;
    first = lo / kBlockN;
    last = max(first, (max(min(q.len, pos0 + tokens), 0) + kBlockN - 1) / kBlockN);
  }
  __device__ __forceinline__ int steps(const KvSeq& q, int blk) const {
    int first, last;
    range(q, blk, first, last);
    return last - first;
  }
  // Bounds of them over the blocks: no more than that, and no fewer where there are any.
  __device__ __forceinline__ int most(const KvSeq& q) const {
    const int all = (q.len + kBlockN - 1) / kBlockN;
    return max(1, window > 0 ? min(all, (window + block_tokens - 2) / kBlockN + 2) : all);
  }
  // (Without a window the first block sees the fewest; with one a block that does not begin at key 0 sees one tile less or
  // more than its neighbours, the last block apart.)
  __device__ __forceinline__ int fewest(const KvSeq& q) const {
    const int ends = min(steps(q, 0), steps(q, blocks(q) - 1));
    return max(1, window > 0 ? min(ends, most(q) - 2) : ends);
  }
};

struct Shares {
  uint32_t whole, shares;  // claims: whole pairs, then shares of the rest of the line
  uint32_t pairs;          // of the line
  int seqs;                // listed
  int per_step;            // see cost_of
  uint32_t from, cost;     // where the rest begins in the line, and what it costs
};

// In shared memory: the sequences, and those that have new tokens in the line's order.
struct ShareLists {
  KvSeq seqs[kKvMaxSeqs];      // of the launch
  uint32_t pairs[kKvMaxSeqs];  // before the sequence's
  uint32_t cost[kKvMaxSeqs];   // of the pairs before the sequence's
  uint16_t index[kKvMaxSeqs];  // in seqs
  __device__ __forceinline__ const KvSeq& at(int s) const { return seqs[index[s]]; }
};

// What a pair costs, in eighths of a step: its steps, and kPieceSteps of them for its start and end, less where a CTA's
// share is so small (per_step) that the number of pairs says little about its time.
template <int kPieceSteps>
__device__ __forceinline__ uint32_t cost_of(int most, int per_step) {
  return 8u * static_cast<uint32_t>(most + min(kPieceSteps, per_step * most));
}

// A place inside a pair, `in` of its cost w, as one of its steps: in * steps / w, rounded down, with in and w in 11 bits so that
// 32 are enough for the product.  Places that are step_cost or more apart are different steps.
__device__ __forceinline__ int scale_of(uint32_t w) { return max(0, 21 - __clz(static_cast<int>(w))); }
__device__ __forceinline__ int step_at(uint32_t in, uint32_t w, int steps) {
  const int s = scale_of(w);
  return static_cast<int>(divide((in >> s) * static_cast<uint32_t>(steps), s > 0 ? (w >> s) + 1u : w));
}
__device__ __forceinline__ uint32_t step_cost(uint32_t w, int fewest) {
  const int s = scale_of(w);
  return divide(w + static_cast<uint32_t>(fewest) - 1u, static_cast<uint32_t>(fewest)) + (s > 0 ? 1u << s : 0u);
}

// The last entry of first[s .. n - 1] that is not above x; first[s] is not.
__device__ __forceinline__ int last_not_above(const uint32_t* first, int n, uint32_t x, int s) {
  if (s + 1 >= n || first[s + 1] > x) return s;
  for (int hi = n - 1; s < hi;) {
    const int mid = (s + hi + 1) >> 1;
    if (first[mid] <= x)
      s = mid;
    else
      hi = mid - 1;
  }
  return s;
}

// One whole warp calls it.  Estimates are in fp32, the same in every CTA; what says where a share begins is in whole
// numbers.
template <int kPieceSteps, int kCtas>
__device__ __forceinline__ Shares make_shares(const KvSeqs& p, int heads, const RowCut& cut, ShareLists& lists) {
  const int lane = threadIdx.x & 31;
  uint32_t sum = 0, block_sum = 0;  // of a lane no more than 2^26
  int most = 1;
  KvSeq mine{};
  int my_blocks = 0, my_most = 0;  // of the lane's last sequence, its only one where there are no more than 32
#pragma unroll 1
  for (int b = lane; b < p.B; b += 32) {
    mine = lists.seqs[b] = kv_seq(p, b);
    my_blocks = cut.blocks(mine);
    my_most = cut.most(mine);
    if (my_blocks > 0) {
      most = max(most, my_most);
      block_sum = min(block_sum + static_cast<uint32_t>(my_blocks), 1u << 26);
      sum = static_cast<uint32_t>(
          fminf(static_cast<float>(sum) + static_cast<float>(my_blocks) * static_cast<float>(my_most), 67108864.f));
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const float per_cta = __fdividef(static_cast<float>(heads), static_cast<float>(gridDim.x));
  const float steps = static_cast<float>(__reduce_add_sync(0xffffffffu, sum)) * per_cta;  // a CTA's, evenly
  Shares r;
  r.per_step = max(0, min(static_cast<int>(fminf(steps, 100.f)) - 1, kPieceSteps));
  const uint32_t all_blocks = __reduce_add_sync(0xffffffffu, block_sum);
  const float all_rounds = static_cast<float>(all_blocks) * per_cta;
  const float even = steps + all_rounds * kPieceSteps;
  // the line, in two passes: the long sequences, then the others
  uint32_t pairs = 0, long_pairs = 0, finest = 8, cost = 0;
  int listed = 0;
  bool all = false;
#pragma unroll 1
  for (int pass = 0; pass < 2 && !all; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      if (p.B > 32 && b < p.B) {
        mine = lists.seqs[b];  // (the lane wrote it)
        my_blocks = cut.blocks(mine);
        my_most = cut.most(mine);
      }
      const bool has = b < p.B && my_blocks > 0, here = has && (10 * my_most >= 9 * most) == (pass == 0);
      const uint32_t some = __ballot_sync(0xffffffffu, here);
      all = p.B <= 32 && some == __ballot_sync(0xffffffffu, has);
      if (some == 0) continue;
      const uint32_t n = here ? static_cast<uint32_t>(my_blocks) * static_cast<uint32_t>(heads) : 0u;
      const uint32_t w = here ? cost_of<kPieceSteps>(my_most, r.per_step) : 0u;
      if (here) finest = max(finest, step_cost(w, cut.fewest(mine)));
      uint32_t in = n, ic = n * w;
      if ((some & (some - 1u)) != 0) {  // more than one
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const uint32_t on = __shfl_up_sync(0xffffffffu, in, m), oc = __shfl_up_sync(0xffffffffu, ic, m);
          if (lane >= m) in += on, ic += oc;
        }
      }
      if (here) {
        const int at = listed + __popc(some & ((1u << lane) - 1u));
        lists.index[at] = static_cast<uint16_t>(b);
        lists.pairs[at] = pairs + in - n;
        lists.cost[at] = cost + ic - n * w;
      }
      const int last = 31 - __clz(some);
      pairs += __shfl_sync(0xffffffffu, in, last);
      cost += __shfl_sync(0xffffffffu, ic, last);
      listed += __popc(some);
    }
    if (pass == 0) long_pairs = pairs;
  }
  __syncwarp();
  finest = __reduce_max_sync(0xffffffffu, finest);
  r.pairs = pairs;
  r.seqs = listed;
  // as many full rounds of long pairs as there are, and the rest in shares
  const uint32_t rounds = long_pairs < gridDim.x ? 0 : divide(long_pairs, gridDim.x);
  r.whole = rounds * gridDim.x;
  r.from = 0;
  if (r.whole > 0) {
    const int s = last_not_above(lists.pairs, listed, r.whole, 0);
    r.from = lists.cost[s] + (r.whole - lists.pairs[s]) * cost_of<kPieceSteps>(cut.most(lists.at(s)), r.per_step);
  }
  r.cost = cost - r.from;
  r.shares = min(gridDim.x, divide(r.cost, finest));
  const float piece = static_cast<float>(most + kPieceSteps);
  // A last round that leaves every SM one of its two CTAs is shorter: 0.65 of one (four 2K chunks at 32K, window 1024: 223 us, as
  // with 0.5 and 0.8; with a whole one 236).  Whole pairs that are not alike end unevenly, half a piece later on average (a
  // chunk beside 15 single tokens: 265 us in shares, which it takes by that, and 292 whole; with a whole piece as with half).
  const float last = all_rounds - floorf(all_rounds);
  const float uncut = all_rounds <= 1.f        ? fmaxf(piece, even)
                      : long_pairs == pairs ? (kCtas == 2 && last <= 0.5f ? floorf(all_rounds) + 0.65f : ceilf(all_rounds)) * piece
                                            : fmaxf(piece, even) + 0.5f * piece;
  // a share's time: its steps, and the start and end of its pieces
  const float wholes = static_cast<float>(rounds), spread = __fdividef(static_cast<float>(gridDim.x), static_cast<float>(r.shares));
  const float share = fmaxf(0.f, steps - wholes * static_cast<float>(most)) * spread +
                      (fmaxf(0.f, all_rounds - wholes) * spread + 1.f) * kPieceSteps;
  // Shares of many long pairs each would have all heads' keys read at once; and costs are counted in 32 bits.  (Of 44 calls
  // the limit of 3 pieces decides in none, as without it all take the same time.  256 sequences up to 4096 tokens, one new each,
  // would be faster whole, as with a limit of 2: 105 us, in shares 141.)
  if (r.shares == 0 || wholes * piece + share >= uncut || share > 3.f * piece || steps * static_cast<float>(gridDim.x) > 6e7f)
    r.whole = pairs, r.shares = 0;
  // Row ranges that overlap can make more pairs than can be counted (those of a call that is in order are below 2^29 and its
  // blocks below 2^26): no work then.
  if (all_blocks >= 1u << 26 || all_rounds * static_cast<float>(gridDim.x) > 1.0e9f) r.whole = r.shares = 0;
  return r;
}

// Where share k begins, from the place where the first one does.
__device__ __forceinline__ uint32_t share_begin(const Shares& sh, uint32_t k) {
  const uint32_t each = divide(sh.cost, sh.shares), more = sh.cost - each * sh.shares;
  return k * each + divide(k * more, sh.shares);  // (k and more are below 2^9)
}

// The same as step `step` of pair `pair`; at the end of the line one past its last pair.
struct ShareStart {
  uint32_t pair;
  int step;
};
template <int kPieceSteps>
__device__ __forceinline__ ShareStart share_start(const ShareLists& lists, const Shares& sh, const RowCut& cut, uint32_t k) {
  ShareStart r{sh.pairs, 0};
  if (k >= sh.shares) return r;
  const uint32_t x = sh.from + share_begin(sh, k);
  const int s = last_not_above(lists.cost, sh.seqs, x, 0);
  const KvSeq q = lists.at(s);
  const uint32_t w = cost_of<kPieceSteps>(cut.most(q), sh.per_step), o = x - lists.cost[s], local = divide(o, w);
  const uint32_t blocks = static_cast<uint32_t>(cut.blocks(q));
  const uint32_t blk = blocks == 1 ? 0u : blocks - 1u - (local - divide(local, blocks) * blocks);
  r.pair = lists.pairs[s] + local;
  r.step = step_at(o - local * w, w, cut.steps(q, static_cast<int>(blk)));
  return r;
}

// The last share that begins before the end of pair g, of listed sequence s.
template <int kPieceSteps>
__device__ __forceinline__ uint32_t last_share(const ShareLists& lists, const Shares& sh, const RowCut& cut, uint32_t g, int s) {
  const uint32_t w = cost_of<kPieceSteps>(cut.most(lists.at(s)), sh.per_step);
  const uint32_t end = lists.cost[s] + (g - lists.pairs[s] + 1u) * w - sh.from;
  // from an estimate that is not too low, and off by one or two at most
  uint32_t k = min(sh.shares - 1u, static_cast<uint32_t>(__fdividef(static_cast<float>(end), static_cast<float>(sh.cost)) *
                                                         static_cast<float>(sh.shares)) + 1u);
  while (k > 0 && share_begin(sh, k) >= end) --k;
  return k;
}

}  // namespace slope
