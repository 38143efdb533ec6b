// Attention of each sequence's newest tokens over its pages of the 16-bit cache: single tokens (a decode step), chunks
// of prompts, or both in one launch.
//
// out_i = sum_j 2^(x_ij - m_i) v_j / l_i, l_i = sum_j 2^(x_ij - m_i), x_ij = scale log2(e) q_i . k_j over the keys j that
// token i sees, with a running maximum m and sum l; lse_i = (m_i + log2 l_i) ln 2.
//
// A Q tile is 128 rows: as many tokens as fit times all query heads of a KV head, token by token, so a key tile is
// read once for the whole group and a chunk's diagonal wastes a few tokens' worth, whatever the group's size.  Q is
// loaded by TMA boxes of {64 channels, heads, tokens}; a key tile of 128 positions by boxes of one page (or 128 of its
// rows), each lane of the producer warp looking its pages up and starting its own boxes.  Pages that no row of the
// tile needs, and pages out of range, are boxes past the tensor's end, which read 0 without touching memory.
//
// Roles as in the prefill's kernel (attn_partial.cu): S = Q K^T (tcgen05, both operands in shared memory) into TMEM,
// one row per softmax thread, P back into TMEM, O += P V with P from TMEM.  With 64-wide heads two CTAs of one Q tile
// share an SM; wider heads have one CTA with two Q tiles, which take the same key tiles.  Warps whose 32 rows are all empty
// (a decode step has 8 rows, say) skip the softmax.
//
// The work: a pair is (sequence, KV head, row block), its steps the key tiles that its rows see.  The lengths are on the
// device, so every CTA works out the same shares of all pairs (kv_share.cuh) and claims them from a counter until none is
// left.  Pieces of a pair that lies in several shares leave (m, l, O) in the workspace, and a second launch, queued as a
// programmatic dependent, joins them in order; which CTA computes a share changes no bit.  Equal pieces of each pair, about as
// many as fill the rounds over the grid, in place of equal shares of the line: 2K chunk at 16K, 32 heads of 192/128, 559
// -> 502 us; 32/4 heads of 128/128 494 -> 439; a 1000-token chunk at 16K and 15 decoding sequences, 64/8 heads of 64,
// 292 -> 265; 1 x 1000 tokens 11.2 -> 11.7 (the shares take longer to work out).  The join inside this kernel by the CTA that
// is last at a pair was faster for one short sequence (10.9) and slower elsewhere (the mixed step by 35).
//
// What bounds it, on one GB300: long chunks the tensor cores with the softmax beside them (64/8 heads of 64, 4096 tokens at
// 64K: 3640 us, 1.17 PFLOP/s; if a 64-wide PV takes as long as a 128-wide one, 90% of the tensor pipe's time); decode steps
// HBM (8 x 102400 tokens: 255 us, 6.58 TB/s of the 6.68 of a copy; 32 ragged up to 32K: 65 us, 4.4 TB/s); short ones latencies
// (1 x 1000: 11.7 us, of which the join's launch 3, lengths and shares 2).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "kv_share.cuh"
#include "sm103_ptx.cuh"
#include "waits.cuh"

namespace slope {
namespace {

constexpr uint32_t kChunkBytes = 128 * 128;  // 128 rows x 64 bf16
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: the running maximum moves when a score passes it by this
constexpr int kPieceSteps = 5;             // what a piece's start and end cost, in steps
constexpr int kHoles = 8;                  // ring of the steps' missing pages: more than the K tiles in flight
constexpr int kJoinThreads = 512;

// A pair of which several pieces are joined.
struct KvPair {
  int32_t row0, tokens, head0, heads, slot, pieces, pad[2];
};

struct KvAttnParams {
  KvSeqs seqs;
  int32_t Hkv, group;
  RowTile tile;
  int32_t window;
  float scale_log2;
  void* out;
  int64_t out_srow, out_shead;
  int32_t out_bf16;
  float* lse;  // may be null
  int64_t lse_srow, lse_shead;
  int32_t rows_cap;  // rows of a piece in the workspace
  int32_t max_slots;
  int32_t* n_pairs;  // workspace: pairs that are joined
  KvPair* pairs;     // workspace: those
  float2* ml;        // workspace: m and l of a piece's rows
  float* part;       // workspace: O of its rows, not normalised
  int* status;
  uint32_t* tile_counter;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// ---------------------------------------------------------------- pieces

// A piece: steps [j0, j1) of a pair.
struct Piece {
  int32_t tokens;  // of the row block; -1: no pieces left
  int32_t row0;    // q row of its first token
  int32_t pos0;    // position of its first token
  int32_t j0, j1;  // key tiles
  int32_t len;     // tokens of the sequence
  int32_t kvh, head0, heads;
  int32_t slot;    // in the workspace; -1: the whole pair
  int32_t b;
  int32_t flo[2], fhi[2];  // steps [flo, fhi) that every row of Q tile t sees in full
};

// Steps [from, to) of pair g of the line; `to` may lie past its last.  s: a sequence of the list not behind the pair's, set to
// that one.
__device__ __forceinline__ Piece make_piece(const KvAttnParams& p, const ShareLists& lists, const Shares& shares,
                                            const RowCut& cut, uint32_t g, int from, int to, uint32_t share, int& s) {
  Piece r;
  s = last_not_above(lists.pairs, shares.seqs, g, s);
  const int block_tokens = cut.block_tokens;
  const KvSeq q = lists.at(s);
  // local = head * blocks + (blocks - 1 - block)
  const uint32_t blocks = static_cast<uint32_t>(cut.blocks(q)), local = g - lists.pairs[s];
  const int h = static_cast<int>(blocks == 1 ? local : divide(local, blocks));
  const int blk = static_cast<int>(blocks - 1 - (local - h * blocks));
  r.b = p.seqs.b0 + lists.index[s];
  r.kvh = p.tile.parts == 1 ? h : h / p.tile.parts;
  const int first = (h - r.kvh * p.tile.parts) * p.tile.heads;
  r.head0 = r.kvh * p.group + first;
  r.heads = min(p.tile.heads, p.group - first);
  r.tokens = min(block_tokens, q.n - blk * block_tokens);
  r.row0 = q.row0 + blk * block_tokens;
  r.pos0 = q.len - q.n + blk * block_tokens;
  r.len = q.len;
  int j_lo, j_hi;
  cut.range(q, blk, j_lo, j_hi);
  r.j0 = j_lo + from;
  r.j1 = min(j_hi, j_lo + to);
  r.slot = from > 0 ? 2 * static_cast<int32_t>(share) : r.j1 < j_hi ? 2 * static_cast<int32_t>(share) + 1 : -1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tile_tokens = p.tile.tokens, qa = r.pos0 + t * tile_tokens, rows = min(tile_tokens, r.tokens - t * tile_tokens);
    r.fhi[t] = min(r.len, qa + 1) >> 7;  // (of a negative position: below every step)
    r.flo[t] = p.window > 0 ? max(0, (qa + rows - 1 - p.window + kBlockN) >> 7) : 0;
  }
  return r;
}

template <int DQK, int DV, int QT>
struct Cfg {
  static constexpr int kTmaWarp = 4 * QT, kMmaWarp = kTmaWarp + 1;
  static constexpr int kThreads = 32 * (5 * QT + 1);
  static constexpr int kCtas = QT == 1 && DQK == 64 && DV == 64 ? 2 : 1;  // on an SM
  static constexpr uint32_t kTmemCols = 512 / kCtas;
  static constexpr int kQChunks = DQK / 64, kVChunks = DV / 64;
  static constexpr int kQTileBytes = kQChunks * kChunkBytes;
  static constexpr int kKTileBytes = kQTileBytes, kVTileBytes = kVChunks * kChunkBytes;
  // Steps whose K and V tiles fit: with one Q tile and wide heads (decode steps) two or more, so that the copies keep an
  // SM's share of HBM busy.
  static constexpr int kRoom = (kCtas == 2 ? 115712 : 232448) - 16384 - QT * kQTileBytes;
  static constexpr int kStages = kRoom / (kKTileBytes + kVTileBytes) < 4 ? kRoom / (kKTileBytes + kVTileBytes) : 4;
  static constexpr int kSlots = 2 * kStages;  // K tiles in even ones, V tiles in odd ones
  static_assert(kStages >= 1 && kStages + 2 <= kHoles, "the holes' ring");
  static constexpr int kNumBars = 2 + 2 * kSlots + 7 * QT + 4 * QT + 4;
  static constexpr int kSlotOffset = QT * kQTileBytes;
  static constexpr int kRestOffset = kSlotOffset + kStages * (kKTileBytes + kVTileBytes);
  __device__ static constexpr int slot_offset(uint32_t slot) {  // from kSlotOffset
    return static_cast<int>(slot / 2) * (kKTileBytes + kVTileBytes) + (slot % 2 ? kKTileBytes : 0);
  }
  struct Rest {  // behind the tiles
    uint64_t bars[kNumBars];
    Piece piece[2];
    uint16_t rows[kBlockM];  // of a Q tile: token << 8 | head
    uint32_t holes[kHoles];  // of a step's 16-token runs, those without a page
    uint32_t tmem;
    int abort;
    ShareLists lists;
  };
  static constexpr int kSmemBytes = kRestOffset + static_cast<int>(sizeof(Rest));
  static constexpr uint32_t kColO = QT * kBlockN, kColP = kColO + QT * DV;
  static constexpr bool kSepP = kColP + QT * (kBlockN / 2) <= kTmemCols;
  __device__ static constexpr uint32_t col_p(int t) { return kSepP ? kColP + t * (kBlockN / 2) : t * kBlockN; }
  // Where P overwrites S (dv = 128) the two softmax warps of an SM sub-partition take turns on their exponentials.
  static constexpr bool kTurns = QT == 2 && !kSepP;
  static_assert(kSmemBytes <= (kCtas == 1 ? 232448 : 115712), "shared memory budget");
  static_assert(kColO + QT * DV <= kTmemCols, "TMEM budget");
};

template <int DQK, int DV, int QT>
__global__ void __launch_bounds__(Cfg<DQK, DV, QT>::kThreads, Cfg<DQK, DV, QT>::kCtas)
    kv_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ KvAttnParams p) {
  using C = Cfg<DQK, DV, QT>;
  // All of the shared memory is dynamic and starts on a tile's boundary, so that its addresses are constants: computed
  // ones took registers that the softmax needs.
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const sQ = smem;
  uint8_t* const sSlot = smem + C::kSlotOffset;
  typename C::Rest& sh = *reinterpret_cast<typename C::Rest*>(smem + C::kRestOffset);
  uint64_t* const bar_q = sh.bars;
  uint64_t* const bar_qempty = bar_q + 1;
  uint64_t* const bar_full = bar_q + 2;
  uint64_t* const bar_empty = bar_full + C::kSlots;
  uint64_t* const bar_s = bar_empty + C::kSlots;
  uint64_t* const bar_sfree = bar_s + QT;  // softmax t has loaded S_t into registers
  uint64_t* const bar_p = bar_sfree + QT;
  uint64_t* const bar_p2 = bar_p + QT;  // P over S: the last quarter of P_t
  uint64_t* const bar_o = bar_p2 + QT;
  uint64_t* const bar_ofree = bar_o + QT;
  uint64_t* const bar_drain = bar_ofree + QT;
  uint64_t* const bar_turn = bar_drain + QT;     // [t * 4 + quarter]: that softmax warp may exponentiate
  uint64_t* const bar_wfull = bar_turn + 4 * QT;  // a piece is there
  uint64_t* const bar_wfree = bar_wfull + 2;      // every role is done with it
  volatile int* const cta_abort = &sh.abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowCut cut{QT * p.tile.tokens, p.window};
  const uint64_t limit = p.wait_limit_ns;

  pdl_launch_dependents();  // the join may be scheduled as this grid's CTAs leave
  if (threadIdx.x == C::kTmaWarp * 32) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (threadIdx.x < kBlockM)
    sh.rows[threadIdx.x] = static_cast<uint16_t>(threadIdx.x / p.tile.heads << 8 | threadIdx.x % p.tile.heads);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&sh.tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == C::kMmaWarp * 32) {
    mbar_init(bar_q, 1);
    mbar_init(bar_qempty, QT);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], QT);  // one commit per MMA issuer
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_sfree[t], 4);
      mbar_init(&bar_p[t], 4);
      mbar_init(&bar_p2[t], 4);
      mbar_init(&bar_o[t], 1);
      mbar_init(&bar_ofree[t], 4);
      mbar_init(&bar_drain[t], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&bar_turn[4 * t + q], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_wfull[i], 1);
      mbar_init(&bar_wfree[i], 5 * QT);  // the MMA issuers and the softmax warps
    }
    fence_barrier_init();
  }
  pdl_wait();               // the kernels before this one are done; nothing above touches memory
  uint32_t claimed = 0;     // the producer's first claim, on its way during the cut
  if (threadIdx.x == C::kTmaWarp * 32) claimed = atomicAdd(p.tile_counter, 1u);
  if (threadIdx.x == 0) *cta_abort = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // The k-th piece of the CTA, once it is there; false if the wait ran out.
  auto take_piece = [&](int k) -> bool { return wait_bounded(&bar_wfull[k & 1], (k >> 1) & 1, cta_abort, p.status, limit, 31); };

  if (warp == C::kTmaWarp) {
    // ================================================================ producer: pieces, pages, loads
    const Shares shares = make_shares<kPieceSteps, C::kCtas>(p.seqs, p.Hkv * p.tile.parts, cut, sh.lists);
    if (lane == 0 && blockIdx.x == 0) *p.n_pairs = static_cast<int32_t>(shares.shares);
    const uint32_t total = shares.whole + shares.shares;
    const uint32_t q_bytes = static_cast<uint32_t>(p.tile.heads * p.tile.tokens) * 128 * C::kQChunks;
    const int boxes_log = max(0, 7 - p.seqs.page_shift);  // log2 of the boxes of 64 channels of a key tile
    const int boxes = 1 << boxes_log, box_rows = kBlockN >> boxes_log;
    const int no_page = static_cast<int>(p.seqs.n_pages);  // reads 0
    const int shift = p.seqs.page_shift;
    uint32_t w = 0, next = claimed;  // the claim being worked on, and (in lane 0) the one after it,
    bool fresh = true;               // which has not been looked at
    uint32_t cnt = 0;   // K and V tiles loaded
    uint32_t step = 0;  // steps loaded
    int wt = 0;         // Q tiles loaded
    bool ok = *cta_abort == 0;
    // Entry e of the piece's block table: no_page where no row sees a key, -1 for a page out of range where one does.
    auto page_of = [&](const Piece& pc, int e) -> int {
      const int64_t first = static_cast<int64_t>(e) << shift;
      const int lo = p.window > 0 ? pc.pos0 - p.window + 1 : 0;  // positions [lo, hi) that some row sees
      const int hi = min(pc.len, pc.pos0 + pc.tokens);
      if (first >= hi || first + (int64_t(1) << shift) <= lo) return no_page;
      const int pg = p.seqs.table[pc.b * p.seqs.table_stride + e];
      return pg >= 0 && pg < no_page ? pg : -1;
    };
    // What is left of the claim: from step `step0` of pair `pair` to step `end_step` of pair `end`.
    uint32_t pair = 0, end = 0, share = 0;
    int step0 = 0, end_step = 0, seq = 0;
    bool over = false;  // w is past the last claim
    // A piece, and its first 64 pages: entry e0 + lane of the table in each lane, and the 32 after them on their way.  The next
    // one is made out while the first loads of this one are under way.
    struct Work {
      Piece pc;
      uint32_t pair, share;
      int seq, e0, page, ahead;
    };
    auto used_up = [&]() { return pair > end || (pair == end && step0 >= end_step); };
    auto prepare = [&](Work& q) -> bool {
      while (used_up()) {
        if (!fresh && lane == 0) next = atomicAdd(p.tile_counter, 1u);
        fresh = false;
        w = __shfl_sync(0xffffffffu, next, 0);
        if (w >= total) {
          over = true;
          return false;
        }
        if (w < shares.whole) {
          pair = w, end = w + 1, step0 = end_step = 0;
          continue;
        }
        share = w - shares.whole;
        const ShareStart at = share_start<kPieceSteps>(sh.lists, shares, cut, share + (lane & 1));  // its start and its end
        pair = __shfl_sync(0xffffffffu, at.pair, 0), end = __shfl_sync(0xffffffffu, at.pair, 1);
        step0 = __shfl_sync(0xffffffffu, at.step, 0), end_step = __shfl_sync(0xffffffffu, at.step, 1);
        // no pair begins in this share and goes on in others
        if (lane == 0 && (end_step == 0 || (end == pair && step0 > 0))) p.pairs[share].pieces = 0;
      }
      q.pc = make_piece(p, sh.lists, shares, cut, pair, step0, pair == end ? end_step : INT_MAX / 2, share, seq);
      q.pair = pair, q.share = share, q.seq = seq;
      ++pair, step0 = 0;
      q.e0 = (q.pc.j0 * kBlockN) >> shift;
      q.page = q.pc.j1 > q.pc.j0 ? page_of(q.pc, q.e0 + lane) : no_page;
      q.ahead = q.pc.j1 > q.pc.j0 ? page_of(q.pc, q.e0 + 32 + lane) : no_page;
      return true;
    };
    Work now{}, then{};
    bool more = true;
    for (int k = -1; ok; ++k) {  // (before the first piece there is only the next one to be made out)
      if (k >= 2) ok = warp_all(wait_bounded(&bar_wfree[k & 1], ((k >> 1) - 1) & 1, cta_abort, p.status, limit, 32));
      if (!ok) break;
      if (!more) {
        if (lane == 0) {
          sh.piece[k & 1].tokens = -1;
          mbar_arrive(&bar_wfull[k & 1]);
        }
        break;
      }
      if (k >= 0 && used_up()) {  // the next claim, on its way while this piece loads
        fresh = true;
        if (lane == 0) next = atomicAdd(p.tile_counter, 1u);
      }
      const Piece& pc = now.pc;
      if (lane == 0 && k >= 0) {
        sh.piece[k & 1] = pc;
        mbar_arrive(&bar_wfull[k & 1]);
      }
      auto load_rows = [&]() -> bool {
        // Q of the previous piece is in use until its last S MMAs are done
        if (wt > 0 && !warp_all(wait_bounded(bar_qempty, (wt - 1) & 1, cta_abort, p.status, limit, 33))) return false;
        if (lane == 0) {
          const int nt = QT == 2 && pc.tokens > p.tile.tokens ? 2 : 1;
          mbar_arrive_expect_tx(bar_q, nt * q_bytes);
          for (int t = 0; t < nt; ++t)
            for (int ch = 0; ch < C::kQChunks; ++ch)
              tma_load_3d(sQ + t * C::kQTileBytes + ch * kChunkBytes, &tm_q, bar_q, 64 * ch, pc.head0,
                          pc.row0 + t * p.tile.tokens);
        }
        ++wt;
        return true;
      };
      const bool rows_first = wt == 0;
      if (rows_first && pc.j1 > pc.j0) ok = load_rows();
      bool prepared = false;
      for (int j = pc.j0; ok; ++j, ++step) {
        if (!prepared && (j == pc.j0 + 2 || j >= pc.j1)) {
          prepared = true;
          more = prepare(then);
        }
        if (j >= pc.j1) break;
        const int e = (j * kBlockN) >> shift;
        if (e >= now.e0 + 32) {
          now.e0 += 32;
          now.page = now.ahead;
          now.ahead = page_of(pc, now.e0 + 32 + lane);
        }
        // lane i loads box i % boxes of channel chunk i / boxes
        const int mine = __shfl_sync(0xffffffffu, now.page, (e - now.e0) + (lane & (boxes - 1)));
        const uint32_t missing = __ballot_sync(0xffffffffu, mine < 0) & ((1u << boxes) - 1);
        const int pg = mine < 0 ? no_page : mine;
        const int in_page = boxes_log > 0 ? 0 : (j * kBlockN) & ((1 << shift) - 1);
        const int chunk = lane >> boxes_log;
        const uint32_t at = static_cast<uint32_t>(chunk) * kChunkBytes + (lane & (boxes - 1)) * box_rows * 128;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const uint32_t slot = cnt % C::kSlots, ph = (cnt / C::kSlots) & 1;
          ok = warp_all(wait_bounded(&bar_empty[slot], ph ^ 1, cta_abort, p.status, limit, 34 + kv));
          if (!ok) break;
          if (lane == 0) {
            if (kv == 0) {  // bit i: positions 16 i .. 16 i + 15 of the tile have no page
              uint32_t m = 0;
              for (int i = 0; missing != 0 && i < 8; ++i) m |= ((missing >> ((i << boxes_log) >> 3)) & 1u) << i;
              sh.holes[step % kHoles] = m;
            }
            mbar_arrive_expect_tx(&bar_full[slot], kv == 0 ? C::kKTileBytes : C::kVTileBytes);
          }
          __syncwarp();
          if (chunk < (kv == 0 ? C::kQChunks : C::kVChunks))
            tma_load_4d(sSlot + C::slot_offset(slot) + at, kv == 0 ? &tm_k : &tm_v, &bar_full[slot], 64 * chunk, in_page,
                        pc.kvh, pg);
          ++cnt;
        }
        // the first keys need not wait for the previous piece's rows to be done with
        if (ok && !rows_first && j == pc.j0) ok = load_rows();
      }
      // The pair that begins here and goes on in other shares (looked up after the loads, which should not wait for it).
      if (lane == 0 && k >= 0 && pc.slot == 2 * static_cast<int32_t>(now.share) + 1) {
        const int n = static_cast<int>(last_share<kPieceSteps>(sh.lists, shares, cut, now.pair, now.seq) - now.share) + 1;
        p.pairs[now.share] = KvPair{pc.row0, pc.tokens, pc.head0, pc.heads, pc.slot, n, {0, 0}};
      }
      now = then;
    }
    if (!over && fresh) w = __shfl_sync(0xffffffffu, next, 0);  // (given up before)
    if (lane == 0) {
      release_pieces(p.tile_counter, total, w);
      if (!ok) {
        // let the loads already issued land before the CTA gives up its shared memory
        if (wt > 0) wait_final(bar_q, (wt - 1) & 1, limit);
        for (uint32_t i = 0; i < C::kSlots && i < cnt; ++i) {
          const uint32_t last = i + ((cnt - 1 - i) / C::kSlots) * C::kSlots;
          wait_final(&bar_full[i], (last / C::kSlots) & 1, limit);
        }
      }
    }
  } else if (warp >= C::kMmaWarp) {
    // ================================================================ MMA issuers, one for each Q tile
    // Per step j issuer t issues S_t(j) = Q_t K(j)^T and then, with P in columns of its own, O_t += P_t(j-1) V(j-1); with
    // P over S_t, O_t += P_t(j) V(j) once softmax t has written P_t(j).  Every issuer commits once per K and V tile and per
    // piece, whether or not its Q tile has rows.
    if (lane == 0) {
      const int t = warp - C::kMmaWarp;
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, DV, 0, 1);
      constexpr uint32_t kDescHi = smem_desc_hi(1024, kSwizzle128B);
      const uint32_t qlo = smem_desc_lo(smem_u32(sQ + t * C::kQTileBytes), 16);
      const uint32_t d_s = tmem + t * kBlockN, d_o = tmem + C::kColO + t * DV, a_p = tmem + C::col_p(t);
      uint32_t cnt = 0;
      int n = 0;    // S MMAs issued for this Q tile
      int pvw = 0;  // pieces whose first PV into O_t has been issued
      int wt = 0;   // Q tiles waited for
      bool pend = false, pend_first = false;  // the previous step's PV is due
      uint32_t pend_vslot = 0, pend_vph = 0;

      auto issue_qk = [&](uint32_t kslot) {
        const uint32_t klo = smem_desc_lo(smem_u32(sSlot + C::slot_offset(kslot)), 16);
#pragma unroll
        for (int kk = 0; kk < DQK / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
          mma_ss_lh(d_s, qlo + off, kDescHi, klo + off, kDescHi, idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit(&bar_s[t]);
      };
      // The first PV of a piece overwrites O_t: it waits until the epilogue of the one before has read it.
      auto issue_pv = [&](uint32_t vslot, bool first) -> bool {
        if (first) {
          if (pvw > 0) {
            if (!wait_bounded(&bar_ofree[t], (pvw - 1) & 1, cta_abort, p.status, limit, 36)) return false;
            tc_fence_after_sync();
          }
          ++pvw;
        }
        const uint32_t vlo = smem_desc_lo(smem_u32(sSlot + C::slot_offset(vslot)), kChunkBytes);
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk) {
          if (!C::kSepP && kk == 6) {  // the last quarter of P may still have been on its way
            if (!wait_bounded(&bar_p2[t], n & 1, cta_abort, p.status, limit, 50)) return false;
            tc_fence_after_sync();
          }
          mma_ts_lh(d_o, a_p + kk * 8, vlo + ((kk * 2048) >> 4), kDescHi, idesc_pv, (!first || kk > 0) ? 1u : 0u);
        }
        mma_commit(&bar_o[t]);
        return true;
      };
      // The pending step's PV, and its V slot's release.  (An issuer waits for every fill it releases, used or not, so
      // that it never commits for a later fill of a slot before the other issuer has released the earlier one.)
      auto flush = [&](bool part) -> bool {
        if (!pend) return true;
        if (!wait_bounded(&bar_full[pend_vslot], pend_vph, cta_abort, p.status, limit, 37)) return false;
        if (part) {
          if (!wait_bounded(&bar_p[t], (n - 1) & 1, cta_abort, p.status, limit, 38)) return false;
          tc_fence_after_sync();
          if (!issue_pv(pend_vslot, pend_first)) return false;
        }
        mma_commit(&bar_empty[pend_vslot]);
        pend = false;
        return true;
      };

      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!take_piece(k)) break;
        const volatile Piece& pc = sh.piece[k & 1];
        const int tokens = pc.tokens, j0 = pc.j0, j1 = pc.j1, len = pc.len;
        mbar_arrive(&bar_wfree[k & 1]);
        if (tokens < 0) break;
        if (j1 <= j0) continue;
        const bool part = t == 0 || tokens > p.tile.tokens;
        if (!wait_bounded(bar_q, wt & 1, cta_abort, p.status, limit, 39)) break;
        ++wt;
        tc_fence_after_sync();
        bool first = true, keys_there = false;
        for (int j = j0; ok && j < j1; ++j) {
          const uint32_t kslot = cnt % C::kSlots, kph = (cnt / C::kSlots) & 1;
          const uint32_t vslot = (cnt + 1) % C::kSlots, vph = ((cnt + 1) / C::kSlots) & 1;
          cnt += 2;
          if (!keys_there) ok = wait_bounded(&bar_full[kslot], kph, cta_abort, p.status, limit, 40);
          keys_there = false;
          if (!ok) break;
          // With S_t the softmax clears the end of this step's V slot, and has to find the slot's previous fill gone:
          // of two slots, that is the V whose PV is pending.
          if (C::kSepP && C::kSlots == 2 && (j + 1) * kBlockN > len) ok = flush(part);
          if (ok && part) {
            // S_t is free once softmax t has loaded it into registers, or, with P over it, once the PV has read P
            if (n > 0) ok = wait_bounded(C::kSepP ? &bar_sfree[t] : &bar_o[t], (n - 1) & 1, cta_abort, p.status, limit, 41);
            if (ok) {
              tc_fence_after_sync();
              issue_qk(kslot);
            }
          }
          if (!ok) break;
          mma_commit(&bar_empty[kslot]);
          if (C::kSepP) {
            ok = flush(part);
            if (!ok) break;
            pend = true;
            pend_first = first;
            pend_vslot = vslot;
            pend_vph = vph;
            if (part) ++n;
          } else {
            ok = wait_bounded(&bar_full[vslot], vph, cta_abort, p.status, limit, 42);
            // (looked at here, where the issuer waits anyway, the next keys need no look between the products)
            if (ok && part && j + 1 < j1) keys_there = mbar_try_wait(&bar_full[cnt % C::kSlots], (cnt / C::kSlots) & 1);
            if (ok && part) {
              ok = wait_bounded(&bar_p[t], n & 1, cta_abort, p.status, limit, 43);
              if (ok) {
                tc_fence_after_sync();
                ok = issue_pv(vslot, first);
              }
              ++n;
            }
            if (!ok) break;
            mma_commit(&bar_empty[vslot]);
          }
          first = false;
        }
        mma_commit(bar_qempty);  // this issuer's S MMAs of the piece are issued
        if (ok && C::kSepP) ok = flush(part);  // the last PV goes out now: the epilogue waits for it
      }
      // every MMA of this issuer, and the arrivals that its commits make, completes before the CTA leaves
      mma_commit(&bar_drain[t]);
      wait_final(&bar_drain[t], 0, limit);
    }
  } else {
    // ================================================================ softmax and epilogue, a row to a thread
    const int t = QT == 2 ? warp >> 2 : 0;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * kBlockN;
    const uint32_t tP = tmem + lane_base + C::col_p(t);
    const uint32_t tO = tmem + lane_base + C::kColO + t * DV;
    const float sl2 = p.scale_log2;
    // Turn k of tile 0 waits for tile 1's turn k - 1, turn k of tile 1 for tile 0's turn k; both take one turn a step of
    // the pieces that have rows in both tiles.
    int turn = 0;
    auto take_turn = [&]() -> bool {
      if (t == 0 && turn == 0) return true;
      const uint32_t par = static_cast<uint32_t>(t == 0 ? turn - 1 : turn) & 1u;
      return warp_all(wait_bounded(&bar_turn[t * 4 + wq], par, cta_abort, p.status, limit, 44));
    };
    auto pass_turn = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_turn[(t ^ 1) * 4 + wq]);
      ++turn;
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int n = 0;      // steps of this Q tile
    int skipped = 0;  // steps of the CTA that this Q tile had no rows in
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!warp_all(take_piece(k))) break;
      // The piece's fields are read again where they are needed, rather than kept in registers across the steps, which
      // need every one of them.
      const volatile Piece& pc = sh.piece[k & 1];
      int j = pc.j0;
      bool idle, turns;
      {
        const int tokens = pc.tokens, rows_t = min(tokens - t * p.tile.tokens, p.tile.tokens);  // of this Q tile
        if (tokens < 0) break;
        if (QT == 2 && rows_t <= 0) {
          skipped += pc.j1 - j;
          arrive(&bar_wfree[k & 1]);
          continue;
        }
        turns = C::kTurns && tokens > p.tile.tokens;
        idle = (wq * 32) / p.tile.heads >= rows_t;  // none of the warp's rows exists
      }
      float m_used = -INFINITY;  // running maximum, log2 units
      float l = 0.f;             // running sum of exp2(s * sl2 - m_used)
      for (; ok && j < pc.j1; ++j, ++n) {
        const bool inside = j >= pc.flo[t] && j < pc.fhi[t];
        ok = warp_all(wait_bounded(&bar_s[t], n & 1, cta_abort, p.status, limit, 45));
        if (!ok) break;
        if (!inside && (j + 1) * kBlockN > pc.len) {
          // The sequence ends inside this tile.  The V rows behind it have a weight of 0, but 0 times a NaN there would
          // still be NaN: clear them before this Q tile's PV may read them.  S_t is there, so the issuer has waited for
          // every earlier fill of the slot, and the parity can only mean this one.
          const uint32_t vcnt = 2 * static_cast<uint32_t>(n + skipped) + 1, vslot = vcnt % C::kSlots;
          ok = warp_all(wait_bounded(&bar_full[vslot], (vcnt / C::kSlots) & 1, cta_abort, p.status, limit, 46));
          if (!ok) break;
          uint8_t* const sv0 = sSlot + C::slot_offset(vslot);
          for (int c = 0; c < C::kVChunks; ++c)
            for (int off = (pc.len - j * kBlockN) * 128 + row * 16; off < static_cast<int>(kChunkBytes); off += 128 * 16)
              *reinterpret_cast<uint4*>(sv0 + c * kChunkBytes + off) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_shared();
        }
        if (idle) {
          if (C::kSepP) {
            arrive(&bar_sfree[t]);
            // not before the others can be done with the step before
            if (n > 0) ok = warp_all(wait_bounded(&bar_o[t], (n - 1) & 1, cta_abort, p.status, limit, 47));
          }
          if (ok && turns) {
            ok = take_turn();
            if (ok) pass_turn();
          }
          if (!ok) break;
          arrive(&bar_p[t]);
          if (!C::kSepP) arrive(&bar_p2[t]);
          continue;
        }
        const uint32_t holes = *const_cast<volatile uint32_t*>(&sh.holes[static_cast<uint32_t>(n + skipped) % kHoles]);
        tc_fence_after_sync();
        uint32_t r0[32], r1[32], r2[32], r3[32];
        float q0 = tmem_ld32_max(tS + 0, r0);
        float q1 = tmem_ld32_max(tS + 32, r1);
        float q2 = tmem_ld32_max(tS + 64, r2);
        float q3 = tmem_ld32_max(tS + 96, r3);
        tmem_ld_wait();
        reg_fence(r0);
        reg_fence(r1);
        reg_fence(r2);
        reg_fence(r3);
        reg_fence(q0);
        reg_fence(q1);
        reg_fence(q2);
        reg_fence(q3);
        float qm[4] = {q0, q1, q2, q3};
        if (!inside || holes != 0) {
          // The row's visible columns are one interval, less the missing pages.  A quarter of 32 columns that every row
          // of the warp sees keeps its maximum and its scores.
          const int kpos = j * kBlockN;
          const int q_pos = pc.pos0 + t * p.tile.tokens + (sh.rows[row] >> 8);
          const int lo = p.window > 0 ? q_pos - kpos - p.window + 1 : 0;
          const int hi = min(pc.len - kpos - 1, q_pos - kpos);
          auto mask = [&](uint32_t(&r)[32], float& most, int first) {
            const int a = lo - first, b = hi - first;
            const uint32_t gone = (holes >> (first / 16)) & 3u;
            if (!__any_sync(0xffffffffu, a > 0 || b < 31 || gone != 0)) return;
            // (a branch of its own for a quarter that nobody sees made ptxas spill 1.7 KB)
            // visible: a <= c <= b
            const int from = max(a, 0);
            const uint32_t span = static_cast<uint32_t>(max(-1, min(b, 31) - from) + 1);  // columns
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (static_cast<uint32_t>(c - from) >= span || ((gone >> (c / 16)) & 1u)) r[c] = 0xff800000u;  // -inf
            float x = fmax3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]));
            float y = fmax3(__uint_as_float(r[3]), __uint_as_float(r[4]), __uint_as_float(r[5]));
#pragma unroll
            for (int c = 6; c < 30; c += 4) {
              x = fmax3(x, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
              y = fmax3(y, __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
            }
            most = fmax3(x, y, fmaxf(__uint_as_float(r[30]), __uint_as_float(r[31])));
          };
          mask(r0, qm[0], 0);
          mask(r1, qm[1], 32);
          mask(r2, qm[2], 64);
          mask(r3, qm[3], 96);
        }
        const float mx = fmax3(qm[0], qm[1], fmaxf(qm[2], qm[3]));
        float sv[128];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          sv[i] = __uint_as_float(r0[i]);
          sv[32 + i] = __uint_as_float(r1[i]);
          sv[64 + i] = __uint_as_float(r2[i]);
          sv[96 + i] = __uint_as_float(r3[i]);
        }
        const float m_new = mx * sl2;
        const bool need = m_new > m_used + kRescaleThreshold;
        const float alpha = need ? ex2_approx(m_used - m_new) : 1.f;
        m_used = need ? m_new : m_used;
        l *= alpha;
        const float msub = (m_used == -INFINITY) ? 0.f : m_used;
        // O_t holds the previous PV's result: with P in columns of its own once the wait for them is over, with P over S
        // because the issuer waited for that PV before it sent S_t.
        auto rescale = [&]() {
          if (!__any_sync(0xffffffffu, need) || j <= pc.j0) return;
#pragma unroll 1
          for (int c = 0; c < DV / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + c * 16, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tO + c * 16, o);
          }
        };
        if (!C::kSepP) rescale();
        if (turns) {
          ok = take_turn();
          if (!ok) break;
        }
        // p = exp2(s * sl2 - m), packed to bf16 pairs; the row's sum in fp32 before that rounding
        const uint64_t sl2v = pack_f32x2(sl2, sl2), negm = pack_f32x2(-msub, -msub);
        uint64_t acc[4] = {0, 0, 0, 0};
        uint32_t pk[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          pk[i] = softmax_pair(sv[2 * i], sv[2 * i + 1], sl2v, negm, acc[i & 3]);
          if (C::kSepP && i == 15) {  // S_t is in registers: the next S MMA may overwrite it
            tc_fence_before_sync();
            arrive(&bar_sfree[t]);
          }
          if (!C::kSepP && i == 55) {  // three quarters of P are there: the PV may begin
            tmem_st_wait();
            tc_fence_before_sync();
            arrive(&bar_p[t]);
          }
          if ((i & 15) == 15) {
            const int c = i >> 4;
            if constexpr (!C::kSepP) {
              tmem_st16(tP + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[16 * c]));
            } else if (c == 2) {
              if (n > 0) {  // the previous PV has read P
                ok = warp_all(wait_bounded(&bar_o[t], (n - 1) & 1, cta_abort, p.status, limit, 48));
                if (!ok) break;
                tc_fence_after_sync();
              }
#pragma unroll
              for (int cc = 0; cc < 3; ++cc)
                tmem_st16(tP + cc * 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[16 * cc]));
            } else if (c == 3) {
              tmem_st16(tP + 48, *reinterpret_cast<const uint32_t(*)[16]>(&pk[48]));
            }
          }
        }
        if (!ok) break;
        const float2 c0 = unpack_f32x2(acc[0]), c1 = unpack_f32x2(acc[1]);
        const float2 c2 = unpack_f32x2(acc[2]), c3 = unpack_f32x2(acc[3]);
        l += ((c0.x + c0.y) + (c1.x + c1.y)) + ((c2.x + c2.y) + (c3.x + c3.y));
        if (turns) pass_turn();
        if (C::kSepP) rescale();
        tmem_st_wait();
        tc_fence_before_sync();
        arrive(C::kSepP ? &bar_p[t] : &bar_p2[t]);
      }
      if (!ok) break;

      // ---- epilogue
      const bool steps = pc.j1 > pc.j0;
      const int slot = pc.slot, head0 = pc.head0;
      const int my_token = sh.rows[row] >> 8, my_head = sh.rows[row] & 255;
      const bool valid_row = my_token < min(pc.tokens - t * p.tile.tokens, p.tile.tokens) && my_head < pc.heads;
      const int64_t tok = static_cast<int64_t>(pc.row0) + t * p.tile.tokens + my_token;
      arrive(&bar_wfree[k & 1]);
      if (steps) {
        ok = warp_all(wait_bounded(&bar_o[t], (n - 1) & 1, cta_abort, p.status, limit, 49));
        if (!ok) break;
        tc_fence_after_sync();
      }
      // (a row that saw nothing gives 0 whatever O holds, and a sum that is NaN gives NaN)
      const float inv = slot >= 0 || l == 0.f ? 1.f : 1.f / l;
      const uint32_t keep = l == 0.f ? 0u : ~0u;
      const uint64_t inv2 = pack_f32x2(inv, inv);
      const int64_t at = tok * p.out_srow + static_cast<int64_t>(head0 + my_head) * p.out_shead;
      const int64_t prow = static_cast<int64_t>(slot) * p.rows_cap + t * p.tile.tokens * p.tile.heads + row;
      if (valid_row) {
        if (slot >= 0)
          p.ml[prow] = make_float2(m_used, l);
        else if (p.lse != nullptr)
          p.lse[tok * p.lse_srow + static_cast<int64_t>(head0 + my_head) * p.lse_shead] =
              l > 0.f ? (m_used + lg2_approx(l)) * kLn2 : l == 0.f ? -INFINITY : l;
      }
#pragma unroll 1
      for (int c = 0; c < DV / 32; ++c) {
        // (not left undefined: the compiler kept room for it through the steps, and spilled 160 bytes there)
        uint32_t o[32] = {};
        if (steps && !idle) {
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait();
          reg_fence(o);
        }
        if (c == DV / 32 - 1 && steps) {  // O_t is read
          tc_fence_before_sync();
          arrive(&bar_ofree[t]);
        }
        if (!valid_row) continue;
        float f[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = unpack_f32x2(mul_f32x2(
              pack_f32x2(__uint_as_float(o[2 * i] & keep), __uint_as_float(o[2 * i + 1] & keep)), inv2));
          f[2 * i] = x.x, f[2 * i + 1] = x.y;
        }
        if (slot >= 0) {
          float4* const dst = reinterpret_cast<float4*>(p.part + prow * DV + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else if (p.out_bf16) {
          uint4* const dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at + c * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7]));
        } else {
          float4* const dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the pieces of the pairs that were cut, in their order.  A lane has four channels of a row.  Few pieces (many rows:
// a chunk's pairs): every thread has a row's channels of its own and all of its pieces in flight.  More (few rows: a
// decode step): the CTA's four groups of 128 threads take every fourth piece, four in flight, and join at the end.
// (32 heads of 192/128, 4 chunks of 777: 15 us for 28 MB from HBM and more from L2.  A CTA for each part of a share, most of
// them without work, cost 2 us a thousand.)
template <int DV>
__global__ void __launch_bounds__(kJoinThreads, 2) kv_attn_join_kernel(const __grid_constant__ KvAttnParams p) {
  constexpr int kGroups = kJoinThreads / 128, kAhead = 4;
  __shared__ float s_m[kGroups][128], s_l[kGroups][128];
  __shared__ float4 s_v[kGroups][128];
  __shared__ KvPair s_pairs[2 * kKvMaxSms];
  __shared__ int16_t s_list[2 * kKvMaxSms];
  __shared__ int s_count[kJoinThreads / 32];
  const int chunks = (p.rows_cap * (DV / 4) + kJoinThreads - 1) / kJoinThreads;
  const int grp = threadIdx.x >> 7, lane = threadIdx.x & 127;
  pdl_wait();
  // (the first record is read along with what says whether it counts)
  KvPair e = p.pairs[min(static_cast<int>(blockIdx.x), p.max_slots / 2 - 1)];
  const int shares = min(*p.n_pairs, p.max_slots / 2);
  if (*reinterpret_cast<volatile int*>(p.status) != 0) return;  // pieces may be missing
  int n = shares;  // of the list
  if (chunks > 1) {
    // the shares in which a pair begins that goes on in others
    static_assert(2 * kKvMaxSms <= kJoinThreads, "a share to a thread");
    const int t = threadIdx.x, w = t >> 5;
    KvPair r{};
    if (t < shares) r = p.pairs[t];
    const bool mine = r.pieces > 0;
    const uint32_t some = __ballot_sync(0xffffffffu, mine);
    if ((t & 31) == 0) s_count[w] = __popc(some);
    __syncthreads();
    int at = 0;
    n = 0;
    for (int i = 0; i < kJoinThreads / 32; ++i) {
      if (i == w) at = n;
      n += s_count[i];
    }
    if (mine) {
      at += __popc(some & ((1u << (t & 31)) - 1u));
      s_list[at] = static_cast<int16_t>(t);
      s_pairs[at] = r;
    }
    __syncthreads();
  }
  for (int item = blockIdx.x; item < n * chunks; item += gridDim.x) {
    int share = item, chunk = 0;
    if (chunks > 1) {
      const int i = item / chunks;
      share = s_list[i], chunk = item - i * chunks;
      e = s_pairs[i];
    } else if (item != static_cast<int>(blockIdx.x)) {
      e = p.pairs[share];
    }
    const int rows = e.tokens * p.tile.heads;
    if (e.pieces <= 0 || e.slot != 2 * share + 1 || 2 * (share + e.pieces) > p.max_slots || e.row0 < 0 ||
        e.row0 + e.tokens > p.seqs.T || rows > p.rows_cap)
      continue;
    auto slot_of = [&](int c) { return c == 0 ? e.slot : 2 * (share + c); };
    float mm = -INFINITY, ll = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    // a piece whose row saw nothing has m = -inf and l = 0, and a NaN anywhere stays one
    auto add = [&](float m, float l, float4 v, float to) {
      const float f = m == -INFINITY ? 0.f : ex2_approx(m - to);
      ll = fmaf(f, l, ll);
      sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
    };
    auto move = [&](float to) {
      const float alpha = mm == -INFINITY ? 1.f : ex2_approx(mm - to);
      mm = to;
      ll *= alpha;
      sum.x *= alpha, sum.y *= alpha, sum.z *= alpha, sum.w *= alpha;
    };
    // pieces c0, c0 + stride, ... of row rr
    auto gather = [&](int rr, int ch, int c0, int stride) {
      for (; c0 < e.pieces; c0 += kAhead * stride) {
        float2 ml[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int64_t prow = static_cast<int64_t>(slot_of(c0 + k * stride)) * p.rows_cap + rr;
          ml[k] = make_float2(-INFINITY, 0.f), v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c0 + k * stride >= e.pieces) continue;
          ml[k] = p.ml[prow];
          v[k] = *reinterpret_cast<const float4*>(p.part + prow * DV + ch);
        }
        float now = mm;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) now = fmaxf(now, ml[k].x);
        move(now);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (c0 + k * stride < e.pieces) add(ml[k].x, ml[k].y, v[k], now);
      }
    };
    auto store = [&](int rr, int ch) {
      const int token = rr / p.tile.heads, head = rr - token * p.tile.heads;
      if (head >= e.heads) return;
      const int64_t tok = static_cast<int64_t>(e.row0) + token, h = e.head0 + head;
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      const int64_t at = tok * p.out_srow + h * p.out_shead + ch;
      if (p.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
            make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
            make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
      if (ch == 0 && p.lse != nullptr)
        p.lse[tok * p.lse_srow + h * p.lse_shead] = ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * kLn2;
    };
    if (e.pieces <= kAhead) {
      const int i = chunk * kJoinThreads + threadIdx.x, rr = i / (DV / 4), ch = (i % (DV / 4)) * 4;
      if (rr < rows) {
        gather(rr, ch, 0, 1);
        store(rr, ch);
      }
      continue;
    }
    for (int c = 0; c < kJoinThreads / 128; ++c) {
      const int i0 = chunk * kJoinThreads + c * 128, i = i0 + lane;
      if (i0 / (DV / 4) >= rows) break;  // the same for every thread
      const int rr = min(i / (DV / 4), rows - 1), ch = (i % (DV / 4)) * 4;
      mm = -INFINITY, ll = 0.f;
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
      gather(rr, ch, grp, kGroups);
      __syncthreads();
      s_m[grp][lane] = mm, s_l[grp][lane] = ll, s_v[grp][lane] = sum;
      __syncthreads();
      if (grp != 0) continue;
      float now = mm;
#pragma unroll
      for (int g = 1; g < kGroups; ++g) now = fmaxf(now, s_m[g][lane]);
      move(now);
#pragma unroll
      for (int g = 1; g < kGroups; ++g) add(s_m[g][lane], s_l[g][lane], s_v[g][lane], now);
      if (i / (DV / 4) < rows) store(rr, ch);
    }
  }
}

// ---------------------------------------------------------------- launches

// CTAs of a grid that fills a device of so many SMs.
int grid_of(int dqk, int dv, int sms) { return sms * (dqk == 64 && dv == 64 ? 2 : 1); }

struct Workspace {
  int64_t rows_cap, max_slots;
  size_t pairs, ml, part, total;  // offsets
};
Workspace workspace_of(int64_t T, int64_t group, int dqk, int dv, int32_t q_len) {
  const RowTile tile = row_tile(group);
  const int64_t tiles = dqk == 64 && dv == 64 ? 1 : 2;
  const int64_t most = std::max<int64_t>(1, q_len > 0 ? q_len : T);  // new tokens of a sequence
  Workspace w;
  w.rows_cap = std::min<int64_t>(tiles * tile.tokens, most) * tile.heads;
  w.max_slots = 2 * grid_of(dqk, dv, kKvMaxSms);  // a share has two pieces that are joined at most
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.pairs = 256;
  w.ml = w.pairs + up(w.max_slots * sizeof(KvPair));
  w.part = w.ml + up(w.max_slots * w.rows_cap * sizeof(float2));
  w.total = w.part + up(w.max_slots * w.rows_cap * dv * sizeof(float));
  return w;
}

template <int DQK, int DV, int QT>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, KvAttnParams p, int grid,
                   cudaStream_t stream) {
  using C = Cfg<DQK, DV, QT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];  // the kernel's attributes are set on the device
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_attn_kernel<DQK, DV, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv_attn_kernel<DQK, DV, QT>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  if ((e = claim_cache_counter(stream, &p.tile_counter)) != cudaSuccess) return e;
  e = launch_early(kv_attn_kernel<DQK, DV, QT>, dim3(static_cast<unsigned>(grid)), C::kThreads, C::kSmemBytes, stream, tq, tk,
                   tv, p);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(grid * ((p.rows_cap * (DV / 4) + kJoinThreads - 1) / kJoinThreads), 2 * kv_sm_count());
  return launch_early(kv_attn_join_kernel<DV>, dim3(static_cast<unsigned>(ctas)), kJoinThreads, 0, stream, p);
}

// `few`: the sequences have no more new tokens than a Q tile, on average.  Then wide heads too take one Q tile to a CTA,
// and the room of the second one for keys and values (4 sequences of 8192 tokens, 32 heads of 192/128 with a query head
// each, one new token: 159 -> 132 us; 8 of 16384, 32/8 heads of 128: 113 -> 95 us).
cudaError_t launch_kv_attn(int dqk, int dv, bool few, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const KvAttnParams& p, int grid, cudaStream_t stream) {
  if (dqk == 64 && dv == 64) return launch<64, 64, 1>(tq, tk, tv, p, grid, stream);
  if (few) {
    if (dqk == 64 && dv == 128) return launch<64, 128, 1>(tq, tk, tv, p, grid, stream);
    if (dqk == 128 && dv == 64) return launch<128, 64, 1>(tq, tk, tv, p, grid, stream);
    if (dqk == 128 && dv == 128) return launch<128, 128, 1>(tq, tk, tv, p, grid, stream);
    if (dqk == 192 && dv == 64) return launch<192, 64, 1>(tq, tk, tv, p, grid, stream);
    if (dqk == 192 && dv == 128) return launch<192, 128, 1>(tq, tk, tv, p, grid, stream);
  }
  if (dqk == 64 && dv == 128) return launch<64, 128, 2>(tq, tk, tv, p, grid, stream);
  if (dqk == 128 && dv == 64) return launch<128, 64, 2>(tq, tk, tv, p, grid, stream);
  if (dqk == 128 && dv == 128) return launch<128, 128, 2>(tq, tk, tv, p, grid, stream);
  if (dqk == 192 && dv == 64) return launch<192, 64, 2>(tq, tk, tv, p, grid, stream);
  if (dqk == 192 && dv == 128) return launch<192, 128, 2>(tq, tk, tv, p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace slope

using namespace slope;

extern "C" {

size_t slope_kv_attn_workspace_size(int64_t T, int64_t Hq, const slope_kv_cache* cache, int32_t q_len) {
  if (cache == nullptr || !attn_partial_supported(cache->dqk, cache->dv)) return 0;
  if (T < 0 || T >= kKvMaxTokens || cache->Hkv < 1 || Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0 || q_len < 0) return 0;
  return workspace_of(T, Hq / cache->Hkv, cache->dqk, cache->dv, q_len).total;
}

slope_status slope_kv_attn(const slope_tensor* q, const slope_kv_cache* cache, const slope_kv_batch* batch,
                           int64_t window, float scale, slope_tensor* out, slope_tensor* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const CallRange range("slope_kv_attn");
  slope_status st;
  if ((st = check_kv_cache(cache)) != SLOPE_OK || (st = check_kv_q(q, cache)) != SLOPE_OK) return st;
  const int64_t T = q->shape[0], Hq = q->shape[1];
  if (window < 0 || window > (int64_t(1) << 30)) return SLOPE_ERR_SHAPE;
  if ((st = check_kv_batch(batch, cache, T)) != SLOPE_OK) return st;
  if ((st = check_out(out, T, Hq, cache->dv, true)) != SLOPE_OK) return st;
  if (lse != nullptr && (st = check_lse(lse, Hq, T)) != SLOPE_OK) return st;
  if (T == 0 || batch->B == 0) return SLOPE_OK;
  const int64_t vec = out->dtype == SLOPE_BF16 ? 8 : 4;
  if (out->stride[0] % vec || out->stride[1] % vec || !aligned(out->data, 16)) return SLOPE_ERR_STRIDE;

  KvAttnParams p{};
  p.Hkv = cache->Hkv;
  p.group = static_cast<int32_t>(Hq / cache->Hkv);
  p.tile = row_tile(p.group);
  // pairs of a launch are counted in 32 bits, with room for the pieces
  const int64_t pairs = (T / p.tile.tokens + kKvMaxSeqs) * p.Hkv * p.tile.parts;
  if (pairs >= (int64_t(1) << 29)) return SLOPE_ERR_UNSUPPORTED;
  const bool few = T <= batch->B * p.tile.tokens;
  const Workspace w = workspace_of(T, p.group, cache->dqk, cache->dv, batch->cu_q != nullptr ? 0 : batch->q_len);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return SLOPE_ERR_WORKSPACE;
  const int grid = grid_of(cache->dqk, cache->dv, kv_sm_count());
  if (grid <= 0) return cuda_fail("device attributes");
  p.seqs = kv_seqs(batch, cache, T);
  p.window = static_cast<int32_t>(window);
  p.scale_log2 = resolve_scale(scale, cache->dqk) * 1.44269504088896340736f;
  p.out = out->data;
  p.out_srow = out->stride[0];
  p.out_shead = out->stride[1];
  p.out_bf16 = out->dtype == SLOPE_BF16 ? 1 : 0;
  if (lse != nullptr) {
    p.lse = static_cast<float*>(lse->data);
    p.lse_srow = lse->stride[1];
    p.lse_shead = lse->stride[0];
  }
  char* const ws = static_cast<char*>(workspace);
  p.rows_cap = static_cast<int32_t>(w.rows_cap);
  p.max_slots = static_cast<int32_t>(w.max_slots);
  p.n_pairs = reinterpret_cast<int32_t*>(ws);
  p.pairs = reinterpret_cast<KvPair*>(ws + w.pairs);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.status = device_status_ptr();
  if (p.status == nullptr) return cuda_fail("device status word (cudaGetSymbolAddress)");
  p.wait_limit_ns = wait_limit_ns();
  CUtensorMap tq, tk, tv;
  if (!make_q_map(&tq, q, p.tile.heads, p.tile.tokens) || !make_page_map(&tk, cache->k, cache, cache->dqk, cache->k_stride) ||
      !make_page_map(&tv, cache->v, cache, cache->dv, cache->v_stride))
    return cuda_fail("cuTensorMapEncodeTiled");
  for (int64_t b = 0; b < batch->B; b += kKvMaxSeqs) {
    p.seqs.b0 = static_cast<int32_t>(b);
    p.seqs.B = static_cast<int32_t>(std::min<int64_t>(kKvMaxSeqs, batch->B - b));
    const cudaError_t e =
        launch_kv_attn(cache->dqk, cache->dv, few, tq, tk, tv, p, grid, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("cache attention kernel launch", e);
  }
  return SLOPE_OK;
}

}  // extern "C"
