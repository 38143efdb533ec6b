// The attention weight that each cached token got from the newest queries, summed over them and over the query heads of
// its key head:
//   w_j = sum_r 2^(scale log2(e) q_r . k_j - lse_r log2(e)) over the rows r = (token, head) that see j.
//
// The score products are computed transposed, S^T = K Q^T: a key is an accumulator row (one softmax thread) and the query
// rows are its columns, so a thread sums its own key's weights in registers and nothing is reduced across threads.  K stays
// in shared memory, 256 keys to a CTA (two M = 128 tiles, four TMEM accumulators of 128 columns so that the products
// of the next rows run under the exponentials of these), and the row tiles of 128 (token, head) pairs stream past:
// both key tiles use each, which halves what the rows cost to load.  Beside the exponential a weight takes half a
// packed multiply-add and half a packed add, and no maximum, no sum across lanes and no second product: the bound is the
// MUFU unit, at 4 cycles a warp's 32 exponentials (128 x 256 of them take 1024 cycles of an SM).
//
// The work: where the new rows fill many tiles, a pair is (sequence, KV head, 256 keys) and its steps the row tiles
// that see one of the keys; pairs of many rows and few keys are cut (kv_cut.cuh), and the pieces leave 256 sums each in the
// workspace, which a second launch adds in order.  Where the rows are few tiles (a decode step, the last queries of a prompt),
// a pair is (sequence, KV head) and its steps run along the blocks of 256 keys: the rows stay and the keys stream past, read
// once, and nothing is joined.
// Sixteen softmax warps: the four warps of (buffer, key tile) take every second row tile, or of few rows every second key
// block, so that each SM sub-partition has four warps with exponentials to issue.
//
// On one GB300, 64/8 heads of 64: every query of a 2K chunk at 16K 339 us, 70% of the MUFU unit's rate (eight softmax warps and one
// MMA issuer, which was the bound, 571); the last 64 queries of 32K 35.7 (38 before the keys' pieces were as short as gives
// no CTA two); a decode step of 16 x 8K 32 us and of 8 x 100K 147, 5.9 TB/s of keys (70 and 394 before the rows stayed), 36 and
// 162 where the sums are added to what is there.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kv_cut.cuh"
#include "sm103_ptx.cuh"
#include "waits.cuh"

namespace slope {
namespace {

constexpr uint32_t kChunkBytes = 128 * 128;  // 128 rows x 64 bf16
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kKeys = 2 * kBlockN;  // of a CTA's block
constexpr int kPieceSteps = 2;      // what a piece's start and end cost, in steps
constexpr int kFine = 4;            // (kv_cut.cuh: a piece leaves only 1 KB, so they may be short)
constexpr int kLseSlots = 8;
constexpr int kPieces = 4;          // pieces that the producer may be ahead

struct KvWeightsParams {
  KvSeqs seqs;
  int32_t Hkv, group;
  RowTile tile;
  int32_t window, accumulate;
  float scale_log2;
  const float* lse;
  int64_t lse_srow, lse_shead;
  float* weights;
  int64_t w_spage, w_shead;
  int32_t max_slots;
  int32_t* n_pairs;  // workspace: pairs that are joined
  int4* pairs;       // workspace: {sequence, KV head << 16 | pieces, key block, first piece}
  float* part;       // workspace: their sums
  int* status;
  uint32_t* tile_counter;
  uint64_t wait_limit_ns;
};

constexpr int kSoftmaxWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kLseWarp = 19;  // two MMA issuers
constexpr int kThreads = 32 * 20;                                                   // five warps to a sub-partition

// A piece: of a pair of many row tiles, those numbered [i0, i1) among the `count` of every part that see one of the block's
// keys; of few, key blocks [i0, i1), of which those from `seen` on are seen, and the `count` row tiles of every part.
struct Piece {
  int32_t b;  // sequence; -1: no pieces left
  int32_t few;
  int32_t kvh, key0, len;  // (key0: of the block)
  int32_t row0, n, pos0;   // of the sequence: first q row, new tokens, position of the first
  int32_t blk0, count;     // first row block, and how many
  int32_t i0, i1, seen;
  int32_t slot;
};

template <int DQK>
struct Cfg {
  static constexpr int kChunks = DQK / 64;
  static constexpr int kTileBytes = kChunks * kChunkBytes;             // 128 rows of K or Q
  static constexpr int kKSlots = DQK == 64 ? 8 : DQK == 128 ? 4 : 2;   // of 128 keys
  static constexpr int kQSlots = DQK == 64 ? 4 : 2;
  static constexpr int kFew = DQK == 64 ? 4 : DQK == 128 ? 2 : 1;     // row tiles that may stay
  static_assert(kFew <= kQSlots && (kFew == 1 || kKSlots >= 4), "they stay beside two key blocks");
  static constexpr int kQOffset = kKSlots * kTileBytes;
  static constexpr int kRestOffset = kQOffset + kQSlots * kTileBytes;
  struct Rest {  // behind the tiles
    float lse[kLseSlots][128];      // -lse log2(e) of a row tile's columns
    float few_lse[kPieces][kFew][128];  // of a piece's few row tiles
    float sums[kPieces][2][kBlockN];  // [piece][key tile]: what the second buffer's warps found
    int none[kLseSlots], few_none[kPieces][kFew];  // the tile has rows of -inf: the caller's, or heads past the group
    uint64_t kfull[kKSlots], kempty[kKSlots], qfull[kQSlots], qempty[kQSlots], lfull[kLseSlots], lempty[kLseSlots];
    uint64_t s[4], sfree[4];  // [2 * buffer + key tile]
    uint64_t wfull[kPieces], wfree[kPieces], few_full[kPieces], sums_full[kPieces][2], drain[2];
    Piece piece[kPieces];
    uint32_t tmem;
    int abort;
    CutLists lists;
  };
  static constexpr int kSmemBytes = kRestOffset + static_cast<int>(sizeof(Rest));
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// acc += {2^(s0 sl2 + n0), 2^(s1 sl2 + n1)}
__device__ __forceinline__ void exp_pair(uint32_t s0, uint32_t s1, uint64_t sl2, uint64_t n, uint64_t& acc) {
  asm("{\n\t.reg .b64 s, x;\n\t.reg .f32 x0, x1;\n\t"
      "mov.b64 s, {%1, %2};\n\t"
      "fma.rn.f32x2 x, s, %3, %4;\n\t"
      "mov.b64 {x0, x1}, x;\n\t"
      "ex2.approx.ftz.f32 x0, x0;\n\t"
      "ex2.approx.ftz.f32 x1, x1;\n\t"
      "mov.b64 x, {x0, x1};\n\t"
      "add.rn.f32x2 %0, %0, x;\n\t}"
      : "+l"(acc)
      : "r"(s0), "r"(s1), "l"(sl2), "l"(n));
}

// Key blocks of a sequence, and the row tiles that one of them meets at most (those of a group of more than 128 heads are
// its parts', one part after another); with few row tiles, one block for all keys.
struct KeyCut {
  RowTile tile;
  int few;
  bool accumulate;
  __device__ __forceinline__ int row_tiles(const KvSeq& s) const {
    return (s.n + tile.tokens - 1) / tile.tokens * tile.parts;
  }
  __device__ __forceinline__ SeqCut operator()(const KvSeq& s) const {
    const int rows = row_tiles(s), keys = (s.len + kKeys - 1) / kKeys;
    SeqCut c;
    c.join = rows > few;
    c.blocks = c.join ? keys : keys > 0 && !(rows == 0 && accumulate) ? 1 : 0;
    c.steps = c.join ? rows : keys * max(rows, 1);
    return c;
  }
};

__device__ __forceinline__ Piece make_piece(const KvWeightsParams& p, int per, const CutLists& lists, uint32_t w,
                                            const KeyCut& cut_of, int& join, int& pieces) {
  Piece r;
  const int b = seq_of(lists, p.seqs.B, w);
  const KvSeq q = lists.seqs[b];
  const SeqCut cut = cut_of(q);
  pieces = pieces_of(cut.steps, per);
  // local = (head * pieces + c) * blocks + block
  const uint32_t local = w - lists.units[b], rest = cut.blocks == 1 ? local : divide(local, cut.blocks);
  const int blk = static_cast<int>(local - rest * cut.blocks);
  r.kvh = static_cast<int>(pieces == 1 ? rest : divide(rest, pieces));
  const int c = static_cast<int>(rest) - r.kvh * pieces;
  join = -1;
  r.b = p.seqs.b0 + b;
  r.few = cut.join ? 0 : 1;
  r.len = q.len;
  r.row0 = q.row0;
  r.n = q.n;
  r.pos0 = q.len - q.n;
  r.slot = -1;
  r.seen = 0;
  if (r.few) {
    piece_steps((q.len + kKeys - 1) / kKeys, pieces, c, r.i0, r.i1);
    r.key0 = 0;
    r.blk0 = 0;
    r.count = (q.n + p.tile.tokens - 1) / p.tile.tokens;
    if (p.window > 0) r.seen = max(0, r.pos0 - p.window + 1) / kKeys;
    if (r.count == 0) r.seen = r.i1;
    return r;
  }
  r.key0 = blk * kKeys;
  // tokens [lo, hi) see one of the keys [key0, last]
  const int last = min(q.len, r.key0 + kKeys) - 1;
  const int lo = min(q.n, max(0, r.key0 - r.pos0));
  const int hi = p.window > 0 ? max(lo, min(q.n, last + p.window - r.pos0)) : q.n;
  r.blk0 = lo / p.tile.tokens;
  r.count = hi > lo ? (hi + p.tile.tokens - 1) / p.tile.tokens - r.blk0 : 0;
  piece_steps(r.count * p.tile.parts, pieces, c, r.i0, r.i1);
  if (pieces > 1) {
    const int pair = r.kvh * cut.blocks + blk;
    r.slot = static_cast<int32_t>(lists.slots[b]) + pair * pieces + c;
    if (c == 0) join = static_cast<int32_t>(lists.joins[b]) + pair;  // the first piece lists the pair
  }
  return r;
}

// Row tile i of a piece.
struct Rows {
  int token, tokens;  // first token among the sequence's new ones, and how many
  int head, heads;    // first head in the group, and how many
};
__device__ __forceinline__ Rows rows_of(const KvWeightsParams& p, int i, const Piece& pc) {
  Rows r;
  const int part = p.tile.parts > 1 ? i / pc.count : 0;
  r.token = (pc.blk0 + i - part * pc.count) * p.tile.tokens;
  r.tokens = min(p.tile.tokens, pc.n - r.token);
  r.head = part * p.tile.heads;
  r.heads = min(p.tile.heads, p.group - r.head);
  return r;
}

template <int DQK>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ KvWeightsParams p) {
  using C = Cfg<DQK>;
  extern __shared__ __align__(1024) uint8_t smem[];  // all of the shared memory: it starts on a tile's boundary
  uint8_t* const sK = smem;
  uint8_t* const sQ = smem + C::kQOffset;
  typename C::Rest& sh = *reinterpret_cast<typename C::Rest*>(smem + C::kRestOffset);
  volatile int* const cta_abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  const KeyCut cut_of{p.tile, C::kFew, p.accumulate != 0};

  pdl_launch_dependents();
  if (threadIdx.x == kTmaWarp * 32) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == kMmaWarp * 32) {
    for (int i = 0; i < C::kKSlots; ++i) mbar_init(&sh.kfull[i], 1), mbar_init(&sh.kempty[i], 1);
    for (int i = 0; i < C::kQSlots; ++i) mbar_init(&sh.qfull[i], 1), mbar_init(&sh.qempty[i], 2);
    for (int i = 0; i < kLseSlots; ++i) mbar_init(&sh.lfull[i], 1), mbar_init(&sh.lempty[i], kSoftmaxWarps / 2);
    for (int i = 0; i < 4; ++i) mbar_init(&sh.s[i], 1), mbar_init(&sh.sfree[i], 4);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&sh.wfull[i], 1);
      mbar_init(&sh.wfree[i], 3 + kSoftmaxWarps);
      mbar_init(&sh.few_full[i], 1);
      for (int t = 0; t < 2; ++t) mbar_init(&sh.sums_full[i][t], 4);
    }
    for (int t = 0; t < 2; ++t) mbar_init(&sh.drain[t], 1);
    fence_barrier_init();
  }
  // The rows of a Q slot that no box fills stay 0, and their scores too.
  for (int i = threadIdx.x; i < C::kQSlots * C::kChunks * 128 * 8; i += kThreads)
    if (((i >> 3) & 127) >= p.tile.heads * p.tile.tokens) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  pdl_wait();  // the kernels before this one are done; nothing above touches memory
  uint32_t claimed = 0;
  if (threadIdx.x == kTmaWarp * 32) claimed = atomicAdd(p.tile_counter, 1u);
  if (threadIdx.x == 0) *cta_abort = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
    return wait_bounded(bar, parity & 1, cta_abort, p.status, limit, site);
  };
  auto take_piece = [&](int k) -> bool { return wait(&sh.wfull[k % kPieces], k / kPieces, 61); };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == kTmaWarp) {
    // ================================================================ producer: pieces, pages, loads
    const Cut cut = make_cut<kPieceSteps, kFine>(p.seqs, p.Hkv, cut_of, sh.lists);
    if (lane == 0 && blockIdx.x == 0) *p.n_pairs = static_cast<int32_t>(cut.joins);
    const uint32_t total = cut.total;
    const uint32_t q_bytes = static_cast<uint32_t>(p.tile.heads * p.tile.tokens) * 128 * C::kChunks;
    const int shift = p.seqs.page_shift;
    const int boxes_log = max(0, 7 - shift);  // log2 of the boxes of 64 channels of 128 keys
    const int boxes = 1 << boxes_log, box_rows = kBlockN >> boxes_log;
    const int no_page = static_cast<int>(p.seqs.n_pages);  // reads 0
    uint32_t w = __shfl_sync(0xffffffffu, claimed, 0);
    int kcnt = 0, qcnt = 0;  // key tiles and row tiles loaded
    bool ok = *cta_abort == 0;
    for (int k = 0; ok; ++k) {
      if (k >= kPieces) ok = warp_all(wait(&sh.wfree[k % kPieces], k / kPieces - 1, 62));
      if (!ok) break;
      if (w >= total) {
        if (lane == 0) {
          sh.piece[k % kPieces].b = -1;
          mbar_arrive(&sh.wfull[k % kPieces]);
        }
        break;
      }
      uint32_t next = 0;
      if (lane == 0) next = atomicAdd(p.tile_counter, 1u);
      int join, pieces;
      const Piece pc = make_piece(p, cut.per, sh.lists, w, cut_of, join, pieces);
      if (lane == 0) {
        sh.piece[k % kPieces] = pc;
        mbar_arrive(&sh.wfull[k % kPieces]);
        if (join >= 0) p.pairs[join] = make_int4(pc.b, pc.kvh << 16 | pieces, pc.key0 / kKeys, pc.slot);
      }
      const int32_t* const row = p.seqs.table + pc.b * p.seqs.table_stride;
      // page of the keys of box `lane` of a key block (two tiles of `boxes` each)
      auto page_of = [&](int key0) -> int {
        const int64_t at = static_cast<int64_t>(key0) + lane * box_rows;
        if (lane >= 2 * boxes || at >= pc.len) return no_page;
        const int pg = row[at >> shift];
        return pg >= 0 && pg < no_page ? pg : no_page;
      };
      auto load_keys = [&](int key0, int page) -> bool {
        for (int t = 0; t < 2; ++t, ++kcnt) {
          const int slot = kcnt % C::kKSlots;
          if (!warp_all(wait(&sh.kempty[slot], kcnt / C::kKSlots + 1, 63))) return false;
          if (lane == 0) mbar_arrive_expect_tx(&sh.kfull[slot], C::kTileBytes);
          // lane i loads box i % boxes of channel chunk i / boxes
          const int box = lane & (boxes - 1), chunk = lane >> boxes_log;
          const int pg = __shfl_sync(0xffffffffu, page, t * boxes + box);
          if (chunk < C::kChunks)
            tma_load_4d(sK + slot * C::kTileBytes + chunk * kChunkBytes + box * box_rows * 128, &tm_k, &sh.kfull[slot],
                        64 * chunk, (key0 + t * kBlockN + box * box_rows) & ((1 << shift) - 1), pc.kvh, pg);
        }
        return true;
      };
      auto load_rows = [&](int i) -> bool {
        const int qs = qcnt % C::kQSlots;
        if (!warp_all(wait(&sh.qempty[qs], qcnt / C::kQSlots + 1, 64))) return false;
        if (lane == 0) {
          const Rows r = rows_of(p, i, pc);
          mbar_arrive_expect_tx(&sh.qfull[qs], q_bytes);
          for (int ch = 0; ch < C::kChunks; ++ch)
            tma_load_3d(sQ + qs * C::kTileBytes + ch * kChunkBytes, &tm_q, &sh.qfull[qs], 64 * ch,
                        pc.kvh * p.group + r.head, pc.row0 + r.token);
        }
        ++qcnt;
        return true;
      };
      if (pc.few) {
        const int first = max(pc.i0, pc.seen), tiles = pc.count * p.tile.parts;
        int page = first < pc.i1 ? page_of(first * kKeys) : no_page;
        for (int i = 0; ok && i < tiles && first < pc.i1; ++i) ok = load_rows(i);
        for (int i = first; ok && i < pc.i1; ++i) {
          const int ahead = i + 1 < pc.i1 ? page_of((i + 1) * kKeys) : no_page;
          ok = load_keys(i * kKeys, page);
          page = ahead;
        }
      } else if (pc.i1 > pc.i0) {
        ok = load_keys(pc.key0, page_of(pc.key0));
        for (int i = pc.i0; ok && i < pc.i1; ++i) ok = load_rows(i);
      }
      w = __shfl_sync(0xffffffffu, next, 0);
    }
    if (lane == 0) {
      release_pieces(p.tile_counter, total, w);
      if (!ok) {
        // the loads already issued land before the CTA gives up its shared memory
        for (int i = 0; i < C::kKSlots && i < kcnt; ++i)
          wait_final(&sh.kfull[i], ((kcnt - 1 - i) / C::kKSlots) & 1, limit);
        for (int i = 0; i < C::kQSlots && i < qcnt; ++i)
          wait_final(&sh.qfull[i], ((qcnt - 1 - i) / C::kQSlots) & 1, limit);
      }
    }
  } else if (warp == kLseWarp) {
    // ================================================================ the rows' lse, next to their tile
    // (The next one's loads are on their way while this one waits for a slot.)
    int tokens[4], heads[4];  // of the lane's four columns
    int64_t offset[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tokens[j] = (lane + 32 * j) / p.tile.heads;
      heads[j] = lane + 32 * j - tokens[j] * p.tile.heads;
      offset[j] = heads[j] * p.lse_shead + tokens[j] * p.lse_srow;
    }
    int cnt = 0;  // ring slots filled
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!warp_all(take_piece(k))) break;
      const Piece pc = sh.piece[k % kPieces];
      if (pc.b < 0) break;
      const int t0 = pc.few ? 0 : pc.i0;
      const int tiles = pc.few ? (pc.seen < pc.i1 ? pc.count * p.tile.parts : 0) : pc.i1 - pc.i0;
      float next[4];
      int have = 0;  // tokens of that tile
      auto fetch = [&](int i) {
        const Rows r = rows_of(p, i, pc);
        const float* const at = p.lse + (static_cast<int64_t>(pc.kvh) * p.group + r.head) * p.lse_shead +
                                (static_cast<int64_t>(pc.row0) + r.token) * p.lse_srow;
        have = r.tokens;
#pragma unroll
        for (int j = 0; j < 4; ++j) next[j] = tokens[j] < r.tokens && heads[j] < r.heads ? at[offset[j]] : -INFINITY;
      };
      if (tiles > 0) fetch(t0);
      for (int i = 0; i < tiles; ++i) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = next[j] == -INFINITY ? next[j] : -next[j] * kLog2e;
        bool none = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) none |= tokens[j] < have && v[j] == -INFINITY;
        const int some = __any_sync(0xffffffffu, none);
        if (i + 1 < tiles) fetch(t0 + i + 1);
        // (that of few row tiles has a place of its own, which lasts as long as the piece)
        const int slot = cnt % kLseSlots;
        if (!pc.few) ok = warp_all(wait(&sh.lempty[slot], cnt / kLseSlots + 1, 65));
        if (!ok) break;
        float* const dst = pc.few ? sh.few_lse[k % kPieces][i] : sh.lse[slot];
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[lane + 32 * j] = v[j];
        if (lane == 0) (pc.few ? sh.few_none[k % kPieces][i] : sh.none[slot]) = some;
        __syncwarp();
        if (!pc.few) {
          if (lane == 0) mbar_arrive(&sh.lfull[slot]);
          ++cnt;
        }
      }
      if (ok && lane == 0) mbar_arrive(&sh.few_full[k % kPieces]);
      arrive(&sh.wfree[k % kPieces]);
    }
  } else if (warp >= kMmaWarp) {
    // ================================================================ MMA issuers, one for each key tile
    // (Beside sixteen busy warps an issuer's own instructions count: with one for both tiles a step took 2400 cycles.)
    if (lane == 0) {
      const int t = warp - kMmaWarp;
      constexpr uint32_t kDescHi = smem_desc_hi(1024, kSwizzle128B);
      int kcnt = 0, qcnt = 0, used[2] = {0, 0};  // key tiles and row tiles taken, uses of each buffer
      // S^T of the key tile at klo and the row tile at qlo (descriptors)
      auto product = [&](int buf, uint32_t klo, uint32_t qlo, uint32_t idesc) -> bool {
        const int b = 2 * buf + t;
        int& n = buf == 0 ? used[0] : used[1];
        if (!wait(&sh.sfree[b], n + 1, 68)) return false;
        ++n;
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < DQK / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
          mma_ss_lh(tmem + b * 128, klo + off, kDescHi, qlo + off, kDescHi, idesc, kk > 0 ? 1u : 0u);
        }
        mma_commit(&sh.s[b]);
        return true;
      };
      const uint32_t klo0 = smem_desc_lo(smem_u32(sK), 16), qlo0 = smem_desc_lo(smem_u32(sQ), 16);
      auto idesc_of = [](int cols) { return idesc_bf16_f32(kBlockM, 0, 0, 0) | (static_cast<uint32_t>(cols >> 3) << 17); };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!take_piece(k)) break;
        const Piece& pc = sh.piece[k % kPieces];
        const int b = pc.b, few = pc.few, i0 = pc.i0, i1 = pc.i1, first = max(i0, pc.seen);
        const int tiles = pc.count * p.tile.parts, tokens = pc.n;
        mbar_arrive(&sh.wfree[k % kPieces]);
        if (b < 0) break;
        if (few) {
          if (first >= i1) continue;
          // (128 columns in every step would cost a decode step time)
          const uint32_t idesc = idesc_of(tiles == 1 ? (tokens * p.tile.heads + 31) & ~31 : 128);
          bool rows_there = false;
          for (int m = i0; ok && m < i1; m += 2) {  // two blocks at a time, one to each buffer
            for (int r = 0; ok && r < tiles; ++r) {
              const int qs = (qcnt + r) % C::kQSlots;
              if (!rows_there) ok = wait(&sh.qfull[qs], (qcnt + r) / C::kQSlots, 67);
#pragma unroll
              for (int buf = 0; buf < 2; ++buf) {
                if (!ok || m + buf < first || m + buf >= i1) continue;
                const int at = kcnt + 2 * (m + buf - first) + t, kslot = at % C::kKSlots;
                if (r == 0) ok = wait(&sh.kfull[kslot], at / C::kKSlots, 66);
                if (ok) ok = product(buf, klo0 + kslot * (C::kTileBytes >> 4), qlo0 + qs * (C::kTileBytes >> 4), idesc);
                if (ok && r == tiles - 1) mma_commit(&sh.kempty[kslot]);
              }
            }
            rows_there = true;
          }
          for (int r = 0; ok && r < tiles; ++r) mma_commit(&sh.qempty[(qcnt + r) % C::kQSlots]);
          kcnt += 2 * (i1 - first);
          qcnt += tiles;
        } else if (i1 > i0) {
          const uint32_t idesc = idesc_of(128);
          const int kslot = (kcnt + t) % C::kKSlots;
          ok = wait(&sh.kfull[kslot], (kcnt + t) / C::kKSlots, 66);
          for (int i = i0; ok && i < i1; ++i, ++qcnt) {
            const int qs = qcnt % C::kQSlots;
            ok = wait(&sh.qfull[qs], qcnt / C::kQSlots, 67) &&
                 product((i - i0) & 1, klo0 + kslot * (C::kTileBytes >> 4), qlo0 + qs * (C::kTileBytes >> 4), idesc);
            if (ok) mma_commit(&sh.qempty[qs]);
          }
          if (ok) mma_commit(&sh.kempty[kslot]);
          kcnt += 2;
        }
      }
      mma_commit(&sh.drain[t]);
      wait_final(&sh.drain[t], 0, limit);
    }
  } else {
    // ================================================================ a key to a thread
    const int buf = warp >> 3, t = (warp >> 2) & 1;
    const int row = (warp & 3) * 32 + lane, key = t * kBlockN + row;  // in the block
    const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (2 * buf + t) * 128;
    const uint64_t sl2 = pack_f32x2(p.scale_log2, p.scale_log2);
    int lcnt = 0, used = 0;  // row tiles' lse taken, uses of this buffer
    bool ok = true;
    auto scores_there = [&](int step) -> bool {
      if (!warp_all(wait(&sh.s[2 * buf + t], step, 70))) return false;
      tc_fence_after_sync();
      return true;
    };
    // The sum over a row tile's columns, all of which count (one without a row has a score of 0 and an lse of inf): each 32
    // columns' load runs under the exponentials of the 32 before.
    auto all_columns = [&](const float* lse) -> float {
      uint64_t acc[2] = {0, 0};
      uint32_t s[2][32];
      tmem_ld32(tS, s[0]);
      tmem_ld_wait();
      reg_fence(s[0]);
#pragma unroll
      for (int c = 0; c < kBlockN; c += 32) {
        uint32_t(&now)[32] = s[(c / 32) & 1], (&then)[32] = s[(c / 32 + 1) & 1];
        if (c + 32 < kBlockN) tmem_ld32(tS + c + 32, then);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(lse + c + 4 * e);
          exp_pair(now[4 * e], now[4 * e + 1], sl2, n.x, acc[0]);
          exp_pair(now[4 * e + 2], now[4 * e + 3], sl2, n.y, acc[1]);
        }
        if (c + 32 < kBlockN) {
          tmem_ld_wait();
          reg_fence(then);
        }
        if (c + 64 == kBlockN) {  // the scores are in registers
          tc_fence_before_sync();
          arrive(&sh.sfree[2 * buf + t]);
        }
      }
      const float2 a = unpack_f32x2(acc[0]), z = unpack_f32x2(acc[1]);
      return (a.x + a.y) + (z.x + z.y);
    };
    // Whether row tile i is full and all its rows see all of the warp's keys.
    auto seen_by_all = [&](const Piece& pc, int i, int pos) -> bool {
      const Rows r = rows_of(p, i, pc);
      const int kfirst = pos - row, qa = pc.pos0 + r.token;
      return r.tokens == p.tile.tokens && r.heads == p.tile.heads && kfirst + kBlockN - 1 <= qa &&
             (p.window == 0 || qa + r.tokens - 1 - kfirst < p.window);
    };
    // The sum over row tile i's columns that see the key at position pos.  (any tile; none: of its rows some add nothing)
    auto columns = [&](const Piece& pc, int i, int pos, const float* lse, int none) -> float {
      const Rows r = rows_of(p, i, pc);
      const int cols = r.tokens * p.tile.heads, qa = pc.pos0 + r.token, qb = qa + r.tokens - 1;
      // tokens from the key's position on, and up to the window's end
      const int lo = min(max(0, pos - qa), r.tokens) * p.tile.heads;
      const int hi = p.window > 0 && pos + p.window - 1 < qb ? max(0, pos + p.window - qa) * p.tile.heads : cols;
      const int kfirst = pos - row, klast = kfirst + kBlockN - 1;
      const bool all = klast <= qa && (p.window == 0 || qb - kfirst < p.window);  // every row sees every key
      uint64_t acc[2] = {0, 0};
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t s[32];
        tmem_ld32(tS + c, s);
        tmem_ld_wait();
        reg_fence(s);
        if (c + 32 >= cols) {  // the scores are in registers
          tc_fence_before_sync();
          arrive(&sh.sfree[2 * buf + t]);
        }
        float x[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 n = *reinterpret_cast<const float4*>(lse + c + 4 * e);
          const float2 a = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[4 * e]), __uint_as_float(s[4 * e + 1])), sl2,
                                                  pack_f32x2(n.x, n.y)));
          const float2 z = unpack_f32x2(fma_f32x2(
              pack_f32x2(__uint_as_float(s[4 * e + 2]), __uint_as_float(s[4 * e + 3])), sl2, pack_f32x2(n.z, n.w)));
          x[4 * e] = a.x, x[4 * e + 1] = a.y, x[4 * e + 2] = z.x, x[4 * e + 3] = z.y;
        }
        if (!(all && c + 32 <= cols)) {  // whatever hidden rows and columns without a row hold does not count
          const uint32_t span = static_cast<uint32_t>(max(0, hi - lo));
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (static_cast<uint32_t>(c + e - lo) >= span) x[e] = -INFINITY;
        }
        if (none != 0) {  // (a score that is not finite may have made them NaN)
          const uint32_t out = __ballot_sync(0xffffffffu, lse[c + lane] == -INFINITY);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((out >> e) & 1u) x[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          acc[e & 1] = add_f32x2(acc[e & 1], pack_f32x2(ex2_approx(x[2 * e]), ex2_approx(x[2 * e + 1])));
      }
      const float2 a = unpack_f32x2(acc[0]), z = unpack_f32x2(acc[1]);
      return (a.x + a.y) + (z.x + z.y);
    };
    for (int k = 0; ok; ++k) {
      if (!warp_all(take_piece(k))) break;
      const Piece pc = sh.piece[k % kPieces];
      if (pc.b < 0) break;
      // The page of a key's weight, looked up ahead of the sums and first looked at when they are there.
      auto page_of = [&](int pos) -> int {
        return pos < pc.len ? p.seqs.table[pc.b * p.seqs.table_stride + (pos >> p.seqs.page_shift)] : -1;
      };
      auto put = [&](int pg, int pos, float sum) {
        if (pg < 0 || pg >= p.seqs.n_pages || (p.accumulate && sum == 0.f)) return;
        float* const dst = p.weights + pg * p.w_spage + pc.kvh * p.w_shead + (pos & ((1 << p.seqs.page_shift) - 1));
        *dst = p.accumulate ? *dst + sum : sum;
      };
      if (pc.few) {
        const int tiles = pc.count * p.tile.parts;
        ok = warp_all(wait(&sh.few_full[k % kPieces], k / kPieces, 71));
        const int first = pc.i0 + buf;  // this buffer's first block
        int next = first < pc.i1 ? page_of(first * kKeys + key) : -1;
        for (int i = first; ok && i < pc.i1; i += 2) {
          const int pg = next, pos = i * kKeys + key;
          next = i + 2 < pc.i1 ? page_of((i + 2) * kKeys + key) : -1;
          float total = 0.f;
          for (int r = 0; ok && i >= pc.seen && r < tiles; ++r, ++used) {
            const float* const lse = sh.few_lse[k % kPieces][r];
            const int none = sh.few_none[k % kPieces][r];
            const bool all = tiles > 1 && seen_by_all(pc, r, pos);
            ok = scores_there(used);
            if (ok) total += all && none == 0 ? all_columns(lse) : columns(pc, r, pos, lse, none);
          }
          if (!ok) break;
          put(pg, pos, total);
        }
        if (!ok) break;
      } else {
        const int pos = pc.key0 + key;
        const int pg = buf == 0 && pc.slot < 0 ? page_of(pos) : -1;
        // row tiles [f0, f1) are full, and all their rows see all of the warp's keys (of a group in parts none is taken as such)
        int f0 = 0, f1 = 0;
        if (p.tile.parts == 1) {
          const int kfirst = pos - row, klast = kfirst + kBlockN - 1, tokens = p.tile.tokens;
          f0 = (max(0, klast - pc.pos0) + tokens - 1) / tokens - pc.blk0;
          f1 = pc.n / tokens - pc.blk0;
          if (p.window > 0) f1 = min(f1, max(0, kfirst + p.window - pc.pos0) / tokens - pc.blk0);
        }
        float total = 0.f;
        for (int i = pc.i0 + buf; i < pc.i1; i += 2, ++used) {  // this buffer's
          const int at = lcnt + (i - pc.i0), slot = at % kLseSlots;
          ok = warp_all(wait(&sh.lfull[slot], at / kLseSlots, 69));
          if (!ok) break;
          const int none = sh.none[slot];  // (on its way during the wait)
          ok = scores_there(used);
          if (!ok) break;
          total += i >= f0 && i < f1 && none == 0 ? all_columns(sh.lse[slot]) : columns(pc, i, pos, sh.lse[slot], none);
          arrive(&sh.lempty[slot]);
        }
        if (!ok) break;
        lcnt += pc.i1 - pc.i0;
        if (buf == 1) {
          sh.sums[k % kPieces][t][row] = total;
        } else {
          ok = warp_all(wait(&sh.sums_full[k % kPieces][t], k / kPieces, 72));
          if (!ok) break;
          total += sh.sums[k % kPieces][t][row];
          if (pc.slot >= 0)
            p.part[static_cast<int64_t>(pc.slot) * kKeys + key] = total;
          else
            put(pg, pos, total);
        }
      }
      if (buf == 1) arrive(&sh.sums_full[k % kPieces][t]);
      arrive(&sh.wfree[k % kPieces]);
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the sums of the pieces of the pairs that were cut, in their order.
__global__ void __launch_bounds__(kKeys) kv_weights_join_kernel(const __grid_constant__ KvWeightsParams p) {
  pdl_wait();
  if (*reinterpret_cast<volatile int*>(p.status) != 0) return;  // pieces may be missing
  const int n_pairs = min(*p.n_pairs, p.max_slots);
  for (int pair = blockIdx.x; pair < n_pairs; pair += gridDim.x) {
    const int4 e = p.pairs[pair];
    const int pieces = e.y & 0xffff, kvh = static_cast<int>(static_cast<uint32_t>(e.y) >> 16);
    if (e.w < 0 || e.w + pieces > p.max_slots || e.x < p.seqs.b0 || e.x >= p.seqs.b0 + p.seqs.B || kvh >= p.Hkv) continue;
    const int pos = e.z * kKeys + threadIdx.x;
    const KvSeq s = kv_seq(p.seqs, e.x - p.seqs.b0);
    if (pos >= s.len) continue;
    const int pg = p.seqs.table[e.x * p.seqs.table_stride + (pos >> p.seqs.page_shift)];
    if (pg < 0 || pg >= p.seqs.n_pages) continue;
    float sum = 0.f;
#pragma unroll 8
    for (int c = 0; c < pieces; ++c) sum += p.part[static_cast<int64_t>(e.w + c) * kKeys + threadIdx.x];
    float* const dst = p.weights + pg * p.w_spage + kvh * p.w_shead + (pos & ((1 << p.seqs.page_shift) - 1));
    if (!(p.accumulate && sum == 0.f)) *dst = p.accumulate ? *dst + sum : sum;
  }
}

// ---------------------------------------------------------------- launches

struct Workspace {
  int64_t max_slots;
  size_t pairs, part, total;  // offsets
};
Workspace workspace_of() {
  Workspace w;
  w.max_slots = max_joined<kFine>(kKvMaxSms);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.pairs = 256;
  w.part = w.pairs + up(w.max_slots * sizeof(int4));
  w.total = w.part + up(w.max_slots * kKeys * sizeof(float));
  return w;
}

template <int DQK>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, KvWeightsParams p, int64_t tiles, cudaStream_t stream) {
  using C = Cfg<DQK>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];  // the kernel's attribute is set on the device
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_weights_kernel<DQK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  if ((e = claim_cache_counter(stream, &p.tile_counter)) != cudaSuccess) return e;
  const int sms = kv_sm_count();
  e = launch_early(kv_weights_kernel<DQK>, dim3(static_cast<unsigned>(sms)), kThreads, C::kSmemBytes, stream, tq, tk, p);
  if (e != cudaSuccess || tiles <= C::kFew) return e;  // (no sequence's rows fill more tiles: nothing is joined)
  return launch_early(kv_weights_join_kernel, dim3(static_cast<unsigned>(2 * sms)), kKeys, 0, stream, p);
}

}  // namespace
}  // namespace slope

using namespace slope;

extern "C" {

size_t slope_kv_attn_weights_workspace_size(int64_t T, int64_t Hq, const slope_kv_cache* cache, int32_t q_len) {
  if (cache == nullptr || !attn_partial_supported(cache->dqk, cache->dv)) return 0;
  if (T < 0 || T >= kKvMaxTokens || cache->Hkv < 1 || Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0 || q_len < 0) return 0;
  return workspace_of().total;
}

slope_status slope_kv_attn_weights(const slope_tensor* q, const slope_kv_cache* cache, const slope_kv_batch* batch,
                                   const slope_tensor* lse, int64_t window, float scale, int accumulate,
                                   slope_tensor* weights, void* workspace, size_t workspace_bytes, void* stream) {
  const CallRange range("slope_kv_attn_weights");
  slope_status st;
  if ((st = check_kv_cache(cache)) != SLOPE_OK || (st = check_kv_q(q, cache)) != SLOPE_OK) return st;
  const int64_t T = q->shape[0], Hq = q->shape[1];
  if (window < 0 || window > (int64_t(1) << 30)) return SLOPE_ERR_SHAPE;
  if ((st = check_kv_batch(batch, cache, T)) != SLOPE_OK) return st;
  if ((st = check_lse(lse, Hq, T)) != SLOPE_OK) return st;
  if ((st = check_kv_weights(weights, cache)) != SLOPE_OK) return st;
  if (batch->B == 0 || (T == 0 && accumulate)) return SLOPE_OK;

  KvWeightsParams p{};
  p.Hkv = cache->Hkv;
  p.group = static_cast<int32_t>(Hq / cache->Hkv);
  p.tile = row_tile(p.group);
  // pieces of a launch are counted in 32 bits
  const int64_t blocks = (batch->max_pages * cache->page_size + kKeys - 1) / kKeys;
  if (std::min<int64_t>(batch->B, kKvMaxSeqs) * blocks * p.Hkv >= (int64_t(1) << 31)) return SLOPE_ERR_UNSUPPORTED;
  if ((T + p.tile.tokens) / p.tile.tokens * p.tile.parts >= (int64_t(1) << 30)) return SLOPE_ERR_UNSUPPORTED;
  const Workspace w = workspace_of();
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return SLOPE_ERR_WORKSPACE;
  if (kv_sm_count() <= 0) return cuda_fail("device attributes");
  p.seqs = kv_seqs(batch, cache, T);
  p.window = static_cast<int32_t>(window);
  p.accumulate = accumulate ? 1 : 0;
  p.scale_log2 = resolve_scale(scale, cache->dqk) * kLog2e;
  p.lse = static_cast<const float*>(lse->data);
  p.lse_srow = lse->stride[1];
  p.lse_shead = lse->stride[0];
  p.weights = static_cast<float*>(weights->data);
  p.w_spage = weights->stride[0];
  p.w_shead = weights->stride[1];
  char* const ws = static_cast<char*>(workspace);
  p.max_slots = static_cast<int32_t>(w.max_slots);
  p.n_pairs = reinterpret_cast<int32_t*>(ws);
  p.pairs = reinterpret_cast<int4*>(ws + w.pairs);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.status = device_status_ptr();
  if (p.status == nullptr) return cuda_fail("device status word (cudaGetSymbolAddress)");
  p.wait_limit_ns = wait_limit_ns();
  CUtensorMap tq, tk;
  if (!make_page_map(&tk, cache->k, cache, cache->dqk, cache->k_stride)) return cuda_fail("cuTensorMapEncodeTiled");
  if (T == 0)
    tq = tk;  // no row is loaded
  else if (!make_q_map(&tq, q, p.tile.heads, p.tile.tokens))
    return cuda_fail("cuTensorMapEncodeTiled");
  // row tiles of a sequence at most
  const int64_t most = batch->cu_q != nullptr ? T : batch->q_len;
  const int64_t tiles = (most + p.tile.tokens - 1) / p.tile.tokens * p.tile.parts;
  for (int64_t b = 0; b < batch->B; b += kKvMaxSeqs) {
    p.seqs.b0 = static_cast<int32_t>(b);
    p.seqs.B = static_cast<int32_t>(std::min<int64_t>(kKvMaxSeqs, batch->B - b));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dqk == 64    ? launch<64>(tq, tk, p, tiles, s)
                          : cache->dqk == 128 ? launch<128>(tq, tk, p, tiles, s)
                                              : launch<192>(tq, tk, p, tiles, s);
    if (e != cudaSuccess) return cuda_fail("cache weights kernel launch", e);
  }
  return SLOPE_OK;
}

}  // extern "C"
