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
// The work: a pair is (sequence, KV head, 256 keys), its steps the row tiles (attention over few rows, a decode step,
// has one or two, and then this kernel reads K at the copy rate, up to four key blocks ahead).  Pairs of many rows and
// few keys are cut (kv_cut.cuh); their pieces leave 256 sums each in the workspace, which a second launch adds in order.
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
  int32_t* n_slots;  // workspace: pieces that are joined
  int4* pairs;       // workspace, for each of them: {sequence, KV head, key block, pieces (0 but in the first)}
  float* part;       // workspace: their sums
  int* status;
  uint32_t* tile_counter;
  uint64_t wait_limit_ns;
};

template <int DQK>
struct Cfg {
  static constexpr int kChunks = DQK / 64;
  static constexpr int kTileBytes = kChunks * kChunkBytes;  // 128 rows of K or Q
  static constexpr int kKSlots = DQK == 64 ? 4 : DQK == 128 ? 2 : 1;  // of 256 keys
  static constexpr int kQSlots = DQK == 64 ? 4 : 2;
  static constexpr int kQOffset = kKSlots * 2 * kTileBytes;
  static constexpr int kLseOffset = kQOffset + kQSlots * kTileBytes;
  static constexpr int kListOffset = kLseOffset + kQSlots * 128 * 4;
  static constexpr int kSmemBytes = 1024 + kListOffset + static_cast<int>(sizeof(CutLists));
  static_assert(kSmemBytes <= 231424, "shared memory budget");
};
constexpr int kSoftmaxWarps = 8, kTmaWarp = 8, kMmaWarp = 9, kLseWarp = 10, kLseWarps = 2;
constexpr int kThreads = 32 * (kLseWarp + kLseWarps);

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// Key blocks of a sequence, and the row tiles that one of them meets at most.  (The row tiles of a group of more than
// 128 heads are those of its parts, one part after another.)
struct KeyCut {
  RowTile tile;
  __device__ __forceinline__ SeqCut operator()(const KvSeq& s) const {
    SeqCut c;
    c.blocks = (s.len + kKeys - 1) / kKeys;
    c.steps = (s.n + tile.tokens - 1) / tile.tokens * tile.parts;
    return c;
  }
};

// A piece: row tiles [i0, i1) of a key block, numbered from 0 among the `count` of every part that see one of its keys.
struct Piece {
  int32_t b;  // sequence; -1: no pieces left
  int32_t kvh, key0, len;
  int32_t row0, n, pos0;  // of the sequence: first q row, new tokens, position of the first
  int32_t blk0, count;    // first row block that sees a key, and how many
  int32_t i0, i1;
  int32_t slot;
};

__device__ __forceinline__ Piece make_piece(const KvWeightsParams& p, int per, const CutLists& lists, uint32_t w,
                                            const KeyCut& cut_of, int& pieces, int& c) {
  Piece r;
  const int b = seq_of(lists, p.seqs.B, w);
  const KvSeq q = lists.seqs[b];
  const SeqCut cut = cut_of(q);
  pieces = pieces_of(cut.steps, per);
  uint32_t local = w - lists.units[b];
  const int blk = static_cast<int>(local % cut.blocks);
  local /= cut.blocks;
  c = static_cast<int>(local % pieces);
  r.kvh = static_cast<int>(local / pieces);
  r.b = p.seqs.b0 + b;
  r.key0 = blk * kKeys;
  r.len = q.len;
  r.row0 = q.row0;
  r.n = q.n;
  r.pos0 = q.len - q.n;
  // tokens [lo, hi) see one of the keys [key0, last]
  const int last = min(q.len, r.key0 + kKeys) - 1;
  const int lo = min(q.n, max(0, r.key0 - r.pos0));
  const int hi = p.window > 0 ? max(lo, min(q.n, last + p.window - r.pos0)) : q.n;
  r.blk0 = lo / p.tile.tokens;
  r.count = hi > lo ? (hi + p.tile.tokens - 1) / p.tile.tokens - r.blk0 : 0;
  piece_steps(r.count * p.tile.parts, pieces, c, r.i0, r.i1);
  r.slot = pieces > 1 ? static_cast<int32_t>(lists.slots[b]) + (r.kvh * cut.blocks + blk) * pieces + c : -1;
  return r;
}

// Row tile i of a piece.
struct Rows {
  int token, tokens;  // first token among the sequence's new ones, and how many
  int head, heads;    // first head in the group, and how many
};
__device__ __forceinline__ Rows rows_of(const KvWeightsParams& p, int i, int blk0, int count, int n) {
  Rows r;
  const int part = p.tile.parts > 1 ? i / count : 0;
  r.token = (blk0 + i - part * count) * p.tile.tokens;
  r.tokens = min(p.tile.tokens, n - r.token);
  r.head = part * p.tile.heads;
  r.heads = min(p.tile.heads, p.group - r.head);
  return r;
}

template <int DQK>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ KvWeightsParams p) {
  using C = Cfg<DQK>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Piece s_piece[kPieces];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint64_t bar_kfull[C::kKSlots], bar_kempty[C::kKSlots], bar_qfull[C::kQSlots], bar_qempty[C::kQSlots];
  __shared__ uint64_t bar_s[4], bar_sfree[4];  // [2 * buffer + key tile]
  __shared__ uint64_t bar_wfull[kPieces], bar_wfree[kPieces], bar_drain;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sK = smem;
  uint8_t* const sQ = smem + C::kQOffset;
  float* const sLse = reinterpret_cast<float*>(smem + C::kLseOffset);  // [slot][column]: -lse log2(e)
  CutLists& lists = *reinterpret_cast<CutLists*>(smem + C::kListOffset);
  volatile int* const cta_abort = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  const KeyCut cut_of{p.tile};

  pdl_launch_dependents();
  uint32_t claimed = 0;
  if (threadIdx.x == kTmaWarp * 32) {
    claimed = atomicAdd(p.tile_counter, 1u);
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
  }
  if (threadIdx.x == 0) *cta_abort = *reinterpret_cast<volatile int*>(p.status) != 0 ? 1 : 0;
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == kMmaWarp * 32) {
    for (int i = 0; i < C::kKSlots; ++i) mbar_init(&bar_kfull[i], 1), mbar_init(&bar_kempty[i], 1);
    for (int i = 0; i < C::kQSlots; ++i) {
      mbar_init(&bar_qfull[i], 2);                   // the loads, and the lse
      mbar_init(&bar_qempty[i], 1 + kSoftmaxWarps);  // the products, and the lse's readers
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bar_s[i], 1), mbar_init(&bar_sfree[i], 4);
    for (int i = 0; i < kPieces; ++i) mbar_init(&bar_wfull[i], 1), mbar_init(&bar_wfree[i], 1 + kLseWarps + kSoftmaxWarps);
    mbar_init(&bar_drain, 1);
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
    return wait_bounded(bar, parity & 1, cta_abort, p.status, limit, site);
  };
  auto take_piece = [&](int k) -> bool { return wait(&bar_wfull[k % kPieces], k / kPieces, 61); };

  if (warp == kTmaWarp) {
    // ================================================================ producer: pieces, pages, loads
    const Cut cut = make_cut<kPieceSteps>(p.seqs, p.Hkv, cut_of, lists);
    if (lane == 0 && blockIdx.x == 0) *p.n_slots = static_cast<int32_t>(cut.slots);
    const uint32_t total = cut.total;
    const uint32_t q_bytes = static_cast<uint32_t>(p.tile.heads * p.tile.tokens) * 128 * C::kChunks;
    const int shift = p.seqs.page_shift;
    const int boxes_log = max(0, 7 - shift);  // log2 of the boxes of 64 channels of 128 keys
    const int boxes = 1 << boxes_log, box_rows = kBlockN >> boxes_log;
    const int no_page = static_cast<int>(p.seqs.n_pages);  // reads 0
    uint32_t w = __shfl_sync(0xffffffffu, claimed, 0);
    int kcnt = 0, qcnt = 0;  // K blocks and row tiles loaded
    bool ok = *cta_abort == 0;
    for (int k = 0; ok; ++k) {
      if (k >= kPieces) ok = warp_all(wait(&bar_wfree[k % kPieces], k / kPieces - 1, 62));
      if (!ok) break;
      if (w >= total) {
        if (lane == 0) {
          s_piece[k % kPieces].b = -1;
          mbar_arrive(&bar_wfull[k % kPieces]);
        }
        break;
      }
      uint32_t next = 0;
      if (lane == 0) next = atomicAdd(p.tile_counter, 1u);
      int pieces, c;
      const Piece pc = make_piece(p, cut.per, lists, w, cut_of, pieces, c);
      if (lane == 0) {
        s_piece[k % kPieces] = pc;
        mbar_arrive(&bar_wfull[k % kPieces]);
        if (pc.slot >= 0) p.pairs[pc.slot] = make_int4(pc.b, pc.kvh, pc.key0 / kKeys, c == 0 ? pieces : 0);
      }
      if (pc.i1 > pc.i0) {
        // ---- the keys: lane i looks up page i of the block, then loads boxes lane, lane + 32, ...
        const int slot = kcnt % C::kKSlots;
        const int32_t* const row = p.seqs.table + pc.b * p.seqs.table_stride;
        const int64_t at = static_cast<int64_t>(pc.key0) + lane * box_rows;
        int page = no_page;
        if (lane < 2 * boxes && at < pc.len) {
          const int pg = row[at >> shift];
          if (pg >= 0 && pg < no_page) page = pg;
        }
        ok = warp_all(wait(&bar_kempty[slot], kcnt / C::kKSlots + 1, 63));
        if (ok) {
          if (lane == 0) mbar_arrive_expect_tx(&bar_kfull[slot], 2 * C::kTileBytes);
          __syncwarp();
          for (int i0 = 0; i0 < 2 * boxes * C::kChunks; i0 += 32) {
            const int i = i0 + lane, box = i & (2 * boxes - 1), chunk = i >> (boxes_log + 1);
            const int pg = __shfl_sync(0xffffffffu, page, box);
            if (chunk < C::kChunks) {
              const int tile = box >> boxes_log, in_tile = box & (boxes - 1);
              tma_load_4d(sK + (slot * 2 + tile) * C::kTileBytes + chunk * kChunkBytes + in_tile * box_rows * 128, &tm_k,
                          &bar_kfull[slot], 64 * chunk, (pc.key0 + box * box_rows) & ((1 << shift) - 1), pc.kvh, pg);
            }
          }
          ++kcnt;
        }
        for (int i = pc.i0; ok && i < pc.i1; ++i, ++qcnt) {
          const int qs = qcnt % C::kQSlots;
          ok = warp_all(wait(&bar_qempty[qs], qcnt / C::kQSlots + 1, 64));
          if (!ok) break;
          if (lane == 0) {
            const Rows r = rows_of(p, i, pc.blk0, pc.count, pc.n);
            mbar_arrive_expect_tx(&bar_qfull[qs], q_bytes);
            for (int ch = 0; ch < C::kChunks; ++ch)
              tma_load_3d(sQ + qs * C::kTileBytes + ch * kChunkBytes, &tm_q, &bar_qfull[qs], 64 * ch,
                          pc.kvh * p.group + r.head, pc.row0 + r.token);
          }
        }
      }
      w = __shfl_sync(0xffffffffu, next, 0);
    }
    if (lane == 0) {
      release_pieces(p.tile_counter, total, w);
      if (!ok) {
        // the loads already issued land before the CTA gives up its shared memory (the row tiles' barriers also count
        // the lse's arrival, which may never come: their bytes are waited for as long as the limit says)
        for (int i = 0; i < C::kKSlots && i < kcnt; ++i)
          wait_final(&bar_kfull[i], ((kcnt - 1 - i) / C::kKSlots) & 1, limit);
        for (int i = 0; i < C::kQSlots && i < qcnt; ++i)
          wait_final(&bar_qfull[i], ((qcnt - 1 - i) / C::kQSlots) & 1, limit);
      }
    }
  } else if (warp >= kLseWarp) {
    // ================================================================ the rows' lse, next to their tile
    // Each warp takes every second row tile, and has its next one's loads on their way while it waits for a slot.
    int qcnt = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!warp_all(take_piece(k))) break;
      const Piece pc = s_piece[k % kPieces];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_wfree[k % kPieces]);
      if (pc.b < 0) break;
      float next[4];
      auto fetch = [&](int i) {
        const Rows r = rows_of(p, i, pc.blk0, pc.count, pc.n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = lane + 32 * j, token = col / p.tile.heads, head = col - token * p.tile.heads;
          next[j] = -INFINITY;
          if (i < pc.i1 && token < r.tokens && head < r.heads)
            next[j] = p.lse[(static_cast<int64_t>(pc.kvh) * p.group + r.head + head) * p.lse_shead +
                            (static_cast<int64_t>(pc.row0) + r.token + token) * p.lse_srow];
        }
      };
      const int first = pc.i0 + ((qcnt ^ (warp - kLseWarp)) & 1);
      if (first < pc.i1) fetch(first);
      for (int i = first; i < pc.i1; i += kLseWarps) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = next[j];
        fetch(min(i + kLseWarps, pc.i1 - 1));
        const int at = qcnt + (i - pc.i0), qs = at % C::kQSlots;
        ok = warp_all(wait(&bar_qempty[qs], at / C::kQSlots + 1, 65));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) sLse[qs * 128 + lane + 32 * j] = v[j] == -INFINITY ? v[j] : -v[j] * kLog2e;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfull[qs]);
      }
      qcnt += pc.i1 - pc.i0;
    }
  } else if (warp == kMmaWarp) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kDescHi = smem_desc_hi(1024, kSwizzle128B);
      int kcnt = 0, qcnt = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!take_piece(k)) break;
        const Piece pc = s_piece[k % kPieces];
        mbar_arrive(&bar_wfree[k % kPieces]);
        if (pc.b < 0) break;
        if (pc.i1 <= pc.i0) continue;
        const int kslot = kcnt % C::kKSlots;
        if (!wait(&bar_kfull[kslot], kcnt / C::kKSlots, 66)) break;
        ++kcnt;
        for (int i = pc.i0; ok && i < pc.i1; ++i, ++qcnt) {
          const int qs = qcnt % C::kQSlots;
          ok = wait(&bar_qfull[qs], qcnt / C::kQSlots, 67);
          if (!ok) break;
          const Rows r = rows_of(p, i, pc.blk0, pc.count, pc.n);
          const int cols = (r.tokens * p.tile.heads + 15) & ~15;  // 128 at most
          const uint32_t idesc = idesc_bf16_f32(kBlockM, 0, 0, 0) | (static_cast<uint32_t>(cols >> 3) << 17);
          const uint32_t qlo = smem_desc_lo(smem_u32(sQ + qs * C::kTileBytes), 16);
          for (int t = 0; t < 2 && ok; ++t) {
            const int buf = 2 * (qcnt & 1) + t;
            ok = wait(&bar_sfree[buf], (qcnt >> 1) + 1, 68);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t klo = smem_desc_lo(smem_u32(sK + (kslot * 2 + t) * C::kTileBytes), 16);
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
              mma_ss_lh(tmem + buf * 128, klo + off, kDescHi, qlo + off, kDescHi, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bar_s[buf]);
          }
          if (ok) mma_commit(&bar_qempty[qs]);
        }
        if (ok) mma_commit(&bar_kempty[kslot]);
      }
      mma_commit(&bar_drain);
      wait_final(&bar_drain, 0, limit);
    }
  } else {
    // ================================================================ a key to a thread
    const int t = warp >> 2;
    const int key = t * kBlockN + (warp & 3) * 32 + lane;  // in the block
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint64_t sl2 = pack_f32x2(p.scale_log2, p.scale_log2);
    int qcnt = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!warp_all(take_piece(k))) break;
      const Piece pc = s_piece[k % kPieces];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_wfree[k % kPieces]);
      if (pc.b < 0) break;
      const int pos = pc.key0 + key;
      // the place of the key's weight, looked up ahead of the sums
      float* dst = nullptr;
      if (pc.slot < 0 && pos < pc.len) {
        const int pg = p.seqs.table[pc.b * p.seqs.table_stride + (pos >> p.seqs.page_shift)];
        if (pg >= 0 && pg < p.seqs.n_pages)
          dst = p.weights + pg * p.w_spage + pc.kvh * p.w_shead + (pos & ((1 << p.seqs.page_shift) - 1));
      }
      const int kfirst = pc.key0 + t * kBlockN, klast = kfirst + kBlockN - 1;
      float total = 0.f;
      for (int i = pc.i0; ok && i < pc.i1; ++i, ++qcnt) {
        const int qs = qcnt % C::kQSlots, buf = 2 * (qcnt & 1) + t;
        const Rows r = rows_of(p, i, pc.blk0, pc.count, pc.n);
        const int cols = r.tokens * p.tile.heads, qa = pc.pos0 + r.token, qb = qa + r.tokens - 1;
        // the columns whose rows see this key: tokens from its position on, and up to the window's end
        const int lo = max(0, pos - qa) * p.tile.heads;
        const int hi = p.window > 0 && pos + p.window - 1 < qb ? (pos + p.window - qa) * p.tile.heads : cols;
        const bool all = klast <= qa && (p.window == 0 || qb - kfirst < p.window);  // every row sees every key
        ok = warp_all(wait(&bar_qfull[qs], qcnt / C::kQSlots, 69)) && warp_all(wait(&bar_s[buf], qcnt >> 1, 70));
        if (!ok) break;
        tc_fence_after_sync();
        const float4* const lse = reinterpret_cast<const float4*>(sLse + qs * 128);
        uint64_t acc[2] = {0, 0};
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t s[32];
          tmem_ld32(tmem + lane_base + buf * 128 + c, s);
          tmem_ld_wait();
          reg_fence(s);
          if (c + 32 >= cols) {  // the scores are in registers
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_sfree[buf]);
          }
          float x[32];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 n = lse[c / 4 + e];
            const float2 a = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[4 * e]), __uint_as_float(s[4 * e + 1])),
                                                    sl2, pack_f32x2(n.x, n.y)));
            const float2 b = unpack_f32x2(fma_f32x2(
                pack_f32x2(__uint_as_float(s[4 * e + 2]), __uint_as_float(s[4 * e + 3])), sl2, pack_f32x2(n.z, n.w)));
            x[4 * e] = a.x, x[4 * e + 1] = a.y, x[4 * e + 2] = b.x, x[4 * e + 3] = b.y;
          }
          if (!(all && c + 32 <= cols)) {  // whatever hidden rows and columns without a row hold does not count
            const uint32_t span = static_cast<uint32_t>(max(0, hi - lo));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (static_cast<uint32_t>(c + e - lo) >= span) x[e] = -INFINITY;
          }
          if (r.heads < p.tile.heads) {  // the last part of a group of more than 128 heads
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((c + e) % p.tile.heads >= r.heads) x[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[e & 1] = add_f32x2(acc[e & 1], pack_f32x2(ex2_approx(x[2 * e]), ex2_approx(x[2 * e + 1])));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qempty[qs]);
        const float2 a = unpack_f32x2(acc[0]), b = unpack_f32x2(acc[1]);
        total += (a.x + a.y) + (b.x + b.y);
      }
      if (!ok) break;
      if (pc.slot >= 0)
        p.part[static_cast<int64_t>(pc.slot) * kKeys + key] = total;
      else if (dst != nullptr && !(p.accumulate && total == 0.f))
        *dst = p.accumulate ? *dst + total : total;
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
  const int n_slots = min(*p.n_slots, p.max_slots);
  for (int slot = blockIdx.x; slot < n_slots; slot += gridDim.x) {
    const int4 e = p.pairs[slot];
    if (e.w <= 0 || slot + e.w > n_slots || e.x < p.seqs.b0 || e.x >= p.seqs.b0 + p.seqs.B) continue;
    const int pos = e.z * kKeys + threadIdx.x;
    const KvSeq s = kv_seq(p.seqs, e.x - p.seqs.b0);
    if (pos >= s.len) continue;
    const int pg = p.seqs.table[e.x * p.seqs.table_stride + (pos >> p.seqs.page_shift)];
    if (pg < 0 || pg >= p.seqs.n_pages) continue;
    float sum = 0.f;
#pragma unroll 8
    for (int c = 0; c < e.w; ++c) sum += p.part[static_cast<int64_t>(slot + c) * kKeys + threadIdx.x];
    float* const dst = p.weights + pg * p.w_spage + e.y * p.w_shead + (pos & ((1 << p.seqs.page_shift) - 1));
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
  w.max_slots = max_joined(kv_sm_count());
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  w.pairs = 256;
  w.part = w.pairs + up(w.max_slots * sizeof(int4));
  w.total = w.part + up(w.max_slots * kKeys * sizeof(float));
  return w;
}

template <int DQK>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, KvWeightsParams p, cudaStream_t stream) {
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
  p.tile_counter = claim_tile_counter();
  if (p.tile_counter == nullptr) return cudaErrorInvalidDevice;
  const int sms = kv_sm_count();
  kv_weights_kernel<DQK><<<sms, kThreads, C::kSmemBytes, stream>>>(tq, tk, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * sms));
  cfg.blockDim = dim3(kKeys);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_weights_join_kernel, p);
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
  if (kv_sm_count() <= 0) return cuda_fail("device attributes");
  const Workspace w = workspace_of();
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return SLOPE_ERR_WORKSPACE;
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
  p.n_slots = reinterpret_cast<int32_t*>(ws);
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
  for (int64_t b = 0; b < batch->B; b += kKvMaxSeqs) {
    p.seqs.b0 = static_cast<int32_t>(b);
    p.seqs.B = static_cast<int32_t>(std::min<int64_t>(kKvMaxSeqs, batch->B - b));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dqk == 64    ? launch<64>(tq, tk, p, s)
                          : cache->dqk == 128 ? launch<128>(tq, tk, p, s)
                                              : launch<192>(tq, tk, p, s);
    if (e != cudaSuccess) return cuda_fail("cache weights kernel launch", e);
  }
  return SLOPE_OK;
}

}  // extern "C"
