// RMS norm of every query and key head and the rotation by position, in one
// pass: y = x / sqrt(mean(x^2) + eps) * w, then the pairs (a, b) of the rotated
// channels become (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq.
//
// Bandwidth-bound: every value is read once and written once.  A lane has two words of eight channels (16
// bytes of bf16) of a head, one and the one half a rotation away, so the pairs that the rotation mixes need no
// other lane and no second load, whatever part of the head is rotated; words that are not rotated are paired
// as they come.  A head of 64 channels takes 4 lanes, of 128 8, of 192 12 of 16.  A warp takes one token
// and runs over its heads, two or three groups of them at a time with the next ones' loads in flight, and then,
// where that pays, over further tokens.  The weights and the token's sines and cosines are the same for every head
// of a lane, and stay in its registers as
//   y_e = (x_e A_e + x_partner B_e) / rms,   A = w cos, B = -+ w_partner sin.
//
// Measured, bf16: 32768 tokens, 64/8 heads of 64, all rotated, 101 us = 6.0 TB/s (88% of the copy rate); 8191 tokens,
// 128/128 heads of 192, 273 us = 5.9 TB/s; 16384 tokens, 32/8 heads of 128, 58 us.  With eight lanes to a head of
// any size, the other half fetched again or by shuffles, these took 118, 295 to 364 and 83 us; one group at
// a time at the same registers 131 us; six CTAs an SM instead of four spill.  16 tokens: 2.9 us, which is the launch.
// fp32, 16384 tokens, 64/8 heads of 64: 94 us = 6.4 TB/s; bf16 to fp32 73 us, fp32 to bf16 76 us.
//
// Angles: position * inv_freq loses everything in fp32 at far positions (at
// position 10^6 an fp32 angle is off by 0.06 radians).  The frequency is kept as
// turns per position in 64-bit fixed point, so the product's low 64 bits are the
// fraction of a turn, exactly, with no reduction.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.cuh"
#include "kernels.cuh"
#include "slope_serving.h"
#include "sm103_ptx.cuh"

namespace slope {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxHalf = 96;  // rotated pairs of a head

// Lanes that share a head (of 192 channels 12 of 16), and the heads that a warp's load covers.
__host__ __device__ constexpr int lanes_per_head(int d) { return d == 64 ? 4 : d == 128 ? 8 : 16; }
__host__ __device__ constexpr int heads_per_pass(int d) { return 32 / lanes_per_head(d); }

struct NormRopeSide {
  const void* x;
  void* y;
  const void* w;  // NULL: 1
  int64_t x_srow, x_shead, y_srow, y_shead, w_shead;
  int32_t w_bf16;
  int32_t H;  // 0: absent
};

struct NormRopeParams {
  NormRopeSide side[2];  // queries, keys
  int64_t T;
  const int32_t* positions;  // NULL: pos0 + row
  int64_t pos0;
  float eps;
  int32_t norm, rotate, interleaved, begin, half;
  float factor;
  int32_t heads;   // of a warp (of side[0].H + side[1].H)
  int32_t splits;  // warps of a token
  uint64_t turns[kMaxHalf];  // inv_freq / 2 pi modulo 1, times 2^64
};

// Eight channels as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  // channels 2 i and 2 i + 1
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t u = (&r[0].x)[i];
      return pack_f32x2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
      return pack_f32x2(__uint_as_float((&r[i / 2].x)[i % 2 * 2]), __uint_as_float((&r[i / 2].x)[i % 2 * 2 + 1]));
    }
  }
};
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
  const float2 f = unpack_f32x2(v);
  return pack_f32x2(f.y, f.x);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const uint64_t (&v)[4]) {
  const float2 a = unpack_f32x2(v[0]), b = unpack_f32x2(v[1]), c = unpack_f32x2(v[2]), d = unpack_f32x2(v[3]);
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(c.x, c.y, d.x, d.y);
  }
}

__device__ __forceinline__ float weight_at(const NormRopeSide& s, int64_t i) {
  return s.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(s.w)[i]) : static_cast<const float*>(s.w)[i];
}
__device__ __forceinline__ uint64_t weight_pair(const NormRopeSide& s, int64_t i) {
  return pack_f32x2(weight_at(s, i), weight_at(s, i + 1));
}

// kInter: the channels of a pair are neighbours, else half a rotation apart.  kLoop: the warps go on to further
// tokens, whose first heads are fetched during the last pass of the one before.
template <typename TI, typename TO, int D, bool kInter, bool kLoop>
__global__ void __launch_bounds__(kThreads, sizeof(TI) == 2 ? 4 : 3) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ __align__(16) float s_cos[kWarps][kMaxHalf], s_sin[kWarps][kMaxHalf];  // of the warp's token
  __shared__ __align__(16) float s_w[2][D];  // weights shared by every head of a side, else 1
  constexpr int kLanes = lanes_per_head(D), kHeads = heads_per_pass(D), kUsed = D / 16;
  constexpr int kWide = D == 192 && sizeof(TI) == 2 ? 3 : 2;  // groups of kHeads in a pass
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int li = min(lane % kLanes, kUsed - 1), sub = lane / kLanes;
  const bool used = lane % kLanes < kUsed;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps, tasks = p.T * p.splits;
  int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp;  // a token's heads, or a part of them
  int64_t tok = 0;
  // the task's heads of either side, and the passes they take
  int h_begin[2], h_end[2], n_pass[2];
  auto take = [&]() {
    tok = p.splits == 1 ? task : task / p.splits;
    const int first = static_cast<int>(task - tok * p.splits) * p.heads;
    const int last = tok < p.T ? min(first + p.heads, p.side[0].H + p.side[1].H) : first;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int base = w ? p.side[0].H : 0;
      h_begin[w] = max(first - base, 0);
      h_end[w] = min(last - base, p.side[w].H);
      n_pass[w] = h_begin[w] < h_end[w] ? (h_end[w] - h_begin[w] + kHeads * kWide - 1) / (kHeads * kWide) : 0;
    }
  };
  // The lane's two words: a word and the one half a rotation away, the first lanes of a head; then the words that
  // are not rotated.  Interleaved: neighbours.
  int ch[2];
  bool rot[2];
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ch[i] = 16 * li + 8 * i;
      rot[i] = p.rotate && ch[i] >= p.begin && ch[i] < p.begin + 2 * p.half;
    }
  } else {
    const int n = p.rotate ? p.half / 8 : 0;  // pairs of rotated words
    rot[0] = rot[1] = li < n;
    const int a = 2 * (li - n);               // among the words that are not rotated
    ch[0] = li < n ? p.begin + 8 * li : 8 * a + (8 * a < p.begin ? 0 : 16 * n);
    ch[1] = li < n ? ch[0] + p.half : 8 * a + 8 + (8 * a + 8 < p.begin ? 0 : 16 * n);
  }
  Raw8<TI> v[kWide][2];
  auto fetch = [&](int pass, Raw8<TI>(&fv)[kWide][2]) {
    const int w = pass >= n_pass[0] ? 1 : 0;
    const NormRopeSide& s = p.side[w];
    const int h0 = w ? h_begin[1] + (pass - n_pass[0]) * (kHeads * kWide) : h_begin[0] + pass * (kHeads * kWide);
    const TI* const x = static_cast<const TI*>(s.x) + tok * s.x_srow;
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
      // past the last head: its values once more, which are not stored
      const int h = min(h0 + k * kHeads + sub, (w ? h_end[1] : h_end[0]) - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) fv[k][i].load(x + h * s.x_shead + ch[i]);
    }
  };
  auto position = [&](int64_t t) -> int64_t {
    return !p.rotate || t >= p.T ? 0 : p.positions != nullptr ? p.positions[t] : p.pos0 + t;
  };
  take();
  int64_t pos = kLoop ? position(tok) : 0;
  if (n_pass[0] + n_pass[1] > 0) fetch(0, v);

  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const NormRopeSide& s = p.side[i / D];
    s_w[i / D][i % D] = s.w != nullptr && s.w_shead == 0 ? weight_at(s, i % D) : 1.f;
  }
  auto turn = [&]() {  // the token's sines and cosines
    if (!p.rotate) return;
    const int64_t at = kLoop ? pos : position(tok);
    for (int f = lane; f < p.half; f += 32) {
      // the fraction of a turn, rounded to 32 bits and taken in [-1/2, 1/2)
      const uint64_t frac = p.turns[f] * static_cast<uint64_t>(at) + 0x80000000ull;
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &sn, &cs);
      s_cos[warp][f] = cs * p.factor;
      s_sin[warp][f] = sn * p.factor;
    }
  };
  if (!kLoop) turn();
  __syncthreads();

  // y_e = (x_e fa_e + x_partner fb_e) / rms
  uint64_t fa[2][4], fb[2][4];
  auto set_factors = [&](int which) {
    float a[2][8], b[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&s_w[which][ch[i] + e]);
        a[i][e] = w.x, a[i][e + 1] = w.y, a[i][e + 2] = w.z, a[i][e + 3] = w.w;
        b[i][e] = b[i][e + 1] = b[i][e + 2] = b[i][e + 3] = 0.f;
      }
    if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!rot[i]) continue;
        const float4 cs = *reinterpret_cast<const float4*>(&s_cos[warp][(ch[i] - p.begin) / 2]);
        const float4 sn = *reinterpret_cast<const float4*>(&s_sin[warp][(ch[i] - p.begin) / 2]);
        const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          b[i][2 * e] = -a[i][2 * e + 1] * s4[e];
          b[i][2 * e + 1] = a[i][2 * e] * s4[e];
          a[i][2 * e] *= c4[e];
          a[i][2 * e + 1] *= c4[e];
        }
      }
    } else if (rot[0]) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 cs = *reinterpret_cast<const float4*>(&s_cos[warp][8 * li + e]);
        const float4 sn = *reinterpret_cast<const float4*>(&s_sin[warp][8 * li + e]);
        const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b[0][e + j] = -a[1][e + j] * s4[j];
          b[1][e + j] = a[0][e + j] * s4[j];
          a[0][e + j] *= c4[j];
          a[1][e + j] *= c4[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        fa[i][e] = pack_f32x2(a[i][2 * e], a[i][2 * e + 1]);
        fb[i][e] = pack_f32x2(b[i][2 * e], b[i][2 * e + 1]);
      }
  };

  for (;;) {
    if constexpr (kLoop) {
      __syncwarp();  // the last token's sines and cosines are read
      turn();
      __syncwarp();
    }
    const int passes = n_pass[0] + n_pass[1];
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
      const int which = pass >= n_pass[0] ? 1 : 0;
      const NormRopeSide& s = p.side[which];
      const int h0 = which ? h_begin[1] + (pass - n_pass[0]) * (kHeads * kWide) : h_begin[0] + pass * (kHeads * kWide);
      const int end = which ? h_end[1] : h_end[0];
      const bool per_head = s.w_shead != 0;
      if (pass == 0 || pass == n_pass[0]) set_factors(which);
      // the next pass's loads are in flight during this one (its heads are others, so in place they are unwritten)
      Raw8<TI> nv[kWide][2];
#pragma unroll
      for (int k = 0; k < kWide; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) nv[k][i] = v[k][i];
      const int64_t row = tok;
      if (pass + 1 < passes) {
        fetch(pass + 1, nv);
      } else if (kLoop && task + stride < tasks) {  // the next task's first
        task += stride;
        take();
        task -= stride;
        pos = position(tok);
        fetch(0, nv);
      }
      TO* const y = static_cast<TO*>(s.y) + row * s.y_srow;
#pragma unroll
      for (int k = 0; k < kWide; ++k) {
        uint64_t x[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = v[k][i].pair(e);
        float scale = 1.f;
        if (p.norm) {
          uint64_t sq2 = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sq2 = fma_f32x2(x[i][e], x[i][e], sq2);
          const float2 sq = unpack_f32x2(sq2);
          float sum = used ? sq.x + sq.y : 0.f;
#pragma unroll
          for (int m = 1; m < kLanes; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          scale = rsqrtf(fmaf(sum, 1.f / D, p.eps));
        }
        const int h = h0 + k * kHeads + sub;
        if (h >= end || !used) continue;
        if (per_head) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = mul_f32x2(x[i][e], weight_pair(s, h * s.w_shead + ch[i] + 2 * e));
        }
        const uint64_t scale2 = pack_f32x2(scale, scale);
        TO* const yh = y + h * s.y_shead;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint64_t out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = mul_f32x2(x[i][e], fa[i][e]);
          if (rot[i]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = fma_f32x2(kInter ? swapped(x[i][e]) : x[1 - i][e], fb[i][e], out[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = mul_f32x2(out[e], scale2);
          store8(yh + ch[i], out);
        }
      }
#pragma unroll
      for (int k = 0; k < kWide; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) v[k][i] = nv[k][i];
    }
    if (!kLoop || (task += stride) >= tasks) break;
  }
}

// CTAs that fit on the GPU (four on each of 152 SMs).
constexpr int64_t kResident = 608;

template <typename TI, typename TO, int D, bool kLoop>
void launch_one(const NormRopeParams& p, int64_t ctas, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(kLoop ? kResident : ctas));
  if (p.interleaved)
    qk_norm_rope_kernel<TI, TO, D, true, kLoop><<<grid, kThreads, 0, stream>>>(p);
  else
    qk_norm_rope_kernel<TI, TO, D, false, kLoop><<<grid, kThreads, 0, stream>>>(p);
}

// bf16 heads of 64 and 128 channels loop where there are more tokens than the GPU holds warps: 32768 tokens of 64/8
// heads of 64 take 101 us so and 107 with a CTA for every four tokens, 16000 of 8/1 19 and 20.  Heads of 192 have
// no registers for it (291 and 273 us for 8191 tokens of 128/128), fp32 gains nothing, small calls lose 0.3 us.
template <typename TI, typename TO, int D>
cudaError_t launch_d(const NormRopeParams& p, int64_t ctas, cudaStream_t stream) {
  if constexpr (sizeof(TI) == 2 && D != 192) {
    if (ctas > kResident) {
      launch_one<TI, TO, D, true>(p, ctas, stream);
      return cudaGetLastError();
    }
  }
  launch_one<TI, TO, D, false>(p, ctas, stream);
  return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t launch(const NormRopeParams& p, int d, int64_t ctas, cudaStream_t stream) {
  if (d == 64) return launch_d<TI, TO, 64>(p, ctas, stream);
  if (d == 128) return launch_d<TI, TO, 128>(p, ctas, stream);
  return launch_d<TI, TO, 192>(p, ctas, stream);
}

bool strides8(const slope_tensor* t) {
  return t->stride[2] == 1 && t->stride[0] > 0 && t->stride[1] > 0 && t->stride[0] % 8 == 0 && t->stride[1] % 8 == 0 &&
         aligned(t->data, 16);
}

// An input and its output, of the same shape.
slope_status check_pair(const slope_tensor* x, const slope_tensor* y) {
  if (y == nullptr) return SLOPE_ERR_NULL;
  for (const slope_tensor* t : {x, y}) {
    if (t->dtype != SLOPE_BF16 && t->dtype != SLOPE_F32) return SLOPE_ERR_DTYPE;
    if (t->ndim != 3) return SLOPE_ERR_SHAPE;
  }
  for (int i = 0; i < 3; ++i)
    if (x->shape[i] != y->shape[i]) return SLOPE_ERR_SHAPE;
  if (x->shape[0] < 0 || x->shape[0] > (int64_t(1) << 30) || x->shape[1] <= 0 || x->shape[1] > 65535)
    return SLOPE_ERR_SHAPE;
  const int64_t d = x->shape[2];
  if (d != 64 && d != 128 && d != 192) return SLOPE_ERR_UNSUPPORTED;
  if (x->shape[0] == 0) return SLOPE_OK;
  if (x->data == nullptr || y->data == nullptr) return SLOPE_ERR_NULL;
  if (!strides8(x) || !strides8(y)) return SLOPE_ERR_STRIDE;
  // in place means element for element; anything else a thread could overwrite unread values with
  if (x->data == y->data &&
      (x->dtype != y->dtype || x->stride[0] != y->stride[0] || x->stride[1] != y->stride[1]))
    return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

slope_status check_weight(const slope_tensor* w, int norm, int64_t H, int64_t d) {
  if (w == nullptr) return SLOPE_OK;
  if (!norm) return SLOPE_ERR_UNSUPPORTED;
  if (w->dtype != SLOPE_BF16 && w->dtype != SLOPE_F32) return SLOPE_ERR_DTYPE;
  if (w->ndim != 2 || (w->shape[0] != 1 && w->shape[0] != H) || w->shape[1] != d) return SLOPE_ERR_SHAPE;
  if (w->data == nullptr) return SLOPE_ERR_NULL;
  if (w->stride[1] != 1 || (w->shape[0] > 1 && w->stride[0] <= 0)) return SLOPE_ERR_STRIDE;
  if (!aligned(w->data, w->dtype == SLOPE_F32 ? 4 : 2)) return SLOPE_ERR_STRIDE;
  return SLOPE_OK;
}

}  // namespace
}  // namespace slope

using namespace slope;

extern "C" slope_status slope_qk_norm_rope(const slope_tensor* q, const slope_tensor* k, const slope_tensor* q_weight,
                                           const slope_tensor* k_weight, int norm, float eps, const slope_rope* rope,
                                           const int32_t* positions, int64_t pos0, slope_tensor* q_out,
                                           slope_tensor* k_out, void* stream) {
  const CallRange range("slope_qk_norm_rope");
  const slope_tensor* x[2] = {q, k};
  const slope_tensor* w[2] = {q_weight, k_weight};
  slope_tensor* y[2] = {q_out, k_out};
  if (q == nullptr && k == nullptr) return SLOPE_ERR_NULL;
  const slope_tensor *first = nullptr, *first_out = nullptr;
  NormRopeParams p{};
  for (int i = 0; i < 2; ++i) {
    if (x[i] == nullptr) {
      if (y[i] != nullptr || w[i] != nullptr) return SLOPE_ERR_NULL;
      continue;
    }
    slope_status st = check_pair(x[i], y[i]);
    if (st != SLOPE_OK) return st;
    if ((st = check_weight(w[i], norm, x[i]->shape[1], x[i]->shape[2])) != SLOPE_OK) return st;
    if (first == nullptr) {
      first = x[i];
      first_out = y[i];
    } else {
      if (x[i]->dtype != first->dtype || y[i]->dtype != first_out->dtype) return SLOPE_ERR_DTYPE;
      if (x[i]->shape[0] != first->shape[0] || x[i]->shape[2] != first->shape[2]) return SLOPE_ERR_SHAPE;
    }
    NormRopeSide& s = p.side[i];
    s.x = x[i]->data;
    s.y = y[i]->data;
    s.x_srow = x[i]->stride[0], s.x_shead = x[i]->stride[1];
    s.y_srow = y[i]->stride[0], s.y_shead = y[i]->stride[1];
    s.H = static_cast<int32_t>(x[i]->shape[1]);
    if (w[i] != nullptr) {
      s.w = w[i]->data;
      s.w_bf16 = w[i]->dtype == SLOPE_BF16 ? 1 : 0;
      s.w_shead = w[i]->shape[0] > 1 ? w[i]->stride[0] : 0;
    }
  }
  if (norm && !(eps >= 0.f && std::isfinite(eps))) return SLOPE_ERR_SHAPE;
  const int64_t T = first->shape[0];
  const int d = static_cast<int>(first->shape[2]);
  if (rope != nullptr) {
    if (rope->inv_freq == nullptr) return SLOPE_ERR_NULL;
    if (rope->dim < 16 || rope->dim % 16 != 0 || rope->begin < 0 || rope->begin % 8 != 0 || rope->begin > d - rope->dim)
      return SLOPE_ERR_SHAPE;
    if (!std::isfinite(rope->attention_factor)) return SLOPE_ERR_SHAPE;
    constexpr int64_t kPos = int64_t(1) << 31;
    if (positions == nullptr && (pos0 < -kPos || pos0 > kPos - T)) return SLOPE_ERR_SHAPE;
    p.rotate = 1;
    p.begin = rope->begin;
    p.half = rope->dim / 2;
    p.interleaved = rope->interleaved != 0 ? 1 : 0;
    p.factor = rope->attention_factor;
    for (int i = 0; i < p.half; ++i) {
      if (!std::isfinite(rope->inv_freq[i])) return SLOPE_ERR_SHAPE;
      const double t = rope->inv_freq[i] / 6.283185307179586476925286766559;
      const double turns = (t - std::floor(t)) * 0x1p64;
      p.turns[i] = turns < 0x1p64 ? static_cast<uint64_t>(turns) : 0;
    }
  }
  if (T == 0) return SLOPE_OK;
  if (!aligned(positions, 4)) return SLOPE_ERR_STRIDE;
  p.T = T;
  p.positions = positions;
  p.pos0 = pos0;
  p.eps = eps;
  p.norm = norm != 0 ? 1 : 0;
  const int64_t H = p.side[0].H + p.side[1].H;
  // A warp to a token once there are enough tokens to fill the GPU (about 32 warps on each of 152 SMs),
  // else several warps, down to the heads of one pass each, for the shortest call.
  const int64_t want = (H * T + 4863) / 4864;
  const int64_t at_once = d == 192 ? 6 : heads_per_pass(d);
  p.heads = static_cast<int32_t>(std::min((H + at_once - 1) / at_once, (want + at_once - 1) / at_once) * at_once);
  p.splits = static_cast<int32_t>((H + p.heads - 1) / p.heads);
  const int64_t ctas = (T * p.splits + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffLL) return SLOPE_ERR_SHAPE;
  auto s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (first->dtype == SLOPE_BF16)
    e = first_out->dtype == SLOPE_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, d, ctas, s)
                                       : launch<__nv_bfloat16, float>(p, d, ctas, s);
  else
    e = first_out->dtype == SLOPE_BF16 ? launch<float, __nv_bfloat16>(p, d, ctas, s)
                                       : launch<float, float>(p, d, ctas, s);
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("norm and rotation kernel launch", e);
}
