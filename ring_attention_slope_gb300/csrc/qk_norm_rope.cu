// RMS norm of every query and key head and the rotation by position, in one
// pass: y = x / sqrt(mean(x^2) + eps) * w, then the pairs (a, b) of the rotated
// channels become (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq.
//
// Bandwidth-bound: every value is read once and written once.  Eight lanes
// share a head, each with 16-byte loads of 8 channels (d / 64 of them), so a
// warp's load instruction covers four heads' consecutive 128 bytes.  A CTA
// takes a few tokens and first puts the sines and cosines of their angles in
// shared memory, where all heads use them; the angles are the only arithmetic
// that would show (two of them per pair of channels would cost more than the
// memory pass).
//
// Angles: position * inv_freq loses everything in fp32 at far positions (at
// position 10^6 an fp32 angle is off by 0.06 radians).  The frequency is kept as
// turns per position in 64-bit fixed point, so the product's low 64 bits are the
// fraction of a turn, exactly, with no reduction.
//
// Halves layout: a lane needs the channels half a rotation away, which another
// lane loads too.  It loads them again (they hit L1) rather than shuffle, since
// with rotated parts of any size they may sit in any lane and register.
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

constexpr int kThreads = 256;
constexpr int kLanesPerHead = 8;
constexpr int kRowsPerPass = kThreads / kLanesPerHead;  // heads a CTA takes at a time
constexpr int kMaxHalf = 96;                            // rotated pairs of a head
constexpr int kMaxTokens = 4;                           // tokens of a CTA

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
  int32_t tokens;  // of a CTA
  int32_t heads;   // of a CTA (of side[0].H + side[1].H)
  uint64_t turns[kMaxHalf];  // inv_freq / 2 pi modulo 1, times 2^64
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 r = *reinterpret_cast<const float4*>(p + 4 * i);
      v[4 * i] = r.x, v[4 * i + 1] = r.y, v[4 * i + 2] = r.z, v[4 * i + 3] = r.w;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float weight_at(const NormRopeSide& s, int64_t i) {
  if (s.w == nullptr) return 1.f;
  return s.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(s.w)[i]) : static_cast<const float*>(s.w)[i];
}

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ __align__(16) float s_cos[kMaxTokens * kMaxHalf], s_sin[kMaxTokens * kMaxHalf];
  __shared__ __align__(16) float s_w[2 * D];  // weights shared by every head of a side
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - t0));
  const int h0 = blockIdx.y * p.heads;
  const int n_heads = min(p.heads, p.side[0].H + p.side[1].H - h0);

  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const NormRopeSide& s = p.side[i / D];
    s_w[i] = s.w_shead == 0 ? weight_at(s, i % D) : 1.f;
  }
  if (p.rotate) {
    for (int i = threadIdx.x; i < n_tok * p.half; i += kThreads) {
      const int tok = i / p.half, f = i - tok * p.half;
      const int64_t pos = p.positions != nullptr ? p.positions[t0 + tok] : p.pos0 + t0 + tok;
      // the fraction of a turn, rounded to 32 bits and taken in [-1/2, 1/2)
      const uint64_t frac = p.turns[f] * static_cast<uint64_t>(pos) + 0x80000000ull;
      const int32_t turn = static_cast<int32_t>(frac >> 32);
      float sn, cs;
      sincospif(static_cast<float>(turn) * 0x1p-31f, &sn, &cs);
      s_cos[tok * kMaxHalf + f] = cs * p.factor;
      s_sin[tok * kMaxHalf + f] = sn * p.factor;
    }
  }
  __syncthreads();

  constexpr int kChunks = D / 64;
  const int lane8 = threadIdx.x % kLanesPerHead;
  const int n_rows = n_tok * n_heads;
  // every thread runs every pass: the shuffles below need whole warps
  for (int r0 = 0; r0 < n_rows; r0 += kRowsPerPass) {
    const int r = r0 + threadIdx.x / kLanesPerHead;
    const bool live = r < n_rows;
    const int tok = live ? r / n_heads : 0;
    const int hh = h0 + (live ? r - tok * n_heads : 0);
    const int which = hh >= p.side[0].H ? 1 : 0;
    const NormRopeSide& s = p.side[which];
    const int h = which ? hh - p.side[0].H : hh;
    const TI* x = static_cast<const TI*>(s.x) + (t0 + tok) * s.x_srow + h * s.x_shead;
    float v[kChunks][8], o[kChunks][8];  // own channels, and their partners in the halves layout
    int side_of[kChunks];                // 0 not rotated, 1 first half, 2 second half, 3 interleaved
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = c * 64 + lane8 * 8;
      side_of[c] = 0;
      if (live) {
        load8(x + e, v[c]);
        if (p.rotate && e >= p.begin && e < p.begin + 2 * p.half) {
          side_of[c] = p.interleaved ? 3 : e < p.begin + p.half ? 1 : 2;
          if (!p.interleaved) load8(x + (side_of[c] == 1 ? e + p.half : e - p.half), o[c]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(v[c][i], v[c][i], sq);
    }
    float scale = 1.f;
    if (p.norm) {
#pragma unroll
      for (int m = 1; m < kLanesPerHead; m <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
      scale = rsqrtf(sq * (1.f / D) + p.eps);
    }
    __syncwarp();  // in place: every lane has read what it needs of the head
    if (!live) continue;
    TO* y = static_cast<TO*>(s.y) + (t0 + tok) * s.y_srow + h * s.y_shead;
    const float* sw = s_w + which * D;
    const bool per_head = s.w_shead != 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = c * 64 + lane8 * 8;
      auto apply = [&](float (&a)[8], int at) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          a[i] *= scale * (per_head ? weight_at(s, h * s.w_shead + at + i) : sw[at + i]);
      };
      if (p.norm) apply(v[c], e);
      if (side_of[c] == 1 || side_of[c] == 2) {
        const int po = side_of[c] == 1 ? e + p.half : e - p.half;
        if (p.norm) apply(o[c], po);
        const int f0 = tok * kMaxHalf + (side_of[c] == 1 ? e : po) - p.begin;
        const float sign = side_of[c] == 1 ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = fmaf(sign * o[c][i], s_sin[f0 + i], v[c][i] * s_cos[f0 + i]);
      } else if (side_of[c] == 3) {
        const int f0 = tok * kMaxHalf + (e - p.begin) / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = v[c][2 * i], b = v[c][2 * i + 1];
          v[c][2 * i] = fmaf(-b, s_sin[f0 + i], a * s_cos[f0 + i]);
          v[c][2 * i + 1] = fmaf(a, s_sin[f0 + i], b * s_cos[f0 + i]);
        }
      }
      store8(y + e, v[c]);
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_d(const NormRopeParams& p, int d, dim3 grid, cudaStream_t stream) {
  if (d == 64) qk_norm_rope_kernel<TI, TO, 64><<<grid, kThreads, 0, stream>>>(p);
  if (d == 128) qk_norm_rope_kernel<TI, TO, 128><<<grid, kThreads, 0, stream>>>(p);
  if (d == 192) qk_norm_rope_kernel<TI, TO, 192><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
      p.turns[i] = static_cast<uint64_t>(std::ldexp(t - std::floor(t), 64) < 0x1p64 ? std::ldexp(t - std::floor(t), 64) : 0.0);
    }
  }
  if (T == 0) return SLOPE_OK;
  p.T = T;
  p.positions = positions;
  p.pos0 = pos0;
  p.eps = eps;
  p.norm = norm != 0 ? 1 : 0;
  const int64_t H = p.side[0].H + p.side[1].H;
  // Few heads in all: one token and one pass of heads to a CTA, for the shortest call.  Else several
  // tokens with all their heads, so that the angles and weights are fetched once for many passes.
  const int64_t passes = (H + kRowsPerPass - 1) / kRowsPerPass;
  const bool small = T * passes <= 1216;  // a wave of 8 CTAs on each of the 152 SMs
  p.tokens = small ? 1 : kMaxTokens;
  p.heads = small ? kRowsPerPass : static_cast<int32_t>(H);
  const dim3 grid(static_cast<unsigned>((T + p.tokens - 1) / p.tokens),
                  static_cast<unsigned>((H + p.heads - 1) / p.heads));
  auto s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (first->dtype == SLOPE_BF16)
    e = first_out->dtype == SLOPE_BF16 ? launch_d<__nv_bfloat16, __nv_bfloat16>(p, d, grid, s)
                                       : launch_d<__nv_bfloat16, float>(p, d, grid, s);
  else
    e = first_out->dtype == SLOPE_BF16 ? launch_d<float, __nv_bfloat16>(p, d, grid, s)
                                       : launch_d<float, float>(p, d, grid, s);
  return e == cudaSuccess ? SLOPE_OK : cuda_fail("norm and rotation kernel launch", e);
}
