// RMS norm of every query and key head and the rotation by position, in one
// pass: y = x / sqrt(mean(x^2) + eps) * w, then the pairs (a, b) of the rotated
// channels become (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq.
//
// Bandwidth-bound: every value is read once and written once.  Eight lanes
// share a head, each with 16-byte loads of 8 channels (d / 64 of them), so a
// warp's load instruction covers four heads' consecutive 128 bytes.  A warp takes
// one token and runs over its heads: the weights and the token's sines and cosines
// are then the same for every head of a lane, and stay in its registers as
//   y_e = (x_e A_e + x_partner B_e) / rms,   A = w cos, B = -+ w_partner sin.
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

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kLanesPerHead = 8;
constexpr int kHeadsPerPass = 32 / kLanesPerHead;  // heads a warp takes at a time
constexpr int kMaxHalf = 96;                       // rotated pairs of a head

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

// A lane's factors for its channels: y_e = (x_e a_e + x_partner b_e) / rms.
template <int kChunks>
struct Factors {
  uint64_t a[kChunks][4], b[kChunks][4];
};

// kInter: pairs are neighbours (and a pair's partner is in the same lane's channels), else halves.
template <typename TI, typename TO, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, D == 64 ? 6 : 4)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ __align__(16) float s_cos[kWarps][kMaxHalf], s_sin[kWarps][kMaxHalf];  // of the warp's token
  __shared__ __align__(16) float s_w[2][D];  // weights shared by every head of a side, else 1
  constexpr int kChunks = D / 64;
  constexpr int kWide = D == 64 && sizeof(TI) == 2 ? 2 : 1;  // groups of four heads in a pass
  // a 64-channel bf16 head lies in one 16-byte word of its eight lanes: the other half comes by shuffle
  constexpr bool kShuffle = D == 64 && sizeof(TI) == 2 && !kInter;
  constexpr bool kLoadPartner = !kInter && !kShuffle;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int lane8 = lane % kLanesPerHead, sub = lane / kLanesPerHead;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t tok = task / p.splits;
  const bool here = tok < p.T;
  const int split = static_cast<int>(task - tok * p.splits);
  const int first = split * p.heads, last = here ? min(first + p.heads, p.side[0].H + p.side[1].H) : first;
  // the warp's heads of either side, and the passes they take
  int h_begin[2], h_end[2], n_pass[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int base = w ? p.side[0].H : 0;
    h_begin[w] = max(first - base, 0);
    h_end[w] = min(last - base, p.side[w].H);
    n_pass[w] = h_begin[w] < h_end[w] ? (h_end[w] - h_begin[w] + kHeadsPerPass * kWide - 1) / (kHeadsPerPass * kWide) : 0;
  }
  // elements from a chunk of the lane to the other half of its pairs (0: not rotated; 1: neighbours)
  int partner[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int off = c * 64 + lane8 * 8 - p.begin;
    partner[c] = !p.rotate || off < 0 || off >= 2 * p.half ? 0 : kInter ? 1 : off < p.half ? p.half : -p.half;
  }
  Raw8<TI> v[kWide][kChunks], o[kWide][kChunks];
#pragma unroll
  for (int k = 0; k < kWide; ++k)
#pragma unroll
    for (int c = 0; c < kChunks; ++c) o[k][c] = Raw8<TI>{};
  auto fetch = [&](int pass, Raw8<TI>(&fv)[kWide][kChunks], Raw8<TI>(&fo)[kWide][kChunks]) {
    const int w = pass >= n_pass[0] ? 1 : 0;
    const NormRopeSide& s = p.side[w];
    const int h0 = w ? h_begin[1] + (pass - n_pass[0]) * (kHeadsPerPass * kWide) : h_begin[0] + pass * (kHeadsPerPass * kWide);
    const TI* const x = static_cast<const TI*>(s.x) + tok * s.x_srow + lane8 * 8;
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
      // past the last head: its values once more, which are not stored
      const int h = min(h0 + k * kHeadsPerPass + sub, (w ? h_end[1] : h_end[0]) - 1);
      const TI* const xh = x + h * s.x_shead;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        fv[k][c].load(xh + c * 64);
        if (kLoadPartner && partner[c] != 0) fo[k][c].load(xh + c * 64 + partner[c]);
      }
    }
  };
  const int passes = n_pass[0] + n_pass[1];
  if (passes > 0) fetch(0, v, o);

  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const NormRopeSide& s = p.side[i / D];
    s_w[i / D][i % D] = s.w != nullptr && s.w_shead == 0 ? weight_at(s, i % D) : 1.f;
  }
  if (here && p.rotate) {
    const int64_t pos = p.positions != nullptr ? p.positions[tok] : p.pos0 + tok;
    for (int f = lane; f < p.half; f += 32) {
      // the fraction of a turn, rounded to 32 bits and taken in [-1/2, 1/2)
      const uint64_t frac = p.turns[f] * static_cast<uint64_t>(pos) + 0x80000000ull;
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &sn, &cs);
      s_cos[warp][f] = cs * p.factor;
      s_sin[warp][f] = sn * p.factor;
    }
  }
  __syncthreads();

  Factors<kChunks> f;
  auto set_factors = [&](int which) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = c * 64 + lane8 * 8, off = e - p.begin;
      const bool in = partner[c] != 0;
      float fa[8], fb[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&s_w[which][e + i]);
        fa[i] = w.x, fa[i + 1] = w.y, fa[i + 2] = w.z, fa[i + 3] = w.w;
        fb[i] = fb[i + 1] = fb[i + 2] = fb[i + 3] = 0.f;
      }
      if (in && kInter) {
        const float4 cs = *reinterpret_cast<const float4*>(&s_cos[warp][off / 2]);
        const float4 sn = *reinterpret_cast<const float4*>(&s_sin[warp][off / 2]);
        const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fb[2 * i] = -fa[2 * i + 1] * s4[i];
          fb[2 * i + 1] = fa[2 * i] * s4[i];
          fa[2 * i] *= c4[i];
          fa[2 * i + 1] *= c4[i];
        }
      } else if (in) {
        const int at = off < p.half ? off : off - p.half;
        const float sign = off < p.half ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 cs = *reinterpret_cast<const float4*>(&s_cos[warp][at + i]);
          const float4 sn = *reinterpret_cast<const float4*>(&s_sin[warp][at + i]);
          const float4 w = *reinterpret_cast<const float4*>(&s_w[which][e + i + partner[c]]);
          fb[i] = sign * sn.x * w.x, fb[i + 1] = sign * sn.y * w.y, fb[i + 2] = sign * sn.z * w.z, fb[i + 3] = sign * sn.w * w.w;
          fa[i] *= cs.x, fa[i + 1] *= cs.y, fa[i + 2] *= cs.z, fa[i + 3] *= cs.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f.a[c][i] = pack_f32x2(fa[2 * i], fa[2 * i + 1]);
        f.b[c][i] = pack_f32x2(fb[2 * i], fb[2 * i + 1]);
      }
    }
  };

#pragma unroll 1
  for (int pass = 0; pass < passes; ++pass) {
    const int which = pass >= n_pass[0] ? 1 : 0;
    const NormRopeSide& s = p.side[which];
    const int h0 = which ? h_begin[1] + (pass - n_pass[0]) * (kHeadsPerPass * kWide) : h_begin[0] + pass * (kHeadsPerPass * kWide);
    const int end = which ? h_end[1] : h_end[0];
    const bool per_head = s.w_shead != 0;
    if (pass == 0 || pass == n_pass[0]) set_factors(which);
    // the next pass's loads are in flight during this one (its heads are others, so in place they are unwritten)
    Raw8<TI> nv[kWide][kChunks], no[kWide][kChunks];
#pragma unroll
    for (int k = 0; k < kWide; ++k)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) nv[k][c] = v[k][c], no[k][c] = o[k][c];
    if (pass + 1 < passes) fetch(pass + 1, nv, no);
    float scale[kWide];
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
      scale[k] = 1.f;
      if (p.norm) {
        uint64_t sq2 = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) sq2 = fma_f32x2(v[k][c].pair(i), v[k][c].pair(i), sq2);
        const float2 sq = unpack_f32x2(sq2);
        float sum = sq.x + sq.y;
#pragma unroll
        for (int m = 1; m < kLanesPerHead; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        scale[k] = rsqrtf(fmaf(sum, 1.f / D, p.eps));
      }
    }
    if constexpr (kShuffle) {
      const int from = lane + partner[0] / 8;  // lanes that are not rotated get their own, and do not use it
#pragma unroll
      for (int k = 0; k < kWide; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) (&o[k][0].r[0].x)[i] = __shfl_sync(0xffffffffu, (&v[k][0].r[0].x)[i], from);
    }
    __syncwarp();  // in place: every lane has read what it needs of these heads
    TO* const y = static_cast<TO*>(s.y) + tok * s.y_srow + lane8 * 8;
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
      const int h = h0 + k * kHeadsPerPass + sub;
      if (h >= end) continue;
      const uint64_t scale2 = pack_f32x2(scale[k], scale[k]);
      TO* const yh = y + h * s.y_shead;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint64_t vv[4], oo[4], out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vv[i] = v[k][c].pair(i);
          oo[i] = kInter ? swapped(vv[i]) : o[k][c].pair(i);
        }
        if (per_head) {
          const int64_t wi = h * s.w_shead + c * 64 + lane8 * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vv[i] = mul_f32x2(vv[i], weight_pair(s, wi + 2 * i));
            if (!kInter && partner[c] != 0) oo[i] = mul_f32x2(oo[i], weight_pair(s, wi + 2 * i + partner[c]));
            if (kInter) oo[i] = swapped(vv[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = mul_f32x2(vv[i], f.a[c][i]);
        if (partner[c] != 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = fma_f32x2(oo[i], f.b[c][i], out[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = mul_f32x2(out[i], scale2);
        store8(yh + c * 64, out);
      }
    }
#pragma unroll
    for (int k = 0; k < kWide; ++k)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) v[k][c] = nv[k][c], o[k][c] = no[k][c];
  }
}

template <typename TI, typename TO>
cudaError_t launch_d(const NormRopeParams& p, int d, dim3 grid, cudaStream_t stream) {
  if (d == 64)
    p.interleaved ? qk_norm_rope_kernel<TI, TO, 64, true><<<grid, kThreads, 0, stream>>>(p)
                  : qk_norm_rope_kernel<TI, TO, 64, false><<<grid, kThreads, 0, stream>>>(p);
  else if (d == 128)
    p.interleaved ? qk_norm_rope_kernel<TI, TO, 128, true><<<grid, kThreads, 0, stream>>>(p)
                  : qk_norm_rope_kernel<TI, TO, 128, false><<<grid, kThreads, 0, stream>>>(p);
  else
    p.interleaved ? qk_norm_rope_kernel<TI, TO, 192, true><<<grid, kThreads, 0, stream>>>(p)
                  : qk_norm_rope_kernel<TI, TO, 192, false><<<grid, kThreads, 0, stream>>>(p);
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
  if (!aligned(positions, 4)) return SLOPE_ERR_STRIDE;
  p.T = T;
  p.positions = positions;
  p.pos0 = pos0;
  p.eps = eps;
  p.norm = norm != 0 ? 1 : 0;
  const int64_t H = p.side[0].H + p.side[1].H;
  // A warp to a token once there are enough tokens to fill the GPU (about 32 warps on each of 152 SMs),
  // else several warps, down to one pass of four heads each, for the shortest call.
  const int64_t want = (H * T + 4863) / 4864;
  p.heads = static_cast<int32_t>(std::min<int64_t>(
      (H + kHeadsPerPass - 1) / kHeadsPerPass, (want + kHeadsPerPass - 1) / kHeadsPerPass) * kHeadsPerPass);
  p.splits = static_cast<int32_t>((H + p.heads - 1) / p.heads);
  const int64_t ctas = (T * p.splits + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffLL) return SLOPE_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(ctas));
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
