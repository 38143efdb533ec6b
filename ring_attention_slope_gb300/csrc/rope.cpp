// Rotation frequencies on the host (slope_rope_inv_freq).
//
// Plain: inv_freq[i] = base^(-2 i / dim), radians per position.  The scalings
// stretch them for contexts longer than a model was trained on; each is its
// published formula, in doubles.
#include <algorithm>
#include <cmath>

#include "slope_serving.h"

namespace {
constexpr double kTwoPi = 6.283185307179586476925286766559;
}

extern "C" slope_status slope_rope_inv_freq(int32_t dim, double base, slope_rope_scaling scaling, double factor,
                                            double original, double fast, double slow, double* inv_freq,
                                            double* attention_factor) {
  if (inv_freq == nullptr) return SLOPE_ERR_NULL;
  if (dim < 4 || dim > 512 || dim % 2 != 0) return SLOPE_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return SLOPE_ERR_SHAPE;
  const int kind = static_cast<int>(scaling);
  if (kind < SLOPE_ROPE_PLAIN || kind > SLOPE_ROPE_YARN) return SLOPE_ERR_UNSUPPORTED;
  if (kind != SLOPE_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return SLOPE_ERR_SHAPE;
  const bool ramped = kind == SLOPE_ROPE_BANDS || kind == SLOPE_ROPE_YARN;
  if (ramped && !(original > 0.0 && std::isfinite(original) && slow > 0.0 && fast > slow && std::isfinite(fast)))
    return SLOPE_ERR_SHAPE;

  const int half = dim / 2;
  if (kind == SLOPE_ROPE_NTK) base *= std::pow(factor, static_cast<double>(dim) / (dim - 2));
  // YaRN's ramp ends: the (fractional) channel index whose frequency turns `n` times in `original` positions
  auto index_of = [&](double n) { return dim * std::log(original / (n * kTwoPi)) / (2.0 * std::log(base)); };
  double lo = 0.0, hi = 0.0;
  if (kind == SLOPE_ROPE_YARN) {
    lo = std::max(0.0, std::floor(index_of(fast)));
    hi = std::min(static_cast<double>(dim - 1), std::ceil(index_of(slow)));
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < half; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (kind == SLOPE_ROPE_LINEAR) {
      f /= factor;
    } else if (kind == SLOPE_ROPE_BANDS) {
      const double turns = original * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
      f = f * keep + f / factor * (1.0 - keep);
    } else if (kind == SLOPE_ROPE_YARN) {
      const double stretch = std::min(1.0, std::max(0.0, (i - lo) / (hi - lo)));
      f = f * (1.0 - stretch) + f / factor * stretch;
    }
    inv_freq[i] = f;
  }
  if (attention_factor != nullptr) *attention_factor = kind == SLOPE_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return SLOPE_OK;
}
