// scout_rope_turns: the frequencies of rotary positions as fractions of 2^64 of a turn (host code).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "scout.h"

namespace {
constexpr double kTwoPi = 6.283185307179586476925286766559;
bool positive(double v) { return std::isfinite(v) && v > 0.0; }
}  // namespace

extern "C" int scout_rope_turns(double base, int rot_dim, const scout_rope_scaling* scaling, uint64_t* turns,
                                float* amplitude) {
  if (turns == nullptr || amplitude == nullptr || !std::isfinite(base) || !(base > 1.0)) return SCOUT_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16 != 0) return SCOUT_ERR_UNSUPPORTED;
  const int pairs = rot_dim / 2;
  const int kind = scaling != nullptr ? scaling->kind : 0;
  double amp = 1.0, first = 0.0, last = 1.0;  // INDEX: the pairs between which the slowing sets in
  if (scaling != nullptr) {
    const scout_rope_scaling& s = *scaling;
    if (kind < SCOUT_ROPE_LINEAR || kind > SCOUT_ROPE_DIVISORS) return SCOUT_ERR_INVALID_ARG;
    if (kind != SCOUT_ROPE_DIVISORS && !positive(s.factor)) return SCOUT_ERR_INVALID_ARG;
    if ((kind == SCOUT_ROPE_ROTATIONS || kind == SCOUT_ROPE_INDEX) &&
        (!positive(s.original) || !positive(s.low) || !std::isfinite(s.high) || !(s.high > s.low)))
      return SCOUT_ERR_INVALID_ARG;
    if (kind == SCOUT_ROPE_DIVISORS) {
      if (s.divisors == nullptr) return SCOUT_ERR_INVALID_ARG;
      for (int i = 0; i < pairs; ++i)
        if (!positive(s.divisors[i])) return SCOUT_ERR_INVALID_ARG;
    }
    if (!std::isfinite(s.amplitude) || s.amplitude < 0.0) return SCOUT_ERR_INVALID_ARG;
    if (s.amplitude > 0.0)
      amp = s.amplitude;
    else if (kind == SCOUT_ROPE_INDEX && s.factor > 1.0)
      amp = 0.1 * std::log(s.factor) + 1.0;
    if (kind == SCOUT_ROPE_NTK) base *= std::pow(s.factor, (double)rot_dim / (rot_dim - 2));
    if (kind == SCOUT_ROPE_INDEX) {
      auto at = [&](double n) { return rot_dim * std::log(s.original / (kTwoPi * n)) / (2.0 * std::log(base)); };
      first = std::fmax(std::floor(at(s.high)), 0.0);
      last = std::fmin(std::ceil(at(s.low)), rot_dim - 1.0);
    }
  }
  if (!std::isfinite(base) || amp > (double)std::numeric_limits<float>::max()) return SCOUT_ERR_INVALID_ARG;
  uint64_t made[64];
  for (int i = 0; i < pairs; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    switch (kind) {
      case SCOUT_ROPE_LINEAR: f /= scaling->factor; break;
      case SCOUT_ROPE_ROTATIONS: {
        const double k = (scaling->original * f / kTwoPi - scaling->low) / (scaling->high - scaling->low);
        const double keep = std::fmin(std::fmax(k, 0.0), 1.0);
        f = keep * f + (1.0 - keep) * f / scaling->factor;
        break;
      }
      case SCOUT_ROPE_INDEX: {
        const double slow = std::fmin(std::fmax((i - first) / std::fmax(last - first, 1e-3), 0.0), 1.0);
        f = (1.0 - slow) * f + slow * f / scaling->factor;
        break;
      }
      case SCOUT_ROPE_DIVISORS: f /= scaling->divisors[i]; break;
      default: break;
    }
    const double t = f / kTwoPi;
    if (!std::isfinite(t)) return SCOUT_ERR_INVALID_ARG;  // a factor or divisor too small for its frequency
    // below 2^64: t - floor(t) is at most 1 - 2^-53
    made[i] = (uint64_t)std::ldexp(t - std::floor(t), 64);
  }
  std::copy(made, made + pairs, turns);
  *amplitude = (float)amp;
  return SCOUT_OK;
}
