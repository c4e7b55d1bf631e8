// Host frequencies of the rotary position embedding.
//
// Pair i of a head's rotated part turns by position * theta_i radians, theta_i
// = base^(-2i/rotary_dim), theta changed for contexts longer than the model
// was trained on (pa_rope_scaling).  The kernels take the frequencies as
// 64-bit fixed-point turns per position: position * turns modulo 2^64 is the
// fraction of a turn, exactly, at any position, where the product of a
// position of 10^5 and a 32-bit theta is off by 10^-2 radians.
//
// All arithmetic is in double, so the result does not depend on the host.
#include <cmath>
#include <cstdint>

#include "pa_kv.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool positive(double x) { return std::isfinite(x) && x > 0.0; }

// turns per position as a fraction of 2^64 (whole turns leave no trace).  Of a
// negative theta, the complement of -theta's: t - floor(t) would round a small
// one to 53 bits next to 1, off by 2^-54 of a turn at every position.
uint64_t fixed_turns(double theta) {
    const double t = std::fabs(theta) / kTwoPi;
    const double frac = std::floor(std::ldexp(t - std::floor(t), 64) + 0.5);
    const uint64_t turns = frac >= 18446744073709551616.0 ? 0ull : static_cast<uint64_t>(frac);
    return theta < 0.0 ? 0ull - turns : turns;
}

}  // namespace

extern "C" pa_status pa_rope_frequencies(int32_t rotary_dim, double base, const pa_rope_scaling* scaling,
                                         double* inv_freq, uint64_t* turns, float* rope_factor) {
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || inv_freq == nullptr || turns == nullptr || rope_factor == nullptr)
        return PA_ERR_INVALID_ARG;
    const int n = rotary_dim / 2;
    const pa_rope_scaling none = {PA_ROPE_NONE, 1.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    const pa_rope_scaling& s = scaling != nullptr ? *scaling : none;
    const int kind = static_cast<int>(s.kind);
    if (kind < PA_ROPE_NONE || kind > PA_ROPE_GIVEN) return PA_ERR_UNSUPPORTED;
    *rope_factor = 1.f;
    if (kind == PA_ROPE_GIVEN) {
        for (int i = 0; i < n; ++i)
            if (!std::isfinite(inv_freq[i])) return PA_ERR_INVALID_ARG;
        for (int i = 0; i < n; ++i) turns[i] = fixed_turns(inv_freq[i]);
        return PA_OK;
    }
    if (!positive(base) || base <= 1.0) return PA_ERR_INVALID_ARG;
    if (kind != PA_ROPE_NONE && !(positive(s.factor) && s.factor >= 1.0)) return PA_ERR_INVALID_ARG;
    if ((kind == PA_ROPE_YARN || kind == PA_ROPE_BANDED) && !positive(s.original_max_position))
        return PA_ERR_INVALID_ARG;
    double b = base;
    if (kind == PA_ROPE_NTK) {
        // the base grows so that the slowest pair is stretched by `factor`
        // and the fastest one not at all
        if (rotary_dim <= 2) return PA_ERR_INVALID_ARG;
        b = base * std::pow(s.factor, rotary_dim / (rotary_dim - 2.0));
    }
    double lo = 0.0, hi = 0.0;
    if (kind == PA_ROPE_YARN) {
        // pair index at which the original context holds beta turns; between
        // the two indices the frequencies go linearly from kept to divided
        if (!positive(s.beta_fast) || !positive(s.beta_slow) || s.beta_fast < s.beta_slow) return PA_ERR_INVALID_ARG;
        const double per = rotary_dim / (2.0 * std::log(base));
        lo = std::floor(per * std::log(s.original_max_position / (s.beta_fast * kTwoPi)));
        hi = std::ceil(per * std::log(s.original_max_position / (s.beta_slow * kTwoPi)));
        lo = lo < 0.0 ? 0.0 : lo;
        hi = hi > rotary_dim - 1.0 ? rotary_dim - 1.0 : hi;
        *rope_factor = static_cast<float>(0.1 * std::log(s.factor) + 1.0);
    }
    if (kind == PA_ROPE_BANDED && !(positive(s.low_freq_factor) && positive(s.high_freq_factor) &&
                                    s.high_freq_factor > s.low_freq_factor))
        return PA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        double th = std::pow(b, -2.0 * i / rotary_dim);
        if (kind == PA_ROPE_LINEAR) {
            th /= s.factor;
        } else if (kind == PA_ROPE_YARN) {
            const double span = hi - lo > 0.001 ? hi - lo : 0.001;
            double r = (i - lo) / span;
            r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
            th = th / s.factor * r + th * (1.0 - r);
        } else if (kind == PA_ROPE_BANDED) {
            // turns of this pair over the original context
            const double c = s.original_max_position * th / kTwoPi;
            double w = (c - s.low_freq_factor) / (s.high_freq_factor - s.low_freq_factor);
            w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
            th = (1.0 - w) * th / s.factor + w * th;
        }
        inv_freq[i] = th;
        turns[i] = fixed_turns(th);
    }
    return PA_OK;
}
