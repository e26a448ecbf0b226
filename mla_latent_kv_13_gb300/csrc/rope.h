// rope.h -- host side of the rotation's frequencies, and the rotation of heads.
#pragma once

#include <cmath>

#include "common.cuh"

namespace mla {

// theta^(-2i/64), i = 0..31, in double
inline RopeFreqs rope_freqs(float theta) {
    RopeFreqs r;
    for (int i = 0; i < D_ROPE / 2; ++i)
        r.f[i] = std::pow(static_cast<double>(theta), -2.0 * i / static_cast<double>(D_ROPE));
    return r;
}

// Rotation of each pair per position, in turns: the fraction as a 64-bit fixed-point number, so
// that a position's angle modulo a turn is one integer product, exact but for the constant's own
// 2^-65 (fp64, which would do for the product, is slow on this part: it took half the kernel's time).
template <int N>
struct TurnTable {
    uint64_t f[N];
};
using TurnFreqs = TurnTable<D_ROPE / 2>;
inline uint64_t turn_freq(double w) {
    // w / (2 pi) as two doubles, then its fraction
    const double hi = w * 0.15915494309189535;
    const double lo = std::fma(w, 0.15915494309189535, -hi) + w * -9.839338337591243e-18;
    const double frac = hi - std::floor(hi);
    return static_cast<uint64_t>(frac * 0x1p64) +
           static_cast<uint64_t>(static_cast<int64_t>((lo - std::floor(lo + 0.5)) * 0x1p64));
}
inline TurnFreqs turn_freqs(float theta) {
    const RopeFreqs w = rope_freqs(theta);
    TurnFreqs r;
    for (int i = 0; i < D_ROPE / 2; ++i) r.f[i] = turn_freq(w.f[i]);
    return r;
}
template <int N>
inline TurnTable<N> turn_table(const mla_rope_t &plan) {
    TurnTable<N> r{};
    for (int i = 0; i < plan.rot / 2 && i < N; ++i) r.f[i] = turn_freq(plan.freq[i]);
    return r;
}
// whether a plan's fields can be used (its frequencies up to rot / 2)
inline bool plan_ok(const mla_rope_t &plan) {
    if (plan.rot < 2 || plan.rot > MLA_ROPE_MAX || plan.rot % 2 ||
        (plan.layout != MLA_ROPE_INTERLEAVED && plan.layout != MLA_ROPE_HALF) ||
        !std::isfinite(plan.magnitude))
        return false;
    for (int i = 0; i < plan.rot / 2; ++i)
        if (!(plan.freq[i] >= 0. && plan.freq[i] <= MLA_ROPE_MAX_FREQ)) return false;
    return true;
}

struct RopeParams {
    const uint16_t *x;  // [tokens][heads][width], strides in values
    long x_token, x_head;
    int tokens, heads, width, offset;
    const int32_t *pos;
    uint16_t *y;  // [tokens][heads][rot]
    long y_token, y_head;
    uint16_t *rest;  // [tokens][heads][width - rot], or null
    long rest_token, rest_head;
};
cudaError_t launch_rope(const RopeParams &p, const mla_rope_t &plan, cudaStream_t stream);

}  // namespace mla
