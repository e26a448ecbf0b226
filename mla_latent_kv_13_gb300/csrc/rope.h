// rope.h -- host side of the rotation's frequencies.
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

}  // namespace mla
