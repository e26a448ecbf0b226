// turn.cuh -- cos and sin of a position's angles.
#pragma once

#include <stdint.h>

namespace mla {

// cos and sin of `at` (in turns, as a 64-bit fraction) to about half an ulp. The angle is reduced to a
// quarter turn and at most pi / 4 (kept as two floats); there the Taylor polynomials to degrees 13 and
// 12 (remainders under 2^-40), whose leading terms take the rounding errors of x and x^2 along.
__device__ __forceinline__ void turn_by(uint64_t at, float &c, float &s) {
    at += 1ull << 61;
    const int q = static_cast<int>(at >> 62);  // nearest quarter; the rest as 24 + 24 bits
    const int64_t rest = static_cast<int64_t>(at & ((1ull << 62) - 1)) - (1ll << 61);
    const float a = static_cast<float>(static_cast<int>(rest >> 38));
    const float b = static_cast<float>(static_cast<int>(rest >> 14 & 0xFFFFFF));
    constexpr float PI2 = 6.2831854820251465f, PI2_LO = -1.7484555314695172e-07f;  // 2 pi
    constexpr float E26 = 1.f / (1 << 26), E50 = E26 / (1 << 24);
    const float p = a * (PI2 * E26);
    const float e = fmaf(b, PI2 * E50, fmaf(a, PI2_LO * E26, fmaf(a, PI2 * E26, -p)));
    const float x = p + e, xl = e - (x - p);
    const float z = x * x;
    // x^2 = z + zl
    const float zl = fmaf(2.f * x, xl, fmaf(x, x, -z));
    float ps = 1.60590438e-10f;           // 1 / 13!
    ps = fmaf(ps, z, -2.50521084e-8f);    // 1 / 11!
    ps = fmaf(ps, z, 2.75573192e-6f);     // 1 / 9!
    ps = fmaf(ps, z, -1.98412698e-4f);    // 1 / 7!
    ps = fmaf(ps, z, 8.33333333e-3f);     // 1 / 5!
    ps = fmaf(ps, z, -0.166666667f);      // 1 / 3!
    const float sn = x + fmaf(ps * z, x, fmaf(-0.5f * z, xl, xl));
    float pc = 2.08767570e-9f;            // 1 / 12!
    pc = fmaf(pc, z, -2.75573192e-7f);    // 1 / 10!
    pc = fmaf(pc, z, 2.48015873e-5f);     // 1 / 8!
    pc = fmaf(pc, z, -1.38888889e-3f);    // 1 / 6!
    pc = fmaf(pc, z, 4.16666667e-2f);     // 1 / 4!
    const float h = 0.5f * z, w = 1.f - h;
    const float cs = w + (((1.f - w) - h) + fmaf(pc * z, z, -0.5f * zl));
    const float u = q & 1 ? sn : cs, v = q & 1 ? cs : sn;
    c = q == 1 || q == 2 ? -u : u;
    s = q >= 2 ? -v : v;
}
// the same of pos turns of f
__device__ __forceinline__ void turn(uint32_t pos, uint64_t f, float &c, float &s) {
    turn_by(f * pos, c, s);
}

}  // namespace mla
