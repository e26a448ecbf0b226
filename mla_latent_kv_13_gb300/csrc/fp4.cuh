// fp4.cuh -- the 4-bit latent cache: e2m1 codes with an e4m3 scale for each 16 latent values of a
// token and one exponent for the token.
//
//   value = level(code) * scale * 2^e,  levels 0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives
// A level has two significant bits and a scale four, so a value has six at most: it is exactly a bf16
// value (at and above 2^-130: 2^-1 * 2^-9 * 2^-120).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "fp8.cuh"

namespace mla {

constexpr int FP4_GROUP = 16;                    // latent values of a scale
constexpr int FP4_GROUPS = D_C / FP4_GROUP;      // 32: one for each lane of a warp
constexpr int FP4_E_MIN = -120, FP4_E_MAX = 117;  // exponents that finite bf16 rows give

struct Fp4Group {
    uint2 codes;  // the first value in the lowest four bits
    uint8_t scale;
};

// Exponent of a token from its largest magnitude mx (finite, exactly a bf16 value): the smallest e
// with mx <= 6 * 448 * 2^e, 6 * 448 = 0.65625 * 2^12.
__device__ __forceinline__ int fp4_row_exp(float mx) {
    if (!(mx > 0.f)) return 0;
    int k;
    const float f = frexpf(mx, &k);
    return max(f <= 0.65625f ? k - 12 : k - 11, FP4_E_MIN);
}

// e2m1 codes of two floats, nearest, ties to even, saturating at 6: lo in the lower four bits.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float hi, float lo) {
    uint32_t r;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n mov.b32 %0, {t, 0, 0, 0};\n}\n"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// 16 values of a token (bf16 values, at most 6 * 448 in magnitude once scaled by down = 2^-e), of
// largest magnitude mx; ok: they are all finite (else the group reads back as NaN).
//
// The scale is e4m3(mx down / 6), the quotient rounded to fp32 first, which decides nothing: mx has 8
// significant bits, and a number of that kind that is not on the border of two scales is 2^-8 or more
// away from it. The codes are e2m1(v down / scale). v down times the reciprocal of the scale is within
// 2^-21 of that, and rounded to a multiple of 2^-14 (by adding and taking off 768) it is on the border
// of two codes exactly where the quotient is: else it is at least 2^-10 away from it.
__device__ __forceinline__ Fp4Group fp4_quantize(const float (&v)[FP4_GROUP], float mx, bool ok, int e,
                                                 float down) {
    float want = __fdiv_rn(mx * down, 6.f);
    if (e == FP4_E_MAX) want = fminf(want, 320.f);  // 6 * 352 * 2^117 would not be a bf16 number
    const uint16_t two = f32x2_to_e4m3x2(0.f, ok ? want : 0.f);
    Fp4Group g;
    g.scale = ok ? static_cast<uint8_t>(two & 0xFF) : 0x7F;
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(two))));
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = fmaf(v[8 * h + 2 * k] * down, inv, 768.f) - 768.f;
            const float b = fmaf(v[8 * h + 2 * k + 1] * down, inv, 768.f) - 768.f;
            w[h] |= f32x2_to_e2m1x2(b, a) << (8 * k);
        }
        if (!ok) w[h] = 0;
    }
    g.codes = make_uint2(w[0], w[1]);
    return g;
}

// 8 codes of a group as bf16: four pairs. up = scale * 2^e.
__device__ __forceinline__ void fp4_widen8(uint32_t codes, float up, uint32_t (&out)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h;
        asm("{\n .reg .b8 t, u, v, w;\n mov.b32 {t, u, v, w}, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n"
            : "=r"(h)
            : "r"(codes >> (8 * k)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        out[k] = pack_bf16x2(f.x * up, f.y * up);
    }
}
__device__ __forceinline__ float fp4_factor(uint8_t scale, int e) {
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(scale))));
    return s * exp2_int(e < FP4_E_MIN ? FP4_E_MIN : e);
}

}  // namespace mla
