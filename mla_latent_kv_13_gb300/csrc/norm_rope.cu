// norm_rope.cu -- the latent norms of a ragged batch's new tokens, the rotation of their keys
// and the write into the paged cache, in one pass over the down-projection's output.
//
//   x = [c_q | c_kv | k_r];  rms(v) = v / sqrt(mean v^2 + eps)
//   c_q out = rms(c_q) w_q;  cache row = [rms(c_kv) w_kv | RoPE(k_r, position)]
// Everything is fp32 (the angles 64-bit fixed point) with one rounding at the store, to bf16 or, for
// an FP8 cache, to e4m3 codes of the row's power-of-two scale. A code next to the border of two steps
// shows every fp32 rounding before it, so the FP8 row is carried further: sum of squares and
// factor as two floats each, one rounding to fp32, then one to e4m3. The 4-bit cache's row (fp4.cuh)
// is the exact norm's 512 values to the nearest bf16, quantised: from the FP8 row's sums and factors, so that
// nearly no code depends on how they were formed (a bf16 cache's own row, with fp32's roundings, may be a step
// off it next to a border).
//
// One warp per token for the key side and one for the query side: a row stays in the warp's
// registers (16-byte pieces, at most 6 of them per lane; a longer c_q is read twice), its sum
// of squares is one shuffle reduction, and no warp waits for another. Bound by memory for many
// tokens, by the chain of one row's loads for few.
#include <limits.h>

#include "common.cuh"
#include "fp4.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "rope.h"
#include "serve.h"
#include "turn.cuh"

namespace mla {

namespace {

constexpr int WARPS = 2;
constexpr int KEEP = 6;  // 16-byte pieces of c_q a lane keeps in registers

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
// 1 / sqrt(mean), each step correctly rounded: a value is off by about two fp32 roundings in all
// (the product of a bf16 value and its bf16 weight is exact in fp32)
__device__ __forceinline__ float rms_factor(float mean) { return 1.f / sqrtf(mean); }
// Where fp32 cannot hold the squares of a row the row is scaled by a power of two first (and eps by
// its square), which the norm takes out again: 1 where mean = sum / n + eps is well inside the
// range. A row of up to 2^16 values below 2^128 times 2^-76 has a sum below 2^120; where the
// mean is below 2^-90 no value is above 2^-37, and bf16's smallest, 2^-133, has a square left.
// (The same in every lane, the sums being commutative at every step of the exchange.)
__device__ __forceinline__ float range_scale(float mean) {
    return mean < 0x1p-90f ? 0x1p100f : mean < 0x1p124f ? 1.f : 0x1p-76f;
}
// hi + lo, an unevaluated sum of two floats
struct Two {
    float hi, lo;
};
// a + b with its rounding error carried (the error of a floating sum is a float; Knuth)
__device__ __forceinline__ Two two_add(const Two &a, float b_hi, float b_lo) {
    const float t = a.hi + b_hi, d = t - a.hi;
    return {t, a.lo + b_lo + ((a.hi - (t - d)) + (b_hi - d))};
}
__device__ __forceinline__ Two mean_two(Two sum, float eps) {
    static_assert(D_C == 512, "an exact scale");
    return two_add({sum.hi * (1.f / D_C), sum.lo * (1.f / D_C)}, eps, 0.f);
}
// 1 / sqrt(v) to about 2^-44: the hardware's root and one step of Newton's method whose
// residual 1 - v y^2 is formed with fused products
__device__ __forceinline__ Two rsqrt_two(Two v) {
    const float y = rsqrtf(v.hi + v.lo), p = v.hi * y;
    float r = fmaf(-p, y, 1.f);
    r -= fmaf(v.hi, y, -p) * y;
    r -= v.lo * y * y;
    return {y, 0.5f * y * r};
}

__device__ __forceinline__ float square_sum(const float (&f)[8]) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(f[k], f[k], s);
    return s;
}

// Token t's sequence b (the last one that begins at or before it), by the whole warp, and its
// position; b = -1: none. Up to 128 sequences their starts, ends and lengths are loaded
// together, one round trip to memory; more than that are narrowed down to 128 first.
struct Place {
    int b;
    long pos;
};
__device__ __forceinline__ Place find_place(const NormParams &p, int t, int lane) {
    const int32_t *starts = p.q_starts;
    int lo = 0, len = p.B;
    while (len > 128) {  // 128 probes a round
        const int step = (len + 127) >> 7;
        int k = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (32 * j + lane) * step;
            k += __popc(__ballot_sync(0xffffffffu, at < len && starts[lo + at] <= t));
        }
        if (k == 0) return {-1, 0};
        lo += (k - 1) * step;
        len = min(step, len - (k - 1) * step);
    }
    int s[4], e[4], n[4], b = -1, end = 0, length = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (32 * j < len) {
            const int at = 32 * j + lane;
            const bool there = at < len;
            s[j] = there ? starts[lo + at] : INT_MAX;
            e[j] = there ? starts[lo + at + 1] : 0;
            n[j] = there ? p.seqlens[lo + at] : 0;
        }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (32 * j < len) {
            const unsigned begun = __ballot_sync(0xffffffffu, s[j] <= t);
            if (begun) {
                const int k = 31 - __clz(begun);
                b = lo + 32 * j + k;
                end = __shfl_sync(0xffffffffu, e[j], k);
                length = __shfl_sync(0xffffffffu, n[j], k);
            }
        }
    if (b < 0) return {-1, 0};
    if (t >= end) return {-1, 0};  // a padded batch's token
    return {b, (long)length - end + t};
}

// a row whose squares fp32 cannot hold, scaled by sc
__device__ __noinline__ void norm_query_scaled(const uint4 *src, const uint4 *wq, uint4 *dst, int q_lora,
                                               float eps, float sc, int lane) {
    float sum = 0.f, f[8], w[8];
#pragma unroll 1
    for (int i = lane; i < q_lora / 8; i += 32) {
        unpack8(src[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= sc;
        sum += square_sum(f);
    }
    const float inv = rms_factor(warp_sum(sum) / q_lora + eps * sc * sc);
#pragma unroll 1
    for (int i = lane; i < q_lora / 8; i += 32) {
        unpack8(src[i], f);
        unpack8(wq[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * sc * w[k] * inv;
        dst[i] = pack8(f);
    }
}

__device__ void norm_query(const NormParams &p, int t, int lane) {
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + t * p.ldx);
    const uint4 *wq = reinterpret_cast<const uint4 *>(p.w_q);
    uint4 *dst = reinterpret_cast<uint4 *>(p.c_q + (size_t)t * p.q_lora);
    const int pieces = p.q_lora / 8;
    uint4 v[KEEP];
    float sum = 0.f, f[8];
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        v[k] = lane + 32 * k < pieces ? src[lane + 32 * k] : make_uint4(0u, 0u, 0u, 0u);
    // tokens outside every sequence are left alone (looked up beside the row's loads)
    if (t < p.q_starts[0] || t >= p.q_starts[p.B]) return;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        unpack8(v[k], f);
        sum += square_sum(f);
    }
    for (int i = lane + 32 * KEEP; i < pieces; i += 32) {
        unpack8(src[i], f);
        sum += square_sum(f);
    }
    const float mean = warp_sum(sum) / p.q_lora + p.eps, sc = range_scale(mean);
    if (sc != 1.f) return norm_query_scaled(src, wq, dst, p.q_lora, p.eps, sc, lane);
    const float inv = rms_factor(mean);
    auto put = [&](int i, const uint4 &u) {
        float w[8];
        unpack8(u, f);
        unpack8(wq[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * w[k] * inv;
        dst[i] = pack8(f);
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (lane + 32 * k < pieces) put(lane + 32 * k, v[k]);
    for (int i = lane + 32 * KEEP; i < pieces; i += 32) put(i, src[i]);
}

// The 16 latent values of this lane (a group of a 4-bit cache) of a row whose products or factor are
// near the ends of fp32's range, in 64 bits: to the nearest bf16, by way of the fp32 number that is
// odd in its last place where it is not the value itself.
struct Group16 {
    float v[16];
};
__device__ __noinline__ Group16 latents_of_any_size(const uint16_t *src, const uint16_t *w, float eps,
                                                    int lane) {
    double sum = 0.;
#pragma unroll 1
    for (int k = 0; k < 16; ++k) {
        const double x = bf16_to_f32(src[16 * lane + k]);
        sum += x * x;
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const double inv = 1. / sqrt(sum / D_C + static_cast<double>(eps));
    Group16 g;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const double r = static_cast<double>(bf16_to_f32(src[16 * lane + k])) *
                         static_cast<double>(bf16_to_f32(w[16 * lane + k])) * inv;
        float f = __double2float_rz(r);
        if (static_cast<double>(f) != r && isfinite(r)) f = __uint_as_float(__float_as_uint(f) | 1u);
        g.v[k] = bf16_to_f32(f32_to_bf16(f));
    }
    return g;
}

// where the row goes
enum Format { BF16, FP8, FP4 };

// F: the cache's format. PLAN: the rotation of a plan (its layout, and a magnitude for the rotated
// values) instead of pairs (2i, 2i + 1).
template <int F, bool PLAN>
__device__ void norm_key(const NormParams &p, const TurnFreqs &freqs, int t, int lane) {
    const uint16_t *src = p.x + t * p.ldx + p.q_lora;
    // the 16-byte pieces of a lane: lane and lane + 32; for a 4-bit cache a group of 16 values
    const int i0 = F == FP4 ? 2 * lane : lane, i1 = F == FP4 ? 2 * lane + 1 : lane + 32;
    const uint4 u0 = reinterpret_cast<const uint4 *>(src)[i0];
    const uint4 u1 = reinterpret_cast<const uint4 *>(src)[i1];
    const bool half = PLAN && p.half_layout;
    uint32_t kr;
    if (half) kr = src[D_C + lane] | static_cast<uint32_t>(src[D_C + 32 + lane]) << 16;
    else kr = reinterpret_cast<const uint32_t *>(src + D_C)[lane];
    const uint4 w0 = reinterpret_cast<const uint4 *>(p.w_kv)[i0];
    const uint4 w1 = reinterpret_cast<const uint4 *>(p.w_kv)[i1];
    const Place at = find_place(p, t, lane);
    if (at.b < 0) return;  // a padded batch's token
    const int b = at.b;
    const long pos = at.pos;
    int blk = -1;
    if (pos >= 0 && pos < (long)p.max_blocks * BLOCK)
        blk = p.block_table[(size_t)b * p.max_blocks + pos / BLOCK];
    float a[8], c[8], g[8];
    unpack8(u0, a);
    unpack8(u1, c);
    float eps = p.eps;
    auto rescale = [&](float sc) {
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] *= sc, c[k] *= sc;
        eps = eps * sc * sc;
    };
    float factor = 1.f;
    if (F != BF16) {
        Two mean;
#pragma unroll 1
        for (bool once = true;; once = false) {
            Two sum{0.f, 0.f};  // squares of bf16 values are exact
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum = two_add(sum, a[k] * a[k], 0.f);
                sum = two_add(sum, c[k] * c[k], 0.f);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                sum = two_add(sum, __shfl_xor_sync(0xffffffffu, sum.hi, o),
                              __shfl_xor_sync(0xffffffffu, sum.lo, o));
            mean = mean_two(sum, eps);
            const float sc = range_scale(mean.hi);
            if (sc == 1.f || !once) break;
            rescale(sc);
        }
        const Two inv = rsqrt_two(mean);
        factor = inv.hi;
        auto scaled = [&](float v, float w) {
            const float t = v * w;  // exact
            const float r = fmaf(t, inv.hi, t * inv.lo);
            if (F == FP4 && (__float_as_uint(r) & 0xFFFFu) == 0x8000u) {
                // on the border of two bf16 numbers: which side of it the value itself is on
                const float off = fmaf(t, inv.hi, -r) + t * inv.lo;
                const int away = off == 0.f ? 0 : (off > 0.f) == (r > 0.f) ? 1 : -1;
                return __uint_as_float(__float_as_uint(r) + away);
            }
            return r;
        };
        unpack8(w0, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = scaled(a[k], g[k]);
        unpack8(w1, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = scaled(c[k], g[k]);
    } else {
        float mean;
#pragma unroll 1
        for (bool once = true;; once = false) {
            mean = warp_sum(square_sum(a) + square_sum(c)) / D_C + eps;
            const float sc = range_scale(mean);
            if (sc == 1.f || !once) break;
            rescale(sc);
        }
        const float inv = rms_factor(mean);
        unpack8(w0, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = a[k] * g[k] * inv;
        unpack8(w1, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = c[k] * g[k] * inv;
    }
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b);
        return;
    }
    const float k0 = __uint_as_float(kr << 16), k1 = __uint_as_float(kr & 0xFFFF0000u);
    float co, si;
    turn(static_cast<uint32_t>(pos), freqs.f[lane], co, si);
    if (PLAN) co *= p.magnitude, si *= p.magnitude;
    const float r0 = fmaf(k0, co, -(k1 * si)), r1 = fmaf(k0, si, k1 * co);
    const size_t slot = (size_t)blk * BLOCK + pos % BLOCK;
    auto put_key = [&](uint16_t *to) {
        const uint32_t two = pack_bf16x2(r0, r1);
        if (half)
            to[lane] = static_cast<uint16_t>(two), to[32 + lane] = static_cast<uint16_t>(two >> 16);
        else reinterpret_cast<uint32_t *>(to)[lane] = two;
    };
    if (F == BF16) {
        uint16_t *row = p.cache + slot * D_QK;
        reinterpret_cast<uint4 *>(row)[lane] = pack8(a);
        reinterpret_cast<uint4 *>(row)[lane + 32] = pack8(c);
        put_key(row + D_C);
        return;
    }
    if (F == FP4) {
        float v[FP4_GROUP];
        {
            float f[8];
            unpack8(pack8(a), f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = f[k];
            unpack8(pack8(c), f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[8 + k] = f[k];
        }
        // (as bit patterns, where a NaN is above an infinity)
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < FP4_GROUP; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        // (the same in every lane) a product of a value and its weight may be outside fp32's range or
        // have lost bits: the values are formed anew
        const uint32_t whole = __reduce_max_sync(0xffffffffu, top);
        if (whole >= 0x7F800000u || (whole != 0 && whole < __float_as_uint(0x1p-40f)) ||
            !(factor > 0x1p-40f && factor < 0x1p16f)) {
            const Group16 any = latents_of_any_size(src, p.w_kv, p.eps, lane);
            top = 0;
#pragma unroll
            for (int k = 0; k < FP4_GROUP; ++k) {
                v[k] = any.v[k];
                top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
            }
        }
        const bool ok = top < 0x7F800000u;
        const int e = fp4_row_exp(__uint_as_float(__reduce_max_sync(0xffffffffu, ok ? top : 0u)));
        const Fp4Group q = fp4_quantize(v, __uint_as_float(top), ok, e, exp2_int(-e));
        reinterpret_cast<uint2 *>(p.codes + slot * (D_C / 2))[lane] = q.codes;
        p.scales[slot * FP4_GROUPS + lane] = q.scale;
        if (lane == 0) p.exps[slot] = static_cast<int8_t>(e);
        put_key(p.keys + slot * D_ROPE);
        return;
    }
    float mx = fmaxf(fabsf(r0), fabsf(r1));
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fmaxf(fabsf(a[k]), fabsf(c[k])));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int e = row_scale_exp(mx);
    const float s = exp2_int(-e);
    auto codes4 = [&](const float *f) {
        return static_cast<uint32_t>(f32x2_to_e4m3x2(f[1] * s, f[0] * s)) |
               static_cast<uint32_t>(f32x2_to_e4m3x2(f[3] * s, f[2] * s)) << 16;
    };
    uint8_t *row = p.codes + slot * D_QK;
    reinterpret_cast<uint2 *>(row)[lane] = make_uint2(codes4(a), codes4(a + 4));
    reinterpret_cast<uint2 *>(row)[lane + 32] = make_uint2(codes4(c), codes4(c + 4));
    const uint16_t two = f32x2_to_e4m3x2(r1 * s, r0 * s);
    if (half)
        row[D_C + lane] = static_cast<uint8_t>(two), row[D_C + 32 + lane] = static_cast<uint8_t>(two >> 8);
    else reinterpret_cast<uint16_t *>(row + D_C)[lane] = two;
    if (lane == 0) p.exps[slot] = static_cast<int8_t>(e);
}

// token ranges that do not ascend within [0, tokens] are recorded: sequence b's
__device__ __forceinline__ void check_starts(const NormParams &p, int b) {
    if (b < p.B && (p.q_starts[b] < 0 || p.q_starts[b + 1] < p.q_starts[b] || p.q_starts[b + 1] > p.tokens))
        flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b);
}

// CTA c behind the first `checks`: key and query side of token c (a warp each), or the key side of tokens
// 2c and 2c + 1 alone; the first ones look over the token ranges, a sequence a thread (a CTA for all 4096 took
// 40 us; told apart by a division in the kernel 17.5 us where this takes 17.1). Small CTAs, so that a place is
// free as soon as its two warps are done: 9.7k tokens of q_lora 1536 into an FP8 cache (76 MB) take 17.1 us
// from memory, 4.5 TB/s (CTAs of eight warps 17.7; half as many warps an SM 24.4; a quarter more, with
// registers spilled, 16.9; a persistent grid with the next row on its way 17.5, rows streamed through
// shared memory 27.8). The key side's instructions are the longer half: without it 13.8.
template <int F, bool PLAN>
__global__ void __launch_bounds__(32 * WARPS, 16) norm_rope_kernel(NormParams p, TurnFreqs freqs,
                                                                   int checks) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x < static_cast<unsigned>(checks)) {
        check_starts(p, blockIdx.x * 32 * WARPS + threadIdx.x);
        return;
    }
    const int per = p.q_lora > 0 ? WARPS / 2 : WARPS;
    const int t = (blockIdx.x - checks) * per + warp % per;
    if (t >= p.tokens) return;
    if (warp < per) norm_key<F, PLAN>(p, freqs, t, lane);
    else norm_query(p, t, lane);
}

}  // namespace

cudaError_t launch_norm_rope(const NormParams &p, float theta, const mla_rope_t *plan,
                             cudaStream_t stream) {
    const int per = p.q_lora > 0 ? WARPS / 2 : WARPS;
    const dim3 block(32 * WARPS);
    const int checks = (p.B + 32 * WARPS - 1) / (32 * WARPS);
    const dim3 grid(checks + (p.tokens + per - 1) / per);
    auto go = [&](auto kernel, const TurnFreqs &f) {
        return launch_pdl(kernel, grid, block, 0, stream, p, f, checks);
    };
    if (!plan)
        return p.codes ? go(norm_rope_kernel<FP8, false>, turn_freqs(theta))
                       : go(norm_rope_kernel<BF16, false>, turn_freqs(theta));
    const TurnFreqs f = turn_table<D_ROPE / 2>(*plan);
    return p.scales  ? go(norm_rope_kernel<FP4, true>, f)
           : p.codes ? go(norm_rope_kernel<FP8, true>, f)
                     : go(norm_rope_kernel<BF16, true>, f);
}

}  // namespace mla
