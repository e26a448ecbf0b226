// merge.cuh -- the exact log-sum-exp merge of one output row's parts, by one warp.
#pragma once

#include "common.cuh"

namespace mla {

// Merge np partial rows (fp32 [512], each with its log-sum-exp) into one bf16 row and its
// log-sum-exp, with one warp: lane l holds columns 4l + 128k (k < 4), so every part row is
// read as four coalesced 512-byte segments. Every lane reads every part's log-sum-exp (one
// broadcast load each). The rows of the first two parts are loaded together with the
// log-sum-exps, before the weights are known, so that merging two parts (a sequence cut
// once) takes one memory round trip; further parts follow two at a time. Parts are
// accumulated in order. A part with lse = -inf (an empty range) contributes nothing.
__device__ __forceinline__ void merge_row_warp(const float *o0, size_t ostride, const float *l0,
                                               size_t lstride, int np, uint16_t *orow,
                                               float *orow32, float *lse_out, int lane) {
    auto load_row = [&](int s, float4 (&v)[4]) {
        const float *row = o0 + (size_t)s * ostride + lane * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __ldcs(reinterpret_cast<const float4 *>(row + 128 * k));
    };
    float4 va[4], vb[4];
    const float la = np > 0 ? l0[0] : -INFINITY;
    const float lb = np > 1 ? l0[lstride] : -INFINITY;
    if (np > 0) load_row(0, va);
    if (np > 1) load_row(1, vb);
    float m = fmaxf(la, lb);
    for (int s = 2; s < np; ++s) m = fmaxf(m, l0[s * lstride]);
    float tot = -INFINITY;
    if (m != -INFINITY) {
        float den = 0.f;
        if (la != -INFINITY) den += __expf(la - m);
        if (lb != -INFINITY) den += __expf(lb - m);
        for (int s = 2; s < np; ++s) {
            const float l = l0[s * lstride];
            if (l != -INFINITY) den += __expf(l - m);
        }
        tot = m + __logf(den);
    }
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    auto add_row = [&](float l, const float4 (&v)[4]) {
        const float w = l != -INFINITY ? __expf(l - tot) : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            acc[4 * k] += w * v[k].x;
            acc[4 * k + 1] += w * v[k].y;
            acc[4 * k + 2] += w * v[k].z;
            acc[4 * k + 3] += w * v[k].w;
        }
    };
    if (tot != -INFINITY) {
        if (np > 0) add_row(la, va);
        if (np > 1) add_row(lb, vb);
        for (int s = 2; s < np; s += 2) {
            const float l2 = l0[s * lstride];
            const float l3 = s + 1 < np ? l0[(s + 1) * lstride] : -INFINITY;
            load_row(s, va);
            if (s + 1 < np) load_row(s + 1, vb);
            add_row(l2, va);
            if (s + 1 < np) add_row(l3, vb);
        }
    }
    if (orow32) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4 *>(orow32 + lane * 4 + 128 * k) =
                make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint2 *>(orow + lane * 4 + 128 * k) =
                make_uint2(pack_bf16x2(acc[4 * k], acc[4 * k + 1]),
                           pack_bf16x2(acc[4 * k + 2], acc[4 * k + 3]));
    }
    if (lane == 0) *lse_out = tot;
}

}  // namespace mla
