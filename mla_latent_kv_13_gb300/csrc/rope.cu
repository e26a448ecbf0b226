// rope.cu -- rotary positions: part of every head's values, as pairs (2i, 2i + 1) or (i, i + rot / 2),
// turned by position * freq[i] and multiplied by the plan's magnitude; the head's other values are
// copied beside it where that is wanted (a query split for the expanded attention).
//
// Each moved value is read and written once; what is left to save is the angles: a CTA takes some
// tokens with all their heads, forms the cosines and sines of each token once, in shared memory, and
// goes through the heads with a thread for each vector of a head. fp32 throughout (angles in 64-bit
// fixed point), rounded once.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rope.h"
#include "turn.cuh"

namespace mla {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = MLA_ROPE_MAX / 2;
using Turns = TurnTable<MAX_PAIRS>;
constexpr int ANGLES = 2048;  // pairs of a CTA: 16 KB of cosines and sines

template <int V> struct Vec;
template <> struct Vec<1> { using T = uint16_t; };
template <> struct Vec<2> { using T = uint32_t; };
template <> struct Vec<4> { using T = uint2; };
template <> struct Vec<8> { using T = uint4; };

template <int V>
__device__ __forceinline__ void load_vec(const uint16_t *src, uint16_t (&v)[V]) {
    *reinterpret_cast<typename Vec<V>::T *>(v) = *reinterpret_cast<const typename Vec<V>::T *>(src);
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t *dst, const uint16_t (&v)[V]) {
    *reinterpret_cast<typename Vec<V>::T *>(dst) = *reinterpret_cast<const typename Vec<V>::T *>(v);
}

// V: values of a load. HALF: the layout of halves, a step turns V pairs; else pairs side by side, a
// step turns V / 2 (V = 1: one pair as two loads).
template <bool HALF, int V>
__global__ void __launch_bounds__(THREADS) rope_kernel(RopeParams p, int rot, float magnitude, Turns turns,
                                                       int per) {
    __shared__ float cs[ANGLES], sn[ANGLES];
    grid_launch_dependents();
    grid_dependency_wait();
    const int t0 = blockIdx.x * per, n = min(per, p.tokens - t0);
    const int pairs = rot / 2, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int threads = blockDim.x * blockDim.y;
    for (int k = tid; k < n * pairs; k += threads) {
        const int t = k / pairs, i = k - t * pairs;
        const uint64_t at = turns.f[i] * static_cast<uint64_t>(static_cast<int64_t>(p.pos[t0 + t]));
        float c, s;
        turn_by(at, c, s);
        cs[k] = c * magnitude, sn[k] = s * magnitude;
    }
    __syncthreads();
    constexpr int STEP = !HALF && V == 1 ? 2 : V;           // values that a step moves at each of its places
    const int turned = HALF ? pairs / V : rot / STEP;       // steps of a head's rotated values
    const int before = p.rest ? p.offset / V : 0;           // and of the others, before and behind
    const int behind = p.rest ? (p.width - rot - p.offset) / V : 0;
    const int steps = turned + before + behind;
    for (int u = threadIdx.x; u < steps; u += blockDim.x) {
        for (int k = threadIdx.y; k < n * p.heads; k += blockDim.y) {
            const int t = n == 1 ? 0 : k / p.heads, h = k - t * p.heads;
            const uint16_t *x = p.x + (t0 + t) * p.x_token + h * p.x_head;
            if (u >= turned) {
                const int j = u - turned;
                alignas(2 * V) uint16_t v[V];
                load_vec<V>(x + (j < before ? 0 : rot) + j * V, v);
                store_vec<V>(p.rest + (t0 + t) * p.rest_token + h * p.rest_head + j * V, v);
                continue;
            }
            uint16_t *y = p.y + (t0 + t) * p.y_token + h * p.y_head;
            const float *c = cs + t * pairs, *s = sn + t * pairs;
            x += p.offset;
            if (HALF) {
                const int i = u * V;
                alignas(2 * V) uint16_t a[V];
                alignas(2 * V) uint16_t b[V];
                load_vec<V>(x + i, a);
                load_vec<V>(x + pairs + i, b);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float f = bf16_to_f32(a[q]), g = bf16_to_f32(b[q]);
                    a[q] = f32_to_bf16(fmaf(f, c[i + q], -(g * s[i + q])));
                    b[q] = f32_to_bf16(fmaf(f, s[i + q], g * c[i + q]));
                }
                store_vec<V>(y + i, a);
                store_vec<V>(y + pairs + i, b);
            } else {
                const int i = u * STEP;
                alignas(2 * V) uint16_t a[STEP];
                if constexpr (V == 1) a[0] = x[i], a[1] = x[i + 1];
                else load_vec<V>(x + i, a);
#pragma unroll
                for (int q = 0; q < STEP; q += 2) {
                    const float f = bf16_to_f32(a[q]), g = bf16_to_f32(a[q + 1]);
                    const float co = c[(i + q) / 2], si = s[(i + q) / 2];
                    a[q] = f32_to_bf16(fmaf(f, co, -(g * si)));
                    a[q + 1] = f32_to_bf16(fmaf(f, si, g * co));
                }
                if constexpr (V == 1) y[i] = a[0], y[i + 1] = a[1];
                else store_vec<V>(y + i, a);
            }
        }
    }
}

template <bool HALF, int V>
cudaError_t launch(const RopeParams &p, const mla_rope_t &plan, cudaStream_t stream) {
    const int rot = plan.rot;
    const int turned = HALF ? rot / 2 / V : rot / (V == 1 ? 2 : V);
    const int steps = turned + (p.rest ? (p.width - rot) / V : 0);
    const int x = steps < THREADS ? steps : THREADS;
    const dim3 block(x, THREADS / x);
    // tokens of a CTA: about four steps a thread, as far as the angles have room
    const long of_token = (long)steps * p.heads;
    long per = (4 * THREADS + of_token - 1) / of_token;
    if (per > 2 * ANGLES / rot) per = 2 * ANGLES / rot;
    const dim3 grid(static_cast<unsigned>((p.tokens + per - 1) / per));
    return launch_pdl(rope_kernel<HALF, V>, grid, block, 0, stream, p, rot, plan.magnitude,
                      turn_table<MAX_PAIRS>(plan), static_cast<int>(per));
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, const mla_rope_t &plan, cudaStream_t stream) {
    // the widest vectors that every address allows
    const bool half = plan.layout == MLA_ROPE_HALF;
    uint64_t all = reinterpret_cast<uintptr_t>(p.x) / 2 | reinterpret_cast<uintptr_t>(p.y) / 2 |
                   static_cast<uint64_t>(p.offset) | static_cast<uint64_t>(half ? plan.rot / 2 : plan.rot);
    if (p.tokens > 1) all |= static_cast<uint64_t>(p.x_token) | static_cast<uint64_t>(p.y_token);
    if (p.heads > 1) all |= static_cast<uint64_t>(p.x_head) | static_cast<uint64_t>(p.y_head);
    if (p.rest) {
        all |= reinterpret_cast<uintptr_t>(p.rest) / 2 | static_cast<uint64_t>(p.width);
        if (p.tokens > 1) all |= static_cast<uint64_t>(p.rest_token);
        if (p.heads > 1) all |= static_cast<uint64_t>(p.rest_head);
    }
    auto go = [&](auto h) {
        constexpr bool H = decltype(h)::value;
        return all % 8 == 0   ? launch<H, 8>(p, plan, stream)
               : all % 4 == 0 ? launch<H, 4>(p, plan, stream)
               : all % 2 == 0 ? launch<H, 2>(p, plan, stream)
                              : launch<H, 1>(p, plan, stream);
    };
    return half ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace mla
