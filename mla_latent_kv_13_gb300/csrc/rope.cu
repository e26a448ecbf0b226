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

// What a step of one head moves: V values, or of halves V from each (V = 1 side by side: a pair).
template <bool HALF, int V>
struct Step {
    static constexpr int N = HALF || V == 1 ? 2 * V : V;
    alignas(2 * V) uint16_t v[N];
};

// V: values of a load. HALF: the layout of halves, a step turns V pairs; else pairs side by side, a
// step turns V / 2 (V = 1: one pair as two loads). A thread keeps to one step of a head and takes four
// heads at a time, the first four's loads before the angles are there (one head at a time: 88 us where
// this takes 73 for 4096 tokens of 128 heads, split).
template <bool HALF, int V>
__global__ void __launch_bounds__(THREADS) rope_kernel(RopeParams p, int rot, float magnitude, Turns turns,
                                                       int per) {
    __shared__ float cs[ANGLES], sn[ANGLES];
    grid_launch_dependents();
    grid_dependency_wait();
    const int t0 = blockIdx.x * per, n = min(per, p.tokens - t0);
    const int pairs = rot / 2, tid = threadIdx.y * blockDim.x + threadIdx.x;
    constexpr int PLACE = !HALF && V == 1 ? 2 : V;     // values of a step at each of its places
    const int turned = HALF ? pairs / V : rot / PLACE;  // steps of a head's rotated values
    const int before = p.rest ? p.offset / V : 0;       // and of the others, before and behind
    const int steps = turned + before + (p.rest ? (p.width - rot - p.offset) / V : 0);
    const int all = n * p.heads, rows = blockDim.y;
    constexpr int U = 4;
    Step<HALF, V> r[U];
    auto load = [&](int u, int k0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = k0 + i * rows;
            if (k >= all) continue;
            const int t = n == 1 ? 0 : k / p.heads, h = k - t * p.heads;
            const uint16_t *x = p.x + (t0 + t) * p.x_token + h * p.x_head;
            if (u >= turned) {
                const int j = u - turned;
                load_vec<V>(x + (j < before ? 0 : rot) + j * V, *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
            } else {
                x += p.offset + u * PLACE;
                if constexpr (HALF || V == 1) {
                    load_vec<V>(x, *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
                    load_vec<V>(x + (HALF ? pairs : 1), *reinterpret_cast<uint16_t(*)[V]>(r[i].v + V));
                } else {
                    load_vec<V>(x, *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
                }
            }
        }
    };
    auto store = [&](int u, int k0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = k0 + i * rows;
            if (k >= all) continue;
            const int t = n == 1 ? 0 : k / p.heads, h = k - t * p.heads;
            if (u >= turned) {
                store_vec<V>(p.rest + (t0 + t) * p.rest_token + h * p.rest_head + (u - turned) * V,
                             *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
                continue;
            }
            uint16_t *y = p.y + (t0 + t) * p.y_token + h * p.y_head + u * PLACE;
            const int at = t * pairs + (HALF ? u * V : u * PLACE / 2);
            constexpr int PAIRS = HALF ? V : PLACE / 2;
#pragma unroll
            for (int q = 0; q < PAIRS; ++q) {
                const int a = HALF ? q : 2 * q, b = HALF ? V + q : 2 * q + 1;
                const float f = bf16_to_f32(r[i].v[a]), g = bf16_to_f32(r[i].v[b]);
                const float co = cs[at + q], si = sn[at + q];
                r[i].v[a] = f32_to_bf16(fmaf(f, co, -(g * si)));
                r[i].v[b] = f32_to_bf16(fmaf(f, si, g * co));
            }
            store_vec<V>(y, *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
            if constexpr (HALF || V == 1)
                store_vec<V>(y + (HALF ? pairs : 1), *reinterpret_cast<uint16_t(*)[V]>(r[i].v + V));
        }
    };
    int u = threadIdx.x;
    load(u < steps ? u : 0, u < steps ? threadIdx.y : all);
    for (int k = tid; k < n * pairs; k += blockDim.x * rows) {
        const int t = k / pairs, i = k - t * pairs;
        const uint64_t at = turns.f[i] * static_cast<uint64_t>(static_cast<int64_t>(p.pos[t0 + t]));
        float c, s;
        turn_by(at, c, s);
        cs[k] = c * magnitude, sn[k] = s * magnitude;
    }
    __syncthreads();
    for (bool there = true; u < steps; u += blockDim.x)
        for (int k = threadIdx.y; k < all; k += U * rows, there = false) {
            if (!there) load(u, k);
            store(u, k);
        }
}

template <bool HALF, int V>
cudaError_t launch(const RopeParams &p, const mla_rope_t &plan, cudaStream_t stream) {
    const int rot = plan.rot;
    const int turned = HALF ? rot / 2 / V : rot / (V == 1 ? 2 : V);
    const int steps = turned + (p.rest ? (p.width - rot) / V : 0);
    const int x = steps < THREADS ? steps : THREADS;
    const dim3 block(x, THREADS / x);
    // tokens of a CTA: about four steps a thread, as far as the angles have room and every SM has a CTA
    const long of_token = (long)steps * p.heads;
    long per = (4 * THREADS + of_token - 1) / of_token;
    const long spread = p.tokens / device_sm_count();
    if (per > spread) per = spread > 0 ? spread : 1;
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
