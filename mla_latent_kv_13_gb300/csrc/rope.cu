// rope.cu -- rotary positions: part of every head's values, as pairs (2i, 2i + 1) or (i, i + rot / 2),
// turned by position * freq[i] and multiplied by the plan's magnitude; the head's other values are
// copied beside it where that is wanted (a query split for the expanded attention).
//
// Bound by memory: each moved value is read and written once. A thread has one vector of a head for four
// heads (or tokens, where a token has few), all of whose loads are on their way before the CTA forms its
// tokens' cosines and sines, in shared memory. fp32 throughout (angles in 64-bit fixed point), rounded
// once.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rope.h"
#include "turn.cuh"

namespace mla {

namespace {

constexpr int THREADS = 256;
constexpr int U = 4;  // steps of a thread
constexpr int ANGLES = 2048;  // pairs of a CTA: 16 KB of cosines and sines

template <int V> struct Vec;
template <> struct Vec<1> { using T = uint16_t; };
template <> struct Vec<2> { using T = uint32_t; };
template <> struct Vec<4> { using T = uint2; };
template <> struct Vec<8> { using T = uint4; };
struct alignas(32) U8 { uint32_t v[8]; };
template <> struct Vec<16> { using T = U8; };

template <int V>
__device__ __forceinline__ void load_vec(const uint16_t *src, uint16_t (&v)[V]) {
    if constexpr (V == 16) {
        uint32_t *w = reinterpret_cast<uint32_t *>(v);
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                       "=r"(w[7])
                     : "l"(src));
        return;
    } else
    *reinterpret_cast<typename Vec<V>::T *>(v) = *reinterpret_cast<const typename Vec<V>::T *>(src);
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t *dst, const uint16_t (&v)[V]) {
    if constexpr (V == 16) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
        return;
    } else
    *reinterpret_cast<typename Vec<V>::T *>(dst) = *reinterpret_cast<const typename Vec<V>::T *>(v);
}

// What a step of one head moves: V values, or of halves V from each (V = 1 side by side: a pair).
template <bool HALF, int V>
struct Step {
    static constexpr int N = HALF || V == 1 ? 2 * V : V;
    alignas(2 * V) uint16_t v[N];
};

// V: values of a load. HALF: the layout of halves, a step turns V pairs; else pairs side by side, a
// step turns V / 2 (V = 1: one pair as two loads). CTA (x, y): tokens per x .. and heads hc y .., at
// most four steps a thread (256 threads going through all heads of a token, one head at a time: 88 us
// for 4096 tokens of 128 heads, split; four heads at a time 74; in CTAs of their own 71, with 32-byte
// vectors 62: 6.5 TB/s).
template <bool HALF, int V, int PAIRS>
__global__ void __launch_bounds__(THREADS) rope_kernel(RopeParams p, int rot, float magnitude,
                                                       TurnTable<PAIRS> turns, int per, int hc) {
    __shared__ float cs[ANGLES], sn[ANGLES];
    grid_launch_dependents();
    grid_dependency_wait();
    const int t0 = blockIdx.x * per, n = min(per, p.tokens - t0);
    const int pairs = rot / 2, tid = threadIdx.y * blockDim.x + threadIdx.x;
    constexpr int PLACE = !HALF && V == 1 ? 2 : V;     // values of a step at each of its places
    const int turned = HALF ? pairs / V : rot / PLACE;  // steps of a head's rotated values
    const int before = p.rest ? p.offset / V : 0;       // and of the others, before and behind
    const int steps = turned + before + (p.rest ? (p.width - rot - p.offset) / V : 0);
    const int h0 = blockIdx.y * hc, nh = min(hc, p.heads - h0), all = n * nh, rows = blockDim.y;
    Step<HALF, V> r[U];
    auto load = [&](int u) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = threadIdx.y + i * rows;
            if (k >= all) continue;
            const int t = n == 1 ? 0 : k / nh, h = h0 + k - t * nh;
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
    auto store = [&](int u) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = threadIdx.y + i * rows;
            if (k >= all) continue;
            const int t = n == 1 ? 0 : k / nh, h = h0 + k - t * nh;
            if (u >= turned) {
                store_vec<V>(p.rest + (t0 + t) * p.rest_token + h * p.rest_head + (u - turned) * V,
                             *reinterpret_cast<uint16_t(*)[V]>(r[i].v));
                continue;
            }
            uint16_t *y = p.y + (t0 + t) * p.y_token + h * p.y_head + u * PLACE;
            const int at = t * pairs + (HALF ? u * V : u * PLACE / 2);
            constexpr int TURNED = HALF ? V : PLACE / 2;
#pragma unroll
            for (int q = 0; q < TURNED; ++q) {
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
    load(u);
    for (int k = tid; k < n * pairs; k += blockDim.x * rows) {
        const int t = k / pairs, i = k - t * pairs;
        const uint64_t at = turns.f[i] * static_cast<uint64_t>(static_cast<int64_t>(p.pos[t0 + t]));
        float c, s;
        turn_by(at, c, s);
        cs[k] = c * magnitude, sn[k] = s * magnitude;
    }
    __syncthreads();
    store(u);
    for (u += blockDim.x; u < steps; u += blockDim.x) {  // heads of more steps than a CTA has threads
        load(u);
        store(u);
    }
}

template <bool HALF, int V, int PAIRS>
cudaError_t launch(const RopeParams &p, const mla_rope_t &plan, cudaStream_t stream) {
    const int rot = plan.rot;
    const int turned = HALF ? rot / 2 / V : rot / (V == 1 ? 2 : V);
    const int steps = turned + (p.rest ? (p.width - rot) / V : 0);
    const int x = steps < THREADS ? steps : THREADS;
    const dim3 block(x, THREADS / x);
    // heads and tokens of a CTA: one token's, or tokens as far as the angles have room and every SM has
    // a CTA
    const int most = U * block.y, hc = p.heads < most ? p.heads : most;
    int per = p.heads < most ? most / p.heads : 1;
    const int spread = p.tokens / device_sm_count();
    if (per > spread) per = spread > 0 ? spread : 1;
    if (per > 2 * ANGLES / rot) per = 2 * ANGLES / rot;
    const dim3 grid((p.tokens + per - 1) / per, (p.heads + hc - 1) / hc);
    return launch_pdl(rope_kernel<HALF, V, PAIRS>, grid, block, 0, stream, p, rot, plan.magnitude,
                      turn_table<PAIRS>(plan), per, hc);
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
    // (the frequencies are a kernel argument: 32 of them cost the host less than 128)
    auto as_wide = [&](auto h, auto n) {
        constexpr bool H = decltype(h)::value;
        constexpr int N = decltype(n)::value;
        return all % 16 == 0  ? launch<H, 16, N>(p, plan, stream)
               : all % 8 == 0 ? launch<H, 8, N>(p, plan, stream)
               : all % 4 == 0 ? launch<H, 4, N>(p, plan, stream)
               : all % 2 == 0 ? launch<H, 2, N>(p, plan, stream)
                              : launch<H, 1, N>(p, plan, stream);
    };
    auto go = [&](auto h) {
        return plan.rot <= 64 ? as_wide(h, std::integral_constant<int, 32>{})
                              : as_wide(h, std::integral_constant<int, MLA_ROPE_MAX / 2>{});
    };
    return half ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace mla
