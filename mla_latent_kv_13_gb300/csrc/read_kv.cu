// read_kv.cu -- rows of the paged cache read back as bf16, from any of its formats: a ragged gather
// with the codes widened on the way. Every value of an FP8 or 4-bit cache is exactly a bf16 value.
//
// A row is one step of a warp: a lane has 16 latent values (32 bytes of the output, one store; a whole
// group of a 4-bit cache) and two of the key. A warp takes up to 32 rows: its lanes look up the places
// of all of them side by side, and four rows' loads are in flight at a time. Bound by memory.
#include <limits.h>

#include "common.cuh"
#include "fp4.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "serve.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int WARPS = 4;

enum Format { BF16, FP8, FP4 };

template <int F>
struct Piece {
    uint4 a, b;  // bf16: the values; FP8: 16 codes in a; 4-bit: 16 codes in a.x, a.y
    uint32_t key, scale;
    int e;
};

template <int F>
__device__ __forceinline__ void load_piece(const ReadParams &p, long slot, int lane, Piece<F> &r) {
    if (F == BF16) {
        const uint16_t *row = p.cache + slot * D_QK;
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y),
                       "=r"(r.b.z), "=r"(r.b.w)
                     : "l"(row + 16 * lane));
        r.key = __ldg(reinterpret_cast<const uint32_t *>(row + D_C) + lane);
    } else if (F == FP8) {
        const uint8_t *row = p.codes + slot * D_QK;
        r.a = __ldg(reinterpret_cast<const uint4 *>(row) + lane);
        r.key = __ldg(reinterpret_cast<const uint16_t *>(row + D_C) + lane);
        r.e = __ldg(p.exps + slot);
    } else {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(p.codes + slot * (D_C / 2)) + lane);
        r.a.x = c.x, r.a.y = c.y;
        r.scale = __ldg(p.scales + slot * FP4_GROUPS + lane);
        r.key = __ldg(reinterpret_cast<const uint32_t *>(p.keys + slot * D_ROPE) + lane);
        r.e = __ldg(p.exps + slot);
    }
}

template <int F>
__device__ __forceinline__ void store_piece(uint16_t *row, int lane, const Piece<F> &r, bool there) {
    uint32_t w[8], key = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 0;
    if (there) {
        if (F == BF16) {
            w[0] = r.a.x, w[1] = r.a.y, w[2] = r.a.z, w[3] = r.a.w;
            w[4] = r.b.x, w[5] = r.b.y, w[6] = r.b.z, w[7] = r.b.w;
            key = r.key;
        } else if (F == FP8) {
            const float s = exp2_int(max(r.e, -126));
            const uint32_t c[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = e4m3x2_to_bf16x2_scaled(static_cast<uint16_t>(c[k >> 1] >> (16 * (k & 1))), s);
            key = e4m3x2_to_bf16x2_scaled(static_cast<uint16_t>(r.key), s);
        } else {
            const float up = fp4_factor(static_cast<uint8_t>(r.scale), r.e);
            uint32_t h[4];
            fp4_widen8(r.a.x, up, h);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = h[k];
            fp4_widen8(r.a.y, up, h);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 + k] = h[k];
            key = r.key;
        }
    }
    st_global_v8(row + 16 * lane, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    reinterpret_cast<uint32_t *>(row + D_C)[lane] = key;
}

// The last sequence that begins at or before row r, by the whole warp; -1: none.
__device__ __forceinline__ int find_sequence(const ReadParams &p, int r, int lane) {
    int lo = 0, len = p.B;
    while (true) {
        const int step = (len + 31) >> 5, at = lane * step;
        const unsigned begun =
            __ballot_sync(0xffffffffu, at < len && p.row_starts[lo + at] <= r);
        if (!begun) return lo - 1;
        const int k = 31 - __clz(begun);
        lo += k * step;
        if (step == 1) return lo;
        len = min(step, len - k * step);
    }
}

// The same of row r >= the one that `b` was found for, by one lane: steps that double, then halves, so
// that sequences without rows in between cost a few loads and not one each.
__device__ __forceinline__ int next_sequence(const ReadParams &p, int b, int r) {
    if (b + 1 >= p.B || p.row_starts[b + 1] > r) return b;
    int lo = b + 1, step = 1;  // begins at or before r
    while (lo + step < p.B && p.row_starts[lo + step] <= r) lo += step, step *= 2;
    int hi = min(lo + step, p.B);  // the end, or begins behind it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.row_starts[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

constexpr int CHECKS = 4;  // sequences of a thread that looks over row_starts
// row_starts that do not ascend within [0, rows] are recorded
__device__ void check_rows(const ReadParams &p, int b0) {
    int a[CHECKS], e[CHECKS];
#pragma unroll
    for (int k = 0; k < CHECKS; ++k) {
        const int b = b0 + 32 * WARPS * k;
        a[k] = e[k] = 0;
        if (b < p.B) a[k] = p.row_starts[b], e[k] = p.row_starts[b + 1];
    }
#pragma unroll
    for (int k = 0; k < CHECKS; ++k)
        if (a[k] < 0 || e[k] < a[k] || e[k] > p.rows)
            flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b0 + 32 * WARPS * k);
}

template <int F>
__global__ void __launch_bounds__(32 * WARPS) read_kv_kernel(ReadParams p, int per, unsigned readers) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const long r0 = (long)warp * per;
    if (blockIdx.x >= readers) {  // the CTAs behind those that read
        check_rows(p, (blockIdx.x - readers) * 32 * WARPS * CHECKS + threadIdx.x);
        return;
    }
    if (r0 >= p.rows) return;
    const int n = static_cast<int>(min((long)per, p.rows - r0));
    // this lane's row: its slot in the cache; -1 a bad page (zeros), -2 none of a sequence's rows
    long slot = -2;
    {
        const int r = static_cast<int>(r0) + lane;
        int b = find_sequence(p, static_cast<int>(r0), lane);
        if (lane < n) {
            b = next_sequence(p, b, r);
            if (b >= 0) {
                const long at = (long)r - p.row_starts[b];
                if (r < p.row_starts[b + 1]) {
                    const long pos = (p.first ? p.first[b] : 0) + at;
                    slot = -1;
                    if (pos >= 0 && pos < (long)p.max_blocks * BLOCK) {
                        const int id = p.block_table[(size_t)b * p.max_blocks + pos / BLOCK];
                        if (id >= 0 && id < p.num_blocks) slot = (long)id * BLOCK + pos % BLOCK;
                    }
                    if (slot < 0) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b);
                }
            }
        }
    }
    __syncwarp();
    constexpr int U = 4;  // rows in flight
    for (int i0 = 0; i0 < n; i0 += U) {
        Piece<F> v[U];
        long s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = i0 + u < 32 ? __shfl_sync(0xffffffffu, slot, (i0 + u) & 31) : -2;
            if (s[u] >= 0) load_piece<F>(p, s[u], lane, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s[u] != -2) store_piece<F>(p.out + (r0 + i0 + u) * D_QK, lane, v[u], s[u] >= 0);
    }
}

}  // namespace

cudaError_t launch_read_kv(const ReadParams &p, cudaStream_t stream) {
    // rows of a warp: as many as leave every SM some warps
    const int sms = device_sm_count();
    int per = 32;
    while (per > 4 && (long)sms * 4 * WARPS * per > p.rows) per /= 2;
    const auto readers = static_cast<unsigned>(((long)p.rows + per * WARPS - 1) / (per * WARPS));
    const dim3 grid(readers + (p.B + 32 * WARPS * CHECKS - 1) / (32 * WARPS * CHECKS));
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(32 * WARPS), 0, stream, p, per, readers);
    };
    return p.scales ? go(read_kv_kernel<FP4>) : p.codes ? go(read_kv_kernel<FP8>) : go(read_kv_kernel<BF16>);
}

}  // namespace mla
