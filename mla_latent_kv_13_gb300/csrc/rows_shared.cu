// rows_shared.cu -- the merge of the items that the clusters' shares cut, in decode attention over a
// batch whose sequences share prefixes (rows_shared.cuh).
#include "common.cuh"
#include "rows.h"

namespace mla {

namespace {

constexpr int G = 5;  // parts of a thread in flight

__device__ __forceinline__ void ld_v8(const float *src, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                   "=f"(v[7])
                 : "l"(src));
}

// the larger one, or the NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// CTA (x, j) merges 8 columns of 128 half-rows of the items that the ends of the clusters c = j, j + J, ..
// cut first, by the log-sum-exps of their parts (2 c + 1, 2 (c + 1), 2 (c + 2), ..). The parts lie as the
// attention kernel's threads hold them: part [2 CTAs][32 pieces of 8 columns][128 lanes][8], lane l of CTA
// r row 64 r + l % 64 with its columns from 256 (l / 64) on, so a thread keeps to its lane and every load is
// whole lines. Y threads share a lane: parts y, y + Y, .. each, joined at the end. A part whose
// log-sum-exp is NaN makes the row NaN.
template <int Y>
__global__ void __launch_bounds__(128 * Y) shared_merge_kernel(RowsParams p) {
    __shared__ float joined[Y > 1 ? (Y - 1) * 10 * 128 : 1];  // [Y - 1][m, den, acc][128]
    grid_launch_dependents();
    grid_dependency_wait();
    const int tl = threadIdx.x, y = threadIdx.y, lane = tl & 31;
    const int cta = blockIdx.x & 1, piece = blockIdx.x >> 1, r = 64 * cta + (tl & 63);
    const int mine = blockIdx.y + gridDim.y * lane;
    const int4 jobs = mine < p.sh.clusters ? p.sh.jobs[mine] : make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (unsigned todo = __ballot_sync(0xffffffffu, jobs.y > 64 * cta); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, c = blockIdx.y + gridDim.y * from;
        const int row0 = __shfl_sync(0xffffffffu, jobs.x, from);
        const bool live = r < __shfl_sync(0xffffffffu, jobs.y, from);
        const int np = __shfl_sync(0xffffffffu, jobs.z, from);
        // as the parts come: the sums so far belong to the reference m
        float m = -INFINITY, den = 0.f, acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 1
        for (int k0 = y; live && k0 < np; k0 += Y * G) {
            float v[G][8], l[G], top = m;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int k = k0 + Y * g;
                l[g] = -INFINITY;
                if (k < np) {
                    const int id = k == 0 ? 2 * c + 1 : 2 * (c + k);
                    l[g] = p.lse_part[(size_t)id * p.rows_per_item + r];
                    ld_v8(p.o_part + ((size_t)(2 * id + cta) * 32 + piece) * 1024 + 8 * tl, v[g]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) top = max_nan(top, l[g]);
            if (top == -INFINITY) continue;
            const float keep = __expf(m - top);
            den *= keep;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] *= keep;
            m = top;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (l[g] == -INFINITY) continue;
                const float w = __expf(l[g] - m);
                den += w;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(w, v[g][j], acc[j]);
            }
        }
        if constexpr (Y > 1) {
            __syncthreads();  // the item before has been joined
            if (y > 0) {
                float *at = joined + (y - 1) * 1280 + tl;
                at[0] = m, at[128] = den;
#pragma unroll
                for (int j = 0; j < 8; ++j) at[128 * (2 + j)] = acc[j];
            }
            __syncthreads();
            float top = m;
            if (y == 0) {
#pragma unroll
                for (int q = 0; q < Y - 1; ++q) top = max_nan(top, joined[1280 * q + tl]);
            }
            if (y == 0 && top != -INFINITY) {
                const float keep = __expf(m - top);
                den *= keep;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] *= keep;
#pragma unroll
                for (int q = 0; q < Y - 1; ++q) {
                    const float *at = joined + 1280 * q + tl;
                    const float w = __expf(at[0] - top);
                    den = fmaf(w, at[128], den);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[j] = fmaf(w, at[128 * (2 + j)], acc[j]);
                }
                m = top;
            }
        }
        if (y > 0 || !live) continue;
        const float inv = den > 0.f ? 1.f / den : 0.f;
        const size_t row = (size_t)row0 + r;
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
        *reinterpret_cast<uint4 *>(p.out + row * D_C + 256 * (tl >> 6) + 8 * piece) =
            make_uint4(o[0], o[1], o[2], o[3]);
        if (piece == 0 && tl < 64) p.lse[row] = den != 0.f ? m + __logf(den) : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_shared_merge(const RowsParams &p, cudaStream_t stream) {
    // The parts of an item are about its share of the clusters, or its tiles if those are fewer. With ten or
    // more four threads share them, in few CTAs, each for a quarter of the clusters; with fewer (64, 38) CTAs
    // of 128 threads. One item of 23 weights in 19 parts 17.1 us so and 14.4 with four; 12 items in 6 or 7 each
    // 44.0 and 47.4. The host does not know the lengths and takes the tiles of the longest sequence that may
    // be, which is near an item's where its sequences share most of them. Up to three items (24 clusters
    // each) it takes those of all of an item's sequences: 8 samples behind 1000 rows 15.2 -> 13.7, 8
    // sequences of up to 1000 with nothing in common 17.3 -> 15.6. With more items that is worse where they
    // have few tiles: five groups of 8 behind 900 rows 19.0 with one thread and 21.3 with four, seven 18.5 and
    // 22.8.
    const int seqs = 128 / (p.hq * p.s_q), items = p.B / seqs, P = p.sh.clusters;
    const int share = items > 0 ? P / items : P, most = p.B < seqs ? p.B : seqs;
    const int pages = p.max_seqlen / BLOCK + 1, tiles = (pages * (share >= 24 ? most : 1) + 1) / 2;
    if ((share < tiles ? share : tiles) >= 10)
        return launch_pdl(shared_merge_kernel<4>, dim3(64, (P + 18) / 19), dim3(128, 4), 0, stream, p);
    return launch_pdl(shared_merge_kernel<1>, dim3(64, (P + 1) / 2), dim3(128), 0, stream, p);
}

}  // namespace mla
