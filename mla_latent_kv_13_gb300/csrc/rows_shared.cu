// rows_shared.cu -- the merge of the items that the clusters' shares cut, in decode attention over a
// batch whose sequences share prefixes (rows_shared.cuh).
#include "common.cuh"
#include "rows.h"

namespace mla {

namespace {

constexpr int G = 5;  // parts in flight

__device__ __forceinline__ void ld_v8(const float *src, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                   "=f"(v[7])
                 : "l"(src));
}

// CTA (x, c) merges 8 columns of 128 half-rows of the item that cluster c's end cut first, by the
// log-sum-exps of its parts (2 c + 1, 2 (c + 1), 2 (c + 2), ..). The parts lie as the attention
// kernel's threads hold them: part [2 CTAs][32 pieces of 8 columns][128 lanes][8], lane l of CTA r row
// 64 r + l % 64 with its columns from 256 (l / 64) on, so a thread keeps to its lane and every load is
// whole lines (a row by one warp, part after part row-major: 14 us where this takes 5, 76 cuts of 128
// rows). Five parts are in flight at a time (3 to 12, and 16 columns, are within 3%).
__global__ void __launch_bounds__(128) shared_merge_kernel(RowsParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int c = blockIdx.y, tl = threadIdx.x, cta = blockIdx.x & 1, piece = blockIdx.x >> 1;
    const int4 job = p.sh.jobs[c];
    const int r = 64 * cta + (tl & 63);
    if (r >= job.y) return;
    const int np = job.z;
    float v[G][8], l[G];
    auto load = [&](int k0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            l[g] = -INFINITY;
            if (k0 + g < np) {
                const int id = k0 + g == 0 ? 2 * c + 1 : 2 * (c + k0 + g);
                const float *src = p.o_part + ((size_t)(2 * id + cta) * 32 + piece) * 1024 + 8 * tl;
                l[g] = p.lse_part[(size_t)id * p.rows_per_item + r];
                ld_v8(src, v[g]);
            }
        }
    };
    // as the parts come: the sums so far belong to the reference m
    float m = -INFINITY, den = 0.f, acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < np; k0 += G) {
        load(k0);
        float top = m;
#pragma unroll
        for (int g = 0; g < G; ++g) top = fmaxf(top, l[g]);
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
    const float inv = den > 0.f ? 1.f / den : 0.f;
    const size_t row = (size_t)job.x + r;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    *reinterpret_cast<uint4 *>(p.out + row * D_C + 256 * (tl >> 6) + 8 * piece) =
        make_uint4(o[0], o[1], o[2], o[3]);
    if (piece == 0 && tl < 64) p.lse[row] = den > 0.f ? m + __logf(den) : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_merge(const RowsParams &p, cudaStream_t stream) {
    return launch_pdl(shared_merge_kernel, dim3(64, p.sh.clusters), dim3(128), 0, stream, p);
}

}  // namespace mla
