// rows_shared.cu -- the merge of the items that the clusters' shares cut, in decode attention over a
// batch whose sequences share prefixes (rows_shared.cuh).
#include "common.cuh"
#include "rows.h"

namespace mla {

namespace {

constexpr int WARPS = 8;
constexpr int SPLIT = 4;  // warps of a row: 128 columns each, one 16-byte piece a lane

// CTA (x, c) merges two rows of the item that cluster c's end cut first, by the log-sum-exps of its
// parts. A small batch leaves few rows of many parts: a row's columns lie with four warps, and a lane
// has 16 parts in flight, the first ones before the weights are known.
__global__ void __launch_bounds__(32 * WARPS) shared_merge_kernel(RowsParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.y;
    const int4 job = p.sh.jobs[c];
    const int r = blockIdx.x * (WARPS / SPLIT) + warp / SPLIT;
    if (r >= job.y) return;
    const int np = job.z, col = 128 * (warp % SPLIT) + 4 * lane;
    auto row_of = [&](int k) {
        return (size_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * p.rows_per_item + r;
    };
    constexpr int G = 16;
    float4 v[G];
    auto load = [&](int k0) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            v[g] = k0 + g < np ? __ldcs(reinterpret_cast<const float4 *>(p.o_part + row_of(k0 + g) * D_C + col))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float l = lane < np ? p.lse_part[row_of(lane)] : -INFINITY, m = l;
    for (int k = lane + 32; k < np; k += 32) m = fmaxf(m, p.lse_part[row_of(k)]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float den = 0.f;
    if (m != -INFINITY) {
        den = __expf(l - m);
        for (int k = lane + 32; k < np; k += 32) den += __expf(p.lse_part[row_of(k)] - m);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float tot = m != -INFINITY ? m + __logf(den) : -INFINITY;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float w = l != -INFINITY ? __expf(l - tot) : 0.f;  // of part `lane` of the present 32
    for (int k0 = 0; k0 < np; k0 += G) {
        if (k0 > 0) {
            load(k0);
            if (k0 % 32 == 0) {
                l = k0 + lane < np ? p.lse_part[row_of(k0 + lane)] : -INFINITY;
                w = l != -INFINITY ? __expf(l - tot) : 0.f;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float u = __shfl_sync(0xffffffffu, w, (k0 + g) & 31);
            acc.x += u * v[g].x, acc.y += u * v[g].y, acc.z += u * v[g].z, acc.w += u * v[g].w;
        }
    }
    const size_t row = (size_t)job.x + r;
    *reinterpret_cast<uint2 *>(p.out + row * D_C + col) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    if (lane == 0 && warp % SPLIT == 0) p.lse[row] = tot;
}

}  // namespace

cudaError_t launch_shared_merge(const RowsParams &p, cudaStream_t stream) {
    const int rows = WARPS / SPLIT;
    const dim3 grid((p.rows_per_item + rows - 1) / rows, p.sh.clusters);
    return launch_pdl(shared_merge_kernel, grid, dim3(32 * WARPS), 0, stream, p);
}

}  // namespace mla
