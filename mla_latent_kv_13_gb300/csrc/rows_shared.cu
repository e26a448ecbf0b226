// rows_shared.cu -- the work list of decode attention over a batch whose sequences share prefixes
// (rows.h), and the merge of its parts.
//
// A group's queries are multiplied with the pages that its sequences have in common by items of
// 128 / H tokens each, whichever sequences these belong to: the pages are read and multiplied once
// for 128 rows instead of once for every sequence's H. The rest of each sequence is an item of its
// own, and every row joins the parts of both by their log-sum-exps. With H = 128 an item holds one
// token and nothing is won: every sequence is one item then, as it is in a group too small or with
// too short a prefix for the parts to pay.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "rows.h"
#include "scan.cuh"

namespace mla {

namespace {

constexpr int T_MAX = 1024;    // threads of the schedule kernel
constexpr int G_MAX = 4096;    // groups (at most as many as sequences)
// What an item of common pages costs beside its tiles, in tiles: its start, and the writing and
// merging of its parts.
constexpr int PREFIX_COST = ROWS_SEG_COST + 8;

// One CTA: the groups, their items, the items' pieces for the clusters. Items weigh their tiles and
// ROWS_SEG_COST, laid end to end and cut evenly, as in the ragged schedule.
__global__ void __launch_bounds__(T_MAX) shared_schedule_kernel(SharedSchedule s) {
    __shared__ int first_item[G_MAX + 1];
    __shared__ int warp_tot[33];
    __shared__ int bad;
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = T >> 5;
    const int per = 128 / s.hq;
    grid_launch_dependents();
    grid_dependency_wait();
    if (tid == 0) bad = -1;
    for (int c = tid; c < s.clusters; c += T) {
        s.seg_range[2 * c] = s.max_items + s.clusters;
        s.seg_range[2 * c + 1] = 0;
    }
    __syncthreads();

    // ---- what is wrong is recorded; ranges that do not ascend within [0, B] share nothing
    bool broken = false;
    for (int g = tid; g < s.groups; g += T) {
        const int a = s.group_starts[g], e = s.group_starts[g + 1];
        if (a < 0 || e < a || e > s.B) broken = true;
        if (broken || s.prefix_lens[g] < 0) atomicMax(&bad, g);
    }
    for (int b = tid; b < s.B; b += T) {
        const int L = s.seqlens[b];
        if (L < 0 || L > s.max_seqlen) atomicMax(&bad, b);
        s.seq_group[b] = -1;
    }
    broken = __syncthreads_or(broken);
    const int G = broken ? 0 : s.groups;
    if (tid == 0 && bad >= 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, bad);

    // ---- the pages that each group has in common, read through its longest sequence's table (the
    // others' tables end where they do)
    for (int g = warp; g < G; g += warps) {
        const int a = s.group_starts[g], e = s.group_starts[g + 1];
        int best = 0, at = INT_MAX, live = 0;
        for (int b = a + lane; b < e; b += 32) {
            const int L = min(max(s.seqlens[b], 0), s.max_seqlen);
            s.seq_group[b] = g;
            live += L > 0;
            if (L > best) best = L, at = b;
        }
        const int most = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == most ? at : INT_MAX);
        live = __reduce_add_sync(0xffffffffu, live);
        const int pages = min(max(s.prefix_lens[g], 0), most) / BLOCK;
        const long tiles = (pages + 1) / 2;
        const long k = ((long)(e - a) * s.s_q + per - 1) / per;
        const bool split = pages > 0 && k * (tiles + PREFIX_COST) < live * tiles;
        if (lane == 0)
            s.group_rec[g] = split ? make_int4(static_cast<int>(k), pages, at, a) : make_int4(0, 0, 0, a);
    }
    __syncthreads();
    int prefixes = 0;
    for (int g0 = 0; g0 < G; g0 += T) {
        const int g = g0 + tid;
        int total;
        const int at = prefixes + scan_block(g < G ? s.group_rec[g].x : 0, warp_tot, &total);
        if (g < G) s.group_rec[g].x = first_item[g] = at;
        prefixes += total;
    }
    __syncthreads();

    // ---- the items: first those of common pages, then every sequence's own
    const int n = prefixes + s.B;
    int W = 0;
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        int v = 0, first = 0, common = 0;
        if (i < prefixes) {
            int lo = 0, hi = G - 1;  // the last group whose first item is at most i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first_item[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const int4 g = s.group_rec[lo];
            const int tok0 = g.w * s.s_q + (i - g.x) * per;
            v = (g.y + 1) / 2;
            first = ROWS_PREFIX, common = g.y;
            s.items[i] = make_int4(g.z, tok0, min(per, s.group_starts[lo + 1] * s.s_q - tok0),
                                   g.y * BLOCK);
        } else if (i < n) {
            const int b = i - prefixes, g = s.seq_group[b];
            const int L = min(max(s.seqlens[b], 0), s.max_seqlen);
            const int pages = L > 0 ? (L - 1) / BLOCK + 1 : 0;
            common = g >= 0 ? s.group_rec[g].y : 0;
            first = min(common, L / BLOCK);  // a page that is not full is the sequence's own
            v = pages > first ? (pages - first + 1) / 2 : 0;
            s.items[i] = make_int4(b, b * s.s_q, s.s_q, L);
        }
        int total;
        const int at = scan_block(v > 0 ? v + ROWS_SEG_COST : 0, warp_tot, &total);
        if (i < n) s.item_rec[i] = make_int4(v > 0 ? W + at + ROWS_SEG_COST : -1, v, first, common);
        W += total;
    }

    // ---- their pieces; those of an item follow the ones of the items before it
    const int P = min(s.clusters, W);
    int segs = 0, rows = 0;
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        int c0 = 0, k = 0, mine = 0;
        int4 it = make_int4(0, 0, 0, 0), r = make_int4(-1, 0, 0, 0);
        if (i < n) it = s.items[i], r = s.item_rec[i];  // (written by this thread)
        const int w0 = r.x, v = r.y;
        if (v > 0) {
            c0 = cluster_of_tile(w0, W, P);
            k = cluster_of_tile(w0 + v - 1, W, P) - c0 + 1;
        }
        // where pages are in common, their items and the sequences' own are always parts
        const bool part = r.w > 0 || k > 1;
        const int height = it.z * s.hq;
        if (part) mine = k * height;
        int total, rtotal;
        const int at = segs + scan_block(k, warp_tot, &total);
        const int row = rows + scan_block(mine, warp_tot, &rtotal);
        for (int c = c0; c < c0 + k; ++c) {
            const long r0 = (c * (long)W) / P, r1 = ((c + 1) * (long)W) / P;
            RowsSegment g;
            g.b = it.x, g.tok0 = it.y, g.ntok = it.z, g.pos0 = it.w - it.z;
            g.t0 = static_cast<int>(max(r0, (long)w0) - w0);
            g.t1 = static_cast<int>(min(r1, (long)w0 + v) - w0);
            g.part = part ? row + (c - c0) * height : -1;
            g.first = r.z;
            s.segs[at + c - c0] = g;
            atomicMin(&s.seg_range[2 * c], at + c - c0);
            atomicMax(&s.seg_range[2 * c + 1], at + c - c0 + 1);
        }
        if (i < prefixes) {
            s.prefix_parts[i] = make_int4(row, k, height, 0);
        } else if (i < n) {
            int4 q = make_int4(part || k == 0 ? row : -1, k, -1, 0);
            if (r.w > 0) {
                const int4 g = s.group_rec[s.seq_group[it.x]];
                q.z = g.x, q.w = g.w * s.s_q;
            }
            s.seq_parts[it.x] = q;
        }
        segs += total;
        rows += rtotal;
    }
}

constexpr int MERGE_ROWS = 8;  // rows (one warp each) of a CTA

// One warp a row (token, head): its parts of the common pages, then those of the sequence's own, by
// their log-sum-exps. Rows of G parts are in flight together, the first ones before the
// weights are known.
__global__ void __launch_bounds__(32 * MERGE_ROWS)
    shared_merge_kernel(SharedSchedule s, const float *o_part, const float *lse_part, uint16_t *out,
                        float *lse) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long row = (long)blockIdx.x * MERGE_ROWS + (threadIdx.x >> 5);
    const int high = s.s_q * s.hq;  // rows of a sequence
    if (row >= (long)s.B * high) return;
    const int b = static_cast<int>(row / high);
    const int4 q = s.seq_parts[b];
    if (q.x < 0) return;
    int4 pre = make_int4(0, 0, 0, 0);
    int pre_row = 0;
    if (q.z >= 0) {
        const int per = 128 / s.hq;
        const int j = static_cast<int>(row / s.hq) - q.w;
        pre = s.prefix_parts[q.z + j / per];
        pre_row = pre.x + (j % per) * s.hq + static_cast<int>(row % s.hq);
    }
    const int own_row = q.x + static_cast<int>(row % high);
    const int np = pre.y + q.y;
    auto part = [&](int k) {
        return k < pre.y ? (size_t)pre_row + (size_t)k * pre.z
                         : (size_t)own_row + (size_t)(k - pre.y) * high;
    };
    constexpr int G = 4;
    float v[G][16];
    auto load = [&](int k0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const bool there = k0 + g < np;
            const float *src = o_part + (there ? part(k0 + g) : 0) * D_C + lane * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 u = there ? __ldcs(reinterpret_cast<const float4 *>(src + 128 * k))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                v[g][4 * k] = u.x, v[g][4 * k + 1] = u.y, v[g][4 * k + 2] = u.z, v[g][4 * k + 3] = u.w;
            }
        }
    };
    load(0);
    float m = -INFINITY, den = 0.f;
    for (int k = lane; k < np; k += 32) m = fmaxf(m, lse_part[part(k)]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m != -INFINITY)
        for (int k = lane; k < np; k += 32) den += __expf(lse_part[part(k)] - m);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float tot = m != -INFINITY ? m + __logf(den) : -INFINITY;
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    for (int k0 = 0; k0 < np; k0 += G) {
        if (k0 > 0) load(k0);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float l = k0 + g < np ? lse_part[part(k0 + g)] : -INFINITY;
            const float w = l != -INFINITY ? __expf(l - tot) : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] += w * v[g][j];
        }
    }
    uint16_t *dst = out + (size_t)row * D_C;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint2 *>(dst + lane * 4 + 128 * k) =
            make_uint2(pack_bf16x2(acc[4 * k], acc[4 * k + 1]),
                       pack_bf16x2(acc[4 * k + 2], acc[4 * k + 3]));
    if (lane == 0) lse[row] = tot;
}

}  // namespace

cudaError_t launch_shared_schedule(const SharedSchedule &s, cudaStream_t stream) {
    // as many threads as there is work for in one round: barriers of few warps are cheaper
    int most = s.max_items > s.clusters ? s.max_items : s.clusters;
    const int threads = most >= T_MAX ? T_MAX : (most + 31) / 32 * 32;
    return launch_pdl(shared_schedule_kernel, dim3(1), dim3(threads), 0, stream, s);
}

cudaError_t launch_shared_merge(const SharedSchedule &s, const float *o_part, const float *lse_part,
                                uint16_t *out, float *lse, cudaStream_t stream) {
    const long rows = (long)s.B * s.s_q * s.hq;
    return launch_pdl(shared_merge_kernel, dim3((unsigned)((rows + MERGE_ROWS - 1) / MERGE_ROWS)),
                      dim3(32 * MERGE_ROWS), 0, stream, s, o_part, lse_part, out, lse);
}

}  // namespace mla
