// rows_shared.cuh -- the work list of decode attention over a batch whose sequences share prefixes
// (rows.h), worked out by every cluster for itself before its roles begin.
//
// A group's sequences are taken 128 / (H s_q) at a time, as items: the pages that they have in common
// are multiplied once for the rows of all of them, then each one's own pages with the others' rows
// masked, in one pass with one accumulator. A tile takes its 2176 tensor cycles however many of its rows
// are live, so the own pages cost what they would as items of their own, without their start and
// with nothing to merge (128 sequences of 32 heads behind five prompts of up to 6000 rows 72 -> 44 us,
// their own pages as items before). With H s_q > 64 an item is one sequence and the common pages are
// merely found in L2.
//
// Items weigh their tiles and ROWS_SEG_COST, laid end to end and cut evenly over the clusters. A launch
// of its own for the list took 5 us of a small call's 29; the lengths of the whole batch are one round
// trip to memory and the sums a dozen barriers.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "rows.h"
#include "scan.cuh"

namespace mla {

// An item: where its tiles lie (at), how many, its first sequence and number of sequences, pages in
// common.
struct SharedItem {
    int at, tiles, b0, n, common;
};
constexpr int SHARED_MAX_SEQS = 4096;
// shared memory that the work list takes while it is made
constexpr int SHARED_SCRATCH = SHARED_MAX_SEQS * (int)(4 + 4 + 4 + sizeof(SharedItem)) + 1024;

// By all threads of the CTA; returns this cluster's segments, sh.segs[x .. y). `scratch` is shared
// memory (SHARED_SCRATCH bytes) that nothing else uses meanwhile.
__device__ __forceinline__ int2 shared_work(const RowsParams &p, uint8_t *scratch, int cl, bool first_cta) {
    const SharedParams &sh = p.sh;
    const int tid = threadIdx.x, T = blockDim.x, B = p.B;
    int *misc = reinterpret_cast<int *>(scratch);  // warp totals [33], then
    int *from = misc + 40, *to = misc + 41;         // this cluster's first and last item
    int *lens = misc + 64;
    int *gs = lens + B;              // group starts [groups + 1]
    int *first = gs + sh.groups + 1;  // first item of each run of sequences [groups + 3]
    SharedItem *items = reinterpret_cast<SharedItem *>(first + sh.groups + 3);

    // ---- lengths and groups; what is wrong is recorded, and ranges that do not ascend within [0, B]
    // share nothing
    bool broken = false;
    for (int g = tid; g <= sh.groups; g += T) {
        const int a = sh.group_starts[g];
        gs[g] = a;
        broken |= a < 0 || a > B || (g < sh.groups && sh.group_starts[g + 1] < a);
        if (first_cta && (broken || (g < sh.groups && sh.prefix_lens[g] < 0)))
            flag_error(p.err, MLA_ERR_OUT_OF_RANGE, g);
    }
    for (int b = tid; b < B; b += T) {
        const int L = p.seqlens[b];
        lens[b] = min(max(L, 0), p.max_seqlen);
        if (first_cta && lens[b] != L) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, b);
    }
    if (tid == 0) *from = INT_MAX, *to = -1;
    broken = __syncthreads_or(broken);
    const int G = broken ? -1 : sh.groups;

    // ---- runs of sequences: those before the first group, the groups, those behind the last (broken:
    // one run of all)
    const int per = 128 / (p.hq * p.s_q);  // sequences of an item
    auto run_begin = [&](int r) { return r == 0 ? 0 : gs[r - 1]; };
    auto run_end = [&](int r) { return r <= G ? gs[r] : B; };
    int n = 0;
    for (int r0 = 0; r0 < G + 2; r0 += T) {
        const int r = r0 + tid;
        int k = 0;
        if (r < G + 2) k = (run_end(r) - run_begin(r) + per - 1) / per;
        int total;
        const int at = n + scan_block(k, misc, &total);
        if (r < G + 2) first[r] = at;
        n += total;
    }
    __syncthreads();

    // ---- items
    int W = 0;
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        SharedItem it{0, 0, 0, 0, 0};
        if (i < n) {
            int lo = 0, hi = G + 1;  // the last run whose first item is at most i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            it.b0 = run_begin(lo) + (i - first[lo]) * per;
            it.n = min(per, run_end(lo) - it.b0);
            int longest = 0;
            for (int k = 0; k < it.n; ++k) longest = max(longest, lens[it.b0 + k]);
            if (lo >= 1 && lo <= G) it.common = min(max(sh.prefix_lens[lo - 1], 0), longest) / BLOCK;
            int pages = it.common;
            for (int k = 0; k < it.n; ++k) {
                const int L = lens[it.b0 + k];
                pages += (L > 0 ? (L - 1) / BLOCK + 1 : 0) - min(it.common, L / BLOCK);
            }
            it.tiles = (pages + 1) / 2;
        }
        int total;
        const int at = scan_block(i < n ? it.tiles + ROWS_SEG_COST : 0, misc, &total);
        it.at = W + at + ROWS_SEG_COST;
        if (i < n) items[i] = it;
        W += total;
    }
    __syncthreads();

    // ---- this cluster's share [r0, r1) of the weight: the pieces of items in it. An item without tiles
    // is a piece too (its rows are written as empty ones), at the end of its start-up.
    const int P = min(sh.clusters, W);
    const int r0 = cl < P ? static_cast<int>((cl * (long)W) / P) : W;
    const int r1 = cl < P ? static_cast<int>(((cl + 1) * (long)W) / P) : W;
    auto mine = [&](const SharedItem &it) {
        const int a = it.tiles > 0 ? it.at : it.at - 1, e = it.tiles > 0 ? it.at + it.tiles : it.at;
        return a < r1 && e > r0;
    };
    int4 job = make_int4(0, 0, 0, 0);
    bool cut = false;
    for (int i = tid; i < n; i += T) {
        const SharedItem it = items[i];
        if (!mine(it)) continue;
        atomicMin(from, i);
        atomicMax(to, i);
        RowsSegment g;
        g.b = it.b0, g.tok0 = it.b0 * p.s_q, g.ntok = it.n * p.s_q, g.pos0 = it.common;
        g.t0 = max(r0 - it.at, 0);
        g.t1 = min(r1 - it.at, it.tiles);
        const bool begins = it.at >= r0, ends = it.at + it.tiles <= r1;
        g.part = it.tiles == 0 || (begins && ends) ? -1 : begins ? 2 * cl + 1 : 2 * cl;
        if (it.tiles == 0) g.t0 = g.t1 = 0;
        g.at = it.at;
        sh.segs[i + cl] = g;
        if (it.tiles > 0 && begins && !ends) {
            cut = true;
            job = make_int4(g.tok0 * p.hq, g.ntok * p.hq,
                            cluster_of_tile(it.at + it.tiles - 1, W, P) - cl + 1, 0);
        }
    }
    if (cut) sh.jobs[cl] = job;  // one thread's, if any
    if (!__syncthreads_or(cut) && tid == 0) sh.jobs[cl] = job;
    const int i0 = *from, i1 = *to;

    // ---- the pages of its tiles
    for (int w = 2 * r0 + tid; w < 2 * r1; w += T) {
        const int at = w >> 1;
        int lo = i0, hi = i1;  // the last of its items that begins (its start-up) at or before this place
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (items[mid].at - ROWS_SEG_COST <= at) lo = mid;
            else hi = mid - 1;
        }
        if (i1 < 0) break;
        const SharedItem it = items[lo];
        if (at < it.at || at >= it.at + it.tiles) continue;
        int v = 2 * (at - it.at) + (w & 1), row = 0;
        SharedPage g{-2, 0, 0, 0};
        if (v < it.common) {
            // through the table of the longest sequence: the others' end where they do
            int longest = -1;
            for (int k = 0; k < it.n; ++k)
                if (lens[it.b0 + k] > longest) longest = lens[it.b0 + k], row = it.b0 + k;
            g.id = 0, g.base = v * BLOCK, g.rows = BLOCK;
        } else {
            v -= it.common;
            for (int k = 0; k < it.n; ++k) {
                const int L = lens[it.b0 + k], skip = min(it.common, L / BLOCK);
                const int own = (L > 0 ? (L - 1) / BLOCK + 1 : 0) - skip;
                if (v < own) {
                    row = it.b0 + k;
                    g.id = 0, g.owner = k + 1;
                    g.base = (skip + v) * BLOCK, g.rows = min(BLOCK, L - g.base);
                    break;
                }
                v -= own;
            }
        }
        if (g.id == 0) {
            g.id = p.block_table[(size_t)row * p.max_blocks + g.base / BLOCK];
            if (g.id < 0 || g.id >= p.num_blocks) {
                flag_error(p.err, MLA_ERR_OUT_OF_RANGE, row);
                g = SharedPage{-2, 0, 0, 0};
            }
        }
        *reinterpret_cast<int4 *>(sh.pages + w) = make_int4(g.id, g.base, g.owner, g.rows);
    }
    return i1 < 0 ? make_int2(0, 0) : make_int2(i0 + cl, i1 + cl + 1);
}

}  // namespace mla
