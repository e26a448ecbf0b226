// rows_shared.cuh -- the work list of decode attention over a batch whose sequences share prefixes
// (rows.h), worked out by every cluster for itself before its roles begin.
//
// A group's sequences are taken 128 / (H s_q) at a time, as items: the pages that they have in common
// are multiplied once for the rows of all of them, then each one's own pages with the others' rows
// masked, in one pass with one accumulator. A tile takes its 2176 tensor cycles however many of its rows
// are live, so the own pages cost what they would as items of their own, without their starts and
// with nothing to merge (five prompts of up to 6000 rows, 128 sequences of 32 heads: 72 us with items of
// their own, 67.6 so, before the other changes). With H s_q > 64 an item is one sequence and the common
// pages are merely found in L2.
//
// Sequences stay apart although they share an accumulator: a cached row that is not finite would reach the
// others as 0 * NaN. Where some token does not see a whole page (PAGE_APART) the softmax looks at the
// page's scores: such a row's are not finite for any query. Then those who see it get NaN, and what is not
// finite in V becomes zeros for the rest. Looking costs 32 instructions a tile, under 1% (five prompts 53.6
// -> 54.2 us in a replayed graph, drafts over FP8 41.3 -> 41.5, four samples 13.8 -> 13.9).
//
// Items weigh their tiles and ROWS_SEG_COST, laid end to end and cut evenly over the clusters. Every
// cluster works the list out by itself: a launch of its own for it took 5 us of a small call's 29, this
// 2 to 4. Most of that is fetching instructions that run once, hence the rolled loops. The pages are
// looked up beforehand, by all threads, so that the roles read one entry for each.
//
// Bound by the tensor pipe under the power cap where the common pages are many: 96 samples of 64 heads
// behind 16,000 rows take 155 us (140 before the cap comes in, after some 50 ms of them), of which the list
// 4, the first scores 3, the last output 3 and the merge 7; in between 1.68 PFLOP/s. A tile takes 1.3 us
// (1.05 by its cycles at 2.07 GHz): its K and V are 272 KB out of L2 for a pair of CTAs, 16 TB/s over the
// GPU. Not kept: L2 prefetches of the own pages (55 to 57 to 66 us, five prompts, with 16, 32 and all pages
// ahead), shares snapped to the items' ends (45 to 48 and 55 us, drafts over FP8, within 2 and 4 tiles), a
// start-up weight of 6 to 11 (flat to 3% slower).
#pragma once

#include <limits.h>

#include "common.cuh"
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
constexpr int SHARED_SCRATCH = SHARED_MAX_SEQS * (int)(4 * 4 + sizeof(SharedItem)) + 1024;

// pages of a sequence beside the item's common ones
__device__ __forceinline__ int shared_own(int len, int common) {
    return len / BLOCK + (len % BLOCK != 0) - min(common, len / BLOCK);
}
// The pages and tiles of an item of it.n sequences from it.b0 on, whose first `prefix` rows are the same.
__device__ __forceinline__ void shared_tiles(SharedItem &it, const int *lens, int prefix) {
    int L[8], longest = 0;  // (all loads before any of them is looked at)
#pragma unroll
    for (int k = 0; k < 8; ++k) L[k] = k < it.n ? lens[it.b0 + k] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) longest = max(longest, L[k]);
    it.common = min(prefix, longest) / BLOCK;
    int pages = it.common;
#pragma unroll
    for (int k = 0; k < 8; ++k) pages += shared_own(L[k], it.common);
    it.tiles = (pages + 1) / 2;
}
// (one copy: what the list takes is the fetching of instructions that run once)
__device__ __noinline__ int shared_scan(int x, int *warp_tot, int *total) {
    return scan_block(x, warp_tot, total);
}

// The arrays of the list in `scratch` (SHARED_SCRATCH bytes of shared memory that nothing else uses
// meanwhile).
struct SharedList {
    int *misc;           // warp totals [33], then
    int *from, *to;      // this cluster's first and last item
    int *lens;           // [B]
    int *gs;             // group starts [groups + 1]
    int *pre;            // their prefixes [groups]
    int *first;          // first item of each run of sequences [groups + 3]
    SharedItem *items;   // [B]
    int r0, r1;          // this cluster's share of the weight
    __device__ __forceinline__ SharedList(const RowsParams &p, uint8_t *scratch) {
        misc = reinterpret_cast<int *>(scratch);
        from = misc + 40, to = misc + 41;
        lens = misc + 64;
        gs = lens + p.B;
        pre = gs + p.sh.groups + 1;
        first = pre + p.sh.groups;
        items = reinterpret_cast<SharedItem *>(first + p.sh.groups + 3);
    }
};

// By all threads of the CTA: this cluster's segments, sh.segs[x .. y), the first of them in *own (shared
// memory) too. Other threads' results are theirs to read after the next barrier.
__device__ __forceinline__ int2 shared_list(const RowsParams &p, SharedList &l, int cl, bool first_cta,
                                            RowsSegment *own) {
    const SharedParams &sh = p.sh;
    const int tid = threadIdx.x, T = blockDim.x, B = p.B;
    int *const misc = l.misc, *const from = l.from, *const to = l.to, *const lens = l.lens,
               *const gs = l.gs, *const pre = l.pre, *const first = l.first;
    SharedItem *const items = l.items;

    // ---- lengths and groups; what is wrong is recorded, and ranges that do not ascend within [0, B]
    // share nothing. (All loads of a round before any of them is looked at.)
    bool broken = false;
    const int most = max(B, sh.groups + 1);
#pragma unroll 1
    for (int k = tid; k < most; k += T) {
        int L = 0, a = 0, e = 0, prefix = 0;
        if (k < B) L = p.seqlens[k];
        if (k <= sh.groups) a = sh.group_starts[k];
        if (k < sh.groups) e = sh.group_starts[k + 1], prefix = sh.prefix_lens[k];
        if (k < B) {
            lens[k] = min(max(L, 0), p.max_seqlen);
            if (first_cta && lens[k] != L) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, k);
        }
        if (k <= sh.groups) {
            gs[k] = a;
            if (k < sh.groups) pre[k] = max(prefix, 0);
            const bool wrong = a < 0 || a > B || (k < sh.groups && e < a);
            broken |= wrong;
            if (first_cta && (wrong || prefix < 0)) flag_error(p.err, MLA_ERR_OUT_OF_RANGE, k);
        }
    }
    if (tid == 0) *from = INT_MAX, *to = -1;
    broken = __syncthreads_or(broken);
    const int G = broken ? -1 : sh.groups;

    // ---- runs of sequences: those before the first group, the groups, those behind the last (broken:
    // one run of all)
    const int shift = 31 - __clz(128 / (p.hq * p.s_q));  // sequences of an item: 1, 2, 4 or 8
    auto run_begin = [&](int r) { return r == 0 ? 0 : gs[r - 1]; };
    auto run_end = [&](int r) { return r <= G ? gs[r] : B; };
    auto run_items = [&](int r) { return (run_end(r) - run_begin(r) + (1 << shift) - 1) >> shift; };
    auto item = [&](int r, int i) {  // the i-th item of run r
        SharedItem it{0, 0, 0, 0, 0};
        it.b0 = run_begin(r) + (i << shift);
        it.n = min(1 << shift, run_end(r) - it.b0);
        shared_tiles(it, lens, r >= 1 && r <= G ? pre[r - 1] : 0);
        return it;
    };

    // ---- this cluster's share [r0, r1) of the weight W, one more for the first W % P: the pieces of items
    // in it. An item without tiles is a piece too (its rows are written as empty ones), at the end of
    // its start-up.
    int W = 0, share = 0, more = 0, r0 = 0, r1 = 0;
    auto take_share = [&](int least) {
        const int P = min(sh.clusters, (W + least - 1) / least);
        share = W / P, more = W - share * P;
        r0 = min(cl * share + min(cl, more), W);
        r1 = min(r0 + share + (cl < more), W);
    };
    auto mine = [&](const SharedItem &it) {
        const int a = it.tiles > 0 ? it.at : it.at - 1, e = it.tiles > 0 ? it.at + it.tiles : it.at;
        return a < r1 && e > r0;
    };
    // writes item i's piece; whether the share's end cuts it first (then the merge's job too)
    auto put = [&](int i, const SharedItem &it, bool is_first) {
        RowsSegment g;
        g.b = it.b0, g.tok0 = it.b0 * p.s_q, g.ntok = it.n * p.s_q, g.pos0 = it.common;
        g.t0 = max(r0 - it.at, 0);
        g.t1 = min(r1 - it.at, it.tiles);
        const bool begins = it.at >= r0, ends = it.at + it.tiles <= r1;
        g.part = it.tiles == 0 || (begins && ends) ? -1 : begins ? 2 * cl + 1 : 2 * cl;
        if (it.tiles == 0) g.t0 = g.t1 = 0;
        g.at = it.at;
        sh.segs[i + cl] = g;
        if (is_first) *own = g;
        if (it.tiles == 0 || !begins || ends) return false;
        // the cluster that has its last tile
        const int w = it.at + it.tiles - 1, big = more * (share + 1);
        const int last = w < big ? w / (share + 1) : more + (w - big) / share;
        sh.jobs[cl] = make_int4(g.tok0 * p.hq, g.ntok * p.hq, last - cl + 1, 0);
        return true;
    };

    if ((B >> shift) + sh.groups + 2 <= 32) {
        // at most 32 items: one warp, an item a lane, without barriers in between (a small call 17.1 ->
        // 16.8 us, 12 items over FP8 44.3 -> 43.3)
        if (tid < 32) {
            int r = 0, i = tid;
#pragma unroll 1
            for (int k; r < G + 2 && i >= (k = run_items(r)); ++r) i -= k;
            SharedItem it{0, 0, 0, 0, 0};
            int w = 0;
            if (r < G + 2) it = item(r, i), w = it.tiles + ROWS_SEG_COST;
            int sum = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (tid >= o) sum += y;
            }
            W = __shfl_sync(0xffffffffu, sum, 31);
            // Shares of one tile while the items are short; of two from 24 tiles an item on, whose parts would
            // cost the merge more (us with one, two, three: 1 item of 19 tiles 13.7, 14.7, 15.2; one of 62
            // 17.7, 15.9, 16.4; 3 of 31 20.1, 18.8, 18.4).
            const int n = __popc(__ballot_sync(0xffffffffu, w > 0));
            take_share(W >= (24 + ROWS_SEG_COST) * n ? 2 : 1);
            it.at = sum - w + ROWS_SEG_COST;
            if (w > 0) items[tid] = it;
            const unsigned in = __ballot_sync(0xffffffffu, w > 0 && mine(it));
            const bool cut = in >> tid & 1 && put(tid, it, tid == __ffs(in) - 1);
            const bool any = __any_sync(0xffffffffu, cut);
            if (tid == 0) {
                if (!any) sh.jobs[cl] = make_int4(0, 0, 0, 0);
                *from = __ffs(in) - 1, *to = 31 - __clz(in);
                misc[42] = r0, misc[43] = r1;
            }
        }
        __syncthreads();
        r0 = misc[42], r1 = misc[43];
    } else {
        int n = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < G + 2; b0 += T) {
            const int r = b0 + tid;
            int total;
            const int at = n + shared_scan(r < G + 2 ? run_items(r) : 0, misc, &total);
            if (r < G + 2) first[r] = at;
            n += total;
        }
        __syncthreads();
#pragma unroll 1
        for (int b0 = 0; b0 < n; b0 += T) {
            const int i = b0 + tid;
            SharedItem it{0, 0, 0, 0, 0};
            if (i < n) {
                int r = 0, hi = G + 1;  // the last run whose first item is at most i
#pragma unroll 1
                while (r < hi) {
                    const int mid = (r + hi + 1) >> 1;
                    if (first[mid] <= i) r = mid;
                    else hi = mid - 1;
                }
                it = item(r, i - first[r]);
            }
            int total;
            const int at = shared_scan(i < n ? it.tiles + ROWS_SEG_COST : 0, misc, &total);
            it.at = W + at + ROWS_SEG_COST;
            if (i < n) items[i] = it;
            W += total;
        }
        __syncthreads();
        take_share(1);
        bool cut = false;
#pragma unroll 1
        for (int i = tid; i < n; i += T) {
            const SharedItem it = items[i];
            if (!mine(it)) continue;
            atomicMin(from, i);
            atomicMax(to, i);
            cut |= put(i, it, i == 0 || !mine(items[i - 1]));
        }
        if (!__syncthreads_or(cut) && tid == 0) sh.jobs[cl] = make_int4(0, 0, 0, 0);
    }
    l.r0 = r0, l.r1 = r1;
    const int i0 = *from, i1 = *to;
    return i1 < 0 ? make_int2(0, 0) : make_int2(i0 + cl, i1 + cl + 1);
}

// The pages of this cluster's tiles, by `T` threads; `list` is what shared_list gave.
__device__ __forceinline__ void shared_pages(const RowsParams &p, const SharedList &l, int2 list, int cl,
                                             int T) {
    const SharedParams &sh = p.sh;
    if (list.x >= list.y) return;
    const int i0 = list.x - cl, i1 = list.y - 1 - cl;
    const SharedItem *const items = l.items;
    const int *const lens = l.lens;
#pragma unroll 1
    for (int w = 2 * l.r0 + static_cast<int>(threadIdx.x); w < 2 * l.r1; w += T) {
        const int at = w >> 1;
        int lo = i0, hi = i1;  // the last of its items that begins (its start-up) at or before this place
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (items[mid].at - ROWS_SEG_COST <= at) lo = mid;
            else hi = mid - 1;
        }
        const SharedItem it = items[lo];
        if (at < it.at || at >= it.at + it.tiles) continue;
        int v = 2 * (at - it.at) + (w & 1), row = 0;
        SharedPage g{-2, 0, 0, 0};
        if (v < it.common) {
            // through the table of the longest sequence: the others' end where they do
            int longest = -1;
#pragma unroll 1
            for (int k = 0; k < it.n; ++k) {
                const int L = lens[it.b0 + k];
                if (L > longest) longest = L, row = it.b0 + k;
                if (max(L - p.s_q + 1, 0) / BLOCK <= v) g.owner = PAGE_APART;
            }
            g.id = 0, g.base = v * BLOCK, g.rows = BLOCK;
        } else {
            v -= it.common;
#pragma unroll 1
            for (int k = 0; k < it.n; ++k) {
                const int L = lens[it.b0 + k], skip = min(it.common, L / BLOCK);
                const int own = shared_own(L, it.common);
                if (v < own) {
                    row = it.b0 + k;
                    g.id = 0, g.owner = k + 1;
                    g.base = (skip + v) * BLOCK, g.rows = min(BLOCK, L - g.base);
                    if (it.n > 1 || g.base + g.rows > L - p.s_q + 1) g.owner |= PAGE_APART;
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
}

}  // namespace mla
