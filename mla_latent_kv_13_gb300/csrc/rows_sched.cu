// rows_sched.cu -- the work list of the ragged attention (rows.h): items, their balanced shares
// of the tiles over the clusters, and the merge of the items that a share's end cuts.
#include "common.cuh"
#include "kernels.h"
#include "merge.cuh"
#include "rows.h"

namespace mla {

namespace {

constexpr int T_MAX = 1024;  // threads of the schedule kernel

// Exclusive prefix sum of one value per thread over the CTA; *total (optional) the sum.
__device__ __forceinline__ int scan_block(int x, int *warp_tot, int *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[w] = inc;
    __syncthreads();
    if (w == 0) {
        const int v = lane < static_cast<int>(blockDim.x >> 5) ? warp_tot[lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_tot[lane] = s - v;
        if (lane == 31) warp_tot[32] = s;
    }
    __syncthreads();
    const int before = warp_tot[w] + inc - x;
    *total = warp_tot[32];
    __syncthreads();
    return before;
}

// One CTA. Items of all sequences in order (tokens_per_item tokens each, the last one of a
// sequence the rest); an item with v > 0 tiles weighs v + ROWS_SEG_COST, laid end to end (its
// start-up first); cluster c of P takes the weight range [c W / P, (c + 1) W / P) and the tiles
// inside it. An item that lies in several ranges is cut: each piece gives an fp32 part, merged
// afterwards. Everything is written after the dependency wait: the arrays may still be read by
// the call before.
__global__ void __launch_bounds__(T_MAX) rows_schedule_kernel(RowsSchedule s) {
    __shared__ int first_item[4096 + 1];  // of each sequence
    __shared__ int warp_tot[33];
    __shared__ int bad;
    const int tid = threadIdx.x, T = blockDim.x;
    grid_launch_dependents();
    grid_dependency_wait();
    if (tid == 0) bad = -1;
    for (int c = tid; c < s.clusters; c += T) {
        s.seg_range[2 * c] = s.max_items + s.clusters;
        s.seg_range[2 * c + 1] = 0;
        s.jobs[c] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();

    // ---- items of each sequence; token ranges that do not ascend inside [0, tokens] make the
    // whole call void
    int carry = 0;
    bool broken = false;
    for (int b0 = 0; b0 < s.B; b0 += T) {
        const int b = b0 + tid;
        int k = 0;
        if (b < s.B) {
            int q0 = b * s.s_q, q1 = q0 + s.s_q;
            if (s.q_starts) q0 = s.q_starts[b], q1 = s.q_starts[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > s.tokens) atomicMax(&bad, b), broken = true;
            else k = (q1 - q0 + s.tokens_per_item - 1) / s.tokens_per_item;
            const int L = s.seqlens[b];
            if (L < 0 || L > s.max_seqlen) atomicMax(&bad, b);
        }
        int total;
        const int at = scan_block(k, warp_tot, &total);
        if (b < s.B) first_item[b] = carry + at;
        carry += total;
    }
    broken = __syncthreads_or(broken);
    const int n = broken ? 0 : carry;
    if (tid == 0) {
        first_item[s.B] = carry;
        *s.n_items = n;
        if (bad >= 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, bad);
    }
    __syncthreads();

    // ---- the items, their tiles and weight positions (the last round's stay in registers: the
    // only one where there are few)
    int W = 0, v_last = 0, w_last = -1;
    int4 it_last = make_int4(0, 0, 0, 0);
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        int v = 0;
        if (i < n) {
            int lo = 0, hi = s.B - 1;  // the last sequence whose first item is at most i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first_item[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const int q0 = s.q_starts ? s.q_starts[lo] : lo * s.s_q;
            const int q1 = s.q_starts ? s.q_starts[lo + 1] : q0 + s.s_q;
            const int at = (i - first_item[lo]) * s.tokens_per_item;
            const int nt = min(s.tokens_per_item, q1 - q0 - at);
            const int L = min(max(s.seqlens[lo], 0), s.max_seqlen);
            const int pos0 = L - (q1 - q0) + at;
            v = visible_tiles(visible_pages(pos0, nt, s.window, s.sinks));
            s.items[i] = it_last = make_int4(lo, q0 + at, nt, pos0);
        }
        int total;
        const int at = scan_block(v > 0 ? v + ROWS_SEG_COST : 0, warp_tot, &total);
        v_last = v;
        w_last = v > 0 ? W + at + ROWS_SEG_COST : -1;
        if (i < n) s.item_wpos[i] = w_last;
        W += total;
    }

    // ---- segments: the pieces of item i follow those of the items before it
    const int P = min(s.clusters, W);
    int segs = 0, parts = 0;
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        int v = 0, c0 = 0, c1 = 0, w0 = 0;
        int4 it = make_int4(0, 0, 0, 0);
        const bool last = i0 + T >= n;
        w0 = i >= n ? -1 : last ? w_last : s.item_wpos[i];
        if (w0 >= 0) {
            it = last ? it_last : s.items[i];
            v = last ? v_last : visible_tiles(visible_pages(it.w, it.z, s.window, s.sinks));
            c0 = cluster_of_tile(w0, W, P);
            c1 = cluster_of_tile(w0 + v - 1, W, P);
        }
        const int k = v > 0 ? c1 - c0 + 1 : 0;
        int total, ptotal;
        const int at = segs + scan_block(k, warp_tot, &total);
        const int pt = parts + scan_block(k > 1 ? k : 0, warp_tot, &ptotal);
        for (int c = c0; c < c0 + k; ++c) {
            const long r0 = (c * (long)W) / P, r1 = ((c + 1) * (long)W) / P;
            RowsSegment g;
            g.b = it.x, g.tok0 = it.y, g.ntok = it.z, g.pos0 = it.w;
            g.t0 = static_cast<int>(max(r0, (long)w0) - w0);
            g.t1 = static_cast<int>(min(r1, (long)w0 + v) - w0);
            g.part = k > 1 ? pt + c - c0 : -1;
            g.pad = 0;
            s.segs[at + c - c0] = g;
            atomicMin(&s.seg_range[2 * c], at + c - c0);
            atomicMax(&s.seg_range[2 * c + 1], at + c - c0 + 1);
        }
        if (k > 1) s.jobs[c0] = make_int4(it.y * s.hq, it.z * s.hq, pt, k);
        segs += total;
        parts += ptotal;
    }
}

// merge_row_warp for more than two parts: their log-sum-exps by all lanes at once and eight rows in
// flight, so a memory round trip for every eight parts (two parts a trip took 60 us for 76).
__device__ __forceinline__ void merge_row_many(const float *o0, size_t ostride, const float *l0,
                                               size_t lstride, int np, uint16_t *orow,
                                               float *lse_out, int lane) {
    constexpr int G = 8;
    float v[G][16], l[G];
    auto load = [&](int s0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const bool there = s0 + g < np;
            const float *row = o0 + (size_t)(s0 + g) * ostride + lane * 4;
            l[g] = there ? l0[(s0 + g) * lstride] : -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 u = there ? __ldcs(reinterpret_cast<const float4 *>(row + 128 * k))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                v[g][4 * k] = u.x, v[g][4 * k + 1] = u.y, v[g][4 * k + 2] = u.z, v[g][4 * k + 3] = u.w;
            }
        }
    };
    load(0);  // before the weights are known
    float m = -INFINITY, den = 0.f;
    for (int s = lane; s < np; s += 32) m = fmaxf(m, l0[s * lstride]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m != -INFINITY)
        for (int s = lane; s < np; s += 32) den += __expf(l0[s * lstride] - m);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float tot = m != -INFINITY ? m + __logf(den) : -INFINITY;
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    for (int s0 = 0; s0 < np; s0 += G) {
        if (s0 > 0) load(s0);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float w = l[g] != -INFINITY ? __expf(l[g] - tot) : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] += w * v[g][j];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint2 *>(orow + lane * 4 + 128 * k) =
            make_uint2(pack_bf16x2(acc[4 * k], acc[4 * k + 1]),
                       pack_bf16x2(acc[4 * k + 2], acc[4 * k + 3]));
    if (lane == 0) *lse_out = tot;
}
template <bool MANY>
__device__ __forceinline__ void merge_row(const float *o0, size_t ostride, const float *l0,
                                          size_t lstride, int np, uint16_t *orow, float *lse_out,
                                          int lane) {
    if (MANY && np > 2) merge_row_many(o0, ostride, l0, lstride, np, orow, lse_out, lane);
    else merge_row_warp(o0, ostride, l0, lstride, np, orow, nullptr, lse_out, lane);
}

constexpr int MERGE_ROWS = 8;   // rows (one warp each) per CTA
constexpr int EMPTY_CTAS = 16;  // rows of CTAs that look for items that see nothing

// Grid (ceil(rows_per_item / 8), P + EMPTY_CTAS): CTA (x, c < P) merges rows 8 x .. of the item
// cut at the end of cluster c's range; CTA (x, P + j) clears rows 8 x .. of the items without
// tiles among i = j (mod EMPTY_CTAS).
// MANY: items are expected to have more than two parts (the registers for eight rows in flight
// leave an SM one CTA).
template <bool MANY>
__global__ void __launch_bounds__(32 * MERGE_ROWS)
    rows_merge_kernel(RowsSchedule s, const float *o_part, const float *lse_part,
                      int rows_per_item, uint16_t *out, float *lse) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int r = blockIdx.x * MERGE_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (blockIdx.y >= s.clusters) {
        const int n = *s.n_items;
        for (int i = blockIdx.y - s.clusters; i < n; i += EMPTY_CTAS * 32) {
            const int mine = i + EMPTY_CTAS * lane;
            const bool empty = mine < n && s.item_wpos[mine] < 0;
            for (unsigned m = __ballot_sync(0xffffffffu, empty); m; m &= m - 1) {
                const int4 it = s.items[i + EMPTY_CTAS * (__ffs(m) - 1)];
                if (r >= it.z * s.hq) continue;
                const size_t row = (size_t)it.y * s.hq + r;
                uint4 *d = reinterpret_cast<uint4 *>(out + row * D_C);
                d[lane] = d[lane + 32] = make_uint4(0u, 0u, 0u, 0u);
                if (lane == 0) lse[row] = -INFINITY;
            }
        }
        return;
    }
    const int4 job = s.jobs[blockIdx.y];
    if (r >= job.y) return;
    const size_t row = (size_t)job.x + r;
    merge_row<MANY>(o_part + ((size_t)job.z * rows_per_item + r) * D_C, (size_t)rows_per_item * D_C,
                 lse_part + (size_t)job.z * rows_per_item + r, rows_per_item, job.w, out + row * D_C,
                 lse + row, lane);
}

// Fixed ranges: CTA (x, i) merges rows 8 x .. of item i.
__global__ void __launch_bounds__(32 * MERGE_ROWS) rows_merge_items_kernel(RowsParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.y;
    bool broken;
    const int4 it = p.q_starts ? find_item(p.q_starts, p.B, p.tokens, p.s_q, i, &broken)
                               : make_int4(i, i * p.s_q, p.s_q, 0);
    const int r = blockIdx.x * MERGE_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= it.z * p.hq) return;
    const size_t row = (size_t)it.y * p.hq + r;
    const size_t part = (size_t)i * p.num_splits * p.rows_per_item + r;
    merge_row<true>(p.o_part + part * D_C, (size_t)p.rows_per_item * D_C, p.lse_part + part,
                 p.rows_per_item, p.num_splits, p.out + row * D_C, p.lse + row, lane);
}

}  // namespace

cudaError_t launch_rows_merge_items(const RowsParams &p, int max_items, cudaStream_t stream) {
    const dim3 grid((p.rows_per_item + MERGE_ROWS - 1) / MERGE_ROWS, max_items);
    return launch_pdl(rows_merge_items_kernel, grid, dim3(32 * MERGE_ROWS), 0, stream, p);
}

cudaError_t launch_rows_schedule(const RowsSchedule &s, cudaStream_t stream) {
    // as many threads as there is work for in one round: barriers of few warps are cheaper
    int most = s.B > s.max_items ? s.B : s.max_items;
    if (s.clusters > most) most = s.clusters;
    const int threads = most >= T_MAX ? T_MAX : (most + 31) / 32 * 32;
    return launch_pdl(rows_schedule_kernel, dim3(1), dim3(threads), 0, stream, s);
}

cudaError_t launch_rows_merge(const RowsSchedule &s, const float *o_part, const float *lse_part,
                              int rows_per_item, uint16_t *out, float *lse, cudaStream_t stream) {
    const dim3 grid((rows_per_item + MERGE_ROWS - 1) / MERGE_ROWS, s.clusters + EMPTY_CTAS);
    // fewer items than a quarter of the clusters: more than four parts each, if they weigh alike
    // (1 item of 250 tiles 102 -> 55 us; 128 items of 33 tiles 111 us without, 113 with)
    const bool many = s.max_items < s.clusters / 4;
    return launch_pdl(many ? rows_merge_kernel<true> : rows_merge_kernel<false>, grid,
                      dim3(32 * MERGE_ROWS), 0, stream, s, o_part, lse_part, rows_per_item, out, lse);
}

}  // namespace mla
