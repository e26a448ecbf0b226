// pages.cu -- the life of the paged cache's pages, on the device: sequences release their
// pages, take the lowest free ones, fork (full pages shared, the last partial one copied), and
// the pool is compacted.
//
// Results depend on the order of the lists alone, never on the order in which threads run: free
// pages are handed out in ascending order by prefix sums, reference counts are whole numbers.
// Bound by the bytes of the copied pages (each read and written once); the plans' single pass
// over the reference counts costs a few microseconds for pools of some ten thousand pages.
#include "common.cuh"
#include "kernels.h"
#include "serve.h"

namespace mla {

namespace {

constexpr int T = 1024;

// Exclusive prefix sum of one value per thread over a CTA of whole warps.
template <typename N>
__device__ __forceinline__ N scan_block(N x, N *warp_tot, N *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    N inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[w] = inc;
    __syncthreads();
    if (w == 0) {
        const N v = lane < static_cast<int>(blockDim.x >> 5) ? warp_tot[lane] : 0;
        N s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const N y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_tot[lane] = s - v;
        if (lane == 31) warp_tot[32] = s;
    }
    __syncthreads();
    const N before = warp_tot[w] + inc - x;
    *total = warp_tot[32];
    __syncthreads();
    return before;
}

__device__ __forceinline__ int pages_of(int len) {
    return len / BLOCK + (len % BLOCK != 0);
}

// ------------------------------------------------------------------------------- free

// One CTA per list entry. Whoever swaps the row's length for 0 releases its pages, so a row
// that is listed twice is released once.
__global__ void __launch_bounds__(128) pages_free_kernel(PageState s, const int32_t *rows) {
    __shared__ int len_;
    grid_launch_dependents();
    grid_dependency_wait();
    const int row = rows[blockIdx.x];
    if (row < 0 || row >= s.num_seqs) {
        if (threadIdx.x == 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, blockIdx.x);
        return;
    }
    if (threadIdx.x == 0) len_ = atomicExch(s.seqlens + row, 0);
    __syncthreads();
    int len = len_;
    const long cap = (long)s.max_blocks * BLOCK;
    if (len < 0 || len > cap) {
        if (threadIdx.x == 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, blockIdx.x);
        len = len < 0 ? 0 : static_cast<int>(cap);
    }
    int32_t *tab = s.table + (size_t)row * s.max_blocks;
    for (int k = threadIdx.x; k < pages_of(len); k += blockDim.x) {
        const int id = tab[k];
        tab[k] = -1;
        if (id < 0 || id >= s.num_blocks) {
            flag_error(s.err, MLA_ERR_OUT_OF_RANGE, blockIdx.x);
        } else if (atomicSub(s.refs + id, 1) <= 0) {
            atomicAdd(s.refs + id, 1);  // nobody held it
            flag_error(s.err, MLA_ERR_OUT_OF_RANGE, blockIdx.x);
        }
    }
}

// -------------------------------------------------------------------- extend and fork

// Which of the 16 pages from `first` on are free, as bits.
__device__ __forceinline__ unsigned free16(const PageState &s, int first) {
    unsigned mask = 0;
    if (first + 16 <= s.num_blocks && reinterpret_cast<uintptr_t>(s.refs) % 16 == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int4 r = *reinterpret_cast<const int4 *>(s.refs + first + 4 * k);
            mask |= ((r.x <= 0) | (r.y <= 0) << 1 | (r.z <= 0) << 2 | (r.w <= 0) << 3) << 4 * k;
        }
    } else {
        for (int k = 0; k < 16; ++k)
            if (first + k < s.num_blocks && s.refs[first + k] <= 0) mask |= 1u << k;
    }
    return mask;
}

constexpr int PER = PAGE_LIST_MAX / T;      // entries of a thread, at most
constexpr unsigned NO_ENTRY = 0xFFFFFFFFu;  // an empty slot of the table of rows
static_assert(PAGE_LIST_MAX <= 1 << 12, "an entry's index has 12 bits beside the row's 20");
constexpr int FRESH = 1536;                 // fresh pages that an extend keeps in shared memory
__host__ __device__ constexpr int plan_slots(int n) { return n + n / 2 + 32; }

// One CTA: which entries of the list are valid (the first that names a row wins), the fresh
// pages each needs, and the lowest free pages in the list's order.
// extend: args = new lengths, rows grow, here and now (one launch: the pages of a call are few for
// a thousand threads). fork: args = parents, rows = the empty children; writes the plan alone.
//
// Bound by the chain of round trips to memory (rows, then their lengths) and of barriers; so what
// the threads exchange stays in shared memory, 16 reference counts a thread are loaded along with
// the list, one scan sums the pages wanted (high bits) and found (low 25) together, and the CTA has as
// many threads as there is work for. Release, extend and fork of a few sequences on 300 pages take
// 11.6 us together (13.5 with claims and free pages in global memory and 1024 threads).
template <bool FORK>
__global__ void __launch_bounds__(T) pages_plan_kernel(PageState s, PageScratch w,
                                                       const int32_t *rows, const int32_t *args,
                                                       int n) {
    // table of rows by hash: (row << 12 | lowest index of an entry that names it), open addressing;
    // afterwards, for each entry, the table column of page k of its own is off + k
    extern __shared__ unsigned tab[];
    const int slots = plan_slots(n);
    int32_t *at_s = reinterpret_cast<int32_t *>(tab + slots);  // [n] first of the fresh pages
    int32_t *off_s = reinterpret_cast<int32_t *>(tab);         // [n] INT32_MIN: gets none
    __shared__ long warp_tot[33];
    __shared__ int warp_tot_i[33];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int per = (n + nt - 1) / nt, i0 = tid * per;  // this thread's entries
    for (int k = tid; k < slots; k += nt) tab[k] = NO_ENTRY;
    grid_launch_dependents();
    grid_dependency_wait();
    int row[PER], arg[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const bool there = e < per && i0 + e < n;
        row[e] = there ? rows[i0 + e] : -1;
        arg[e] = there ? args[i0 + e] : 0;
    }
    unsigned mask = free16(s, 16 * tid);
    auto in_list = [&](int r) { return r >= 0 && r < s.num_seqs; };
    auto home = [&](int r) {
        return static_cast<int>(__umulhi(static_cast<unsigned>(r) * 2654435769u, slots));
    };
    __syncthreads();
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        if (!in_list(row[e])) continue;
        const unsigned word = static_cast<unsigned>(row[e]) << 12 | (i0 + e);
        for (int h = home(row[e]);; h = h + 1 < slots ? h + 1 : 0) {
            const unsigned old = atomicCAS(tab + h, NO_ENTRY, word);
            if (old == NO_ENTRY) break;
            if (old >> 12 == static_cast<unsigned>(row[e])) {
                atomicMin(tab + h, word);
                break;
            }
        }
    }
    __syncthreads();
    const long cap = (long)s.max_blocks * BLOCK;
    int len[PER], need[PER];
    bool ok[PER];
    long needs = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        ok[e] = in_list(row[e]) && (!FORK || (arg[e] >= 0 && arg[e] < s.num_seqs));
        if (ok[e]) {
            // (a slot that looks empty is the word of the last entry and row that there can be)
            const unsigned word = static_cast<unsigned>(row[e]) << 12 | (i0 + e);
            unsigned got = tab[home(row[e])];
            for (int h = home(row[e]); got != NO_ENTRY && got >> 12 != static_cast<unsigned>(row[e]);
                 got = tab[h])
                h = h + 1 < slots ? h + 1 : 0;
            ok[e] = got == word;
        }
        len[e] = need[e] = 0;
        if (ok[e]) {
            const int old = s.seqlens[row[e]];
            len[e] = FORK ? s.seqlens[arg[e]] : arg[e];
            ok[e] = len[e] >= 0 && len[e] <= cap && (FORK ? old == 0 : old >= 0 && old <= len[e]);
            if (ok[e]) need[e] = FORK ? len[e] % BLOCK != 0 : pages_of(len[e]) - pages_of(old);
        }
        if (!ok[e] && e < per && i0 + e < n) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, i0 + e);
        needs += need[e];
    }
    constexpr int LOW = 25;  // num_blocks <= 2^24; the pages wanted are at most 2^12 2^25
    long total;
    const long before = scan_block<long>(needs << LOW | __popc(mask), warp_tot, &total);
    const long wanted = total >> LOW;
    const int want = static_cast<int>(min(wanted, (long)s.num_blocks));
    // a pool of more than 16 pages a thread: go on counting until there are enough
    int found = static_cast<int>(total & ((1 << LOW) - 1));
    for (int p0 = 16 * nt; found < want && p0 < s.num_blocks; p0 += 16 * nt) {
        int more;
        scan_block<int>(__popc(free16(s, p0 + 16 * tid)), warp_tot_i, &more);
        found += more;
    }
    // entries whose pages are not all there fail, and with them all later ones that need any
    const int have = min(found, want);
    long at = before >> LOW;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = i0 + e;
        if (e < per && i < n) {
            const bool fits = ok[e] && (need[e] == 0 || at + need[e] <= have);
            if (ok[e] && !fits) flag_error(s.err, MLA_ERR_NO_PAGES, i);
            // past the pool's size nothing can be had
            const int first = static_cast<int>(min(at, (long)s.num_blocks));
            if (FORK) {
                w.plan[i] = PageEntry{fits, first, need[e], len[e]};
            } else {
                at_s[i] = first;
                off_s[i] = fits ? pages_of(len[e]) - need[e] - first : INT32_MIN;
                if (fits) s.seqlens[row[e]] = len[e];
            }
        }
        at += need[e];
    }
    if (FORK && tid == 0) w.seg[0] = have;
    __syncthreads();
    // the free pages in order (fork: for the next kernel)
    int32_t *fresh = FORK || have > FRESH ? w.fresh : at_s + n;
    int k = static_cast<int>(before & ((1 << LOW) - 1));
    for (int p0 = 0, done = 0; done < have; p0 += 16 * nt) {
        int count = static_cast<int>(total & ((1 << LOW) - 1));
        if (p0 > 0) {
            mask = free16(s, p0 + 16 * tid);
            k = done + scan_block<int>(__popc(mask), warp_tot_i, &count);
        }
        for (; mask && k < have; mask &= mask - 1, ++k) {
            const int id = p0 + 16 * tid + __ffs(mask) - 1;
            fresh[k] = id;
            if (FORK) w.rank[id] = k;  // which pages the call hands out
        }
        done += count;
    }
    if (FORK) return;
    // page k goes to the last entry whose pages begin at or before it
    __syncthreads();
    for (k = tid; k < have; k += nt) {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at_s[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        if (off_s[lo] == INT32_MIN) continue;
        const int id = fresh[k];
        s.table[(size_t)rows[lo] * s.max_blocks + off_s[lo] + k] = id;
        s.refs[id] = 1;
    }
}

// Copies a page of one layer by the CTA: 16-byte pieces, eight in flight per thread.
__device__ __forceinline__ void copy_page(const mla_page_pool_t &p, int layer, int src, int dst) {
    char *base = static_cast<char *>(p.base) + (size_t)layer * p.layer_stride;
    const uint4 *from = reinterpret_cast<const uint4 *>(base + (size_t)src * p.page_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(base + (size_t)dst * p.page_bytes);
    const int pieces = static_cast<int>(p.page_bytes / 16);
    constexpr int K = 8;
    for (int i0 = threadIdx.x; i0 < pieces; i0 += K * blockDim.x) {
        uint4 v[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (i0 + k * (int)blockDim.x < pieces) v[k] = __ldcs(from + i0 + k * blockDim.x);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (i0 + k * (int)blockDim.x < pieces) __stcs(to + i0 + k * blockDim.x, v[k]);
    }
}

// CTAs 0 .. n - 1: fork i's row, lengths and counts (a parent with a bad page, or one that nobody
// held before the call, is refused whole). The others copy the partial pages: unit (fork, layer,
// pool). A copy for a refused fork goes to a page that stays free.
__global__ void __launch_bounds__(256) pages_fork_kernel(PageState s, PageScratch w,
                                                         const int32_t *parents,
                                                         const int32_t *children, int n,
                                                         PagePools pools, int layers) {
    grid_launch_dependents();
    grid_dependency_wait();
    if (blockIdx.x >= n) {
        const long unit = blockIdx.x - n;
        const int i = static_cast<int>(unit / (layers * pools.n));
        const int l = static_cast<int>(unit / pools.n % layers);
        const mla_page_pool_t &p = pools.p[unit % pools.n];
        const PageEntry e = w.plan[i];
        if (!e.valid || e.need == 0 || l >= p.layers) return;
        const int src = s.table[(size_t)parents[i] * s.max_blocks + e.len / BLOCK];
        if (src >= 0 && src < s.num_blocks) copy_page(p, l, src, w.fresh[e.at]);
        return;
    }
    const int i = blockIdx.x;
    const PageEntry e = w.plan[i];
    if (!e.valid) return;
    const int32_t *from = s.table + (size_t)parents[i] * s.max_blocks;
    int32_t *to = s.table + (size_t)children[i] * s.max_blocks;
    const int held = pages_of(e.len), full = e.len / BLOCK;
    bool bad = false;
    for (int k = threadIdx.x; k < held; k += blockDim.x) {
        const int id = from[k];
        if (id < 0 || id >= s.num_blocks) {
            bad = true;
            continue;
        }
        // a page that this call hands out was free, whatever its count is by now (rank is not
        // cleared between calls: what it says holds where `fresh` agrees)
        const int k_new = w.rank[id];
        bad |= __ldcg(s.refs + id) <= 0 ||
               (k_new >= 0 && k_new < w.seg[0] && w.fresh[k_new] == id);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, i);
        return;
    }
    for (int k = threadIdx.x; k < held; k += blockDim.x) {
        if (k < full) {
            const int id = from[k];
            to[k] = id;
            atomicAdd(s.refs + id, 1);
        } else {
            to[k] = w.fresh[e.at];
            s.refs[w.fresh[e.at]] = 1;
        }
    }
    if (threadIdx.x == 0) s.seqlens[children[i]] = e.len;
}

// ------------------------------------------------------------------------------ compact

// Which of the 16 pages from `first` on are held, as bits.
__device__ __forceinline__ unsigned held16(const PageState &s, int first) {
    const int left = s.num_blocks - first;  // pages there are
    const unsigned there = left >= 16 ? 0xFFFFu : left > 0 ? (1u << left) - 1 : 0u;
    return ~free16(s, first) & there;
}

// live pages of each segment of PAGE_SEG pages
__global__ void __launch_bounds__(T) pages_count_kernel(PageState s, PageScratch w) {
    __shared__ int warp_tot[33];
    grid_launch_dependents();
    grid_dependency_wait();
    int total;
    scan_block<int>(__popc(held16(s, blockIdx.x * PAGE_SEG + 16 * threadIdx.x)), warp_tot, &total);
    if (threadIdx.x == 0) w.seg[blockIdx.x] = total;
}

// With N live pages, the k-th live page at or past N moves into the k-th free page before N.
// rank: k of a page that moves, -1 one that stays, -2 a free one; mover[k], fresh[k] = holes.
__global__ void __launch_bounds__(T) pages_rank_kernel(PageState s, PageScratch w, int segments,
                                                       int32_t *live_out) {
    __shared__ int warp_tot[33];
    const int tid = threadIdx.x;
    grid_launch_dependents();
    grid_dependency_wait();
    const int first = blockIdx.x * PAGE_SEG + 16 * tid;
    const unsigned held = held16(s, first);
    int N, base = 0;
    int at = scan_block<int>(__popc(held), warp_tot, &N);  // live pages before `first`
    if (segments > 1) {  // of all segments, and of those before this one
        int all = 0, before = 0;
        for (int g = tid; g < segments; g += T) {
            const int c = w.seg[g];
            all += c;
            if (g < blockIdx.x) before += c;
        }
        scan_block<int>(all, warp_tot, &N);
        scan_block<int>(before, warp_tot, &base);
        at += base;
    }
    // live pages before page N
    const int edge = N / PAGE_SEG;
    int below = 0;
    if (segments == 1)  // not counted beforehand
        below = edge == 1 ? __popc(held) : 0;
    else
        for (int g = tid; g < edge; g += T) below += w.seg[g];
    const int from = edge * PAGE_SEG + 16 * tid;
    if (from < N) {
        const int left = N - from;
        below += __popc(held16(s, from) & (left >= 16 ? 0xFFFFu : (1u << left) - 1));
    }
    int stay;
    scan_block<int>(below, warp_tot, &stay);
    for (int k = 0; k < 16; ++k) {
        const int id = first + k;
        if (id >= s.num_blocks) break;
        const bool live = held >> k & 1;
        int r = live ? -1 : -2;
        if (live && id >= N) {
            r = at - stay;
            w.mover[r] = id;
        } else if (!live && id < N) {
            w.fresh[id - at] = id;
        }
        w.rank[id] = r;
        at += live;
    }
    if (blockIdx.x == 0 && tid == 0) {
        w.seg[segments] = N;
        w.seg[segments + 1] = N - stay;
        *live_out = N;
    }
}

// CTAs 0 .. num_seqs - 1 rewrite the tables' rows, the next `ref_ctas` the counts, the rest move
// pages: unit (move, layer, pool), as many rounds as there are units. A count is read and
// written by one thread alone (a moved page's and its hole's by the mover's), so refs_out may be
// refs.
__global__ void __launch_bounds__(256) pages_move_kernel(PageState s, PageScratch w, int segments,
                                                         int32_t *refs_out, int32_t *table_out,
                                                         int ref_ctas, PagePools pools, int layers) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int N = w.seg[segments];
    int cta = blockIdx.x;
    if (cta < s.num_seqs) {
        const int len = s.seqlens[cta];
        const bool fine = len >= 0 && len <= (long)s.max_blocks * BLOCK;
        if (!fine && threadIdx.x == 0) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, cta);
        const int held = fine ? pages_of(len) : 0;
        const size_t row = (size_t)cta * s.max_blocks;
        for (int k = threadIdx.x; k < s.max_blocks; k += blockDim.x) {
            int id = s.table[row + k];
            if (k < held) {
                const int r = id >= 0 && id < s.num_blocks ? w.rank[id] : -2;
                if (r >= 0) id = w.fresh[r];
                else if (r == -2) flag_error(s.err, MLA_ERR_OUT_OF_RANGE, cta);
            }
            table_out[row + k] = id;
        }
        return;
    }
    cta -= s.num_seqs;
    if (cta < ref_ctas) {
        for (int id = cta * blockDim.x + threadIdx.x; id < s.num_blocks; id += ref_ctas * blockDim.x) {
            const int r = w.rank[id];
            if (r >= 0) {
                const int v = s.refs[id];
                refs_out[w.fresh[r]] = v;
                refs_out[id] = 0;
            } else if (r == -1) {
                refs_out[id] = s.refs[id];
            } else if (id >= N) {
                refs_out[id] = 0;
            }
        }
        return;
    }
    cta -= ref_ctas;
    const long units = (long)w.seg[segments + 1] * layers * pools.n;
    const int movers = gridDim.x - s.num_seqs - ref_ctas;
    for (long u = cta; u < units; u += movers) {
        const int r = static_cast<int>(u / (layers * pools.n));
        const int l = static_cast<int>(u / pools.n % layers);
        const mla_page_pool_t &p = pools.p[u % pools.n];
        if (l < p.layers) copy_page(p, l, w.mover[r], w.fresh[r]);
    }
}

int most_layers(const PagePools &pools) {
    int l = 0;
    for (int k = 0; k < pools.n; ++k)
        if (pools.p[k].layers > l) l = pools.p[k].layers;
    return l;
}

// threads for 16 pages each, in one CTA
int scan_threads(int pages) {
    const int t = (pages + 511) / 512 * 32;
    return t < T ? t : T;
}

template <bool FORK>
cudaError_t launch_plan(const PageState &s, const PageScratch &w, const int32_t *rows,
                        const int32_t *args, int n, cudaStream_t stream) {
    const int pool = scan_threads(s.num_blocks), list = (n + 31) / 32 * 32;
    const int threads = list > T ? T : pool > list ? pool : list;
    const size_t smem = sizeof(int32_t) * (plan_slots(n) + n + (FORK ? 0 : FRESH));
    static_assert(sizeof(int32_t) * (plan_slots(PAGE_LIST_MAX) + PAGE_LIST_MAX + FRESH) <= 47 * 1024,
                  "shared memory without a request for more");
    return launch_pdl(pages_plan_kernel<FORK>, dim3(1), dim3(threads), smem, stream, s, w, rows, args,
                      n);
}

}  // namespace

cudaError_t launch_pages_free(const PageState &s, const int32_t *rows, int n,
                              cudaStream_t stream) {
    return launch_pdl(pages_free_kernel, dim3(n), dim3(128), 0, stream, s, rows);
}

cudaError_t launch_pages_extend(const PageState &s, const PageScratch &w, const int32_t *rows,
                                const int32_t *new_lens, int n, cudaStream_t stream) {
    return launch_plan<false>(s, w, rows, new_lens, n, stream);
}

cudaError_t launch_pages_fork(const PageState &s, const PageScratch &w, const int32_t *parents,
                              const int32_t *children, int n, const PagePools &pools,
                              cudaStream_t stream) {
    const cudaError_t e = launch_plan<true>(s, w, children, parents, n, stream);
    if (e != cudaSuccess) return e;
    const int layers = most_layers(pools);
    return launch_pdl(pages_fork_kernel, dim3(n + n * layers * pools.n), dim3(256), 0, stream, s, w,
                      parents, children, n, pools, layers);
}

cudaError_t launch_pages_compact(const PageState &s, const PageScratch &w, int32_t *refs_out,
                                 int32_t *table_out, int32_t *live_out, const PagePools &pools,
                                 cudaStream_t stream) {
    const int segments = (s.num_blocks + PAGE_SEG - 1) / PAGE_SEG;
    cudaError_t e = cudaSuccess;
    if (segments > 1)  // one segment is counted where it is ranked
        e = launch_pdl(pages_count_kernel, dim3(segments), dim3(T), 0, stream, s, w);
    if (e != cudaSuccess) return e;
    e = launch_pdl(pages_rank_kernel, dim3(segments), dim3(scan_threads(s.num_blocks)), 0, stream, s, w,
                   segments, live_out);
    if (e != cudaSuccess) return e;
    const int layers = most_layers(pools);
    const int ref_ctas = s.num_blocks < 64 * 256 ? (s.num_blocks + 255) / 256 : 64;
    const long units = (long)s.num_blocks / 2 * layers * pools.n;  // at most half the pages move
    const long room = 8L * device_sm_count();
    const int movers = static_cast<int>(units < room ? units : room);
    return launch_pdl(pages_move_kernel, dim3(s.num_seqs + ref_ctas + movers), dim3(256), 0, stream,
                      s, w, segments, refs_out, table_out, ref_ctas, pools, layers);
}

}  // namespace mla
