// serve.h -- internal interface of what a ragged batch needs beside its attention: the latent
// norms with the cache write, and the pages' life.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla.h"

namespace mla {

struct NormParams {
    const uint16_t *x;  // [tokens][ldx]: c_q (q_lora) | c_kv (512) | k_rope (64)
    long ldx;
    int q_lora;
    const uint16_t *w_q, *w_kv;
    float eps;
    const int32_t *q_starts, *seqlens;
    int B, tokens;
    const int32_t *block_table;
    int max_blocks, num_blocks;
    uint16_t *c_q;    // [tokens][q_lora]
    uint16_t *cache;  // bf16 cache, or null:
    uint8_t *codes;   // FP8 cache
    int8_t *exps;
    uint32_t *err;
};
cudaError_t launch_norm_rope(const NormParams &p, float theta, cudaStream_t stream);

// The pages' state: refs[page] = sequences that hold it (0: free), the block table, and the
// sequences' lengths; a sequence of length L holds the first ceil(L / 64) entries of its row.
struct PageState {
    int32_t *refs;
    int num_blocks;
    int32_t *table;
    int max_blocks;
    int32_t *seqlens;
    int num_seqs;
    uint32_t *err;
};
struct PagePools {
    int n;
    mla_page_pool_t p[MLA_MAX_POOLS];
};
constexpr int PAGE_LIST_MAX = 4096;  // entries of one extend or fork call
struct PageEntry {                   // what the plan decided for one entry of the list
    int32_t valid, at, need, len;    // its fresh pages are fresh[at .. at + need); new length
};
struct PageScratch {
    PageEntry *plan;   // [PAGE_LIST_MAX]
    int32_t *fresh;    // [num_blocks] lowest free pages; compact: the holes
    int32_t *mover;    // [num_blocks]
    int32_t *rank;     // [num_blocks] compact; fork: k of fresh[k] at that page (not cleared)
    int32_t *seg;      // [segments + 2]
};
constexpr int PAGE_SEG = 16384;  // pages counted by one CTA of compact (16 a thread)

cudaError_t launch_pages_free(const PageState &s, const int32_t *rows, int n, cudaStream_t stream);
cudaError_t launch_pages_extend(const PageState &s, const PageScratch &w, const int32_t *rows,
                                const int32_t *new_lens, int n, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageState &s, const PageScratch &w, const int32_t *parents,
                              const int32_t *children, int n, const PagePools &pools,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const PageState &s, const PageScratch &w, int32_t *refs_out,
                                 int32_t *table_out, int32_t *live_out, const PagePools &pools,
                                 cudaStream_t stream);

}  // namespace mla
