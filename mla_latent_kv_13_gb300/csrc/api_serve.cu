// api_serve.cu -- the C ABI of the latent norms with the cache write, and of the pages' life
// (declared in include/mla.h).
#include <limits.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"
#include "rope.h"
#include "serve.h"

using namespace mla;

namespace {

// where the rows go: the fields of one format
struct NormCache {
    mla_bf16_t *cache;
    uint8_t *codes;
    int8_t *exps;
    uint8_t *scales;
    mla_bf16_t *keys;
};

// plan null: the rotation of rope_theta
mla_status_t norm_run(const mla_bf16_t *x, long ldx, int q_lora, const mla_bf16_t *w_q,
                      const mla_bf16_t *w_kv, float eps, const int32_t *q_starts,
                      const int32_t *seqlens, int B, int tokens, const int32_t *block_table,
                      int max_blocks, const NormCache &to, int num_blocks, float rope_theta,
                      const mla_rope_t *plan, mla_bf16_t *c_q, void *workspace, size_t ws_bytes,
                      mla_stream_t stream) {
    if (!x || !w_kv || !q_starts || !seqlens || !block_table || !workspace ||
        (q_lora > 0 && (!w_q || !c_q)))
        return MLA_ERR_INVALID_ARG;
    if (B < 1 || B > 4096 || tokens < 1 || q_lora < 0 || q_lora % 8 || max_blocks < 1 ||
        num_blocks < 1 || ldx < q_lora + D_QK || ldx % 8 || !(eps >= 0.f) || !isfinite(eps) ||
        (plan ? !plan_ok(*plan) || plan->rot != D_ROPE
              : !(rope_theta > 0.f) || !isfinite(rope_theta)))
        return MLA_ERR_INVALID_ARG;
    if (tokens > (1 << 24) || q_lora > (1 << 16) || max_blocks > INT_MAX / BLOCK)
        return MLA_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(w_kv, 16) || !aligned(q_starts, 4) || !aligned(seqlens, 4) ||
        !aligned(block_table, 4) || !aligned(to.cache, 16) || !aligned(to.codes, 16) ||
        !aligned(to.scales, 16) || !aligned(to.keys, 16) ||
        (q_lora > 0 && (!aligned(w_q, 16) || !aligned(c_q, 16))) || !aligned(workspace, 256))
        return MLA_ERR_INVALID_ARG;
    if (ws_bytes < HDR) return MLA_ERR_WORKSPACE;
    NormParams p{};
    p.x = x; p.ldx = ldx; p.q_lora = q_lora; p.w_q = w_q; p.w_kv = w_kv; p.eps = eps;
    p.q_starts = q_starts; p.seqlens = seqlens; p.B = B; p.tokens = tokens;
    p.block_table = block_table; p.max_blocks = max_blocks; p.num_blocks = num_blocks;
    p.c_q = c_q; p.cache = to.cache; p.codes = to.codes; p.exps = to.exps;
    p.scales = to.scales; p.keys = to.keys;
    if (plan) p.half_layout = plan->layout == MLA_ROPE_HALF, p.magnitude = plan->magnitude;
    p.err = err_word(workspace);
    return cuda_status(launch_norm_rope(p, rope_theta, plan, S(stream)));
}

struct PageLayout {
    size_t plan, fresh, mover, rank, seg, total;
};
PageLayout page_layout(int num_blocks) {
    PageLayout L{};
    L.plan = HDR;
    L.fresh = L.plan + align256(PAGE_LIST_MAX * sizeof(PageEntry));
    L.mover = L.fresh + align256((size_t)num_blocks * 4);
    L.rank = L.mover + align256((size_t)num_blocks * 4);
    L.seg = L.rank + align256((size_t)num_blocks * 4);
    L.total = L.seg + align256(((size_t)(num_blocks + PAGE_SEG - 1) / PAGE_SEG + 2) * 4);
    return L;
}

// The checks that every call on the pages shares; on MLA_OK fills in the state and the scratch.
mla_status_t page_state(int32_t *refs, int num_blocks, int32_t *block_table, int max_blocks,
                        int32_t *seqlens, int num_seqs, void *workspace, size_t ws_bytes,
                        PageState &s, PageScratch &w) {
    if (!refs || !block_table || !seqlens || !workspace) return MLA_ERR_INVALID_ARG;
    if (num_blocks < 1 || max_blocks < 1 || num_seqs < 1) return MLA_ERR_INVALID_ARG;
    if (num_blocks > (1 << 24) || num_seqs > (1 << 20) || max_blocks > INT_MAX / BLOCK)
        return MLA_ERR_UNSUPPORTED;
    if (!aligned(refs, 4) || !aligned(block_table, 4) || !aligned(seqlens, 4) ||
        !aligned(workspace, 256))
        return MLA_ERR_INVALID_ARG;
    const PageLayout L = page_layout(num_blocks);
    if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
    char *b = static_cast<char *>(workspace);
    s = PageState{refs, num_blocks, block_table, max_blocks, seqlens, num_seqs, err_word(workspace)};
    w.plan = reinterpret_cast<PageEntry *>(b + L.plan);
    w.fresh = reinterpret_cast<int32_t *>(b + L.fresh);
    w.mover = reinterpret_cast<int32_t *>(b + L.mover);
    w.rank = reinterpret_cast<int32_t *>(b + L.rank);
    w.seg = reinterpret_cast<int32_t *>(b + L.seg);
    return MLA_OK;
}

mla_status_t page_pools(const mla_page_pool_t *pools, int n_pools, int num_blocks, PagePools &out) {
    if (n_pools < 0 || n_pools > MLA_MAX_POOLS || (n_pools > 0 && !pools))
        return MLA_ERR_INVALID_ARG;
    out.n = n_pools;
    for (int k = 0; k < n_pools; ++k) {
        const mla_page_pool_t &p = pools[k];
        if (!p.base || p.layers < 1 || p.page_bytes < 16 || p.page_bytes % 16 || p.layer_stride % 16 ||
            !aligned(p.base, 16) ||
            (p.layers > 1 && p.layer_stride < (size_t)num_blocks * p.page_bytes))
            return MLA_ERR_INVALID_ARG;
        if (p.page_bytes > (1u << 24) || p.layers > 4096) return MLA_ERR_UNSUPPORTED;
        out.p[k] = p;
    }
    return MLA_OK;
}

}  // namespace

extern "C" {

mla_status_t mla_norm_rope_append(const mla_bf16_t *x, long ldx, int q_lora,
                                  const mla_bf16_t *w_q, const mla_bf16_t *w_kv, float eps,
                                  const int32_t *q_starts, const int32_t *seqlens, int B,
                                  int tokens, const int32_t *block_table, int max_blocks,
                                  mla_bf16_t *kv_cache, int num_blocks, float rope_theta,
                                  mla_bf16_t *c_q, void *workspace, size_t ws_bytes,
                                  mla_stream_t stream) {
    if (!kv_cache) return MLA_ERR_INVALID_ARG;
    return norm_run(x, ldx, q_lora, w_q, w_kv, eps, q_starts, seqlens, B, tokens, block_table,
                    max_blocks, {kv_cache}, num_blocks, rope_theta, nullptr, c_q, workspace, ws_bytes,
                    stream);
}

mla_status_t mla_norm_rope_append_fp8(const mla_bf16_t *x, long ldx, int q_lora,
                                      const mla_bf16_t *w_q, const mla_bf16_t *w_kv, float eps,
                                      const int32_t *q_starts, const int32_t *seqlens, int B,
                                      int tokens, const int32_t *block_table, int max_blocks,
                                      uint8_t *kv_codes, int8_t *kv_exps, int num_blocks,
                                      float rope_theta, mla_bf16_t *c_q, void *workspace,
                                      size_t ws_bytes, mla_stream_t stream) {
    if (!kv_codes || !kv_exps) return MLA_ERR_INVALID_ARG;
    return norm_run(x, ldx, q_lora, w_q, w_kv, eps, q_starts, seqlens, B, tokens, block_table,
                    max_blocks, {nullptr, kv_codes, kv_exps}, num_blocks, rope_theta, nullptr, c_q,
                    workspace, ws_bytes, stream);
}

mla_status_t mla_norm_rope_append_scaled(const mla_bf16_t *x, long ldx, int q_lora,
                                         const mla_bf16_t *w_q, const mla_bf16_t *w_kv, float eps,
                                         const int32_t *q_starts, const int32_t *seqlens, int B,
                                         int tokens, const int32_t *block_table, int max_blocks,
                                         mla_bf16_t *kv_cache, int num_blocks,
                                         const mla_rope_t *plan, mla_bf16_t *c_q, void *workspace,
                                         size_t ws_bytes, mla_stream_t stream) {
    if (!kv_cache || !plan) return MLA_ERR_INVALID_ARG;
    return norm_run(x, ldx, q_lora, w_q, w_kv, eps, q_starts, seqlens, B, tokens, block_table,
                    max_blocks, {kv_cache}, num_blocks, 0.f, plan, c_q, workspace, ws_bytes, stream);
}

mla_status_t mla_norm_rope_append_scaled_fp8(const mla_bf16_t *x, long ldx, int q_lora,
                                             const mla_bf16_t *w_q, const mla_bf16_t *w_kv, float eps,
                                             const int32_t *q_starts, const int32_t *seqlens, int B,
                                             int tokens, const int32_t *block_table, int max_blocks,
                                             uint8_t *kv_codes, int8_t *kv_exps, int num_blocks,
                                             const mla_rope_t *plan, mla_bf16_t *c_q,
                                             void *workspace, size_t ws_bytes, mla_stream_t stream) {
    if (!kv_codes || !kv_exps || !plan) return MLA_ERR_INVALID_ARG;
    return norm_run(x, ldx, q_lora, w_q, w_kv, eps, q_starts, seqlens, B, tokens, block_table,
                    max_blocks, {nullptr, kv_codes, kv_exps}, num_blocks, 0.f, plan, c_q, workspace,
                    ws_bytes, stream);
}

mla_status_t mla_norm_rope_append_fp4(const mla_bf16_t *x, long ldx, int q_lora,
                                      const mla_bf16_t *w_q, const mla_bf16_t *w_kv, float eps,
                                      const int32_t *q_starts, const int32_t *seqlens, int B,
                                      int tokens, const int32_t *block_table, int max_blocks,
                                      uint8_t *kv_codes, uint8_t *kv_scales, int8_t *kv_exps,
                                      mla_bf16_t *kv_keys, int num_blocks, const mla_rope_t *plan,
                                      mla_bf16_t *c_q, void *workspace, size_t ws_bytes,
                                      mla_stream_t stream) {
    if (!kv_codes || !kv_scales || !kv_exps || !kv_keys || !plan) return MLA_ERR_INVALID_ARG;
    return norm_run(x, ldx, q_lora, w_q, w_kv, eps, q_starts, seqlens, B, tokens, block_table,
                    max_blocks, {nullptr, kv_codes, kv_exps, kv_scales, kv_keys}, num_blocks, 0.f, plan,
                    c_q, workspace, ws_bytes, stream);
}

mla_status_t mla_pages_workspace_size(int num_blocks, int num_seqs, size_t *bytes) {
    if (!bytes || num_blocks < 1 || num_seqs < 1) return MLA_ERR_INVALID_ARG;
    if (num_blocks > (1 << 24) || num_seqs > (1 << 20)) return MLA_ERR_UNSUPPORTED;
    *bytes = page_layout(num_blocks).total;
    return MLA_OK;
}

mla_status_t mla_pages_free(int32_t *refs, int num_blocks, int32_t *block_table, int max_blocks,
                            int32_t *seqlens, int num_seqs, const int32_t *rows, int n,
                            void *workspace, size_t ws_bytes, mla_stream_t stream) {
    PageState s;
    PageScratch w;
    const mla_status_t v = page_state(refs, num_blocks, block_table, max_blocks, seqlens, num_seqs,
                                      workspace, ws_bytes, s, w);
    if (v != MLA_OK) return v;
    if (n < 0) return MLA_ERR_INVALID_ARG;
    if (n == 0) return MLA_OK;
    if (!rows || !aligned(rows, 4)) return MLA_ERR_INVALID_ARG;
    return cuda_status(launch_pages_free(s, rows, n, S(stream)));
}

mla_status_t mla_pages_extend(int32_t *refs, int num_blocks, int32_t *block_table, int max_blocks,
                              int32_t *seqlens, int num_seqs, const int32_t *rows,
                              const int32_t *new_lens, int n, void *workspace, size_t ws_bytes,
                              mla_stream_t stream) {
    PageState s;
    PageScratch w;
    const mla_status_t v = page_state(refs, num_blocks, block_table, max_blocks, seqlens, num_seqs,
                                      workspace, ws_bytes, s, w);
    if (v != MLA_OK) return v;
    if (n < 0) return MLA_ERR_INVALID_ARG;
    if (n > PAGE_LIST_MAX) return MLA_ERR_UNSUPPORTED;
    if (n == 0) return MLA_OK;
    if (!rows || !new_lens || !aligned(rows, 4) || !aligned(new_lens, 4)) return MLA_ERR_INVALID_ARG;
    return cuda_status(launch_pages_extend(s, w, rows, new_lens, n, S(stream)));
}

mla_status_t mla_pages_fork(int32_t *refs, int num_blocks, int32_t *block_table, int max_blocks,
                            int32_t *seqlens, int num_seqs, const int32_t *parents,
                            const int32_t *children, int n, const mla_page_pool_t *pools,
                            int n_pools, void *workspace, size_t ws_bytes, mla_stream_t stream) {
    PageState s;
    PageScratch w;
    mla_status_t v = page_state(refs, num_blocks, block_table, max_blocks, seqlens, num_seqs,
                                workspace, ws_bytes, s, w);
    if (v != MLA_OK) return v;
    PagePools p;
    if ((v = page_pools(pools, n_pools, num_blocks, p)) != MLA_OK) return v;
    if (n < 0) return MLA_ERR_INVALID_ARG;
    if (n > PAGE_LIST_MAX) return MLA_ERR_UNSUPPORTED;
    if (n == 0) return MLA_OK;
    if (!parents || !children || !aligned(parents, 4) || !aligned(children, 4))
        return MLA_ERR_INVALID_ARG;
    return cuda_status(launch_pages_fork(s, w, parents, children, n, p, S(stream)));
}

mla_status_t mla_pages_compact(int32_t *refs, int num_blocks, int32_t *block_table, int max_blocks,
                               int32_t *seqlens, int num_seqs, int32_t *refs_out,
                               int32_t *table_out, int32_t *live_out, const mla_page_pool_t *pools,
                               int n_pools, void *workspace, size_t ws_bytes, mla_stream_t stream) {
    PageState s;
    PageScratch w;
    mla_status_t v = page_state(refs, num_blocks, block_table, max_blocks, seqlens, num_seqs,
                                workspace, ws_bytes, s, w);
    if (v != MLA_OK) return v;
    PagePools p;
    if ((v = page_pools(pools, n_pools, num_blocks, p)) != MLA_OK) return v;
    if (!refs_out || !table_out || !live_out || !aligned(refs_out, 4) || !aligned(table_out, 4) ||
        !aligned(live_out, 4))
        return MLA_ERR_INVALID_ARG;
    return cuda_status(launch_pages_compact(s, w, refs_out, table_out, live_out, p, S(stream)));
}

}  // extern "C"
