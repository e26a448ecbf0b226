// api_ctx.cu -- the C ABI of rotary positions and of reading a paged cache back (declared in
// include/mla.h).
#include <limits.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"
#include "rope.h"
#include "serve.h"

using namespace mla;

namespace {

mla_status_t read_run(const mla_bf16_t *cache, const uint8_t *codes, const int8_t *exps,
                      const uint8_t *scales, const mla_bf16_t *keys, int num_blocks,
                      const int32_t *block_table, int max_blocks, const int32_t *first,
                      const int32_t *row_starts, int B, int rows, mla_bf16_t *out, void *workspace,
                      size_t ws_bytes, mla_stream_t stream) {
    if (!block_table || !row_starts || !out || !workspace) return MLA_ERR_INVALID_ARG;
    if (num_blocks < 1 || max_blocks < 1 || B < 1 || B > 4096 || rows < 1) return MLA_ERR_INVALID_ARG;
    if (num_blocks > (1 << 24) || max_blocks > INT_MAX / BLOCK || rows > (1 << 30))
        return MLA_ERR_UNSUPPORTED;
    if (!aligned(cache, 32) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(keys, 16) ||
        !aligned(block_table, 4) || !aligned(first, 4) || !aligned(row_starts, 4) ||
        !aligned(out, 32) || !aligned(workspace, 256))
        return MLA_ERR_INVALID_ARG;
    if (ws_bytes < HDR) return MLA_ERR_WORKSPACE;
    ReadParams p{};
    p.cache = cache; p.codes = codes; p.exps = exps; p.scales = scales; p.keys = keys;
    p.num_blocks = num_blocks; p.block_table = block_table; p.max_blocks = max_blocks;
    p.first = first; p.row_starts = row_starts; p.B = B; p.rows = rows; p.out = out;
    p.err = err_word(workspace);
    return cuda_status(launch_read_kv(p, S(stream)));
}

// Whether no two of tokens x heads rows of `width` values share a place.
bool rows_apart(int tokens, int heads, int width, long by_token, long by_head) {
    if ((tokens > 1 && by_token < width) || (heads > 1 && by_head < width)) return false;
    if (tokens == 1 || heads == 1 || by_head <= (by_token - width) / (heads - 1) ||
        by_token <= (by_head - width) / (tokens - 1))
        return true;
    // neither a token's heads nor a head's tokens lie together: j heads on may be i tokens on, or near
    for (int j = 1; j < heads; ++j) {
        const __int128 at = static_cast<__int128>(j) * by_head;
        const __int128 i = at / by_token, off = at % by_token;
        if ((off < width && i < tokens) || (by_token - off < width && i + 1 < tokens)) return false;
    }
    return true;
}

}  // namespace

extern "C" {

mla_status_t mla_rope_plan(int rot, int layout, double theta, int scaling, double factor,
                           int original, double fast, double slow, mla_rope_t *plan) {
    if (!plan || rot < 2 || rot % 2 || (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) ||
        !(theta > 0.) || !isfinite(theta) || scaling < MLA_ROPE_PLAIN || scaling > MLA_ROPE_BANDS)
        return MLA_ERR_INVALID_ARG;
    if (rot > MLA_ROPE_MAX) return MLA_ERR_UNSUPPORTED;
    if (scaling != MLA_ROPE_PLAIN && (!(factor > 0.) || !isfinite(factor))) return MLA_ERR_INVALID_ARG;
    const bool ramp = scaling == MLA_ROPE_YARN || scaling == MLA_ROPE_BANDS;
    if (ramp && (original < 1 || !(slow > 0.) || !(fast > slow) || !isfinite(fast) || !(theta > 1.)))
        return MLA_ERR_INVALID_ARG;
    mla_rope_t r{};
    r.rot = rot;
    r.layout = layout;
    r.magnitude = scaling == MLA_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.) : 1.f;
    const double two_pi = 6.283185307179586476925286766559;
    double base = theta;
    if (scaling == MLA_ROPE_NTK && rot > 2) base *= pow(factor, (double)rot / (rot - 2));
    // the pair that turns `turns` times over the original context, as a real number
    auto index = [&](double turns) {
        return rot * log(original / (turns * two_pi)) / (2. * log(theta));
    };
    double low = 0., high = 0.;
    if (scaling == MLA_ROPE_YARN) {
        low = fmax(floor(index(fast)), 0.);
        high = fmin(ceil(index(slow)), rot - 1.);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2. * i / rot);
        double keep = 1.;  // of the plain frequency, the rest of the one divided by factor
        if (scaling == MLA_ROPE_LINEAR) keep = 0.;
        if (scaling == MLA_ROPE_YARN)
            keep = 1. - fmin(1., fmax(0., (i - low) / fmax(high - low, 0.001)));
        if (scaling == MLA_ROPE_BANDS)
            keep = fmin(1., fmax(0., (original * f / two_pi - slow) / (fast - slow)));
        r.freq[i] = keep == 1. ? f : f * keep + f / factor * (1. - keep);
    }
    if (!plan_ok(r)) return MLA_ERR_INVALID_ARG;
    *plan = r;
    return MLA_OK;
}

mla_status_t mla_rope(const mla_bf16_t *x, long x_token, long x_head, int tokens, int heads,
                      int width, int offset, const mla_rope_t *plan, const int32_t *pos,
                      mla_bf16_t *y, long y_token, long y_head, mla_bf16_t *rest, long rest_token,
                      long rest_head, mla_stream_t stream) {
    if (!x || !plan || !pos || !y || tokens < 1 || heads < 1 || width < 1 || offset < 0 ||
        x_token < 0 || x_head < 0 || y_token < 0 || y_head < 0 || !plan_ok(*plan) ||
        width - offset < plan->rot)
        return MLA_ERR_INVALID_ARG;
    const int others = width - plan->rot;
    if (tokens > (1 << 24) || heads > (1 << 12)) return MLA_ERR_UNSUPPORTED;
    if (!rows_apart(tokens, heads, plan->rot, y_token, y_head) ||
        (rest && others > 0 && !rows_apart(tokens, heads, others, rest_token, rest_head)))
        return MLA_ERR_INVALID_ARG;
    if (width > (1 << 12)) return MLA_ERR_UNSUPPORTED;
    if (!aligned(x, 2) || !aligned(y, 2) || !aligned(rest, 2) || !aligned(pos, 4))
        return MLA_ERR_INVALID_ARG;
    RopeParams p{};
    p.x = x; p.x_token = x_token; p.x_head = x_head;
    p.tokens = tokens; p.heads = heads; p.width = width; p.offset = offset; p.pos = pos;
    p.y = y; p.y_token = y_token; p.y_head = y_head;
    p.rest = others > 0 ? rest : nullptr; p.rest_token = rest_token; p.rest_head = rest_head;
    return cuda_status(launch_rope(p, *plan, S(stream)));
}

mla_status_t mla_read_kv(const mla_bf16_t *kv_cache, int num_blocks, const int32_t *block_table,
                         int max_blocks, const int32_t *first, const int32_t *row_starts, int B,
                         int rows, mla_bf16_t *out, void *workspace, size_t ws_bytes,
                         mla_stream_t stream) {
    if (!kv_cache) return MLA_ERR_INVALID_ARG;
    return read_run(kv_cache, nullptr, nullptr, nullptr, nullptr, num_blocks, block_table, max_blocks,
                    first, row_starts, B, rows, out, workspace, ws_bytes, stream);
}

mla_status_t mla_read_kv_fp8(const uint8_t *kv_codes, const int8_t *kv_exps, int num_blocks,
                             const int32_t *block_table, int max_blocks, const int32_t *first,
                             const int32_t *row_starts, int B, int rows, mla_bf16_t *out,
                             void *workspace, size_t ws_bytes, mla_stream_t stream) {
    if (!kv_codes || !kv_exps) return MLA_ERR_INVALID_ARG;
    return read_run(nullptr, kv_codes, kv_exps, nullptr, nullptr, num_blocks, block_table, max_blocks,
                    first, row_starts, B, rows, out, workspace, ws_bytes, stream);
}

mla_status_t mla_read_kv_fp4(const uint8_t *kv_codes, const uint8_t *kv_scales, const int8_t *kv_exps,
                             const mla_bf16_t *kv_keys, int num_blocks, const int32_t *block_table,
                             int max_blocks, const int32_t *first, const int32_t *row_starts, int B,
                             int rows, mla_bf16_t *out, void *workspace, size_t ws_bytes,
                             mla_stream_t stream) {
    if (!kv_codes || !kv_scales || !kv_exps || !kv_keys) return MLA_ERR_INVALID_ARG;
    return read_run(nullptr, kv_codes, kv_exps, kv_scales, kv_keys, num_blocks, block_table, max_blocks,
                    first, row_starts, B, rows, out, workspace, ws_bytes, stream);
}

}  // extern "C"
