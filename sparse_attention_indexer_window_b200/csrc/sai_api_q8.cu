// C-ABI entry points of the 8-bit indexer operators (declared in
// include/sai.h): argument validation and launch. Nothing here allocates
// device memory or synchronises the stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sai.h"
#include "indexer_q8.h"
#include "sai_host.h"

namespace {

using sai::al16;
using sai::al4;
using sai::cuda_status;
using sai::PageMap;

bool group_ok(int group) { return group == 32 || group == 64 || group == 128 || group == 256 || group == 512; }

// Sizes shared by the calls on a cache; the entries of one sequence are
// numbered with 31 bits, rows of the whole cache with 64.
sai_status check_map(int B, const int32_t *table, int n_pages, int page, int max_pages)
{
    if (n_pages < 1 || page < 1 || max_pages < 1 || (int64_t)max_pages * page > INT32_MAX)
        return SAI_ERR_SHAPE;
    if (!table && (max_pages != 1 || n_pages < B))
        return SAI_ERR_SHAPE;
    if (table && !al4(table))
        return SAI_ERR_ALIGN;
    return SAI_OK;
}

sai_status check_format(int B, int n, int D, int group, int code, int type)
{
    if (type < 0 || type > 2 || code < 0 || code > 1)
        return SAI_ERR_UNSUPPORTED;
    if (B < 1 || n < 1 || D < 1)
        return SAI_ERR_SHAPE;
    if (!group_ok(group))
        return SAI_ERR_UNSUPPORTED;
    if (D % group != 0 || (int64_t)B * n > INT32_MAX || (int64_t)B * n * (D / group) > INT32_MAX)
        return SAI_ERR_SHAPE;
    return SAI_OK;
}

sai_status check_indexer(int B, int S, int H, int D, int P, int cr)
{
    if (B < 1 || S < 1 || H < 1 || D < 1 || P < 1 || cr < 1)
        return SAI_ERR_SHAPE;
    // (the kernels count rows and keys in 32 bits, up to 64 tiles of 128 past the last)
    constexpr int64_t most = INT32_MAX - 16384;
    if ((int64_t)B * S * H > most || (int64_t)B * P > most || (int64_t)P * cr > INT32_MAX)
        return SAI_ERR_SHAPE;
    if (H > 128 || (D != 32 && D != 64 && D != 128))
        return SAI_ERR_UNSUPPORTED;
    return SAI_OK;
}

}  // namespace

extern "C" {

sai_status sai_q8_cache_write(const void *x, int x_type, int64_t stride_b, int64_t stride_n, const int32_t *start,
                              const int32_t *n_new, const int32_t *block_table, int B, int n, int D, int group,
                              int code, int n_pages, int page, int max_pages, void *cache, float *scales,
                              int32_t *d_err, void *stream)
{
    if (!x || !cache || !scales)
        return SAI_ERR_NULL;
    sai_status e = check_format(B, n, D, group, code, x_type);
    if (e == SAI_OK)
        e = check_map(B, block_table, n_pages, page, max_pages);
    if (e != SAI_OK)
        return e;
    if (stride_b < 0 || stride_n < 0)
        return SAI_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(x) & (x_type == SAI_TYPE_FP32 ? 3u : 1u)) || !al16(cache) || !al4(scales) ||
        (start && !al4(start)) || (n_new && !al4(n_new)) || (d_err && !al4(d_err)))
        return SAI_ERR_ALIGN;
    const sai::Q8WriteArgs a = {x, stride_b, stride_n, start, n_new, B, n, D, group, static_cast<uint8_t *>(cache),
                                scales, PageMap{block_table, n_pages, page, max_pages}, d_err};
    return cuda_status(sai::launch_q8_write(a, x_type, code, reinterpret_cast<cudaStream_t>(stream)));
}

sai_status sai_q8_cache_read(const void *cache, const float *scales, const int32_t *idx, const int32_t *start,
                             const int32_t *lens, const int32_t *block_table, int B, int n, int D, int group,
                             int code, int n_pages, int page, int max_pages, void *out, int out_type,
                             int32_t *d_err, void *stream)
{
    if (!cache || !scales || !out)
        return SAI_ERR_NULL;
    sai_status e = check_format(B, n, D, group, code, out_type);
    if (e == SAI_OK)
        e = check_map(B, block_table, n_pages, page, max_pages);
    if (e != SAI_OK)
        return e;
    if (idx && start)
        return SAI_ERR_SHAPE;
    if (!al16(cache) || !al4(scales) || !al16(out) || (idx && !al4(idx)) || (start && !al4(start)) ||
        (lens && !al4(lens)) || (d_err && !al4(d_err)))
        return SAI_ERR_ALIGN;
    const sai::Q8ReadArgs a = {static_cast<const uint8_t *>(cache), scales, idx, start, lens, B, n, D, group,
                               PageMap{block_table, n_pages, page, max_pages}, out, d_err};
    return cuda_status(sai::launch_q8_read(a, out_type, code, reinterpret_cast<cudaStream_t>(stream)));
}

sai_status sai_indexer_scores(const int8_t *q8, const float *q_scale, const float *w, const int8_t *cache,
                              const float *k_scale, const int32_t *block_table, const int32_t *q_start,
                              const int32_t *k_len, const int32_t *doc_start, int B, int S, int H, int D, int P,
                              int n_pages, int page, int max_pages, int cr, float *scores, int32_t *d_err,
                              void *stream)
{
    if (!q8 || !q_scale || !w || !cache || !k_scale || !scores)
        return SAI_ERR_NULL;
    sai_status e = check_indexer(B, S, H, D, P, cr);
    if (e == SAI_OK)
        e = check_map(B, block_table, n_pages, page, max_pages);
    if (e != SAI_OK)
        return e;
    if (P > max_pages * page)
        return SAI_ERR_SHAPE;
    // a 128-key tile starts on a page's first entry or holds whole pages
    if (max_pages > 1 && page % 128 != 0 && page != 64 && page != 32 && page != 16 && page != 8)
        return SAI_ERR_UNSUPPORTED;
    if (!al16(q8) || !al4(q_scale) || !al4(w) || !al16(cache) || !al4(k_scale) || !al4(scores) ||
        (q_start && !al4(q_start)) || (k_len && !al4(k_len)) || (doc_start && !al4(doc_start)) ||
        (d_err && !al4(d_err)))
        return SAI_ERR_ALIGN;
    const sai::ScoresArgs a = {q8, q_scale, w, cache, k_scale, q_start, k_len, doc_start, B, S, H, D, P, cr,
                               PageMap{block_table, n_pages, page, max_pages}, scores, d_err};
    return cuda_status(sai::launch_indexer_scores(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t sai_indexer_scores_backward_workspace_bytes(int B, int S, int H, int D, int P)
{
    if (check_indexer(B, S, H, D, P, 1) != SAI_OK)
        return 0;
    return sai::indexer_scores_bwd_ws_bytes(B, S, H, D, P);
}

sai_status sai_indexer_scores_backward(const float *dscores, const int32_t *idx, const int8_t *q8,
                                       const float *q_scale, const float *w, const int8_t *k8, const float *k_scale,
                                       const int32_t *doc_start, int B, int S, int H, int D, int P, int K, int cr,
                                       int t_begin, uint16_t *dq, uint16_t *dk, float *dw, void *workspace,
                                       size_t ws_bytes, int32_t *d_err, void *stream)
{
    if (!dscores || !q8 || !q_scale || !w || !k8 || !k_scale || !dq || !dk || !dw)
        return SAI_ERR_NULL;
    sai_status e = check_indexer(B, S, H, D, P, cr);
    if (e != SAI_OK)
        return e;
    if (K < 1 || K > P || (!idx && K != P) || t_begin < 0 || (int64_t)t_begin + S > INT32_MAX ||
        (int64_t)B * ((P + 255LL) / 256) * ((S + 127LL) / 128 * sai::padded_heads(H) + 1) > INT32_MAX ||
        (int64_t)B * S + ((int64_t)B * P * (D / 16) + 127) / 128 > INT32_MAX)       // blocks of the first kernel
        return SAI_ERR_SHAPE;
    if (!al4(dscores) || (idx && !al4(idx)) || !al16(q8) || !al4(q_scale) || !al4(w) || !al16(k8) ||
        !al4(k_scale) || !al16(dq) || !al16(dk) || !al4(dw) || (doc_start && !al4(doc_start)) ||
        (d_err && !al4(d_err)))
        return SAI_ERR_ALIGN;
    if (!workspace || !al16(workspace) || ws_bytes < sai::indexer_scores_bwd_ws_bytes(B, S, H, D, P))
        return SAI_ERR_WORKSPACE;
    const sai::ScoresBwdArgs a = {dscores, idx, q8, q_scale, w, k8, k_scale, doc_start, B, S, H, D, P, K, cr,
                                  t_begin, dq, dk, dw, d_err};
    return cuda_status(sai::launch_indexer_scores_bwd(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
