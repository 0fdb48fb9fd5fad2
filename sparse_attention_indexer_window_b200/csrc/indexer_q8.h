// Launch interface of the 8-bit indexer operators: the quantised cache
// (q8_cache.cu), the indexer's scores (indexer_scores.cu) and their gradient
// (indexer_scores_bwd.cu). Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sai {

// Where a sequence's entries live: entry `pos` of sequence b is row pos % page
// of page table[b*max_pages + pos/page] (page b itself when table is NULL).
struct PageMap {
    const int32_t *table;
    int n_pages, page, max_pages;
};

// Row of the cache holding entry pos of sequence b, or -1 when the entry has
// none (pos outside the table's capacity, or a page id outside the cache).
__device__ __forceinline__ int64_t page_row(const PageMap &m, int b, int64_t pos)
{
    if (pos < 0 || pos >= (int64_t)m.max_pages * m.page)
        return -1;
    const int pi = (int)((uint32_t)pos / (uint32_t)m.page);   // the capacity fits 31 bits (checked on the host)
    const int id = m.table ? __ldg(m.table + (int64_t)b * m.max_pages + pi) : b;
    if (id < 0 || id >= m.n_pages)
        return -1;
    return (int64_t)id * m.page + ((uint32_t)pos - (uint32_t)pi * (uint32_t)m.page);
}

struct Q8WriteArgs {
    const void *x;
    int64_t stride_b, stride_n;     // elements
    const int32_t *start, *n_new;   // [B] or NULL (0, n)
    int B, n, D, group;
    uint8_t *cache;
    float *scales;
    PageMap map;
    int32_t *err;
};
cudaError_t launch_q8_write(const Q8WriteArgs &a, int type, int code, cudaStream_t stream);

struct Q8ReadArgs {
    const uint8_t *cache;
    const float *scales;
    const int32_t *idx, *start, *lens;   // [B,n], [B], [B] or NULL
    int B, n, D, group;
    PageMap map;
    void *out;
    int32_t *err;
};
cudaError_t launch_q8_read(const Q8ReadArgs &a, int type, int code, cudaStream_t stream);

struct ScoresArgs {
    const int8_t *q8;        // [B,S,H,D]
    const float *q_scale;    // [B,S,H]
    const float *w;          // [B,S,H]
    const int8_t *cache;     // [n_pages,page,D]
    const float *k_scale;    // [n_pages,page]
    const int32_t *q_start, *k_len, *doc_start;
    int B, S, H, D, P, cr;
    PageMap map;
    float *out;              // [B,S,P]
    int32_t *err;
};
cudaError_t launch_indexer_scores(const ScoresArgs &a, cudaStream_t stream);

// TMA map of 8-bit rows [d2][d1][d0], box d0 x box1 x box2, swizzled over its
// rows; and H rounded up to the power of two that the tensor-core tiles take.
bool make_map_q8(CUtensorMap *m, const void *ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1,
                 uint32_t box2);
int padded_heads(int H);

struct ScoresBwdArgs {
    const float *dscores;    // [B,S,K]
    const int32_t *idx;      // [B,S,K] or NULL (K == P)
    const int8_t *q8;
    const float *q_scale, *w;
    const int8_t *k8;        // [B,P,D]
    const float *k_scale;    // [B,P]
    const int32_t *doc_start;
    int B, S, H, D, P, K, cr, t_begin;
    uint16_t *dq, *dk;       // bf16
    float *dw;
    int32_t *err;
};
size_t indexer_scores_bwd_ws_bytes(int B, int S, int H, int D, int P);
cudaError_t launch_indexer_scores_bwd(const ScoresBwdArgs &a, void *ws, cudaStream_t stream);

}  // namespace sai
