// latent_args.cuh -- arguments of the latent-cache kernels (latent_write.cu, latent_attn.cu,
// latent_simt.cu) and of the page kernels (pages.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "moe_verify.h"

namespace moe {

struct LatentWriteArgs {
    moe_latent_cache_t cache;
    moe_heads_t latent, k, q, q_out;   // q.heads = 0: absent
    moe_rotary_t rot;                  // rot.rot = 0: no rotation
    const int32_t *slots;
    const float *norm;                 // may be null
    int32_t *err;                      // may be null
    int32_t tokens;
    float eps;
};

struct LatentArgs {
    moe_latent_cache_t cache;
    moe_heads_t q, out;
    float *lse;                // may be null
    const int32_t *q_start, *ctx, *page_table;
    const uint64_t *mask;      // may be null: a chain
    int32_t *err;
    void *part;                // partial results (after the workspace header)
    long long wait_limit;
    int32_t seqs, tokens, max_tokens, max_pages, heads;
    int32_t undivided;         // tensor cores: an item is one CTA's (short contexts)
    int32_t divisions;         // CUDA cores: parts of the positions
    float scale_log2;          // scale * log2(e)
};

cudaError_t launch_latent_write(const LatentWriteArgs &a, cudaStream_t s, bool pdl);
// The kernel on the CUDA cores and its workspace after the header.
cudaError_t launch_latent_simt(const LatentArgs &a, cudaStream_t s, bool pdl);
size_t latent_simt_part_bytes(int rank);
// The tensor-core kernel: whether it takes these operands, its workspace after the header, the
// launch (cudaErrorNotSupported: strides that no tensor map describes).
bool latent_attn_supports(const moe_latent_cache_t &c, const moe_heads_t &q, const moe_heads_t &out);
size_t latent_attn_part_bytes();
cudaError_t launch_latent_attn(LatentArgs a, cudaStream_t s, bool pdl);

// Rows of one layer's cache that move from page to page: up to four planes (keys, values, and their
// scales) of `segs` pieces of `bytes` bytes a row.  All strides in bytes.
struct Plane {
    int64_t page_stride, row_stride, seg_stride;
    int32_t segs, bytes;
    int32_t unit, per_seg, per_row;   // bytes moved at a time (16, 4 for scales), units of a piece and of a row
    int32_t dense;                    // a page's rows are one piece
    uint32_t by_seg, by_row;          // floor((2^32 - 1) / per_seg), of per_row
};
constexpr int kPlanes = 4, kLayersLaunch = 64;   // caches of equal shape in one launch
struct PageRows {
    Plane plane[kPlanes];
    int32_t planes, layers;
    void *base[kLayersLaunch][kPlanes];
};
// Pieces of a row (of up to 128 units, all its planes in line) that a CTA of the moving kernel takes.
constexpr int kMove = 128;
inline int move_columns(const PageRows &r) {
    int columns = 0;
    for (int k = 0; k < r.planes; ++k) columns += r.plane[k].per_row;
    return columns;
}
inline int move_slices(const PageRows &r) { return (move_columns(r) + kMove - 1) / kMove; }

struct PageArgs {
    moe_page_pool_t pool;
    int32_t *err;
    uint32_t *forked;          // the header's count of a fork's CTAs
    int32_t *lists;            // workspace after the header: nothing in it outlives a call
    const int32_t *length, *need, *ctx, *path, *count, *src, *ids;
    int32_t *got, *after, *length_out;
    int32_t items, max_path;
};
size_t pages_list_bytes(const moe_page_pool_t &pool);
cudaError_t launch_pages_reserve(const PageArgs &a, const PageRows *rows, int launches, cudaStream_t s, bool pdl);
cudaError_t launch_pages_fork(const PageArgs &a, cudaStream_t s, bool pdl);
cudaError_t launch_pages_accept(const PageArgs &a, const PageRows *rows, int launches, cudaStream_t s, bool pdl);
cudaError_t launch_pages_free(const PageArgs &a, cudaStream_t s, bool pdl);

}  // namespace moe
