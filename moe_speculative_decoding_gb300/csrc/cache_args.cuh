// cache_args.cuh -- arguments of the attention-side kernels (rope_kv.cu, tree_attn_simt.cu,
// tree_attn.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "moe_verify.h"

namespace moe {

// Rows of one launch of the rotary / cache-row kernels.  Row r of a token: q rows, then k, then
// v.  q and k go to dense outputs or (k, v, cached != 0) into the cache.
struct RowArgs {
    moe_heads_t q, q_out, k, k_out, v;   // heads = 0 where absent
    moe_kv_cache_t cache;
    moe_rotary_t rot;                    // rot.rot = 0: no rotation
    const int32_t *slots;                // cached only
    int32_t *err;                        // may be null
    int32_t tokens, dim, cached;
};

struct ReadArgs {
    moe_kv_cache_t cache;
    moe_heads_t k_out, v_out;
    const int32_t *slots;
    int32_t *err;
    int32_t tokens;
};

// Most positions of a sequence: whole tiles of 128 that 31 bits number.
constexpr long long kMaxPositions = (1ll << 31) - 128;

struct TreeArgs {
    moe_kv_cache_t cache;
    moe_heads_t q, out;
    float *lse;                // may be null
    const int32_t *q_start, *ctx, *page_table;
    const uint64_t *mask;      // may be null: a chain
    int32_t *err;
    void *part;                // partial results (after the workspace header)
    long long wait_limit;
    int32_t seqs, tokens, max_tokens, max_pages, group;
    int32_t undivided;         // an item is one CTA's (short contexts)
    float scale_log2;          // scale * log2(e)
};

cudaError_t launch_rope_table(const double *w, int half, double magnitude, int positions, float *table,
                              cudaStream_t s);
cudaError_t launch_rows(const RowArgs &a, cudaStream_t s, bool pdl);
cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t s, bool pdl);
cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t s, bool pdl);
// The tensor-core kernel: whether it takes these operands, its workspace after the header, the
// launch (cudaErrorNotSupported: strides that no tensor map describes).
bool tree_attn_supports(const moe_kv_cache_t &c, const moe_heads_t &q, const moe_heads_t &out);
size_t tree_attn_part_bytes(int dim);
cudaError_t launch_tree_attn(TreeArgs a, cudaStream_t s, bool pdl);
long long current_wait_limit();   // moe_set_wait_limit's, or the default

}  // namespace moe
