// cache_api.cu -- the C ABI of the attention side (declared in include/moe_verify.h): host-side
// validation, the rotary frequencies, and dispatch to the kernels.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_args.cuh"
#include "common.cuh"

using namespace moe;

namespace {

constexpr bool kUsePdl = true;

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

moe_status_t status_of(cudaError_t e) {
    if (e == cudaErrorNotSupported) return MOE_ERR_UNSUPPORTED;
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t check_cache(const moe_kv_cache_t *c) {
    if (c == nullptr || c->reserved != 0) return MOE_ERR_ARG;
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16 && c->dtype != MOE_E4M3) return MOE_ERR_ARG;
    if (c->heads < 1 || c->dim < 1 || c->page < 1 || c->pages < 1) return MOE_ERR_ARG;
    const int es = c->dtype == MOE_F32 ? 4 : (c->dtype == MOE_BF16 ? 2 : 1);
    if (c->dim > 256 || c->dim * es % 16 != 0 || c->heads > 65535) return MOE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c->pages) * c->page >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    if (c->k == nullptr || c->v == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16)) return MOE_ERR_ARG;
    const int64_t strides[] = {c->page_stride, c->token_stride, c->head_stride};
    for (const int64_t st : strides)
        if (st < 0 || st * es % 16 != 0) return MOE_ERR_ARG;
    if (c->dtype == MOE_E4M3 &&
        (c->k_scale == nullptr || c->v_scale == nullptr || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
        return MOE_ERR_ARG;
    return MOE_OK;
}

bool heads_ok(const moe_heads_t *h) {
    if (h == nullptr || h->ptr == nullptr || h->heads < 1) return false;
    if (h->dtype != MOE_F32 && h->dtype != MOE_BF16) return false;
    return aligned(h->ptr, h->dtype == MOE_F32 ? 4 : 2);
}

moe_status_t check_rotary(const moe_rotary_t *r, int dim) {
    if (r == nullptr || r->table == nullptr || r->positions == nullptr || !aligned(r->table, 8) ||
        !aligned(r->positions, 4))
        return MOE_ERR_ARG;
    if (r->rot < 2 || r->rot % 2 != 0 || r->rot > dim || r->table_positions < 1) return MOE_ERR_ARG;
    return MOE_OK;
}

// The rows of a launch are numbered in 31 bits.
bool too_many_rows(int64_t tokens, int64_t rows) { return tokens * rows >= (1ll << 31); }

int32_t *error_word(void *ws) { return ws == nullptr ? nullptr : &static_cast<DeviceWorkspace *>(ws)->error; }

}  // namespace

extern "C" {

moe_status_t moe_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, int32_t original,
                                  double beta_fast, double beta_slow, double *w, double *magnitude) {
    if (w == nullptr || magnitude == nullptr || rot < 2 || rot > 256 || rot % 2 != 0) return MOE_ERR_ARG;
    if (!(base > 1.0) || !(factor >= 1.0) || !std::isfinite(base) || !std::isfinite(factor)) return MOE_ERR_ARG;
    if (scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_BY_PARTS) return MOE_ERR_ARG;
    double lo = 0.0, hi = 0.0;
    if (scaling == MOE_ROPE_BY_PARTS) {
        if (original < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
            return MOE_ERR_ARG;
        const double kTwoPi = 6.283185307179586476925;
        auto index = [&](double turns) { return rot * std::log(original / (kTwoPi * turns)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(index(beta_fast)), 0.0);
        hi = std::min(std::ceil(index(beta_slow)), static_cast<double>(rot - 1));
        if (hi < lo + 0.001) hi = lo + 0.001;
    }
    if (scaling == MOE_ROPE_BASE && rot > 2) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        const double plain = std::pow(base, -2.0 * i / rot);
        w[i] = plain;
        if (scaling == MOE_ROPE_LINEAR) w[i] = plain / factor;
        if (scaling == MOE_ROPE_BY_PARTS) {
            const double ramp = std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);
            w[i] = plain * (ramp / factor + 1.0 - ramp);
        }
    }
    *magnitude = scaling == MOE_ROPE_BY_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return MOE_OK;
}

moe_status_t moe_rope_table(const double *w, int32_t half, double magnitude, int32_t positions, float *table,
                            moe_stream_t s) {
    if (w == nullptr || half < 1 || half > 128 || positions < 0) return MOE_ERR_ARG;
    if (positions == 0) return MOE_OK;
    if (table == nullptr || !aligned(table, 8)) return MOE_ERR_ARG;
    return status_of(launch_rope_table(w, half, magnitude, positions, table, reinterpret_cast<cudaStream_t>(s)));
}

moe_status_t moe_rope(const moe_heads_t *q, const moe_heads_t *q_out, const moe_heads_t *k, const moe_heads_t *k_out,
                      int32_t tokens, int32_t dim, const moe_rotary_t *rotary, void *ws, moe_stream_t s) {
    if (tokens < 0 || dim < 1) return MOE_ERR_ARG;
    if (dim > 256) return MOE_ERR_UNSUPPORTED;
    if (tokens == 0) return MOE_OK;
    moe_status_t st = check_rotary(rotary, dim);
    if (st != MOE_OK) return st;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return MOE_ERR_ARG;
    if (q == nullptr && k == nullptr) return MOE_ERR_ARG;
    if (q != nullptr && (!heads_ok(q) || !heads_ok(q_out) || q->heads != q_out->heads)) return MOE_ERR_ARG;
    if (k != nullptr && (!heads_ok(k) || !heads_ok(k_out) || k->heads != k_out->heads)) return MOE_ERR_ARG;
    if (ws != nullptr && !aligned(ws, 16)) return MOE_ERR_ARG;
    RowArgs a;
    std::memset(&a, 0, sizeof a);
    if (q != nullptr) {
        a.q = *q;
        a.q_out = *q_out;
    }
    if (k != nullptr) {
        a.k = *k;
        a.k_out = *k_out;
    }
    if (too_many_rows(tokens, static_cast<int64_t>(a.q.heads) + a.k.heads)) return MOE_ERR_UNSUPPORTED;
    a.rot = *rotary;
    a.err = error_word(ws);
    a.tokens = tokens;
    a.dim = dim;
    return status_of(launch_rows(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

moe_status_t moe_kv_write(const moe_kv_cache_t *cache, const moe_heads_t *k, const moe_heads_t *v,
                          const int32_t *slots, int32_t tokens, const moe_rotary_t *rotary, const moe_heads_t *q,
                          const moe_heads_t *q_out, void *ws, moe_stream_t s) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    if (tokens < 0) return MOE_ERR_ARG;
    if (tokens == 0) return MOE_OK;
    if (!heads_ok(k) || !heads_ok(v) || k->heads != cache->heads || v->heads != cache->heads) return MOE_ERR_ARG;
    if (slots == nullptr || !aligned(slots, 4) || (ws != nullptr && !aligned(ws, 16))) return MOE_ERR_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && rotary == nullptr)) return MOE_ERR_ARG;
    if (q != nullptr && (!heads_ok(q) || !heads_ok(q_out) || q->heads != q_out->heads)) return MOE_ERR_ARG;
    RowArgs a;
    std::memset(&a, 0, sizeof a);
    if (rotary != nullptr) {
        st = check_rotary(rotary, cache->dim);
        if (st != MOE_OK) return st;
        a.rot = *rotary;
    }
    if (q != nullptr) {
        a.q = *q;
        a.q_out = *q_out;
    }
    if (too_many_rows(tokens, static_cast<int64_t>(a.q.heads) + 2ll * cache->heads)) return MOE_ERR_UNSUPPORTED;
    a.k = *k;
    a.v = *v;
    a.cache = *cache;
    a.slots = slots;
    a.err = error_word(ws);
    a.tokens = tokens;
    a.dim = cache->dim;
    a.cached = 1;
    return status_of(launch_rows(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

moe_status_t moe_kv_read(const moe_kv_cache_t *cache, const int32_t *slots, int32_t tokens, const moe_heads_t *k_out,
                         const moe_heads_t *v_out, void *ws, moe_stream_t s) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    if (tokens < 0) return MOE_ERR_ARG;
    if (tokens == 0) return MOE_OK;
    if (!heads_ok(k_out) || !heads_ok(v_out) || k_out->heads != cache->heads || v_out->heads != cache->heads)
        return MOE_ERR_ARG;
    if (slots == nullptr || !aligned(slots, 4) || (ws != nullptr && !aligned(ws, 16))) return MOE_ERR_ARG;
    if (too_many_rows(tokens, 2ll * cache->heads)) return MOE_ERR_UNSUPPORTED;
    ReadArgs a;
    std::memset(&a, 0, sizeof a);
    a.cache = *cache;
    a.k_out = *k_out;
    a.v_out = *v_out;
    a.slots = slots;
    a.err = error_word(ws);
    a.tokens = tokens;
    return status_of(launch_kv_read(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

size_t moe_tree_attention_workspace_bytes(const moe_kv_cache_t *cache, int32_t tokens, int32_t seqs, int32_t q_heads) {
    if (cache == nullptr || tokens < 0 || seqs < 0 || q_heads < 1) return 0;
    const bool parts = (cache->dtype == MOE_BF16 || cache->dtype == MOE_E4M3) && cache->dim <= 128;
    return kWorkspaceBytes + (parts ? tree_attn_part_bytes(cache->dim) : 0);
}

moe_status_t moe_tree_attention(const moe_kv_cache_t *cache, const moe_heads_t *q, const moe_heads_t *out, float *lse,
                                const int32_t *q_start, const int32_t *ctx, const int32_t *page_table,
                                const uint64_t *mask, int32_t seqs, int32_t tokens, int32_t max_tokens,
                                int32_t max_pages, float scale, void *ws, size_t ws_bytes, moe_stream_t s) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK) return st;
    if (seqs < 0 || tokens < 0 || max_tokens < 1 || max_pages < 1 || !(scale > 0.0f) || !std::isfinite(scale))
        return MOE_ERR_ARG;
    if (max_tokens > MOE_MAX_TREE_TOKENS || seqs > 65535) return MOE_ERR_UNSUPPORTED;
    if (tokens == 0 || seqs == 0) return MOE_OK;
    if (!heads_ok(q) || !heads_ok(out) || q->heads != out->heads || q->dtype != out->dtype) return MOE_ERR_ARG;
    if (q->heads % cache->heads != 0) return MOE_ERR_ARG;
    if (q->heads / cache->heads > 64) return MOE_ERR_UNSUPPORTED;
    if (q_start == nullptr || ctx == nullptr || page_table == nullptr || !aligned(q_start, 4) || !aligned(ctx, 4) ||
        !aligned(page_table, 4) || !aligned(mask, 8) || !aligned(lse, 4))
        return MOE_ERR_ARG;
    if (ws == nullptr || ws_bytes < moe_tree_attention_workspace_bytes(cache, tokens, seqs, q->heads))
        return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return MOE_ERR_ARG;
    TreeArgs a;
    std::memset(&a, 0, sizeof a);
    a.cache = *cache;
    a.q = *q;
    a.out = *out;
    a.lse = lse;
    a.q_start = q_start;
    a.ctx = ctx;
    a.page_table = page_table;
    a.mask = mask;
    a.err = error_word(ws);
    a.part = static_cast<uint8_t *>(ws) + kWorkspaceBytes;
    a.seqs = seqs;
    a.tokens = tokens;
    a.max_tokens = max_tokens;
    a.max_pages = max_pages;
    a.group = q->heads / cache->heads;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.wait_limit = current_wait_limit();
    const cudaStream_t st_ = reinterpret_cast<cudaStream_t>(s);
    if (tree_attn_supports(*cache, *q, *out)) {
        const cudaError_t e = launch_tree_attn(a, st_, kUsePdl);
        if (e != cudaErrorNotSupported) return status_of(e);
    }
    return status_of(launch_tree_simt(a, st_, kUsePdl));
}

}  // extern "C"
