// latent_api.cu -- the C ABI of the latent cache and of the pages (declared in include/moe_verify.h):
// host-side validation and dispatch to the kernels.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_args.cuh"
#include "common.cuh"
#include "latent_args.cuh"

using namespace moe;

namespace {

constexpr bool kUsePdl = true;

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status_t check_latent(const moe_latent_cache_t *c) {
    if (c == nullptr || c->reserved != 0) return MOE_ERR_ARG;
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_ARG;
    if (c->rank < 1 || c->rope < 1 || c->page < 1 || c->pages < 1) return MOE_ERR_ARG;
    const int es = c->dtype == MOE_F32 ? 4 : 2;
    if (c->rank > 512 || c->rope > 128 || c->rank * es % 16 != 0 || c->rope * es % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c->pages) * c->page >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    if (c->rows == nullptr || !aligned(c->rows, 16)) return MOE_ERR_ARG;
    if (c->page_stride < 0 || c->token_stride < 0 || c->page_stride * es % 16 != 0 || c->token_stride * es % 16 != 0)
        return MOE_ERR_ARG;
    return MOE_OK;
}

bool heads_ok(const moe_heads_t *h) {
    if (h == nullptr || h->ptr == nullptr || h->heads < 1) return false;
    if (h->dtype != MOE_F32 && h->dtype != MOE_BF16) return false;
    return aligned(h->ptr, h->dtype == MOE_F32 ? 4 : 2);
}

int32_t *error_word(void *ws) { return ws == nullptr ? nullptr : &static_cast<DeviceWorkspace *>(ws)->error; }

moe_status_t check_pool(const moe_page_pool_t *p) {
    if (p == nullptr || p->pages < 1 || p->page < 1 || p->seqs < 1 || p->max_pages < 1) return MOE_ERR_ARG;
    if (p->refs == nullptr || p->table == nullptr || p->held == nullptr || !aligned(p->refs, 4) || !aligned(p->table, 4) ||
        !aligned(p->held, 4))
        return MOE_ERR_ARG;
    if (static_cast<int64_t>(p->pages) * p->page >= (1ll << 31) || static_cast<int64_t>(p->max_pages) * p->page >= (1ll << 31) ||
        static_cast<int64_t>(p->seqs) * p->max_pages >= (1ll << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t check_ws(const moe_page_pool_t *pool, const void *ws, size_t bytes) {
    if (ws == nullptr || bytes < moe_pages_workspace_bytes(pool)) return MOE_ERR_WORKSPACE;
    return aligned(ws, 16) ? MOE_OK : MOE_ERR_ARG;
}

PageArgs page_args(const moe_page_pool_t *pool, void *ws) {
    PageArgs a;
    std::memset(&a, 0, sizeof a);
    a.pool = *pool;
    a.err = error_word(ws);
    a.forked = &static_cast<DeviceWorkspace *>(ws)->forked;
    a.lists = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + kWorkspaceBytes);
    return a;
}

// A plane whose rows are one piece where they lie together, moved `unit` bytes at a time: 16 where addresses and
// strides are multiples of that, 4 for scales, whose address need not be one (with pages of one position all heads'
// scales are one piece, of any multiple of 4 bytes).
Plane plane_of(int64_t page, int64_t row, int64_t seg, int segs, int bytes, int unit) {
    Plane p;
    std::memset(&p, 0, sizeof p);
    p.page_stride = page;
    p.row_stride = row;
    p.seg_stride = seg;
    p.segs = segs;
    p.bytes = bytes;
    if (segs == 1 || seg == bytes) {
        p.bytes = bytes * segs;
        p.segs = 1;
        p.seg_stride = p.bytes;
    }
    p.unit = unit;
    p.per_seg = p.bytes / p.unit;
    p.per_row = p.per_seg * p.segs;
    p.dense = p.segs == 1 && row == p.bytes;
    p.by_seg = 0xFFFFFFFFu / static_cast<uint32_t>(p.per_seg);
    p.by_row = 0xFFFFFFFFu / static_cast<uint32_t>(p.per_row);
    return p;
}
bool same(const PageRows &a, const PageRows &b) {
    return a.planes == b.planes && std::memcmp(a.plane, b.plane, sizeof a.plane) == 0;
}

// The copying kernel numbers its work, sequences by layers, planes and pieces of up to 1024 units, in 31 bits.
bool too_much(const moe_page_pool_t *pool, const Plane &p) {
    const int64_t pieces = (static_cast<int64_t>(p.per_row) * pool->page + 1023) / 1024;
    return pieces >= (1ll << 21) || pool->seqs * pieces >= (1ll << 31) / (kLayersLaunch * kPlanes);
}

constexpr int kMaxLaunches = 16;   // of the rows' kernel in one call: 1024 caches of equal shape, or 16 shapes

// The caches as launches of up to kLayersLaunch of equal shape.
struct Layers {
    PageRows rows[kMaxLaunches];
    int launches = 0;

    moe_status_t add(const PageRows &shape, void *const (&base)[kPlanes]) {
        int at = launches - 1;   // the last launch of this shape
        while (at >= 0 && !same(rows[at], shape)) --at;
        if (at < 0 || rows[at].layers == kLayersLaunch) {
            if (launches == kMaxLaunches) return MOE_ERR_UNSUPPORTED;
            at = launches++;
            rows[at] = shape;
        }
        PageRows &r = rows[at];
        for (int i = 0; i < kPlanes; ++i) r.base[r.layers][i] = base[i];
        ++r.layers;
        return MOE_OK;
    }
};

// moe_kv_cache_t's own rules, through the call that checks them and enqueues nothing for no tokens.
moe_status_t check_kv(const moe_kv_cache_t *c) { return moe_kv_read(c, nullptr, 0, nullptr, nullptr, nullptr, nullptr); }

moe_status_t collect(const moe_page_pool_t *pool, const moe_page_caches_t *caches, Layers &out) {
    if (caches == nullptr || caches->kv_count < 0 || caches->latent_count < 0) return MOE_ERR_ARG;
    if ((caches->kv_count > 0 && caches->kv == nullptr) || (caches->latent_count > 0 && caches->latent == nullptr)) return MOE_ERR_ARG;
    PageRows shape;
    std::memset(&shape, 0, sizeof shape);
    for (int i = 0; i < caches->kv_count; ++i) {
        const moe_kv_cache_t &c = caches->kv[i];
        const moe_status_t st = check_kv(&c);
        if (st != MOE_OK) return st;
        if (c.pages != pool->pages || c.page != pool->page) return MOE_ERR_ARG;
        const int es = c.dtype == MOE_F32 ? 4 : (c.dtype == MOE_BF16 ? 2 : 1);
        std::memset(&shape, 0, sizeof shape);
        shape.planes = c.dtype == MOE_E4M3 ? 4 : 2;
        shape.plane[0] = shape.plane[1] = plane_of(c.page_stride * es, c.token_stride * es, c.head_stride * es, c.heads, c.dim * es, 16);
        if (c.dtype == MOE_E4M3)
            shape.plane[2] = shape.plane[3] =
                plane_of(static_cast<int64_t>(c.heads) * c.page * 4, 4, static_cast<int64_t>(c.page) * 4, c.heads, 4, 4);
        for (int k = 0; k < shape.planes; ++k)
            if (too_much(pool, shape.plane[k])) return MOE_ERR_UNSUPPORTED;
        void *const base[kPlanes] = {c.k, c.v, c.k_scale, c.v_scale};
        const moe_status_t full = out.add(shape, base);
        if (full != MOE_OK) return full;
    }
    for (int i = 0; i < caches->latent_count; ++i) {
        const moe_latent_cache_t &c = caches->latent[i];
        const moe_status_t st = check_latent(&c);
        if (st != MOE_OK) return st;
        if (c.pages != pool->pages || c.page != pool->page) return MOE_ERR_ARG;
        const int es = c.dtype == MOE_F32 ? 4 : 2;
        std::memset(&shape, 0, sizeof shape);
        shape.planes = 1;
        shape.plane[0] = plane_of(c.page_stride * es, c.token_stride * es, 0, 1, (c.rank + c.rope) * es, 16);
        if (too_much(pool, shape.plane[0])) return MOE_ERR_UNSUPPORTED;
        void *const base[kPlanes] = {c.rows, nullptr, nullptr, nullptr};
        const moe_status_t full = out.add(shape, base);
        if (full != MOE_OK) return full;
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_latent_write(const moe_latent_cache_t *cache, const moe_heads_t *latent, const moe_heads_t *k_rope,
                              const int32_t *slots, int32_t tokens, const float *norm, float eps,
                              const moe_rotary_t *rotary, const moe_heads_t *q, const moe_heads_t *q_out, void *ws,
                              moe_stream_t s) {
    const moe_status_t st = check_latent(cache);
    if (st != MOE_OK) return st;
    if (tokens < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_ARG;
    if (tokens == 0) return MOE_OK;
    if (!heads_ok(latent) || !heads_ok(k_rope) || latent->heads != 1 || k_rope->heads != 1) return MOE_ERR_ARG;
    if (slots == nullptr || !aligned(slots, 4) || !aligned(norm, 4) || (ws != nullptr && !aligned(ws, 16))) return MOE_ERR_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && rotary == nullptr)) return MOE_ERR_ARG;
    if (q != nullptr && (!heads_ok(q) || !heads_ok(q_out) || q->heads != q_out->heads)) return MOE_ERR_ARG;
    LatentWriteArgs a;
    std::memset(&a, 0, sizeof a);
    if (rotary != nullptr) {
        if (rotary->table == nullptr || rotary->positions == nullptr || !aligned(rotary->table, 8) || !aligned(rotary->positions, 4))
            return MOE_ERR_ARG;
        if (rotary->rot < 2 || rotary->rot % 2 != 0 || rotary->rot > cache->rope || rotary->table_positions < 1) return MOE_ERR_ARG;
        a.rot = *rotary;
    }
    if (q != nullptr) {
        a.q = *q;
        a.q_out = *q_out;
    }
    // the rows of a launch are numbered in 31 bits
    if (static_cast<int64_t>(tokens) * (1ll + a.q.heads) >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    a.cache = *cache;
    a.latent = *latent;
    a.k = *k_rope;
    a.latent.head_stride = a.k.head_stride = 0;   // one head: no step
    a.slots = slots;
    a.norm = norm;
    a.eps = eps;
    a.err = error_word(ws);
    a.tokens = tokens;
    return status_of(launch_latent_write(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

size_t moe_latent_attention_workspace_bytes(const moe_latent_cache_t *cache, int32_t tokens, int32_t seqs, int32_t heads) {
    if (cache == nullptr || tokens < 0 || seqs < 0 || heads < 1) return 0;
    if (cache->rank < 1 || cache->rank > 512) return kWorkspaceBytes;
    const size_t simt = latent_simt_part_bytes(cache->rank);
    return kWorkspaceBytes + (cache->dtype == MOE_BF16 ? std::max(latent_attn_part_bytes(), simt) : simt);
}

moe_status_t moe_latent_attention(const moe_latent_cache_t *cache, const moe_heads_t *q, const moe_heads_t *out, float *lse,
                                  const int32_t *q_start, const int32_t *ctx, const int32_t *page_table,
                                  const uint64_t *mask, int32_t seqs, int32_t tokens, int32_t max_tokens,
                                  int32_t max_pages, float scale, void *ws, size_t ws_bytes, moe_stream_t s) {
    const moe_status_t st = check_latent(cache);
    if (st != MOE_OK) return st;
    if (seqs < 0 || tokens < 0 || max_tokens < 1 || max_pages < 1 || !(scale > 0.0f) || !std::isfinite(scale)) return MOE_ERR_ARG;
    if (max_tokens > MOE_MAX_TREE_TOKENS || seqs > 65535) return MOE_ERR_UNSUPPORTED;
    if (tokens == 0 || seqs == 0) return MOE_OK;
    if (!heads_ok(q) || !heads_ok(out) || q->heads != out->heads || q->dtype != out->dtype) return MOE_ERR_ARG;
    if (q->heads > 1024) return MOE_ERR_UNSUPPORTED;
    if (q_start == nullptr || ctx == nullptr || page_table == nullptr || !aligned(q_start, 4) || !aligned(ctx, 4) ||
        !aligned(page_table, 4) || !aligned(mask, 8) || !aligned(lse, 4))
        return MOE_ERR_ARG;
    if (ws == nullptr || ws_bytes < moe_latent_attention_workspace_bytes(cache, tokens, seqs, q->heads)) return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return MOE_ERR_ARG;
    LatentArgs a;
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
    a.heads = q->heads;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.wait_limit = current_wait_limit();
    const cudaStream_t stream = reinterpret_cast<cudaStream_t>(s);
    if (latent_attn_supports(*cache, *q, *out)) {
        const cudaError_t e = launch_latent_attn(a, stream, kUsePdl);
        if (e != cudaErrorNotSupported) return status_of(e);
    }
    return status_of(launch_latent_simt(a, stream, kUsePdl));
}

size_t moe_pages_workspace_bytes(const moe_page_pool_t *pool) {
    if (pool == nullptr || pool->pages < 1 || pool->seqs < 1) return 0;
    return kWorkspaceBytes + pages_list_bytes(*pool);
}

moe_status_t moe_pages_reserve(const moe_page_pool_t *pool, const int32_t *length, const int32_t *need, int32_t *got,
                               const moe_page_caches_t *caches, void *ws, size_t ws_bytes, moe_stream_t s) {
    moe_status_t st = check_pool(pool);
    if (st != MOE_OK) return st;
    if (pool->seqs > MOE_MAX_POOL_SEQS) return MOE_ERR_UNSUPPORTED;
    if (length == nullptr || need == nullptr || !aligned(length, 4) || !aligned(need, 4) || !aligned(got, 4)) return MOE_ERR_ARG;
    Layers layers;
    if ((st = collect(pool, caches, layers)) != MOE_OK || (st = check_ws(pool, ws, ws_bytes)) != MOE_OK) return st;
    PageArgs a = page_args(pool, ws);
    a.length = length;
    a.need = need;
    a.got = got;
    return status_of(launch_pages_reserve(a, layers.rows, layers.launches, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

moe_status_t moe_pages_fork(const moe_page_pool_t *pool, const int32_t *src, const int32_t *dst, int32_t count,
                            int32_t *length, void *ws, size_t ws_bytes, moe_stream_t s) {
    moe_status_t st = check_pool(pool);
    if (st != MOE_OK) return st;
    if (count < 0) return MOE_ERR_ARG;
    if (count > MOE_MAX_POOL_SEQS) return MOE_ERR_UNSUPPORTED;
    if (count == 0) return MOE_OK;
    if (src == nullptr || dst == nullptr || length == nullptr || !aligned(src, 4) || !aligned(dst, 4) || !aligned(length, 4))
        return MOE_ERR_ARG;
    if ((st = check_ws(pool, ws, ws_bytes)) != MOE_OK) return st;
    PageArgs a = page_args(pool, ws);
    a.src = src;
    a.ids = dst;
    a.items = count;
    a.length_out = length;
    return status_of(launch_pages_fork(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

moe_status_t moe_pages_accept(const moe_page_pool_t *pool, const int32_t *ctx, const int32_t *path, const int32_t *count,
                              int32_t max_path, int32_t *after, const moe_page_caches_t *caches, void *ws,
                              size_t ws_bytes, moe_stream_t s) {
    moe_status_t st = check_pool(pool);
    if (st != MOE_OK) return st;
    if (max_path < 1) return MOE_ERR_ARG;
    if (max_path > MOE_MAX_TREE_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (ctx == nullptr || count == nullptr || !aligned(ctx, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(after, 4))
        return MOE_ERR_ARG;
    Layers layers;
    if ((st = collect(pool, caches, layers)) != MOE_OK || (st = check_ws(pool, ws, ws_bytes)) != MOE_OK) return st;
    for (int i = 0; i < layers.launches; ++i)   // the moving kernel numbers sequences by layers and slices in 31 bits
        if (static_cast<int64_t>(pool->seqs) * move_slices(layers.rows[i]) >= (1ll << 31) / kLayersLaunch) return MOE_ERR_UNSUPPORTED;
    PageArgs a = page_args(pool, ws);
    a.ctx = ctx;
    a.path = path;
    a.count = count;
    a.max_path = max_path;
    a.after = after;
    return status_of(launch_pages_accept(a, layers.rows, layers.launches, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

moe_status_t moe_pages_free(const moe_page_pool_t *pool, const int32_t *ids, int32_t count, int32_t *length, void *ws,
                            size_t ws_bytes, moe_stream_t s) {
    moe_status_t st = check_pool(pool);
    if (st != MOE_OK) return st;
    if (count < 0) return MOE_ERR_ARG;
    if (count == 0) return MOE_OK;
    if (ids == nullptr || !aligned(ids, 4) || !aligned(length, 4)) return MOE_ERR_ARG;
    if ((st = check_ws(pool, ws, ws_bytes)) != MOE_OK) return st;
    PageArgs a = page_args(pool, ws);
    a.ids = ids;
    a.items = count;
    a.length_out = length;
    return status_of(launch_pages_free(a, reinterpret_cast<cudaStream_t>(s), kUsePdl));
}

}  // extern "C"
