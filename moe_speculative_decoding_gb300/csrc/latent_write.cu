// latent_write.cu -- the rows of a paged latent cache: normalised latents and rotated rotary channels of a
// pass's tokens, and the rotation of its queries' rotary channels beside them.
//
//     y_i = c_i w_i / sqrt(mean(c^2) + eps),   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Streaming work, a few operations an element: the bound is memory traffic, each row read once and
// written once.  16301 tokens with 32 heads of 64 rotary channels, bf16: 35.5 us, 4.94 TB/s (a copy of the queries'
// bytes alone, 128 of every 384, reaches 5.5); a pass of 16 tokens with 16 heads 2.8 us, the latency of its
// chain of loads (slot and position, table row).  The same for fp32: 76 us, 4.55 TB/s, and 3.4; bf16 rows into an fp32 cache
// 39 us, 4.96 TB/s.  Rows that are not 16-byte pieces take a warp each, an element or two to a lane at a
// time: 109 us in bf16 (1.6 TB/s), 115 in fp32 (3.0), a pass of 16 tokens 5.3.
#include "latent_args.cuh"
#include "row_common.cuh"

namespace moe {
namespace {

// The place of a token's cache row in elements, -1: it takes nothing.
__device__ __forceinline__ int64_t row_at(const LatentWriteArgs &a, int slot) {
    if (slot < 0) return -1;
    const int page = slot / a.cache.page;
    if (page >= a.cache.pages) {
        record_error(a.err, MOE_ERR_BAD_ID);
        return -1;
    }
    return page * a.cache.page_stride + static_cast<int64_t>(slot - page * a.cache.page) * a.cache.token_stride;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ------------------------------------------------------------------ any layout and types
// A warp per row: row 0 of a token is its cache row, row 1 + h its query head h.
__global__ void __launch_bounds__(kRowThreads) latent_any_kernel(const __grid_constant__ LatentWriteArgs a, uint32_t rows, uint32_t total) {
    pdl_wait();
    pdl_trigger();
    const uint32_t g = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (g >= total) return;
    const int64_t t = g / rows;
    const int r = static_cast<int>(g - static_cast<uint32_t>(t) * rows) - 1, lane = static_cast<int>(threadIdx.x & 31);
    const float2 *cs = nullptr;
    if (a.rot.rot > 0) {
        const int p = a.rot.positions[t];
        if (static_cast<uint32_t>(p) >= static_cast<uint32_t>(a.rot.table_positions)) {
            record_error(a.err, MOE_ERR_BAD_ID);
            return;
        }
        cs = reinterpret_cast<const float2 *>(a.rot.table) + static_cast<int64_t>(p) * (a.rot.rot >> 1);
    }
    const void *src;
    void *dst;
    int64_t from, to;
    int src_type, dst_type;
    if (r < 0) {
        const int64_t at = row_at(a, a.slots[t]);
        if (at < 0) return;
        const int64_t c0 = t * a.latent.token_stride;
        float scale = 1.0f;
        if (a.norm != nullptr) {
            float sum = 0.0f;
            for (int i = lane; i < a.cache.rank; i += 32) {
                const float x = load1(a.latent.ptr, a.latent.dtype, c0 + i);
                sum = fmaf(x, x, sum);
            }
            scale = 1.0f / sqrtf(warp_sum(sum) / static_cast<float>(a.cache.rank) + a.eps);
        }
        for (int i = lane; i < a.cache.rank; i += 32) {
            float x = load1(a.latent.ptr, a.latent.dtype, c0 + i);
            if (a.norm != nullptr) x *= scale * a.norm[i];
            store1(a.cache.rows, a.cache.dtype, at + i, x);
        }
        src = a.k.ptr;
        src_type = a.k.dtype;
        from = t * a.k.token_stride;
        dst = a.cache.rows;
        dst_type = a.cache.dtype;
        to = at + a.cache.rank;
    } else {
        src = a.q.ptr;
        src_type = a.q.dtype;
        from = t * a.q.token_stride + r * a.q.head_stride;
        dst = a.q_out.ptr;
        dst_type = a.q_out.dtype;
        to = t * a.q_out.token_stride + r * a.q_out.head_stride;
    }
    const int half = a.rot.rot >> 1;
    for (int i = lane; i < half; i += 32) {   // (a pair is one lane's, so that q_out may be q)
        const int o0 = a.rot.interleaved ? 2 * i : i, o1 = a.rot.interleaved ? 2 * i + 1 : i + half;
        float x = load1(src, src_type, from + o0), y = load1(src, src_type, from + o1);
        const float2 k = cs[i];
        turn_pair(x, y, k.x, a.rot.inverse ? -k.y : k.y);
        store1(dst, dst_type, to + o0, x);
        store1(dst, dst_type, to + o1, y);
    }
    for (int i = 2 * half + lane; i < a.cache.rope; i += 32) store1(dst, dst_type, to + i, load1(src, src_type, from + i));
}

// ------------------------------------------------------------------ 16 bytes at a time
// `share` warps to a token.  A token's groups are its cache row (group 0) and its query heads, 32 / T at a time:
// T threads (a power of two, T * 16 >= rope) hold a row of rotary channels, 16 each, both halves of 8 pairs
// of the half layout or 16 consecutive ones.  A warp takes every share-th group; the token's slot, position
// and table row are found once, and the next group's loads are on their way while it works on one.
template <typename IN>
struct Eight {
    uint4 v[sizeof(IN) / 2];   // 8 channels as they come from memory
};
template <typename IN>
__device__ __forceinline__ void fetch8(const IN *p, Eight<IN> &r) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(IN) / 2); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
}
template <typename IN>
__device__ __forceinline__ void widen(const Eight<IN> &r, float (&x)[8]) {
    const uint32_t *const w = reinterpret_cast<const uint32_t *>(&r);
    if constexpr (sizeof(IN) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
}


// Two chunks of eight channels at o0 and o1: one access of 32 bytes where they are one piece.
template <typename IN>
__device__ __forceinline__ void fetch_pair(const IN *p, int o0, int o1, Eight<IN> (&r)[2]) {
    if constexpr (sizeof(IN) == 2) {
        if (o1 == o0 + 8 && (reinterpret_cast<uintptr_t>(p + o0) & 31u) == 0) {
            uint4 &x = r[0].v[0], &y = r[1].v[0];
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                         : "l"(p + o0)
                         : "memory");
            return;
        }
    }
    fetch8(p + o0, r[0]);
    fetch8(p + o1, r[1]);
}
template <int TYPE>
__device__ __forceinline__ void store_pair(void *base, int64_t at, int o0, int o1, const float (&x)[8], const float (&y)[8]) {
    if constexpr (TYPE == MOE_BF16) {
        uint16_t *const p = static_cast<uint16_t *>(base) + at + o0;
        if (o1 == o0 + 8 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(pack_bf16(x[0], x[1])),
                         "r"(pack_bf16(x[2], x[3])), "r"(pack_bf16(x[4], x[5])), "r"(pack_bf16(x[6], x[7])), "r"(pack_bf16(y[0], y[1])),
                         "r"(pack_bf16(y[2], y[3])), "r"(pack_bf16(y[4], y[5])), "r"(pack_bf16(y[6], y[7]))
                         : "memory");
            return;
        }
    }
    store8(base, TYPE, at + o0, x);
    store8(base, TYPE, at + o1, y);
}

template <typename IN, typename OUT, int T>
__global__ void __launch_bounds__(kRowThreads, 4) latent_vec_kernel(const __grid_constant__ LatentWriteArgs a, uint32_t share, uint32_t total) {
    constexpr int kOut = sizeof(OUT) == 2 ? MOE_BF16 : MOE_F32, kIn = sizeof(IN) == 2 ? MOE_BF16 : MOE_F32;
    constexpr int kRows = 32 / T;
    pdl_wait();
    pdl_trigger();
    const uint32_t g = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (g >= total) return;
    const int64_t t = g / share;
    const int mine = static_cast<int>(g - static_cast<uint32_t>(t) * share), lane = static_cast<int>(threadIdx.x & 31);
    const int c = lane % T, sub = lane / T;
    const int slot = mine == 0 ? __ldg(a.slots + t) : 0;
    const int p = a.rot.rot > 0 ? __ldg(a.rot.positions + t) : 0;
    // what needs no place is on its way beside the slot and the position
    const bool turn = 16 * c < a.rot.rot, split = turn && !a.rot.interleaved, on = 16 * c < a.cache.rope;
    const int o0 = split ? 8 * c : 16 * c, o1 = split ? (a.rot.rot >> 1) + 8 * c : 16 * c + 8;
    Eight<IN> lat[2], key[2], next[2];
    if (mine == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = (j * 32 + lane) * 8;
            if (ch < a.cache.rank) fetch8(static_cast<const IN *>(a.latent.ptr) + t * a.latent.token_stride + ch, lat[j]);
        }
        if (on && sub == 0) {
            const IN *const k = static_cast<const IN *>(a.k.ptr) + t * a.k.token_stride;
            fetch_pair(k, o0, o1, key);
        }
    }
    const int step = static_cast<int>(share) * kRows;   // heads
    int h = (mine == 0 ? static_cast<int>(share) - 1 : mine - 1) * kRows + sub;
    const IN *q = static_cast<const IN *>(a.q.ptr) + t * a.q.token_stride + h * a.q.head_stride;
    if (on && h < a.q.heads) {
        fetch_pair(q, o0, o1, next);
    }
    if (a.rot.rot > 0 && static_cast<uint32_t>(p) >= static_cast<uint32_t>(a.rot.table_positions)) {
        record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    float cs[16];
    if (turn) {
        const float4 *const k = reinterpret_cast<const float4 *>(a.rot.table + static_cast<int64_t>(p) * a.rot.rot) + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(k + i);
            cs[4 * i] = v.x;
            cs[4 * i + 1] = a.rot.inverse ? -v.y : v.y;
            cs[4 * i + 2] = v.z;
            cs[4 * i + 3] = a.rot.inverse ? -v.w : v.w;
        }
    }
    auto rotated = [&](const Eight<IN> (&r)[2], float (&x)[8], float (&y)[8]) {
        widen(r[0], x);
        widen(r[1], y);
        if (!turn) return;
        if (a.rot.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                turn_pair(x[2 * i], x[2 * i + 1], cs[2 * i], cs[2 * i + 1]);
                turn_pair(y[2 * i], y[2 * i + 1], cs[8 + 2 * i], cs[8 + 2 * i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(x[i], y[i], cs[2 * i], cs[2 * i + 1]);
        }
    };
    const int64_t at = mine == 0 ? row_at(a, slot) : -1;
    if (at >= 0) {   // (the whole warp)
        float v[2][8], sum = 0.0f, scale = 1.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if ((j * 32 + lane) * 8 >= a.cache.rank) continue;
            widen(lat[j], v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
        }
        if (a.norm != nullptr) scale = 1.0f / sqrtf(warp_sum(sum) / static_cast<float>(a.cache.rank) + a.eps);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = (j * 32 + lane) * 8;
            if (ch >= a.cache.rank) continue;
            if (a.norm != nullptr) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(a.norm + ch) + i);
                    v[j][4 * i] *= scale * w.x;
                    v[j][4 * i + 1] *= scale * w.y;
                    v[j][4 * i + 2] *= scale * w.z;
                    v[j][4 * i + 3] *= scale * w.w;
                }
            }
            store8(a.cache.rows, kOut, at + ch, v[j]);
        }
        if (on && sub == 0) {
            float x[8], y[8];
            rotated(key, x, y);
            store_pair<kOut>(a.cache.rows, at + a.cache.rank, o0, o1, x, y);
        }
    }
    if (!on) return;
    const int64_t q_step = step * a.q.head_stride, out_step = step * a.q_out.head_stride;
    int64_t to = t * a.q_out.token_stride + h * a.q_out.head_stride;
    for (; h < a.q.heads; h += step, to += out_step) {
        float x[8], y[8];
        rotated(next, x, y);
        q += q_step;
        if (h + step < a.q.heads) {
            fetch_pair(q, o0, o1, next);
        }
        store_pair<kIn>(a.q_out.ptr, to, o0, o1, x, y);
    }
}

// A warp for every group while all of them are resident at once, so that a short call is short; else one to a
// token (16301 tokens with 32 heads: 35.5 us, with two warps to a token 37, with three 41; four CTAs an SM: with
// three, whose threads have 80 registers, 38, with five 42).
template <typename IN, typename OUT, int T>
cudaError_t launch(const LatentWriteArgs &a, cudaStream_t s, bool pdl) {
    constexpr int rows = 32 / T;
    uint32_t share = 1 + (a.q.heads + rows - 1) / rows;
    if (static_cast<int64_t>(share) * a.tokens > 152ll * 32) share = 1;
    const uint32_t total = share * static_cast<uint32_t>(a.tokens);
    return launch_flat(latent_vec_kernel<IN, OUT, T>, (total + kRowThreads / 32 - 1) / (kRowThreads / 32), s, pdl, a, share, total);
}
template <typename IN, typename OUT>
cudaError_t by_rope(const LatentWriteArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.rope <= 32) return launch<IN, OUT, 2>(a, s, pdl);
    return a.cache.rope <= 64 ? launch<IN, OUT, 4>(a, s, pdl) : launch<IN, OUT, 8>(a, s, pdl);
}
template <typename IN>
cudaError_t by_cache(const LatentWriteArgs &a, cudaStream_t s, bool pdl) {
    return a.cache.dtype == MOE_BF16 ? by_rope<IN, uint16_t>(a, s, pdl) : by_rope<IN, float>(a, s, pdl);
}

}  // namespace

cudaError_t launch_latent_write(const LatentWriteArgs &a, cudaStream_t s, bool pdl) {
    const int type = a.latent.dtype;
    const bool vec = a.cache.rank % 8 == 0 && a.cache.rope % 16 == 0 && a.rot.rot % 16 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.rot.table) | reinterpret_cast<uintptr_t>(a.norm)) & 15u) == 0 &&
                     vec_rows(a.latent) && vec_rows(a.k) && vec_rows(a.q) && vec_rows(a.q_out) && a.k.dtype == type &&
                     (a.q.heads == 0 || (a.q.dtype == type && a.q_out.dtype == type));
    if (vec) return type == MOE_BF16 ? by_cache<uint16_t>(a, s, pdl) : by_cache<float>(a, s, pdl);
    const uint32_t rows = 1 + a.q.heads, total = rows * static_cast<uint32_t>(a.tokens);   // the caller keeps it below 2^31
    return launch_flat(latent_any_kernel, (total + kRowThreads / 32 - 1) / (kRowThreads / 32), s, pdl, a, rows, total);
}

}  // namespace moe
