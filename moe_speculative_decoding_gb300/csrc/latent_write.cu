// latent_write.cu -- the rows of a paged latent cache: normalised latents and rotated rotary channels of a
// pass's tokens, and the rotation of its queries' rotary channels beside them.
//
//     y_i = c_i w_i / sqrt(mean(c^2) + eps),   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Streaming work, a few operations an element: the bound is memory traffic, each row read once and
// written once.
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
// A warp takes a token's cache row, or kPasses * 32 / T of its query rows: T threads (a power of two,
// T * 16 >= rope) hold a row of rotary channels, 16 each, both halves of 8 pairs of the half layout or
// 16 consecutive ones, and the token's 8 cosines and sines stay in registers.
constexpr int kPasses = 2;

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

template <typename IN, typename OUT, int T>
__global__ void __launch_bounds__(kRowThreads) latent_vec_kernel(const __grid_constant__ LatentWriteArgs a, uint32_t tasks, uint32_t total) {
    constexpr int kOut = sizeof(OUT) == 2 ? MOE_BF16 : MOE_F32, kIn = sizeof(IN) == 2 ? MOE_BF16 : MOE_F32;
    constexpr int kRows = 32 / T;
    pdl_wait();
    pdl_trigger();
    const uint32_t g = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (g >= total) return;
    const int64_t t = g / tasks;
    const int task = static_cast<int>(g - static_cast<uint32_t>(t) * tasks), lane = static_cast<int>(threadIdx.x & 31);
    const int c = lane % T, sub = lane / T;
    const int slot = task == 0 ? __ldg(a.slots + t) : 0;
    const int p = a.rot.rot > 0 ? __ldg(a.rot.positions + t) : 0;
    // what needs no place is on its way beside the slot and the position
    const bool turn = 16 * c < a.rot.rot, split = turn && !a.rot.interleaved, on = 16 * c < a.cache.rope;
    const int o0 = split ? 8 * c : 16 * c, o1 = split ? (a.rot.rot >> 1) + 8 * c : 16 * c + 8;
    Eight<IN> raw[kPasses][2], lat[2];
    const int h0 = (task - 1) * kPasses * kRows + sub;
    if (task == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = (j * 32 + lane) * 8;
            if (ch < a.cache.rank) fetch8(static_cast<const IN *>(a.latent.ptr) + t * a.latent.token_stride + ch, lat[j]);
        }
        if (on && sub == 0) {
            const IN *const k = static_cast<const IN *>(a.k.ptr) + t * a.k.token_stride;
            fetch8(k + o0, raw[0][0]);
            fetch8(k + o1, raw[0][1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            const int h = h0 + j * kRows;
            if (on && h < a.q.heads) {
                const IN *const q = static_cast<const IN *>(a.q.ptr) + t * a.q.token_stride + h * a.q.head_stride;
                fetch8(q + o0, raw[j][0]);
                fetch8(q + o1, raw[j][1]);
            }
        }
    }
    if (a.rot.rot > 0 && static_cast<uint32_t>(p) >= static_cast<uint32_t>(a.rot.table_positions)) {
        record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    float cs[16];
    if (turn && (task > 0 || sub == 0)) {
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
    if (task == 0) {
        float v[2][8];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if ((j * 32 + lane) * 8 >= a.cache.rank) continue;
            widen(lat[j], v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
        }
        float scale = 1.0f;
        if (a.norm != nullptr) scale = 1.0f / sqrtf(warp_sum(sum) / static_cast<float>(a.cache.rank) + a.eps);
        const int64_t at = row_at(a, slot);
        if (at < 0) return;
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
            rotated(raw[0], x, y);
            store8(a.cache.rows, kOut, at + a.cache.rank + o0, x);
            store8(a.cache.rows, kOut, at + a.cache.rank + o1, y);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
        const int h = h0 + j * kRows;
        if (!on || h >= a.q.heads) continue;
        float x[8], y[8];
        rotated(raw[j], x, y);
        const int64_t to = t * a.q_out.token_stride + h * a.q_out.head_stride;
        store8(a.q_out.ptr, kIn, to + o0, x);
        store8(a.q_out.ptr, kIn, to + o1, y);
    }
}

template <typename IN, typename OUT, int T>
cudaError_t launch(const LatentWriteArgs &a, cudaStream_t s, bool pdl) {
    constexpr int rows = kPasses * 32 / T;
    const uint32_t tasks = 1 + (a.q.heads + rows - 1) / rows, total = tasks * static_cast<uint32_t>(a.tokens);
    return launch_flat(latent_vec_kernel<IN, OUT, T>, (total + kRowThreads / 32 - 1) / (kRowThreads / 32), s, pdl, a, tasks, total);
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
