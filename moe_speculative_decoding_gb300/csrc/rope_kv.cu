// rope_kv.cu -- rotary positions and the rows of a paged key/value cache: rotation of the pass's
// queries and keys, the (quantising) write of its keys and values, and the read back.
//
// A row is one head of one token, `dim` channels.  Rotation multiplies each channel pair (a, b)
// by [[c, -s], [s, c]] with c = m cos(p w_i), s = m sin(p w_i) from a table (its transpose for
// gradients).  A quantised row is codes of x / scale with scale = amax / 448.  All of it is
// streaming work, a few operations per element: the bound is memory traffic, each row read once
// and written once.
#include "cache_args.cuh"
#include "common.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ rotary table
struct TableFreq {
    double w[128];
};

// One thread per (position, frequency); double sine and cosine (a table is made once).
__global__ void __launch_bounds__(kThreads)
rope_table_kernel(const __grid_constant__ TableFreq f, int half, double magnitude, int positions, float2 *table) {
    const long long total = static_cast<long long>(positions) * half;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        double s, c;
        sincos(static_cast<double>(i / half) * f.w[i % half], &s, &c);
        table[i] = make_float2(static_cast<float>(magnitude * c), static_cast<float>(magnitude * s));
    }
}

// ------------------------------------------------------------------ elements
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 consecutive elements, 16-byte aligned, in fp32
__device__ __forceinline__ void load8(const void *p, int dtype, int64_t off, float (&v)[8]) {
    if (dtype == MOE_BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 u = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + off)[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
    }
}
__device__ __forceinline__ void store8(void *p, int dtype, int64_t off, const float (&v)[8]) {
    if (dtype == MOE_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + off) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        float4 *const q = reinterpret_cast<float4 *>(static_cast<float *>(p) + off);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ float load1(const void *p, int dtype, int64_t off) {
    return dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[off])
                             : static_cast<const float *>(p)[off];
}
__device__ __forceinline__ void store1(void *p, int dtype, int64_t off, float v) {
    if (dtype == MOE_BF16)
        static_cast<__nv_bfloat16 *>(p)[off] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[off] = v;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
// the two values of a pair of codes
__device__ __forceinline__ float2 unpack_e4m3x2(uint16_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    float2 r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

// amax / 448, or 1 where that is 0 (a zero row, or one below the smallest scale)
__device__ __forceinline__ float row_scale(float amax) {
    const float s = amax / 448.0f;
    return s > 0.0f ? s : 1.0f;
}

// ------------------------------------------------------------------ where a row comes from and goes
struct Row {
    const void *src;
    void *dst;           // null: the row is not written
    float *scale;        // e4m3 cache rows
    int64_t src_off, dst_off;
    int src_type, dst_type;
    const float2 *cs;    // the token's table row, or null: no rotation
};

__device__ __forceinline__ Row locate(const RowArgs &a, uint32_t g, uint32_t rows) {
    Row w;
    const uint32_t t = g / rows;
    int r = static_cast<int>(g - t * rows);
    w.cs = nullptr;
    w.scale = nullptr;
    w.dst = nullptr;
    w.dst_off = 0;
    bool live = true;
    if (a.rot.rot > 0) {
        const int p = a.rot.positions[t];
        live = static_cast<uint32_t>(p) < static_cast<uint32_t>(a.rot.table_positions);
        if (!live)
            record_error(a.err, MOE_ERR_BAD_ID);
        else
            w.cs = reinterpret_cast<const float2 *>(a.rot.table) + static_cast<int64_t>(p) * (a.rot.rot >> 1);
    }
    const bool is_q = r < a.q.heads;
    if (!is_q) r -= a.q.heads;
    const bool is_v = !is_q && r >= a.k.heads;
    if (is_v) {
        r -= a.k.heads;
        w.cs = nullptr;
    }
    const moe_heads_t &s = is_q ? a.q : (is_v ? a.v : a.k);
    w.src = s.ptr;
    w.src_type = s.dtype;
    w.src_off = t * s.token_stride + r * s.head_stride;
    if (is_q || !a.cached) {
        const moe_heads_t &d = is_q ? a.q_out : a.k_out;
        w.dst_type = d.dtype;
        w.dst_off = t * d.token_stride + r * d.head_stride;
        if (live) w.dst = d.ptr;
    } else {
        const moe_kv_cache_t &c = a.cache;
        const int slot = a.slots[t];
        w.dst_type = c.dtype;
        if (slot >= 0 && live) {
            const int page = slot / c.page;
            if (page >= c.pages) {
                record_error(a.err, MOE_ERR_BAD_ID);
            } else {
                const int at = slot - page * c.page;
                w.dst = is_v ? c.v : c.k;
                w.dst_off = page * c.page_stride + at * c.token_stride + r * c.head_stride;
                if (c.dtype == MOE_E4M3)
                    w.scale = (is_v ? c.v_scale : c.k_scale) +
                              (static_cast<int64_t>(page) * c.heads + r) * c.page + at;
            }
        }
    }
    return w;
}

// A row on T threads (a power of two, T * 16 >= dim), 16 channels each in two chunks of 8: both
// halves of 8 pairs of the half layout, or 16 consecutive channels.
template <int T>
__global__ void __launch_bounds__(kThreads) rows_vec_kernel(const __grid_constant__ RowArgs a, uint32_t rows, uint32_t total) {
    pdl_wait();
    pdl_trigger();
    const int c = static_cast<int>(threadIdx.x) % T;
    const uint32_t g = blockIdx.x * (kThreads / T) + threadIdx.x / T;
    const bool on = g < total && 16 * c < a.dim;
    float x[8], y[8];
    Row w;
    w.dst = nullptr;
    w.scale = nullptr;
    w.dst_type = MOE_F32;
    int o0 = 16 * c, o1 = 16 * c + 8;
    if (on) {
        w = locate(a, g, rows);
        const bool turn = w.cs != nullptr && 16 * c < a.rot.rot;
        if (turn && !a.rot.interleaved) {
            o0 = 8 * c;
            o1 = (a.rot.rot >> 1) + 8 * c;
        }
        if (w.dst != nullptr) {
            load8(w.src, w.src_type, w.src_off + o0, x);
            load8(w.src, w.src_type, w.src_off + o1, y);
            if (turn) {
                float2 cs[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cs[i] = __ldg(w.cs + 8 * c + i);
                    if (a.rot.inverse) cs[i].y = -cs[i].y;
                }
                if (a.rot.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x[2 * i], q = x[2 * i + 1], u = y[2 * i], v = y[2 * i + 1];
                        x[2 * i] = p * cs[i].x - q * cs[i].y;
                        x[2 * i + 1] = q * cs[i].x + p * cs[i].y;
                        y[2 * i] = u * cs[i + 4].x - v * cs[i + 4].y;
                        y[2 * i + 1] = v * cs[i + 4].x + u * cs[i + 4].y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = x[i], q = y[i];
                        x[i] = p * cs[i].x - q * cs[i].y;
                        y[i] = q * cs[i].x + p * cs[i].y;
                    }
                }
            }
        }
    }
    const bool quant = w.dst != nullptr && w.dst_type == MOE_E4M3;
    if (__any_sync(0xFFFFFFFFu, quant)) {   // the row's T threads share a warp
        float mx = 0.0f;
        if (quant) {
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(x[i]), fabsf(y[i])));
        }
#pragma unroll
        for (int off = T / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        if (quant) {
            const float sc = row_scale(mx);
            if (c == 0) *w.scale = sc;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] /= sc;
                y[i] /= sc;
            }
            uint8_t *const d = static_cast<uint8_t *>(w.dst) + w.dst_off;
            *reinterpret_cast<uint2 *>(d + o0) =
                make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
            *reinterpret_cast<uint2 *>(d + o1) =
                make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
        }
    }
    if (w.dst != nullptr && !quant) {
        store8(w.dst, w.dst_type, w.dst_off + o0, x);
        store8(w.dst, w.dst_type, w.dst_off + o1, y);
    }
}

// Any dim, rot and strides: one warp per row, a channel pair (or two unrotated channels) per lane
// and step.
__global__ void __launch_bounds__(kThreads) rows_any_kernel(const __grid_constant__ RowArgs a, uint32_t rows, uint32_t total) {
    pdl_wait();
    pdl_trigger();
    const int lane = static_cast<int>(threadIdx.x & 31);
    const uint32_t g = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (g >= total) return;
    const Row w = locate(a, g, rows);
    if (w.dst == nullptr) return;
    const int half = w.cs != nullptr ? a.rot.rot >> 1 : 0;
    const int steps = half + (a.dim - 2 * half + 1) / 2;
    auto pair = [&](int i, int &o0, int &o1, float &p, float &q) {
        if (i < half) {
            o0 = a.rot.interleaved ? 2 * i : i;
            o1 = a.rot.interleaved ? 2 * i + 1 : i + half;
        } else {
            o0 = 2 * i;
            o1 = 2 * i + 1;
        }
        const float u = load1(w.src, w.src_type, w.src_off + o0);
        const float v = o1 < a.dim ? load1(w.src, w.src_type, w.src_off + o1) : 0.0f;
        p = u;
        q = v;
        if (i < half) {
            const float2 cs = __ldg(w.cs + i);
            const float s = a.rot.inverse ? -cs.y : cs.y;
            p = u * cs.x - v * s;
            q = v * cs.x + u * s;
        }
    };
    float sc = 1.0f;
    if (w.dst_type == MOE_E4M3) {
        float mx = 0.0f;
        for (int i = lane; i < steps; i += 32) {
            int o0, o1;
            float p, q;
            pair(i, o0, o1, p, q);
            mx = fmaxf(mx, fmaxf(fabsf(p), fabsf(q)));
        }
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        sc = row_scale(mx);
        if (lane == 0) *w.scale = sc;
    }
    for (int i = lane; i < steps; i += 32) {
        int o0, o1;
        float p, q;
        pair(i, o0, o1, p, q);
        if (w.dst_type == MOE_E4M3) {
            uint8_t *const d = static_cast<uint8_t *>(w.dst) + w.dst_off;
            d[o0] = f32_to_e4m3(p / sc);
            if (o1 < a.dim) d[o1] = f32_to_e4m3(q / sc);
        } else {
            store1(w.dst, w.dst_type, w.dst_off + o0, p);
            if (o1 < a.dim) store1(w.dst, w.dst_type, w.dst_off + o1, q);
        }
    }
}

// ------------------------------------------------------------------ read back
// 16 channels per thread (VEC, dim a multiple of 16 and aligned outputs) or one.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a, uint32_t per_row, uint64_t total) {
    pdl_wait();
    pdl_trigger();
    const moe_kv_cache_t &c = a.cache;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<uint64_t>(gridDim.x) * kThreads) {
        const uint64_t row = i / per_row;
        const int ch = static_cast<int>(i - row * per_row) * (VEC ? 16 : 1);
        const uint64_t th = row >> 1;
        const bool is_v = row & 1;
        const int64_t t = static_cast<int64_t>(th / c.heads);
        const int h = static_cast<int>(th - t * c.heads);
        const int slot = a.slots[t];
        int page = 0, at = 0;
        bool live = slot >= 0;
        if (live) {
            page = slot / c.page;
            at = slot - page * c.page;
            if (page >= c.pages) {
                live = false;
                record_error(a.err, MOE_ERR_BAD_ID);
            }
        }
        const void *src = is_v ? c.v : c.k;
        const int64_t so = page * c.page_stride + at * c.token_stride + h * c.head_stride + ch;
        const float sc = live && c.dtype == MOE_E4M3
                             ? (is_v ? c.v_scale : c.k_scale)[(static_cast<int64_t>(page) * c.heads + h) * c.page + at]
                             : 1.0f;
        const moe_heads_t &o = is_v ? a.v_out : a.k_out;
        const int64_t off = t * o.token_stride + h * o.head_stride + ch;
        if (VEC) {
            float x[8] = {}, y[8] = {};
            if (live) {
                if (c.dtype == MOE_E4M3) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(src) + so);
                    const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 lo = unpack_e4m3x2(static_cast<uint16_t>(wd[j] & 0xFFFFu));
                        const float2 hi = unpack_e4m3x2(static_cast<uint16_t>(wd[j] >> 16));
                        float *const d = j < 2 ? x + 4 * j : y + 4 * (j - 2);
                        d[0] = lo.x * sc;
                        d[1] = lo.y * sc;
                        d[2] = hi.x * sc;
                        d[3] = hi.y * sc;
                    }
                } else {
                    load8(src, c.dtype, so, x);
                    load8(src, c.dtype, so + 8, y);
                }
            }
            store8(o.ptr, o.dtype, off, x);
            store8(o.ptr, o.dtype, off + 8, y);
        } else {
            float v = 0.0f;
            if (live)
                v = c.dtype == MOE_E4M3 ? unpack_e4m3x2(static_cast<const uint8_t *>(src)[so]).x * sc
                                        : load1(src, c.dtype, so);
            store1(o.ptr, o.dtype, off, v);
        }
    }
}

bool vec_rows(const moe_heads_t &h) {
    const int64_t unit = h.dtype == MOE_BF16 ? 8 : 4;   // elements of 16 bytes
    return h.heads == 0 ||
           ((reinterpret_cast<uintptr_t>(h.ptr) & 15u) == 0 && h.token_stride % unit == 0 && h.head_stride % unit == 0);
}

template <typename K, typename... Args>
cudaError_t launch_flat(K kernel, unsigned grid, cudaStream_t s, bool pdl, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_rope_table(const double *w, int half, double magnitude, int positions, float *table,
                              cudaStream_t s) {
    TableFreq f = {};
    for (int i = 0; i < half; ++i) f.w[i] = w[i];
    const long long total = static_cast<long long>(positions) * half;
    const unsigned grid = static_cast<unsigned>(std::min<long long>((total + kThreads - 1) / kThreads, 152 * 16));
    rope_table_kernel<<<grid, kThreads, 0, s>>>(f, half, magnitude, positions, reinterpret_cast<float2 *>(table));
    return cudaGetLastError();
}

cudaError_t launch_rows(const RowArgs &a, cudaStream_t s, bool pdl) {
    const uint32_t rows = a.q.heads + a.k.heads + a.v.heads;
    const uint32_t total = rows * static_cast<uint32_t>(a.tokens);   // the caller keeps it below 2^31
    const bool vec = a.dim % 16 == 0 && a.rot.rot % 16 == 0 && vec_rows(a.q) && vec_rows(a.q_out) && vec_rows(a.k) &&
                     vec_rows(a.k_out) && vec_rows(a.v);
    auto grid = [&](int per) { return (total + per - 1) / per; };
    if (!vec) return launch_flat(rows_any_kernel, grid(kThreads / 32), s, pdl, a, rows, total);
    if (a.dim > 128) return launch_flat(rows_vec_kernel<16>, grid(kThreads / 16), s, pdl, a, rows, total);
    if (a.dim > 64) return launch_flat(rows_vec_kernel<8>, grid(kThreads / 8), s, pdl, a, rows, total);
    return launch_flat(rows_vec_kernel<4>, grid(kThreads / 4), s, pdl, a, rows, total);
}

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t s, bool pdl) {
    const bool vec = a.cache.dim % 16 == 0 && vec_rows(a.k_out) && vec_rows(a.v_out);
    const uint32_t per_row = vec ? a.cache.dim / 16 : a.cache.dim;
    const uint64_t total = 2ull * a.tokens * a.cache.heads * per_row;
    const unsigned grid = static_cast<unsigned>(std::min<uint64_t>((total + kThreads - 1) / kThreads, 1u << 30));
    return vec ? launch_flat(read_kernel<true>, grid, s, pdl, a, per_row, total)
               : launch_flat(read_kernel<false>, grid, s, pdl, a, per_row, total);
}

}  // namespace moe
