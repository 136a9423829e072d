// rope_kv.cu -- rotary positions and the rows of a paged key/value cache: rotation of the pass's
// queries and keys, the (quantising) write of its keys and values, and the read back.
//
// A row is one head of one token, `dim` channels.  Rotation multiplies each channel pair (a, b)
// by [[c, -s], [s, c]] with c = m cos(p w_i), s = m sin(p w_i) from a table (its transpose for
// gradients).  A quantised row is codes of x / scale with scale = amax / 448.  All of it is
// streaming work, a few operations per element: the bound is memory traffic, each row read once
// and written once.
//
// Rows of 128 channels, against the copy bandwidth of 6.79 TB/s: 16381 tokens x 40 rows of bf16
// rotated 56.4 us (6.02 TB/s), 16300 x 16 rows written as e4m3 codes 20.7 us (4.89), 8190 x 40
// rows rotated and 8 of them written 30.1 us (5.72), 131000 x 16 rows of codes read back as bf16
// 129 us (6.29); a pass of a few tokens 2.3 to 3.1 us, the latency of its chain of loads (position
// or slot, then table row, then channels).  fp32 rows, whose kernels spill 60-150 bytes a thread under
// launch bounds chosen for narrower ones: 16381 x 40 rotated 110 us (6.12), 131000 x 8 rows of 128
// written to an fp32 cache 176 us (6.11) and read back 204 us (5.27).
#include "cache_args.cuh"
#include "common.cuh"
#include "row_common.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = kRowThreads;

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

// x / s, correctly rounded, from r = 1 / s rounded to nearest: q = x r, and one step with the exact
// remainder x - q s (Markstein's theorem, IBM J. Res. Dev. 34 (1990)): three operations where a
// division takes a dozen.  s within 2^+-100, so that neither r nor the remainder leaves the range
// that matters (a quotient below 2^-11 is code 0 whatever its last bit).
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}
// The same for two numbers at a time, in packed operations.  The remainder, which is exact, is formed
// rounding down so that a remainder of zero is -0 (rounding to nearest makes it +0): added to a
// quotient of zero it leaves its sign, and the codes of -0 and of +0 differ.
__device__ __forceinline__ void quotient2(float &x0, float &x1, uint64_t s_neg, uint64_t r) {
    uint64_t x, q, e;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(s_neg), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(r), "l"(q));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(q));
}

// amax / 448, or 1 where that is 0 (a zero row, or one below the smallest scale)
__device__ __forceinline__ float row_scale(float amax) {
    // (an infinite amax: the remainder would be NaN)
    const float s = amax > 7.888609e-31f && amax < 3.4028235e38f ? quotient(amax, 448.0f, 1.0f / 448.0f) : amax / 448.0f;
    return s > 0.0f ? s : 1.0f;
}
// The chunk's eight codes for scale s.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
    float q[8];
    if (s >= 7.888609e-31f && s <= 1.2676506e30f) {
        const float r = __frcp_rn(s);
        uint64_t r2, s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(r2) : "f"(r));
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(-s));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            q[i] = x[i];
            q[i + 1] = x[i + 1];
            quotient2(q[i], q[i + 1], s2, r2);
        }
    } else {   // also infinite and NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = x[i] / s;
    }
    return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
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

// The streaming kernels take a token's rows together, because a row alone costs more instructions
// for finding its place than for its channels (16381 tokens x 40 heads of 128: 76 us with a row per
// thread group and all of its address arithmetic, 96 us with two): `share` groups of T threads (a
// power of two, T * 16 >= dim) share a token, find its position, table row and cache slot once, and
// step through its heads by pointer.  A thread holds 16 channels of a row, in two chunks of 8: both
// halves of 8 pairs of the half layout, or 16 consecutive channels; the token's 8 cosines and sines
// stay in its registers, and the next row's loads are on their way while it works on one.

// Sixteen bf16 channels in one store of 32 bytes where the address allows it: two of 16 bytes write
// every sector in halves (8190 tokens x 40 rows rotated and written: 31.1 us against 30.4).
__device__ __forceinline__ bool at32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
template <int TYPE>   // two chunks of eight channels, o1 apart
__device__ __forceinline__ void store16(void *base, int64_t off, int o1, const float (&x)[8], const float (&y)[8]) {
    if constexpr (TYPE == MOE_BF16) {
        const uint4 a = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        const uint4 b = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        uint16_t *const p = static_cast<uint16_t *>(base) + off;
        if (o1 == 8 && at32(p)) {
            store32(p, a, b);
        } else {
            *reinterpret_cast<uint4 *>(p) = a;
            *reinterpret_cast<uint4 *>(p + o1) = b;
        }
    } else {
        store8(base, TYPE, off, x);
        store8(base, TYPE, off + o1, y);
    }
}

// 16 channels as they come from memory
template <typename E>
struct Raw {
    uint4 v[sizeof(E)];   // 2 bytes: two chunks of 16; 4 bytes: two of 32
};
template <typename E>
__device__ __forceinline__ void load_raw(const E *p, int o1, Raw<E> &r) {
    if constexpr (sizeof(E) == 2) {
        r.v[0] = *reinterpret_cast<const uint4 *>(p);
        r.v[1] = *reinterpret_cast<const uint4 *>(p + o1);
    } else {
        r.v[0] = *reinterpret_cast<const uint4 *>(p);
        r.v[1] = *reinterpret_cast<const uint4 *>(p + 4);
        r.v[2] = *reinterpret_cast<const uint4 *>(p + o1);
        r.v[3] = *reinterpret_cast<const uint4 *>(p + o1 + 4);
    }
}
template <typename E>
__device__ __forceinline__ void from_raw(const Raw<E> &r, float (&x)[8], float (&y)[8]) {
    if constexpr (sizeof(E) == 2) {
        const uint32_t a[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w}, b[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(a[i]);
            x[2 * i + 1] = bf16_hi(a[i]);
            y[2 * i] = bf16_lo(b[i]);
            y[2 * i + 1] = bf16_hi(b[i]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 a = r.v[h], b = r.v[2 + h];
            x[4 * h] = __uint_as_float(a.x);
            x[4 * h + 1] = __uint_as_float(a.y);
            x[4 * h + 2] = __uint_as_float(a.z);
            x[4 * h + 3] = __uint_as_float(a.w);
            y[4 * h] = __uint_as_float(b.x);
            y[4 * h + 1] = __uint_as_float(b.y);
            y[4 * h + 2] = __uint_as_float(b.z);
            y[4 * h + 3] = __uint_as_float(b.w);
        }
    }
}

// One rotation of the thread's pairs.  cs: 8 (cos, sin); a thread with unrotated channels holds
// (1, 0) there and skips nothing: x * 1 - y * 0 would turn an infinity into NaN, so `turn` decides.
__device__ __forceinline__ void turn16(float (&x)[8], float (&y)[8], const float (&cs)[16], bool adjacent) {
    if (adjacent) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn_pair(x[2 * i], x[2 * i + 1], cs[2 * i], cs[2 * i + 1]);
            turn_pair(y[2 * i], y[2 * i + 1], cs[8 + 2 * i], cs[8 + 2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[i], y[i], cs[2 * i], cs[2 * i + 1]);
    }
}

// IN: the rows' type, also of dense outputs.  CT: the cache's type, or -1 for no cache.  ROT: with
// rotation.  At least four CTAs an SM: what is in flight covers the memory's latency.
template <typename IN, int CT, int T, bool ROT>
__global__ void __launch_bounds__(kThreads, 4) rows_vec_kernel(const __grid_constant__ RowArgs a, int share) {
    constexpr int kInType = sizeof(IN) == 2 ? MOE_BF16 : MOE_F32;
    pdl_wait();
    pdl_trigger();
    const int c = static_cast<int>(threadIdx.x) % T, group = static_cast<int>(threadIdx.x) / T, sub = group % share;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / T / share) + group / share;
    const bool here = t < a.tokens && 16 * c < a.dim;
    float cs[16];
    bool turn = false, live = here;
    int o0 = 16 * c, o1 = 8;   // first chunk, and the second's distance from it
    if (ROT && here) {
        const int p = __ldg(a.rot.positions + t);
        live = static_cast<uint32_t>(p) < static_cast<uint32_t>(a.rot.table_positions);
        if (!live) {
            record_error(a.err, MOE_ERR_BAD_ID);
        } else if (16 * c < a.rot.rot) {
            turn = true;
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
    }
    const bool split = ROT && 16 * c < a.rot.rot && !a.rot.interleaved;
    const int q0 = split ? 8 * c : o0, q1 = split ? a.rot.rot >> 1 : o1;   // chunks of rotated rows

    // dense rows: q, and k where there is no cache
    const int dense = a.q.heads + (CT < 0 ? a.k.heads : 0);
    if (live && sub < dense) {
        auto src = [&](int r) {
            const bool q = CT >= 0 || r < a.q.heads;
            const moe_heads_t &h = q ? a.q : a.k;
            return static_cast<const IN *>(h.ptr) + t * h.token_stride + (q ? r : r - a.q.heads) * h.head_stride + q0;
        };
        Raw<IN> next;
        load_raw(src(sub), q1, next);
        for (int r = sub; r < dense; r += share) {
            float x[8], y[8];
            from_raw(next, x, y);
            if (r + share < dense) load_raw(src(r + share), q1, next);
            if (ROT && turn) turn16(x, y, cs, a.rot.interleaved);
            const bool q = CT >= 0 || r < a.q.heads;
            const moe_heads_t &h = q ? a.q_out : a.k_out;
            const int64_t off = t * h.token_stride + (q ? r : r - a.q.heads) * h.head_stride + q0;
            store16<kInType>(h.ptr, off, q1, x, y);
        }
    }
    if constexpr (CT >= 0) {
        // cache rows: k (rotated), then v
        const moe_kv_cache_t &kc = a.cache;
        const int n = 2 * kc.heads;
        const int slot = live ? __ldg(a.slots + t) : -1;
        auto src = [&](int r) {
            const bool k = r < kc.heads;
            const moe_heads_t &h = k ? a.k : a.v;
            return static_cast<const IN *>(h.ptr) + t * h.token_stride + (k ? r : r - kc.heads) * h.head_stride + (k ? q0 : o0);
        };
        Raw<IN> next;
        if (live && sub < n) load_raw(src(sub), sub < kc.heads ? q1 : o1, next);   // beside the slot's load
        int64_t at = -1, sc_at = 0;
        if (slot >= 0) {
            const int page = slot / kc.page, row = slot - page * kc.page;
            if (page >= kc.pages) {
                record_error(a.err, MOE_ERR_BAD_ID);
            } else {
                at = page * kc.page_stride + row * kc.token_stride;
                sc_at = static_cast<int64_t>(page) * kc.heads * kc.page + row;
            }
        }
        // every group of a warp takes the same number of turns: the lanes of a row meet in shuffles
        for (int r = sub; r - sub < n; r += share) {
            const bool on = at >= 0 && r < n, k = r < kc.heads;
            float x[8] = {}, y[8] = {};
            if (on) {
                from_raw(next, x, y);
                if (r + share < n) load_raw(src(r + share), r + share < kc.heads ? q1 : o1, next);
                if (ROT && turn && k) turn16(x, y, cs, a.rot.interleaved);
            }
            const int h = k ? r : r - kc.heads, d0 = k ? q0 : o0, d1 = k ? q1 : o1;
            const int64_t off = at + h * kc.head_stride + d0;
            if constexpr (CT == MOE_E4M3) {
                float mx = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
                for (int o = T / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                if (on) {
                    const float sc = row_scale(mx);
                    if (c == 0) (k ? kc.k_scale : kc.v_scale)[sc_at + static_cast<int64_t>(h) * kc.page] = sc;
                    uint8_t *const d = static_cast<uint8_t *>(k ? kc.k : kc.v) + off;
                    const uint2 lo = codes8(x, sc), hi = codes8(y, sc);
                    if (d1 == 8) {
                        *reinterpret_cast<uint4 *>(d) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    } else {
                        *reinterpret_cast<uint2 *>(d) = lo;
                        *reinterpret_cast<uint2 *>(d + d1) = hi;
                    }
                }
            } else if (on) {
                store8(k ? kc.k : kc.v, CT, off, x);
                store8(k ? kc.k : kc.v, CT, off + d1, y);
            }
        }
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
        p = load1(w.src, w.src_type, w.src_off + o0);
        q = o1 < a.dim ? load1(w.src, w.src_type, w.src_off + o1) : 0.0f;
        if (i < half) {
            const float2 cs = __ldg(w.cs + i);
            turn_pair(p, q, cs.x, a.rot.inverse ? -cs.y : cs.y);
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
// Row r of the read: token r / (2 heads), then head, keys before values.
struct Back {
    const void *src;   // null: zeros
    int64_t src_off, dst_off;
    float scale;
    bool is_v;
};
__device__ __forceinline__ Back locate_back(const ReadArgs &a, uint32_t r) {
    const moe_kv_cache_t &c = a.cache;
    const uint32_t th = r >> 1;
    const int64_t t = th / static_cast<uint32_t>(c.heads);
    const int h = static_cast<int>(th - static_cast<uint32_t>(t) * c.heads);
    Back w;
    w.is_v = r & 1u;
    w.src = nullptr;
    w.src_off = 0;
    w.scale = 1.0f;
    const moe_heads_t &o = w.is_v ? a.v_out : a.k_out;
    w.dst_off = t * o.token_stride + h * o.head_stride;
    const int slot = __ldg(a.slots + t);
    if (slot < 0) return w;
    const int page = slot / c.page, at = slot - page * c.page;
    if (page >= c.pages) {
        record_error(a.err, MOE_ERR_BAD_ID);
        return w;
    }
    w.src = w.is_v ? c.v : c.k;
    w.src_off = page * c.page_stride + at * c.token_stride + h * c.head_stride;
    if (c.dtype == MOE_E4M3) w.scale = __ldg((w.is_v ? c.v_scale : c.k_scale) + (static_cast<int64_t>(page) * c.heads + h) * c.page + at);
    return w;
}

// Tokens shared as by the rows above: the slot is found once, the heads are stepped through, the
// next row's loads on their way.  Six CTAs an SM: 131000 tokens x 16 rows of e4m3 to bf16 take 128.5 us
// (6.3 TB/s), with five (what its registers left) 135.3, with eight, which spill, 131.4.
template <int CT, typename OUT, int T>
__global__ void __launch_bounds__(kThreads, 6) read_vec_kernel(const __grid_constant__ ReadArgs a, int share) {
    constexpr int kOutType = sizeof(OUT) == 2 ? MOE_BF16 : MOE_F32;
    pdl_wait();
    pdl_trigger();
    const moe_kv_cache_t &kc = a.cache;
    const int ch = static_cast<int>(threadIdx.x) % T * 16, group = static_cast<int>(threadIdx.x) / T, sub = group % share;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / T / share) + group / share;
    if (t >= a.tokens || ch >= kc.dim) return;
    const int slot = __ldg(a.slots + t);
    int64_t at = -1, sc_at = 0;
    if (slot >= 0) {
        const int page = slot / kc.page, row = slot - page * kc.page;
        if (page >= kc.pages) {
            record_error(a.err, MOE_ERR_BAD_ID);
        } else {
            at = page * kc.page_stride + row * kc.token_stride + ch;
            sc_at = static_cast<int64_t>(page) * kc.heads * kc.page + row;
        }
    }
    using E = typename std::conditional<CT == MOE_F32, float, uint16_t>::type;   // of a cache that is not codes
    struct Next {
        uint4 q;
        float scale;
        Raw<E> raw;
    } next;
    auto fetch = [&](int r) {
        const bool k = r < kc.heads;
        const int h = k ? r : r - kc.heads;
        const int64_t off = at + h * kc.head_stride;
        if constexpr (CT == MOE_E4M3) {
            next.q = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(k ? kc.k : kc.v) + off);
            next.scale = __ldg((k ? kc.k_scale : kc.v_scale) + sc_at + static_cast<int64_t>(h) * kc.page);
        } else {
            load_raw(static_cast<const E *>(k ? kc.k : kc.v) + off, 8, next.raw);
        }
    };
    const int n = 2 * kc.heads;
    if (at >= 0 && sub < n) fetch(sub);
    for (int r = sub; r < n; r += share) {
        float x[8] = {}, y[8] = {};
        if (at >= 0) {
            if constexpr (CT == MOE_E4M3) {
                const uint32_t wd[4] = {next.q.x, next.q.y, next.q.z, next.q.w};
                const float sc = next.scale;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 lo = unpack_e4m3x2(static_cast<uint16_t>(wd[j] & 0xFFFFu));
                    const float2 hi = unpack_e4m3x2(static_cast<uint16_t>(wd[j] >> 16));
                    float(&d)[8] = j < 2 ? x : y;
                    d[4 * (j & 1)] = lo.x * sc;
                    d[4 * (j & 1) + 1] = lo.y * sc;
                    d[4 * (j & 1) + 2] = hi.x * sc;
                    d[4 * (j & 1) + 3] = hi.y * sc;
                }
            } else {
                from_raw(next.raw, x, y);
            }
            if (r + share < n) fetch(r + share);
        }
        const bool k = r < kc.heads;
        const moe_heads_t &o = k ? a.k_out : a.v_out;
        const int64_t off = t * o.token_stride + (k ? r : r - kc.heads) * o.head_stride + ch;
        store16<kOutType>(o.ptr, off, 8, x, y);
    }
}

// Any dim and output strides: a warp per row.
__global__ void __launch_bounds__(kThreads) read_any_kernel(const __grid_constant__ ReadArgs a, uint32_t total) {
    pdl_wait();
    pdl_trigger();
    const uint32_t r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= total) return;
    const Back w = locate_back(a, r);
    const moe_heads_t &o = w.is_v ? a.v_out : a.k_out;
    for (int ch = static_cast<int>(threadIdx.x & 31); ch < a.cache.dim; ch += 32) {
        float v = 0.0f;
        if (w.src != nullptr)
            v = a.cache.dtype == MOE_E4M3 ? unpack_e4m3x2(static_cast<const uint8_t *>(w.src)[w.src_off + ch]).x * w.scale
                                          : load1(w.src, a.cache.dtype, w.src_off + ch);
        store1(o.ptr, o.dtype, w.dst_off + ch, v);
    }
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

namespace {

// Groups of threads that share a token: one token to a CTA while that leaves SMs free, so that a
// short call is short; else so few that a group has eight rows to step through, since a CTA's first
// row waits for its slot, its table row and its channels in turn.  (Eight groups whatever the rows:
// 16300 tokens x 16 rows of 128, bf16 to e4m3, 23.1 us against 20.7; 131000 x 16 read back 150.9
// against 136.2; 8190 x 40 rotated and written 33.0 against 30.8.)
int share_of(int groups, int64_t tokens, int rows) {
    int share = groups;
    while (share > 1 && rows < 8 * share && tokens * share > 152ll * groups * 4) share /= 2;
    while (share > 1 && share / 2 >= rows) share /= 2;
    return share;
}

template <typename IN, int CT, int T>
cudaError_t launch_vec(const RowArgs &a, int rows, cudaStream_t s, bool pdl) {
    const int share = share_of(kThreads / T, a.tokens, rows), per = kThreads / T / share;
    const unsigned grid = static_cast<unsigned>((a.tokens + per - 1) / per);
    if constexpr (CT >= 0)
        if (a.rot.rot == 0) return launch_flat(rows_vec_kernel<IN, CT, T, false>, grid, s, pdl, a, share);
    return launch_flat(rows_vec_kernel<IN, CT, T, true>, grid, s, pdl, a, share);
}
template <typename IN, int CT>
cudaError_t by_dim(const RowArgs &a, int rows, cudaStream_t s, bool pdl) {
    if (a.dim > 128) return launch_vec<IN, CT, 16>(a, rows, s, pdl);
    return a.dim > 64 ? launch_vec<IN, CT, 8>(a, rows, s, pdl) : launch_vec<IN, CT, 4>(a, rows, s, pdl);
}
template <typename IN>
cudaError_t by_cache(const RowArgs &a, int rows, cudaStream_t s, bool pdl) {
    if (!a.cached) return by_dim<IN, -1>(a, rows, s, pdl);
    if (a.cache.dtype == MOE_E4M3) return by_dim<IN, MOE_E4M3>(a, rows, s, pdl);
    return a.cache.dtype == MOE_BF16 ? by_dim<IN, MOE_BF16>(a, rows, s, pdl) : by_dim<IN, MOE_F32>(a, rows, s, pdl);
}

template <int CT, typename OUT, int T>
cudaError_t launch_read(const ReadArgs &a, cudaStream_t s, bool pdl) {
    const int share = share_of(kThreads / T, a.tokens, 2 * a.cache.heads), per = kThreads / T / share;
    return launch_flat(read_vec_kernel<CT, OUT, T>, static_cast<unsigned>((a.tokens + per - 1) / per), s, pdl, a, share);
}
template <int CT, typename OUT>
cudaError_t read_by_dim(const ReadArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.dim > 128) return launch_read<CT, OUT, 16>(a, s, pdl);
    return a.cache.dim > 64 ? launch_read<CT, OUT, 8>(a, s, pdl) : launch_read<CT, OUT, 4>(a, s, pdl);
}
template <typename OUT>
cudaError_t read_by_cache(const ReadArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.dtype == MOE_E4M3) return read_by_dim<MOE_E4M3, OUT>(a, s, pdl);
    return a.cache.dtype == MOE_BF16 ? read_by_dim<MOE_BF16, OUT>(a, s, pdl) : read_by_dim<MOE_F32, OUT>(a, s, pdl);
}

}  // namespace

cudaError_t launch_rows(const RowArgs &a, cudaStream_t s, bool pdl) {
    const uint32_t rows = a.q.heads + a.k.heads + a.v.heads;
    const uint32_t total = rows * static_cast<uint32_t>(a.tokens);   // the caller keeps it below 2^31
    // the streaming kernel: 16-byte pieces, one type of rows (an absent q has type 0 = fp32, and no say)
    const int type = a.k.heads > 0 ? a.k.dtype : a.q.dtype;
    auto same = [&](const moe_heads_t &h) { return h.heads == 0 || h.dtype == type; };
    const bool vec = a.dim % 16 == 0 && a.rot.rot % 16 == 0 && (reinterpret_cast<uintptr_t>(a.rot.table) & 15u) == 0 &&
                     vec_rows(a.q) && vec_rows(a.q_out) && vec_rows(a.k) && vec_rows(a.k_out) && vec_rows(a.v) &&
                     same(a.q) && same(a.q_out) && same(a.k) && same(a.k_out) && same(a.v);
    if (!vec) return launch_flat(rows_any_kernel, (total + kThreads / 32 - 1) / (kThreads / 32), s, pdl, a, rows, total);
    return type == MOE_BF16 ? by_cache<uint16_t>(a, static_cast<int>(rows), s, pdl) : by_cache<float>(a, static_cast<int>(rows), s, pdl);
}

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.dim % 16 != 0 || !vec_rows(a.k_out) || !vec_rows(a.v_out) || a.k_out.dtype != a.v_out.dtype) {
        const uint32_t total = 2u * static_cast<uint32_t>(a.tokens) * static_cast<uint32_t>(a.cache.heads);   // below 2^31
        return launch_flat(read_any_kernel, (total + kThreads / 32 - 1) / (kThreads / 32), s, pdl, a, total);
    }
    return a.k_out.dtype == MOE_BF16 ? read_by_cache<uint16_t>(a, s, pdl) : read_by_cache<float>(a, s, pdl);
}

}  // namespace moe
