// tree_attn_simt.cu -- attention of drafted tokens over a paged cache on the CUDA cores, in fp32.
//
// s = scale <q, k>, out = softmax(s) v over the positions a token sees, in one pass with a running
// maximum and sum.  Serves fp32 queries, heads wider than 128 channels and layouts the
// tensor-core kernel does not take.
//
// For short contexts: the positions are not divided among CTAs, so a long one is one CTA's work for every
// 16 rows.  16 tokens of two sequences, 32 and 4 heads of 128, pages of 4: 3.1 ms over 4,000 positions;
// over 115,000 144 ms (fp32 queries the same; heads of 256 291 ms), where the same computation in
// elementary tensor operations takes 7 and the tensor-core kernel, where it serves, 0.09.
//
// A CTA takes 16 rows (token, query head of the group) of one (sequence, cache head) and walks
// the positions in tiles of 32: the tile's keys are staged in shared memory as fp32, a lane owns
// one key and forms its dot products with the warp's 4 rows, the softmax statistics go over the
// lanes, and then a lane owns every 32nd channel of the output while the tile's values stream
// from shared memory.
#include "cache_args.cuh"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kRowsWarp = 4;
constexpr int kRows = kWarps * kRowsWarp;
constexpr int kTile = 32;

__device__ __forceinline__ float ld_elem(const void *p, int dtype, int64_t off) {
    if (dtype == MOE_F32) return static_cast<const float *>(p)[off];
    if (dtype == MOE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[off]);
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(static_cast<const uint8_t *>(p)[off])));
    float r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(r) : "r"(h));
    return r;
}

// DC: 32-channel groups of the head (dim <= 32 * DC)
template <int DC>
__global__ void __launch_bounds__(kWarps * 32) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
    extern __shared__ float smem[];
    const int D = a.cache.dim, pitch = D + 1;
    float *const q_s = smem;                       // [kRows][D]
    float *const kv_s = q_s + kRows * D;           // [kTile][pitch]
    int64_t *const off_s = reinterpret_cast<int64_t *>(kv_s + ((kTile * pitch + 1) & ~1));   // [kTile]
    float *const sc_s = reinterpret_cast<float *>(off_s + kTile);                            // [2][kTile]
    pdl_wait();
    pdl_trigger();
    const moe_kv_cache_t &c = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, hk = blockIdx.y, row0 = blockIdx.x * kRows;
    const int t0 = a.q_start[b], n = a.q_start[b + 1] - t0, ctx = a.ctx[b];
    const int64_t len = static_cast<int64_t>(ctx) + n;
    if (ctx < 0 || n < 0 || n > a.max_tokens || t0 < 0 || t0 > a.tokens - n ||
        len > static_cast<int64_t>(a.max_pages) * c.page || len > kMaxPositions) {
        if (threadIdx.x == 0) record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    const int R = n * a.group;
    if (row0 >= R) return;
    for (int i = threadIdx.x; i < kRows * D; i += kWarps * 32) {
        const int r = row0 + i / D;
        q_s[i] = r < R ? ld_elem(a.q.ptr, a.q.dtype, static_cast<int64_t>(t0 + r / a.group) * a.q.token_stride +
                                                         static_cast<int64_t>(hk * a.group + r % a.group) * a.q.head_stride +
                                                         i % D)
                       : 0.0f;
    }
    uint64_t bits[kRowsWarp];
    float m[kRowsWarp], l[kRowsWarp], acc[kRowsWarp][DC];
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        const int r = row0 + warp * kRowsWarp + j;
        const int i = r / a.group;
        bits[j] = r < R ? (a.mask != nullptr ? a.mask[t0 + i] : (2ull << i) - 1ull) : 0ull;
        m[j] = -__int_as_float(0x7f800000);
        l[j] = 0.0f;
#pragma unroll
        for (int d = 0; d < DC; ++d) acc[j][d] = 0.0f;
    }
    for (int64_t p0 = 0; p0 < len; p0 += kTile) {
        __syncthreads();   // the previous tile is done with
        if (threadIdx.x < kTile) {
            const int64_t p = p0 + threadIdx.x;
            int64_t off = -1;
            float ks = 0.0f, vs = 0.0f;
            if (p < len) {
                const int at = static_cast<int>(p % c.page);
                const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p / c.page];
                if (static_cast<uint32_t>(page) < static_cast<uint32_t>(c.pages)) {
                    off = page * c.page_stride + at * c.token_stride + hk * c.head_stride;
                    ks = vs = 1.0f;
                    if (c.dtype == MOE_E4M3) {
                        const int64_t so = (static_cast<int64_t>(page) * c.heads + hk) * c.page + at;
                        ks = c.k_scale[so];
                        vs = c.v_scale[so];
                    }
                } else {
                    record_error(a.err, MOE_ERR_BAD_ID);
                }
            }
            off_s[threadIdx.x] = off;
            sc_s[threadIdx.x] = ks;
            sc_s[kTile + threadIdx.x] = vs;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * D; i += kWarps * 32) {
            const int j = i / D, d = i - j * D;
            kv_s[j * pitch + d] = off_s[j] >= 0 ? ld_elem(c.k, c.dtype, off_s[j] + d) * sc_s[j] : 0.0f;
        }
        __syncthreads();
        float p[kRowsWarp];
#pragma unroll
        for (int j = 0; j < kRowsWarp; ++j) p[j] = 0.0f;
        for (int d = 0; d < D; ++d) {
            const float k = kv_s[lane * pitch + d];
#pragma unroll
            for (int j = 0; j < kRowsWarp; ++j) p[j] = fmaf(q_s[(warp * kRowsWarp + j) * D + d], k, p[j]);
        }
        uint32_t seen[kRowsWarp];
        const int64_t pos = p0 + lane;
#pragma unroll
        for (int j = 0; j < kRowsWarp; ++j) {
            const int64_t d = pos - ctx;
            const bool see = pos < len && (d < 0 || ((bits[j] >> (d & 63)) & 1ull)) && row0 + warp * kRowsWarp + j < R;
            seen[j] = __ballot_sync(0xFFFFFFFFu, see);
            const float s = see ? p[j] * a.scale_log2 : -__int_as_float(0x7f800000);
            float mx = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = fmaxf(m[j], mx);
            const float ref = mn == -__int_as_float(0x7f800000) ? 0.0f : mn;   // nothing seen yet
            const float keep = exp2f(m[j] - ref);
            m[j] = mn;
            p[j] = see ? exp2f(s - ref) : 0.0f;
            float sum = p[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            l[j] = l[j] * keep + sum;
#pragma unroll
            for (int d2 = 0; d2 < DC; ++d2) acc[j][d2] *= keep;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * D; i += kWarps * 32) {
            const int j = i / D, d = i - j * D;
            kv_s[j * pitch + d] = off_s[j] >= 0 ? ld_elem(c.v, c.dtype, off_s[j] + d) * sc_s[kTile + j] : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kTile; ++k) {
            float v[DC];
#pragma unroll
            for (int d = 0; d < DC; ++d) v[d] = d * 32 + lane < D ? kv_s[k * pitch + d * 32 + lane] : 0.0f;
#pragma unroll
            for (int j = 0; j < kRowsWarp; ++j) {
                const float w = __shfl_sync(0xFFFFFFFFu, p[j], k);
                if ((seen[j] >> k) & 1u) {   // warp-uniform: an unseen value is not touched
#pragma unroll
                    for (int d = 0; d < DC; ++d) acc[j][d] = fmaf(w, v[d], acc[j][d]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        const int r = row0 + warp * kRowsWarp + j;
        if (r >= R) continue;
        const int t = t0 + r / a.group, h = hk * a.group + r % a.group;
        const bool none = m[j] == -__int_as_float(0x7f800000) && l[j] == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l[j];
        const int64_t off = static_cast<int64_t>(t) * a.out.token_stride + static_cast<int64_t>(h) * a.out.head_stride;
#pragma unroll
        for (int d = 0; d < DC; ++d) {
            const int ch = d * 32 + lane;
            if (ch >= D) continue;
            const float v = acc[j][d] * inv;
            if (a.out.dtype == MOE_BF16)
                static_cast<__nv_bfloat16 *>(a.out.ptr)[off + ch] = __float2bfloat16_rn(v);
            else
                static_cast<float *>(a.out.ptr)[off + ch] = v;
        }
        if (a.lse != nullptr && lane == 0)
            a.lse[static_cast<int64_t>(t) * a.q.heads + h] =
                none ? -__int_as_float(0x7f800000) : (m[j] + log2f(l[j])) * 0.69314718055994531f;
    }
}

constexpr size_t smem_bytes(int D) {
    return (kRows * D + ((kTile * (D + 1) + 1) & ~1)) * sizeof(float) + kTile * sizeof(int64_t) + 2 * kTile * sizeof(float);
}

template <int DC>
cudaError_t launch(const TreeArgs &a, dim3 grid, cudaStream_t s, bool pdl) {
    const size_t smem = smem_bytes(a.cache.dim);
    // always what the widest head needs: the limit is the function's, and a smaller one, set for this
    // call, could come between another thread's setting and its launch
    cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<DC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes(32 * DC)));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_simt_kernel<DC>, a);
}

}  // namespace

cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t s, bool pdl) {
    const dim3 grid((a.max_tokens * a.group + kRows - 1) / kRows, a.cache.heads, a.seqs);
    if (a.cache.dim <= 64) return launch<2>(a, grid, s, pdl);
    if (a.cache.dim <= 128) return launch<4>(a, grid, s, pdl);
    return launch<8>(a, grid, s, pdl);
}

}  // namespace moe
