// latent_simt.cu -- latent attention on the CUDA cores, in fp32: fp32 rows and the layouts that the
// tensor-core kernel does not take, for short contexts (the positions are not divided among CTAs).
//
// s = scale <q, row>, out = softmax(s) latent over the positions a token sees, in one pass with a
// running maximum and sum.  A CTA takes 16 rows (token, head) of one sequence and walks the positions in
// tiles of 32, staged in shared memory as fp32 once for scores and outputs: a lane owns one position and
// forms its dot products with the warp's 4 rows, then every 32nd channel of the outputs.
#include "cache_args.cuh"
#include "common.cuh"
#include "latent_args.cuh"
#include "row_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kRowsWarp = 4;
constexpr int kRows = kWarps * kRowsWarp;
constexpr int kTile = 32;

// DC: 32-channel groups of the latent (rank <= 32 * DC)
template <int DC>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_kernel(const __grid_constant__ LatentArgs a) {
    extern __shared__ float smem[];
    const moe_latent_cache_t &c = a.cache;
    const int D = c.rank + c.rope, pitch = D + 1;
    float *const q_s = smem;                       // [kRows][D]
    float *const kv_s = q_s + kRows * D;           // [kTile][pitch]
    int64_t *const off_s = reinterpret_cast<int64_t *>(kv_s + ((kTile * pitch + 1) & ~1));   // [kTile]
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, row0 = blockIdx.x * kRows;
    const int t0 = a.q_start[b], n = a.q_start[b + 1] - t0, ctx = a.ctx[b];
    const int64_t len = static_cast<int64_t>(ctx) + n;
    if (ctx < 0 || n < 0 || n > a.max_tokens || t0 < 0 || t0 > a.tokens - n ||
        len > static_cast<int64_t>(a.max_pages) * c.page || len > kMaxPositions) {
        if (threadIdx.x == 0) record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    const int R = n * a.heads;
    if (row0 >= R) return;
    for (int i = threadIdx.x; i < kRows * D; i += kWarps * 32) {
        const int r = row0 + i / D;
        q_s[i] = r < R ? load1(a.q.ptr, a.q.dtype, static_cast<int64_t>(t0 + r / a.heads) * a.q.token_stride +
                                                       static_cast<int64_t>(r % a.heads) * a.q.head_stride + i % D)
                       : 0.0f;
    }
    uint64_t bits[kRowsWarp];
    float m[kRowsWarp], l[kRowsWarp], acc[kRowsWarp][DC];
    const float none = -__int_as_float(0x7f800000);
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        const int r = row0 + warp * kRowsWarp + j, i = r / a.heads;
        bits[j] = r < R ? (a.mask != nullptr ? a.mask[t0 + i] : (2ull << i) - 1ull) : 0ull;
        m[j] = none;
        l[j] = 0.0f;
#pragma unroll
        for (int d = 0; d < DC; ++d) acc[j][d] = 0.0f;
    }
    for (int64_t p0 = 0; p0 < len; p0 += kTile) {
        __syncthreads();   // the previous tile is done with
        if (threadIdx.x < kTile) {
            const int64_t p = p0 + threadIdx.x;
            int64_t off = -1;
            if (p < len) {
                const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p / c.page];
                if (static_cast<uint32_t>(page) < static_cast<uint32_t>(c.pages))
                    off = page * c.page_stride + (p % c.page) * c.token_stride;
                else
                    record_error(a.err, MOE_ERR_BAD_ID);
            }
            off_s[threadIdx.x] = off;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * D; i += kWarps * 32) {
            const int j = i / D, d = i - j * D;
            kv_s[j * pitch + d] = off_s[j] >= 0 ? load1(c.rows, c.dtype, off_s[j] + d) : 0.0f;
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
            const float s = see ? p[j] * a.scale_log2 : none;
            float mx = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = fmaxf(m[j], mx);
            const float ref = mn == none ? 0.0f : mn;   // nothing seen yet
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
        for (int k = 0; k < kTile; ++k) {
            float v[DC];
#pragma unroll
            for (int d = 0; d < DC; ++d) v[d] = d * 32 + lane < c.rank ? kv_s[k * pitch + d * 32 + lane] : 0.0f;
#pragma unroll
            for (int j = 0; j < kRowsWarp; ++j) {
                const float w = __shfl_sync(0xFFFFFFFFu, p[j], k);
                if ((seen[j] >> k) & 1u) {   // warp-uniform: an unseen latent is not touched
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
        const int t = t0 + r / a.heads, h = r % a.heads;
        const bool empty = m[j] == none && l[j] == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / l[j];
        const int64_t off = static_cast<int64_t>(t) * a.out.token_stride + static_cast<int64_t>(h) * a.out.head_stride;
#pragma unroll
        for (int d = 0; d < DC; ++d)
            if (d * 32 + lane < c.rank) store1(a.out.ptr, a.out.dtype, off + d * 32 + lane, acc[j][d] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[static_cast<int64_t>(t) * a.heads + h] = empty ? none : (m[j] + log2f(l[j])) * 0.69314718055994531f;
    }
}

constexpr size_t smem_bytes(int D) {
    return (kRows * D + ((kTile * (D + 1) + 1) & ~1)) * sizeof(float) + kTile * sizeof(int64_t);
}
constexpr int kMaxRope = 128;

template <int DC>
cudaError_t launch(const LatentArgs &a, cudaStream_t s, bool pdl) {
    // always what the widest row needs: the limit is the function's, and a smaller one, set for this
    // call, could come between another thread's setting and its launch
    constexpr size_t most = smem_bytes(32 * DC + kMaxRope);
    static_assert(most <= 232448, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(latent_simt_kernel<DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.max_tokens * a.heads + kRows - 1) / kRows, a.seqs);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem_bytes(a.cache.rank + a.cache.rope);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_simt_kernel<DC>, a);
}

}  // namespace

cudaError_t launch_latent_simt(const LatentArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.rank <= 128) return launch<4>(a, s, pdl);
    return a.cache.rank <= 256 ? launch<8>(a, s, pdl) : launch<16>(a, s, pdl);
}

}  // namespace moe
