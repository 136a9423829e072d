// latent_simt.cu -- latent attention on the CUDA cores, in fp32: fp32 rows and the layouts that the
// tensor-core kernel does not take.
//
// s = scale <q, row>, out = softmax(s) latent over the positions a token sees, in one pass with a
// running maximum and sum.  A CTA takes 16 rows (token, head) of one sequence and walks a part of the positions
// in tiles of 32, staged in shared memory as fp32 once for scores and outputs: a lane owns one position and
// forms its dot products with the warp's 4 rows, four channels at a time, then every 32nd channel of the
// outputs.  Few rows: the positions are divided among CTAs, whose parts (unnormalised output, maximum,
// sum) a second kernel joins in order.
//
// Bound: shared-memory reads, 8 wavefronts for every 16 products' instructions of a score; two CTAs an SM, so
// that one's tile arrives while the other's is worked on.  fp32, 16 tokens, 16 heads of rank 512 and 64 rotary
// channels: 172 us over 300 positions, 291 over 4,000 and 3.5 ms over 100,000 (1.2 ms as products of a
// library's fp32 matrices; undivided, with a channel at a time, 5.3 and 216 ms).
#include <algorithm>

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
constexpr int kParts = 608;       // CTAs that a call of few rows is divided among, at most

__device__ __forceinline__ float none() { return -__int_as_float(0x7f800000); }
// Words from one row to the next: four more than a multiple of 32, so that eight lanes' 16 bytes of
// neighbouring rows meet all banks.
__host__ __device__ constexpr int pitch_of(int D) { return (D + 31) / 32 * 32 + 4; }

// Parts: [seqs][blocks of kRows][divisions] of kRows rows of rank fp32, then as many of kRows (maximum, sum).
__device__ __forceinline__ int64_t part_of(const LatentArgs &a, int b, int blocks, int block, int z) {
    return (static_cast<int64_t>(b) * blocks + block) * a.divisions + z;
}
__device__ __forceinline__ float2 *sums_of(const LatentArgs &a, int blocks) {
    return reinterpret_cast<float2 *>(static_cast<float *>(a.part) + static_cast<int64_t>(a.seqs) * blocks * a.divisions * kRows * a.cache.rank);
}

__device__ __forceinline__ bool lengths(const LatentArgs &a, int b, int &t0, int &n, int &ctx, int64_t &len) {
    t0 = a.q_start[b];
    const long long tokens = static_cast<long long>(a.q_start[b + 1]) - t0;
    ctx = a.ctx[b];
    len = ctx + tokens;
    n = static_cast<int>(tokens);
    return !(ctx < 0 || tokens < 0 || tokens > a.max_tokens || t0 < 0 || t0 > a.tokens - tokens ||
             len > static_cast<int64_t>(a.max_pages) * a.cache.page || len > kMaxPositions);
}

// DC: 32-channel groups of the latent (rank <= 32 * DC)
template <int DC>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_kernel(const __grid_constant__ LatentArgs a) {
    extern __shared__ __align__(16) float smem[];
    const moe_latent_cache_t &c = a.cache;
    const int D = c.rank + c.rope, pitch = pitch_of(D);
    float *const q_s = smem;                       // [kRows][pitch]
    float *const kv_s = q_s + kRows * pitch;       // [kTile][pitch]
    int64_t *const off_s = reinterpret_cast<int64_t *>(kv_s + kTile * pitch);   // [kTile]
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, row0 = blockIdx.x * kRows, Z = a.divisions;
    int t0, n, ctx;
    int64_t len;
    if (!lengths(a, b, t0, n, ctx, len)) {
        if (threadIdx.x == 0) record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    const int R = n * a.heads;
    if (row0 >= R) return;
    const int64_t tiles = (len + kTile - 1) / kTile, per = (tiles + Z - 1) / Z;
    const int64_t p_begin = blockIdx.z * per * kTile, p_end = min(len, (blockIdx.z + 1) * per * kTile);
    for (int j = warp; j < kRows; j += kWarps) {
        const int r = row0 + j;
        const int64_t from = static_cast<int64_t>(t0 + r / a.heads) * a.q.token_stride + static_cast<int64_t>(r % a.heads) * a.q.head_stride;
        for (int d = lane; d < D; d += 32) q_s[j * pitch + d] = r < R ? load1(a.q.ptr, a.q.dtype, from + d) : 0.0f;
    }
    uint64_t bits[kRowsWarp];
    float m[kRowsWarp], l[kRowsWarp], acc[kRowsWarp][DC];
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        const int r = row0 + warp * kRowsWarp + j, i = r / a.heads;
        bits[j] = r < R ? (a.mask != nullptr ? a.mask[t0 + i] : (2ull << i) - 1ull) : 0ull;
        m[j] = none();
        l[j] = 0.0f;
#pragma unroll
        for (int d = 0; d < DC; ++d) acc[j][d] = 0.0f;
    }
    for (int64_t p0 = p_begin; p0 < p_end; p0 += kTile) {
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
        // rows are whole pieces of 16 bytes; a warp takes eight of the tile's, two at a time
        const int chunk = c.dtype == MOE_F32 ? 4 : 8, chunks = D / chunk;
        for (int j = warp * (kTile / kWarps); j < (warp + 1) * (kTile / kWarps); j += 2) {
            const int64_t o0 = off_s[j], o1 = off_s[j + 1];
            for (int i = lane; i < chunks; i += 32) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (c.dtype == MOE_F32) {
                    if (o0 >= 0) x = reinterpret_cast<const uint4 *>(static_cast<const float *>(c.rows) + o0)[i];
                    if (o1 >= 0) y = reinterpret_cast<const uint4 *>(static_cast<const float *>(c.rows) + o1)[i];
                    *reinterpret_cast<uint4 *>(kv_s + j * pitch + 4 * i) = x;
                    *reinterpret_cast<uint4 *>(kv_s + (j + 1) * pitch + 4 * i) = y;
                } else {
                    if (o0 >= 0) x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(c.rows) + o0)[i];
                    if (o1 >= 0) y = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(c.rows) + o1)[i];
                    float4 *const to = reinterpret_cast<float4 *>(kv_s + j * pitch + 8 * i), *const to1 = reinterpret_cast<float4 *>(kv_s + (j + 1) * pitch + 8 * i);
                    to[0] = make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
                    to[1] = make_float4(bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w));
                    to1[0] = make_float4(bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y));
                    to1[1] = make_float4(bf16_lo(y.z), bf16_hi(y.z), bf16_lo(y.w), bf16_hi(y.w));
                }
            }
        }
        __syncthreads();
        float p[kRowsWarp];
#pragma unroll
        for (int j = 0; j < kRowsWarp; ++j) p[j] = 0.0f;
        const float *const mine = kv_s + lane * pitch, *const rows = q_s + warp * kRowsWarp * pitch;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {   // (a multiple of 4)
            const float4 k = *reinterpret_cast<const float4 *>(mine + d);
#pragma unroll
            for (int j = 0; j < kRowsWarp; ++j) {
                const float4 q = *reinterpret_cast<const float4 *>(rows + j * pitch + d);
                p[j] = fmaf(q.x, k.x, p[j]);
                p[j] = fmaf(q.y, k.y, p[j]);
                p[j] = fmaf(q.z, k.z, p[j]);
                p[j] = fmaf(q.w, k.w, p[j]);
            }
        }
        uint32_t seen[kRowsWarp];
        const int64_t pos = p0 + lane;
#pragma unroll
        for (int j = 0; j < kRowsWarp; ++j) {
            const int64_t d = pos - ctx;
            const bool see = pos < p_end && (d < 0 || ((bits[j] >> (d & 63)) & 1ull)) && row0 + warp * kRowsWarp + j < R;
            seen[j] = __ballot_sync(0xFFFFFFFFu, see);
            const float s = see ? p[j] * a.scale_log2 : none();
            float mx = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = fmaxf(m[j], mx);
            const float ref = mn == none() ? 0.0f : mn;   // nothing seen yet
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
    if (Z > 1) {
        const int64_t part = part_of(a, b, gridDim.x, blockIdx.x, blockIdx.z);
#pragma unroll
        for (int j = 0; j < kRowsWarp; ++j) {
            const int64_t r = part * kRows + warp * kRowsWarp + j;
#pragma unroll
            for (int d = 0; d < DC; ++d)
                if (d * 32 + lane < c.rank) static_cast<float *>(a.part)[r * c.rank + d * 32 + lane] = acc[j][d];
            if (lane == 0) sums_of(a, gridDim.x)[r] = make_float2(m[j], l[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        const int r = row0 + warp * kRowsWarp + j;
        if (r >= R) continue;
        const int t = t0 + r / a.heads, h = r % a.heads;
        const bool empty = m[j] == none() && l[j] == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / l[j];
        const int64_t off = static_cast<int64_t>(t) * a.out.token_stride + static_cast<int64_t>(h) * a.out.head_stride;
#pragma unroll
        for (int d = 0; d < DC; ++d)
            if (d * 32 + lane < c.rank) store1(a.out.ptr, a.out.dtype, off + d * 32 + lane, acc[j][d] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[static_cast<int64_t>(t) * a.heads + h] = empty ? none() : (m[j] + log2f(l[j])) * 0.69314718055994531f;
    }
}

// A warp joins a row's parts.
template <int DC>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_join_kernel(const __grid_constant__ LatentArgs a, int blocks) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y, r = blockIdx.x * kWarps + warp, Z = a.divisions;
    int t0, n, ctx;
    int64_t len;
    if (!lengths(a, b, t0, n, ctx, len) || r >= n * a.heads) return;
    const int64_t first = part_of(a, b, blocks, r / kRows, 0) * kRows + r % kRows;   // kRows further: the next part's
    const float2 *const sums = sums_of(a, blocks) + first;
    float m = none();
    for (int z = lane; z < Z; z += 32) m = fmaxf(m, sums[z * kRows].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float ref = m == none() ? 0.0f : m;
    float l = 0.0f, acc[DC];
#pragma unroll
    for (int d = 0; d < DC; ++d) acc[d] = 0.0f;
    for (int z = 0; z < Z; ++z) {
        const float2 s = sums[z * kRows];
        if (s.x == none() && s.y == 0.0f) continue;   // it saw nothing
        const float k = exp2f(s.x - ref);
        l = fmaf(s.y, k, l);
        const float *const o = static_cast<const float *>(a.part) + (first + static_cast<int64_t>(z) * kRows) * a.cache.rank + lane;
#pragma unroll
        for (int d = 0; d < DC; ++d)
            if (d * 32 + lane < a.cache.rank) acc[d] = fmaf(o[d * 32], k, acc[d]);
    }
    const bool empty = m == none() && l == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / l;
    const int t = t0 + r / a.heads, h = r % a.heads;
    const int64_t off = static_cast<int64_t>(t) * a.out.token_stride + static_cast<int64_t>(h) * a.out.head_stride;
#pragma unroll
    for (int d = 0; d < DC; ++d)
        if (d * 32 + lane < a.cache.rank) store1(a.out.ptr, a.out.dtype, off + d * 32 + lane, acc[d] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(t) * a.heads + h] = empty ? none() : (m + log2f(l)) * 0.69314718055994531f;
}

constexpr size_t smem_bytes(int D) { return (kRows + kTile) * pitch_of(D) * sizeof(float) + kTile * sizeof(int64_t); }
constexpr int kMaxRope = 128;

template <int DC>
cudaError_t launch(LatentArgs a, cudaStream_t s, bool pdl) {
    // always what the widest row needs: the limit is the function's, and a smaller one, set for this
    // call, could come between another thread's setting and its launch
    constexpr size_t most = smem_bytes(32 * DC + kMaxRope);
    static_assert(most <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(latent_simt_kernel<DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    const int rows = a.max_tokens * a.heads, blocks = (rows + kRows - 1) / kRows;
    const int64_t tiles = (static_cast<int64_t>(a.max_pages) * a.cache.page + kTile - 1) / kTile, ctas = static_cast<int64_t>(a.seqs) * blocks;
    // two tiles or more to a division
    a.divisions = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((tiles + 1) / 2, kParts / ctas)));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, a.seqs, a.divisions);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem_bytes(a.cache.rank + a.cache.rope);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, latent_simt_kernel<DC>, a);
    if (e != cudaSuccess || a.divisions == 1) return e;
    cfg.gridDim = dim3((rows + kWarps - 1) / kWarps, a.seqs);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_simt_join_kernel<DC>, a, blocks);
}

}  // namespace

size_t latent_simt_part_bytes(int rank) { return static_cast<size_t>(kParts) * kRows * (rank * sizeof(float) + sizeof(float2)); }

cudaError_t launch_latent_simt(const LatentArgs &a, cudaStream_t s, bool pdl) {
    if (a.cache.rank <= 128) return launch<4>(a, s, pdl);
    return a.cache.rank <= 256 ? launch<8>(a, s, pdl) : launch<16>(a, s, pdl);
}

}  // namespace moe
