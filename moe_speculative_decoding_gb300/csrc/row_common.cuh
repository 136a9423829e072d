// row_common.cuh -- what the kernels of cache rows share: elements of either type, the rotation of a
// channel pair, a launch.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

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

// One pair, with its two roundings spelled out: the kernels for any layout and for aligned ones give
// the same numbers.
__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
    const float x = fmaf(a, c, -__fmul_rn(b, s)), y = fmaf(a, s, __fmul_rn(b, c));
    a = x;
    b = y;
}
// rows that can be read and written 16 bytes at a time
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
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace moe
