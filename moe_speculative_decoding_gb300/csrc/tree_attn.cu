// tree_attn.cu -- attention of drafted tokens over a paged cache on the tensor cores (tcgen05 +
// TMA), for bf16 queries over a bf16 or an e4m3 cache, heads of up to 128 channels.
//
//     s = scale <q, k>,  out = sum_p e^(s_p - lse) v_p,  lse = ln sum_p e^(s_p)
//
// Bound: the cache's bytes are read once, 4 * dim * R flops per cached position and head for the R =
// tokens * group rows that share it; up to R of about 256 that is less than the tensor cores do in
// the time of the read, so the kernel is built to stream the cache, and to keep the tensor cores
// busy beyond.
//
// The M = 128 operand is rows (token, query head of the group), so a row of the softmax lies in one
// TMEM lane and is one thread's.  The positions are walked in tiles of 128: S = Q K^T into TMEM,
// the row's running maximum and sum in registers, the weights back into TMEM over S (as the A
// operand, 16 bits), O += P V with V taken as it lies in the cache (positions by channels,
// MN-major).  O is rescaled only when a row's maximum has grown by more than 2^8 (the weights then
// stay below 2^8 and the result is the same ratio), which after the first tiles is rare.
//
// One persistent CTA per SM.  Work is the list of (sequence, cache head, pair of 128-row tiles) x
// tiles of positions, cut into equal contiguous ranges over the CTAs from the lengths on the
// device; a range's part of an item leaves its unnormalised output, maximum and sum in the
// workspace, and a second small kernel joins the parts in order (no atomics: repeats give the same
// bits).  Items that one CTA holds whole are written out directly.
//
// Two softmax warpgroups share a CTA.  With up to 128 rows they take alternate position tiles of
// the same rows, each with its own maximum, sum and O, joined at the end of the item; with more
// they take one 128-row tile each, and every K and V tile serves both.  Either way while one
// forms its weights the other's products run.
//
// e4m3 cache: codes and one fp32 scale per position and head.  K's codes are the B operand as they
// are (kind::f8f6f4): a query row, scaled by a power of two to below 256, is the sum of an e4m3
// number (4 significant bits) and a remainder that e5m2 holds exactly (a multiple of the bf16 unit
// of at most 8), down to 2^-14 of the row's largest; so two products give q k exactly, and the
// key's scale is applied to the column of S in fp32.  V's codes become fp16 (exact) in shared
// memory; the value's scale goes onto the weight in fp32 before the weight is rounded to fp16
// (2^-11; a bf16 cache needs bf16 weights, 2^-8).  The running maximum is then that of the score plus
// the scale's logarithm, so that it is a row's largest weight that lies near 1.
//
// Measured: 8 sequences of 4001-8201 positions, trees of 64 tokens, 8 query heads to each of 4 key
// heads, 128 channels, bf16: 64 us, 753 TFLOP/s.  A tile of K and V serves 256 rows in 3,000 cycles,
// where its four products need 2,050 and its 32,768 exponentials 1,020 (a loop of them alone issues 32 a
// cycle and SM); the rest is the turns and what else a weight takes.  An item's beginning (queries,
// 5,000-8,000 cycles) and end (4,000-5,000) come on top, and the joining kernel: 53-54 and 17-20 us
// one after the other under the profiler.  128 rows over 60-65 thousand positions of e4m3 codes: 167 us,
// twice the floor of their bytes.
//
// Every wait is bounded (an abort flag, MOE_ERR_DEVICE_TIMEOUT, then copies and products are
// drained and TMEM is freed).
#include "tree_common.cuh"

namespace moe {

cudaError_t launch_tree_narrow(const TreeArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, cudaStream_t s, bool pdl);

namespace {

constexpr int kProducerWarp = 8, kMmaWarp = 9;   // two product warps, one per softmax warpgroup
constexpr uint32_t kTmemCols = 512;

// DP: the head's channels rounded up to 64 or 128.
template <bool F8, int DP>
struct Lay {
    static constexpr int kAux = F8 ? 12 : 11;      // V's four converters; the cleaner of its last tiles
    static constexpr int kThreads = F8 ? 512 : 384, kGroups = 1;
    // a thread's registers: the softmax's hold a row's 128 scores; the sum is what is launched with
    static constexpr int kOther = 56, kSoft = F8 ? 200 : 224;
    static constexpr int kRegs = 256 * kSoft + (kThreads - 256) * kOther;
    static constexpr uint32_t kQTile = F8 ? 2 * 16384 : 128 * DP * 2;
    static constexpr uint32_t kKSlot = F8 ? 16384 : 128 * DP * 2;
    static constexpr uint32_t kVSlot = 128 * DP * 2;
    static constexpr uint32_t kStage = F8 ? 16384 : 0;
    // A product warp waits only for its own tiles, every other one when the warpgroups alternate:
    // with two slots these are all of one slot's uses, so that the slot's parity names the use.
    static constexpr int NK = 2, NV = 2, NS = F8 ? 3 : 0, NC = 4;
    // next to the codes: a softmax thread owns a row and weighs all of a tile's scales
    static constexpr bool kLandScales = F8;
    static constexpr int kUsers = 2;               // products that release a slot
    static constexpr int kVReaders = F8 ? 4 : 1;   // arrivals that fill a V slot
    static constexpr uint32_t oK = 2 * kQTile, oV = oK + NK * kKSlot, oS = oV + NV * kVSlot;
    static constexpr uint32_t oSSc = oS + NS * kStage;             // F8: float [NS][ks, vs][128], landing
    static constexpr uint32_t oBar = oSSc + NS * 1024;
    // barriers: k_full, k_empty, v_full, v_empty, st_full, st_empty, sc_full[NC], sc_empty[NC],
    // s_full[2], p_ready[2], q_ready, o_full, v_fix[4], drain
    static constexpr int bKF = 0, bKE = NK, bVF = 2 * NK, bVE = bVF + NV, bSF = bVE + NV, bSE = bSF + NS, bCF = bSE + NS,
                         bCE = bCF + NC, bS = bCE + NC, bP = bS + 2, bQ = bP + 2, bO = bQ + 1, bFix = bO + 1,
                         bDrain = bFix + 4, bW = bDrain + 1, kBars = bW + kRecords;
    static constexpr uint32_t oMisc = oBar + 8 * kBars + 8;        // TMEM address, abort flag, V tiles issued, tiles copied, turns
    static constexpr uint32_t oBad = (oMisc + 32 + 15) & ~15u;     // uint32 [8 items][2 tiles][4]
    static constexpr uint32_t oScale = oBad + 256;                 // F8: float [NC][ks, vs, log2 of vs][128]
    static constexpr uint32_t oTop = oScale + (F8 ? NC * 1536 : 0);  // F8: float [NC][4], the warps' largest log2 of vs so far
    static constexpr uint32_t oQs = oTop + (F8 ? NC * 16 : 0);      // F8: float [2][128], row factors
    static constexpr uint32_t oWalk = (oQs + (F8 ? 1024 : 0) + 7) & ~7u;   // records of walks
    static constexpr uint32_t kSmem = oWalk + kRecords * kRecordBytes;
    static_assert(kSmem <= 232448, "shared memory");
};

// ------------------------------------------------------------------ softmax of a tile
// The largest of a row's 128 scores (times their key scales), unseen ones left out.  LV: in log2 units
// (cs to a score) plus the logarithms of the value scales.  The next 32 columns load while 32 are
// looked at.
template <bool F8, bool EDGE, bool LV>
__device__ __forceinline__ float tile_max(uint32_t s_addr, const float *ks, const float *lv, float cs, const uint32_t (&see)[4]) {
    uint32_t x[2][32];
    const F2 cs2 = f2(cs, cs);
    float m0 = ninf(), m1 = ninf();
    tmem_ld32(s_addr, x[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_wait_ld();
        if (c < 3) tmem_ld32(s_addr + 32 * (c + 1), x[(c + 1) & 1]);
        uint32_t(&y)[32] = x[c & 1];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float a[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = __uint_as_float(y[i + k]);
            if (F8) {
                const float4 q = *reinterpret_cast<const float4 *>(ks + 32 * c + i);
                F2 s0 = f2_mul(f2(a[0], a[1]), f2(q.x, q.y)), s1 = f2_mul(f2(a[2], a[3]), f2(q.z, q.w));
                if (LV) {
                    const float4 z = *reinterpret_cast<const float4 *>(lv + 32 * c + i);
                    s0 = f2_fma(s0, cs2, f2(z.x, z.y));
                    s1 = f2_fma(s1, cs2, f2(z.z, z.w));
                }
                f2_get(s0, a[0], a[1]);
                f2_get(s1, a[2], a[3]);
            }
            if (EDGE) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!(see[c] >> (i + k) & 1u)) a[k] = ninf();
            }
            m0 = fmaxf(fmaxf(m0, a[0]), a[1]);
            m1 = fmaxf(fmaxf(m1, a[2]), a[3]);
        }
    }
    return fmaxf(m0, m1);
}

// Weights 2^(s cs - ref) of the row, summed in fp32, then (times the value scales) rounded to 16
// bits over columns of S that were read before.  Returns the sum.
template <bool F8, bool EDGE>
__device__ __forceinline__ float tile_weights(uint32_t s_addr, const float *ks, const float *vs, float cs, float ref,
                                              const uint32_t (&see)[4]) {
    uint32_t x[2][32];
    F2 l0 = f2(0.0f, 0.0f), l1 = f2(0.0f, 0.0f);
    const F2 cs2 = f2(cs, cs), ref2 = f2(-ref, -ref);
    tmem_ld32(s_addr, x[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_wait_ld();
        if (c < 3) tmem_ld32(s_addr + 32 * (c + 1), x[(c + 1) & 1]);
        uint32_t(&y)[32] = x[c & 1];
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            F2 a = f2(y[i], y[i + 1]), b = f2(y[i + 2], y[i + 3]);
            if (F8) {
                const float4 q = *reinterpret_cast<const float4 *>(ks + 32 * c + i);
                a = f2_mul(a, f2(q.x, q.y));
                b = f2_mul(b, f2(q.z, q.w));
            }
            a = f2_fma(a, cs2, ref2);
            b = f2_fma(b, cs2, ref2);
            float w0, w1, w2, w3;
            f2_get(a, w0, w1);
            f2_get(b, w2, w3);
            w0 = ex2(w0);
            w1 = ex2(w1);
            w2 = ex2(w2);
            w3 = ex2(w3);
            if (EDGE) {
                if (!(see[c] >> i & 1u)) w0 = 0.0f;
                if (!(see[c] >> (i + 1) & 1u)) w1 = 0.0f;
                if (!(see[c] >> (i + 2) & 1u)) w2 = 0.0f;
                if (!(see[c] >> (i + 3) & 1u)) w3 = 0.0f;
            }
            a = f2(w0, w1);
            b = f2(w2, w3);
            l0 = f2_add(l0, a);
            l1 = f2_add(l1, b);
            if (F8) {
                const float4 q = *reinterpret_cast<const float4 *>(vs + 32 * c + i);
                a = f2_mul(a, f2(q.x, q.y));
                b = f2_mul(b, f2(q.z, q.w));
                f2_get(a, w0, w1);
                f2_get(b, w2, w3);
            }
            p[i / 2] = pack2(w0, w1, F8);
            p[i / 2 + 1] = pack2(w2, w3, F8);
        }
        tmem_st16(s_addr + 16 * c, p);
    }
    float s0, s1;
    f2_get(f2_add(l0, l1), s0, s1);
    return s0 + s1;
}

// o[i] += x with i known only at run time, o staying in registers
__device__ __forceinline__ void add_at(float (&o)[32], int i, float x) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (k == i) o[k] += x;
}

// ------------------------------------------------------------------ the kernel
template <bool F8, int DP>
__global__ void __launch_bounds__(Lay<F8, DP>::kThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ TreeArgs a, int box_rows) {
    using L = Lay<F8, DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    volatile int32_t *const abort_flag = reinterpret_cast<volatile int32_t *>(smem + L::oMisc + 4);
    volatile uint32_t *const v_issued = reinterpret_cast<volatile uint32_t *>(smem + L::oMisc + 8), *const copied = v_issued + 1, *const turn_s = v_issued + 3;
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const long long limit = a.wait_limit;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NK; ++i) {
            mbar_init(bar(L::bKF + i), 1);
            mbar_init(bar(L::bKE + i), L::kUsers);
        }
        for (int i = 0; i < L::NV; ++i) {
            mbar_init(bar(L::bVF + i), L::kVReaders);
            mbar_init(bar(L::bVE + i), L::kUsers);
        }
        for (int i = 0; i < L::NS; ++i) {
            mbar_init(bar(L::bSF + i), 1);
            mbar_init(bar(L::bSE + i), 4);
        }
        for (int i = 0; i < L::NC; ++i) {
            mbar_init(bar(L::bCF + i), 4);
            mbar_init(bar(L::bCE + i), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::bS + i), 1);
            mbar_init(bar(L::bP + i), 4);
        }
        mbar_init(bar(L::bQ), 8);
        mbar_init(bar(L::bO), 2);
        for (int i = 0; i < 4; ++i) mbar_init(bar(L::bFix + i), 1);
        mbar_init(bar(L::bDrain), 2);
        for (int i = 0; i < kRecords; ++i) mbar_init(bar(L::bW + i), 1);
        *abort_flag = 0;
        *v_issued = copied[0] = copied[1] = *turn_s = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(base + L::oMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::oMisc);
    Follow follow = {smem + L::oWalk, bar(L::bW), 0};
    const int G = a.group;

    if (warp >= 8) {
        regs_down<L::kOther>();
        pdl_wait();
        pdl_trigger();
        Walk w;
        if (warp == kProducerWarp) {
            walk_begin(a, w, blockIdx.x == 0);
            produce<L, F8, DP, 0, 1>(a, w, &tm_k, &tm_v, smem, box_rows, abort_flag, copied, v_issued, follow);
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---------------------------------------------------------------- products
            // One warp issues both products of one softmax warpgroup's tiles, so that neither waits in
            // line behind the other's, and its O += P V precedes the next S over the same columns.  When
            // the warpgroups share tiles (two M tiles), the warps take turns, O += P V of one tile and S of
            // the next at a time: started together they stay together, and the tensor cores idle while
            // both form weights (4,400 cycles for a K/V tile against 2,900 in turns).
            const int g = warp - kMmaWarp;
            const uint32_t s_col = tmem + g * kTile, o_col = tmem + 256 + g * DP;
            uint32_t base_tile = 0, base_fix = 0, pc = 0, items = 0, turns = 0;   // turns of both, before this item
            bool ok = true;
            while (ok && walk_follow(a, w, follow, abort_flag)) {
                const bool two = w.s.n * G - w.pair * 2 * kTile > kTile;
                const int T = w.hi - w.lo, U = two ? 2 * T : T;
                const int edge0 = max(w.lo, w.s.ctx / kTile);   // the first tile that V's cleaner goes over
                ok = wait_for(bar(L::bQ), items & 1u, abort_flag, a.err, limit);
                const uint64_t q_desc = desc_kmajor_sw128(base + (two ? g : 0) * L::kQTile);
                auto k_ready = [&](int u) {
                    const uint32_t c = base_tile + (two ? u >> 1 : u);
                    return wait_for(bar(L::bKF + c % L::NK), (c / L::NK) & 1u, abort_flag, a.err, limit);
                };
                auto my_turn = [&](int k) { return !two || wait_count(turn_s, turns + k, abort_flag, a.err, limit); };
                auto pass_turn = [&](int k) {
                    if (two && lane == 0) *turn_s = turns + k + 1;
                    __syncwarp();
                };
                auto qk = [&](int u) {
                    const uint32_t c = base_tile + (two ? u >> 1 : u), slot = c % L::NK;
                    tc_fence_after();
                    const uint64_t k_desc = desc_kmajor_sw128(base + L::oK + slot * L::kKSlot);
                    if (elect_one()) {
                        if (F8) {
#pragma unroll
                            for (int i = 0; i < DP / 32; ++i)
                                tc_mma_f8(s_col, q_desc + 2 * i, k_desc + 2 * i, idesc_e4m3_f32(128, 128), i > 0);
#pragma unroll
                            for (int i = 0; i < DP / 32; ++i)
                                tc_mma_f8(s_col, q_desc + 1024 + 2 * i, k_desc + 2 * i, idesc_e5m2_e4m3(128, 128), 1);
                        } else {
#pragma unroll
                            for (int i = 0; i < DP / 16; ++i) {   // 64-channel halves, 16 KB apart
                                const uint32_t o = (i / 4) * 1024 + (i % 4) * 2;
                                tc_mma_bf16(s_col, q_desc + o, k_desc + o, idesc_bf16_f32(128, 128), i > 0);
                            }
                        }
                        tc_commit(bar(L::bKE + slot));
                        if (!two) tc_commit(bar(L::bKE + slot));   // the only user
                        tc_commit(bar(L::bS + g));
                    }
                    __syncwarp();
                };
                if (ok && g < U && (ok = k_ready(g) && my_turn(g))) {
                    qk(g);
                    pass_turn(g);
                }
                for (int u = g; ok && u < U; u += 2) {
                    const int t = two ? u >> 1 : u, tt = w.lo + t;
                    const uint32_t c = base_tile + t, slot = c % L::NV;
                    ok = wait_for(bar(L::bVF + slot), (c / L::NV) & 1u, abort_flag, a.err, limit);
                    if (!F8 && ok && tt >= edge0) {   // V's cleaner has been over it
                        const uint32_t f = base_fix + (tt - edge0);
                        ok = wait_for(bar(L::bFix + (f & 3u)), (f >> 2) & 1u, abort_flag, a.err, limit);
                    }
                    ok = ok && (!two || u + 2 >= U || k_ready(u + 2)) && my_turn(2 + u) &&
                         wait_for(bar(L::bP + g), pc & 1u, abort_flag, a.err, limit);
                    if (!ok) break;
                    ++pc;
                    tc_fence_after();
                    const uint64_t v_desc = desc_mn_sw128(base + L::oV + slot * L::kVSlot, kTile * 128u);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kTile / 16; ++i)   // 16 positions: 2 KB of V, 8 columns of P
                            mma_ts(o_col, s_col + 8 * i, v_desc + 128 * i, idesc_pv(DP, F8 ? 0 : 1), u >= 2 || i > 0);
                        tc_commit(bar(L::bVE + slot));
                        if (!two) tc_commit(bar(L::bVE + slot));
                    }
                    __syncwarp();
                    if (u + 2 < U && (two || (ok = k_ready(u + 2)))) qk(u + 2);
                    pass_turn(2 + u);
                }
                if (two) turns += U + 2;
                if (ok && elect_one()) tc_commit(bar(L::bO));
                __syncwarp();
                base_tile += T;
                base_fix += max(0, w.hi - edge0);
                ++items;
            }
            // every product is done before the CTA leaves
            if (elect_one()) tc_commit(bar(L::bDrain));
            __syncwarp();
            mbar_wait_drain(bar(L::bDrain), 0, kDrain);
            __syncwarp();
        } else if (warp >= L::kAux) {
            if constexpr (F8)
                convert_values<L, DP>(a, w, smem, warp - L::kAux, 0, abort_flag, follow);
            else
                clean_values<L, DP>(a, w, smem, abort_flag, v_issued, follow);
        }
    } else {
        // ---------------------------------------------------------------- softmax, two warpgroups
        regs_up<L::kSoft>();
        Walk w;
        const int g = warp >> 2, r = (warp & 3) * 32 + lane;   // lane quarter = warp % 4
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + g * kTile, o_addr = tmem + lanes + 256 + g * DP;
        float *const qs = reinterpret_cast<float *>(smem + L::oQs);
        const float *const scale_s = reinterpret_cast<const float *>(smem + L::oScale);
        const float4 *const top_s = reinterpret_cast<const float4 *>(smem + L::oTop);
        float2 *const exch = reinterpret_cast<float2 *>(smem);   // [2][128], over Q when Q is done with
        uint32_t sc = 0, scnt = 0;
        bool ok = true;
        pdl_wait();
        while (true) {
            const bool more = walk_follow(a, w, follow, abort_flag);
            // the previous item's exchange has been read; everybody leaves together
            if (softmax_any(!ok || *abort_flag != 0) || !more) break;
            const int R = w.s.n * G, row0 = w.pair * 2 * kTile;
            const bool two = R - row0 > kTile;
            const int T = w.hi - w.lo, U = two ? 2 * T : T;
            // Q rows into shared memory: 16-byte chunks (8 channels), zeros beyond the rows
            {
                constexpr int C = DP / 8;
                const int tiles = two ? 2 : 1;
                const Divisor by_group(G);
                const int c = static_cast<int>(threadIdx.x) % C;   // 256 / C rows a step, eight steps' loads at a time
#pragma unroll 1
                for (int r0 = static_cast<int>(threadIdx.x) / C; r0 < tiles * kTile; r0 += 8 * (256 / C)) {
                    uint4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = row0 + r0 + i * (256 / C);
                        x[i] = make_uint4(0, 0, 0, 0);
                        const int token = static_cast<int>(by_group.quotient(static_cast<uint32_t>(row)));
                        if (row < R && c * 8 < a.cache.dim)
                            x[i] = *reinterpret_cast<const uint4 *>(
                                static_cast<const uint16_t *>(a.q.ptr) + static_cast<int64_t>(w.s.t0 + token) * a.q.token_stride +
                                static_cast<int64_t>(w.hk * G + row - token * G) * a.q.head_stride + c * 8);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = r0 + i * (256 / C), mt = rr / kTile, lr = rr % kTile;
                        if (mt >= tiles) break;
                        float unscale;
                        store_query<F8, DP>(smem + mt * L::kQTile, kTile, lr, c, x[i], unscale);
                        if (F8 && c == 0) qs[mt * 128 + lr] = unscale;
                    }
                }
                fence_proxy_async_smem();
            }
            const int mt = two ? g : 0, row = row0 + mt * kTile + r;
            const bool live = row < R;
            const int token = live ? w.s.t0 + row / G : 0, head = w.hk * G + (live ? row % G : 0);
            uint64_t M = 0;
            if (live) M = a.mask != nullptr ? a.mask[token] : (2ull << (row / G)) - 1ull;
            warp_arrive(bar(L::bQ));
            if (F8) named_barrier(3, 256);   // the row factors, before other threads' are read
            const float cs = F8 ? a.scale_log2 * qs[mt * 128 + r] : a.scale_log2;
            float m = ninf(), l = 0.0f;
            for (int u = g; u < U; u += 2) {
                const int tt = w.lo + (two ? u >> 1 : u);
                const bool edge = (tt + 1) * kTile > w.s.ctx;
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
                if (edge) seen_bits(M, w.s, tt, see);
                const uint32_t tile_no = scnt + (two ? u >> 1 : u), sb = tile_no % L::NC;
                const float *const ks = scale_s + sb * 384, *const vs = ks + 128, *const lv = ks + 256;
                if (F8 && !(ok = wait_for(bar(L::bCF + sb), (tile_no / L::NC) & 1u, abort_flag, a.err, limit))) break;
                if (!(ok = wait_for(bar(L::bS + g), sc & 1u, abort_flag, a.err, limit))) break;
                ++sc;
                tc_fence_after();
                float mx = 0.0f, keep = 1.0f;
                bool look = F8 && (edge || u < 2);
                if (!look) {
                    mx = !F8 && edge ? tile_max<F8, true, false>(s_addr, ks, lv, cs, see) : tile_max<F8, false, false>(s_addr, ks, lv, cs, see);
                    mx *= cs;   // cs > 0; -inf stays
                    // e4m3: with the largest value scale so far this is at or above what counts, a score plus its
                    // own value's; only where that does not do is that one looked for (in every tile: 128 rows
                    // over 60-65 thousand positions 180 us against 170)
                    if (F8) {
                        const float4 t = top_s[sb];
                        look = __any_sync(0xFFFFFFFFu, mx + fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)) - m > kLazy);
                    }
                }
                if (F8 && look) mx = tile_max<F8, true, true>(s_addr, ks, lv, cs, see);
                if ((!F8 || look) && __any_sync(0xFFFFFFFFu, u < 2 || mx - m > kLazy)) {
                    const float mn = fmaxf(m, mx);
                    if (u >= 2) {
                        keep = mn == ninf() ? 1.0f : ex2(m - mn);
                        l *= keep;
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t x[32];
                            tmem_ld32(o_addr + 32 * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * keep);
                            tmem_st32(o_addr + 32 * c, x);
                        }
                    }
                    m = mn;
                }
                const float ref = m == ninf() ? 0.0f : m;   // nothing seen yet: every weight is 0
                l += edge ? tile_weights<F8, true>(s_addr, ks, vs, cs, ref, see)
                          : tile_weights<F8, false>(s_addr, ks, vs, cs, ref, see);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(L::bP + g));
                if (F8) warp_arrive_cnt(bar(L::bCE + sb), two ? 1 : 2);   // the tile's scales are read
            }
            // ------------------------------------------------------------ the item's end
            ok = ok && wait_for(bar(L::bO), static_cast<uint32_t>(w.index) & 1u, abort_flag, a.err, limit);
            tc_fence_after();
            scnt += T;
            constexpr float gain = F8 ? 1.0f / kWeightUp : 1.0f;   // of the accumulator
            float wt[2] = {0.0f, 0.0f}, mm = m, ll = l;
            int c0 = 0, c1 = DP;
            if (!two) {   // both warpgroups hold a part of the same rows: half of the channels each
                exch[g * 128 + r] = make_float2(m, l);
                named_barrier(3, 256);
                const float2 e0 = exch[r], e1 = exch[128 + r];
                mm = fmaxf(e0.x, e1.x);
                const float ref = mm == ninf() ? 0.0f : mm;
                const float k0 = ex2(e0.x - ref), k1 = ex2(e1.x - ref);
                ll = e0.y * k0 + e1.y * k1;
                wt[0] = k0 * gain;
                wt[1] = k1 * gain;
                c0 = g * (DP / 2);
                c1 = c0 + DP / 2;
            } else {
                wt[g] = gain;
            }
            const bool none = mm == ninf() && ll == 0.0f;
            const float inv = none ? 0.0f : 1.0f / ll;
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.index == 0 ? 0 : 1);
            const uint32_t *const bad = reinterpret_cast<const uint32_t *>(smem + L::oBad) + (w.index & 7) * 8;
            uint32_t any_bad = 0;   // of parts that reach past the context: there the products waited for the words
            if (w.hi * kTile > w.s.ctx) {
#pragma unroll
                for (int i = 0; i < 8; ++i) any_bad |= bad[i];
            }
            const int64_t out_off = static_cast<int64_t>(token) * a.out.token_stride + static_cast<int64_t>(head) * a.out.head_stride;
#pragma unroll 1
            for (int c = c0; c < c1; c += 32) {
                __syncwarp();
                float o[32];
                if (two) {
                    uint32_t x[32];
                    tmem_ld32(o_addr + c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(x[i]) * wt[g];
                } else {
                    uint32_t x[32];
                    tmem_ld32(tmem + lanes + 256 + c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(x[i]) * wt[0];
                    if (U > 1) {   // the second warpgroup had a tile
                        tmem_ld32(tmem + lanes + 256 + DP + c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(x[i]), wt[1], o[i]);
                    }
                }
                if (any_bad != 0) {
                    // non-finite values of drafted tokens, for the rows that see them
#pragma unroll 1
                    for (int tt = max(w.lo, w.s.ctx / kTile); tt < w.hi; ++tt) {
                        uint32_t see[4];
                        seen_bits(M, w.s, tt, see);
#pragma unroll 1
                        for (int j = 0; j < kTile; ++j) {
                            if (!(bad[(tt & 1) * 4 + j / 32] >> (j & 31) & 1u) || !(see[j / 32] >> (j & 31) & 1u)) continue;
#pragma unroll 1
                            for (int i = 0; i < 32; ++i) {
                                const float x = c + i < a.cache.dim ? value_at<F8>(a, w.b, w.hk, tt * kTile + j, c + i) : 0.0f;
                                if (!(fabsf(x) <= 3.4028234e38f)) add_at(o, i, x);
                            }
                        }
                    }
                }
                if (live && w.whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (c + i < a.cache.dim)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out.ptr) + out_off + c + i) =
                                make_uint4(pack2(o[i] * inv, o[i + 1] * inv, false), pack2(o[i + 2] * inv, o[i + 3] * inv, false),
                                           pack2(o[i + 4] * inv, o[i + 5] * inv, false), pack2(o[i + 6] * inv, o[i + 7] * inv, false));
                    }
                } else if (live) {
                    float4 *const po = part_out<DP>(a, slot, mt) + r;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) po[static_cast<size_t>((c + i) / 4) * kTile] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            tc_fence_before();   // the next item's products follow this warp's arrival on bQ
            if (live && (two || g == 0)) {
                if (w.whole) {
                    if (a.lse != nullptr)
                        a.lse[static_cast<int64_t>(token) * a.q.heads + head] = none ? ninf() : (mm + log2f(ll)) * 0.69314718055994531f;
                } else {
                    part_ml<DP>(a, gridDim.x, slot, mt)[r] = make_float2(mm, ll);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducerWarp && *abort_flag != 0) drain_copies<L, F8>(smem, copied);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ joining the parts
// For an item that several CTAs of the first kernel shared: out = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i over its parts in order.  The parts lie in L2, so what counts is how many
// loads are in flight: a CTA takes 1024 / DP rows, a thread four channels of one row, its first
// parts on their way while a warp per row forms the weights, a lane per part.
constexpr int kJoinThreads = 256;

template <bool NARROW, int DP>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a, int ctas) {
    constexpr int Q = DP / 4, ROWS = kJoinThreads / Q, AHEAD = 8;
    __shared__ long long red[4][kJoinThreads / 32];
    __shared__ float wt[kMaxCtas][ROWS], inv_s[ROWS];
    const int b = blockIdx.z, hk = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the lengths are no product of the first kernel, which waited for what came before it
    const Seq s = load_seq(a, b);
    const int row0 = blockIdx.x * ROWS, R = s.n * a.group;
    if (row0 >= R) {
        pdl_wait();
        return;
    }
    Work before = {0, 0}, total = {0, 0};
    for (int i = threadIdx.x; i < a.seqs; i += kJoinThreads) {
        const Work x = seq_work(a, load_seq(a, i));
        total.tiles += x.tiles;
        total.items += x.items;
        if (i < b) {
            before.tiles += x.tiles;
            before.items += x.items;
        }
    }
    long long *const sums[4] = {&before.tiles, &before.items, &total.tiles, &total.items};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) *sums[k] += __shfl_xor_sync(0xFFFFFFFFu, *sums[k], o);
        if (lane == 0) red[k][warp] = *sums[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        *sums[k] = 0;
        for (int i = 0; i < kJoinThreads / 32; ++i) *sums[k] += red[k][i];
    }
    const int extra = item_cost(a, total, ctas);
    const long long W = total.tiles + extra * total.items;
    const int pair = row0 / (2 * kTile), mt = row0 / kTile % 2, r0 = row0 % kTile;
    const long long item0 = before.tiles + extra * before.items +
                            (static_cast<long long>(hk) * s.pairs + pair) * (s.tiles + extra);
    const long long first = item0 + extra;   // the unit of the item's first tile
    const int C = used_ctas(W, ctas);
    const int ca = range_of(W, first, C), cb = range_of(W, first + s.tiles - 1, C);
    pdl_wait();
    pdl_trigger();
    if (ca == cb) return;
    // whether the item is the first with tiles in its first CTA's range (the unit before an item is
    // the last tile of the one before)
    const bool head_slot = range_lo(W, ca, C) >= item0;
    auto slot = [&](int i) { return 2 * (ca + i) + (i == 0 && !head_slot ? 1 : 0); };
    const int parts = cb - ca + 1;
    // neighbouring threads read neighbouring 16 bytes of either layout
    const int rr = NARROW ? threadIdx.x / Q : threadIdx.x % ROWS, quad = NARROW ? threadIdx.x % Q : threadIdx.x / ROWS;
    const bool live = row0 + rr < R && quad * 4 < a.cache.dim;
    auto part = [&](int i) {
        return NARROW ? *reinterpret_cast<const float4 *>(narrow_out<DP>(a, slot(i)) + (r0 + rr) * DP + quad * 4)
                      : part_out<DP>(a, slot(i), mt)[static_cast<size_t>(quad) * kTile + r0 + rr];
    };
    float4 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (live && i < parts) x[i] = part(i);
    for (int r = warp; r < ROWS; r += kJoinThreads / 32) {
        if (row0 + r >= R) continue;
        auto ml = [&](int i) { return NARROW ? narrow_ml<DP>(a, ctas, slot(i))[r0 + r] : part_ml<DP>(a, ctas, slot(i), mt)[r0 + r]; };
        float m = ninf(), l = 0.0f;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, ml(i).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float ref = m == ninf() ? 0.0f : m;
        for (int i = lane; i < parts; i += 32) {
            const float2 y = ml(i);
            const float k = ex2(y.x - ref);
            l += y.y * k;
            wt[i][r] = k;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0) {
            const bool none = m == ninf() && l == 0.0f;
            inv_s[r] = none ? 0.0f : 1.0f / l;
            const int row = row0 + r;
            if (a.lse != nullptr)
                a.lse[static_cast<int64_t>(s.t0 + row / a.group) * a.q.heads + hk * a.group + row % a.group] =
                    none ? ninf() : (m + log2f(l)) * 0.69314718055994531f;
        }
    }
    __syncthreads();
    if (!live) return;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < parts; i0 += AHEAD) {
        if (i0 > 0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (i0 + i < parts) x[i] = part(i0 + i);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i0 + i >= parts) continue;
            const float k = wt[i0 + i][rr];
            o.x = fmaf(x[i].x, k, o.x);
            o.y = fmaf(x[i].y, k, o.y);
            o.z = fmaf(x[i].z, k, o.z);
            o.w = fmaf(x[i].w, k, o.w);
        }
    }
    const float inv = inv_s[rr];
    const int row = row0 + rr;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out.ptr) + static_cast<int64_t>(s.t0 + row / a.group) * a.out.token_stride +
                               static_cast<int64_t>(hk * a.group + row % a.group) * a.out.head_stride + quad * 4) =
        make_uint2(pack2(o.x * inv, o.y * inv, false), pack2(o.z * inv, o.w * inv, false));
}

// ------------------------------------------------------------------ host side
std::mutex g_mu;
struct Device {
    int sms = 0;
    bool set[4] = {false, false, false, false};
} g_dev[64];

int sm_count(int dev) {
    std::lock_guard<std::mutex> lock(g_mu);
    Device &d = g_dev[dev & 63];
    if (d.sms == 0) cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    return std::min(d.sms, kMaxCtas);
}

template <bool F8, int DP>
cudaError_t launch_wide(const TreeArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                        cudaStream_t s, bool pdl) {
    using L = Lay<F8, DP>;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        bool &set = g_dev[dev & 63].set[(F8 ? 2 : 0) + (DP == 128 ? 1 : 0)];
        if (!set) {
            cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<F8, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
            if (e == cudaSuccess) e = check_registers(tree_attn_kernel<F8, DP>, L::kThreads, L::kRegs);
            if (e != cudaSuccess) return e;
            set = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<F8, DP>, tm_k, tm_v, a, rows);
}

template <bool NARROW, int DP>
cudaError_t launch_join(const TreeArgs &a, int ctas, cudaStream_t s, bool pdl) {
    constexpr int ROWS = kJoinThreads / (DP / 4);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.max_tokens * a.group + ROWS - 1) / ROWS, a.cache.heads, a.seqs);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<NARROW, DP>, a, ctas);
}

bool wide16(const moe_heads_t &h) {
    return (reinterpret_cast<uintptr_t>(h.ptr) & 15u) == 0 && h.token_stride % 8 == 0 && h.head_stride % 8 == 0;
}

}  // namespace

bool tree_attn_supports(const moe_kv_cache_t &c, const moe_heads_t &q, const moe_heads_t &out) {
    return q.dtype == MOE_BF16 && out.dtype == MOE_BF16 && (c.dtype == MOE_BF16 || c.dtype == MOE_E4M3) && c.dim <= 128 &&
           c.page % 8 == 0 && wide16(q) && wide16(out) &&
           (c.dtype == MOE_BF16 || ((reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) & 15u) == 0);
}

// A workspace serves whichever kernel a call runs on, on the device that is current when its size is
// asked for (room for kMaxCtas CTAs' parts would be more than any call there touches): a larger
// device refuses it.
size_t tree_attn_part_bytes(int dim) {
    int dev = 0;
    int sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        const int n = sm_count(dev);
        if (n > 0) sms = n;
    }
    return static_cast<size_t>(sms) * 2 * 2 * kTile * (dim_padded(dim) * sizeof(float) + sizeof(float2));
}

cudaError_t launch_tree_attn(TreeArgs a, cudaStream_t s, bool pdl) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = sm_count(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const bool f8 = a.cache.dtype == MOE_E4M3, wide_head = a.cache.dim > 64;
    const int rows = box_rows_of(a.cache.page);
    CUtensorMap tm_k, tm_v;
    if (!encode(&tm_k, a.cache, a.cache.k, rows, true) || !encode(&tm_v, a.cache, a.cache.v, rows, !f8))
        return cudaErrorNotSupported;
    // Short contexts: an item's few tiles one after the other take less time than another end of an
    // item and the launch that joins the parts.  8 heads of 128, 4 rows, one sequence: 7.9 us
    // undivided against 8.8 at two tiles, 8.6 and 8.9 at three, 9.3 and 8.9 at four (and 2 us less
    // for the host), 12.2 and 9.2 at eight; 256 rows, four sequences: 24.0 and 30.8 at eight.  With
    // enough items for the SMs (16 sequences, e4m3): 16.7 and 24.8 at eight, 22.6 and 24.4 at twelve,
    // 27.4 and 26.9 at sixteen.
    // (a table may be wider than any sequence is long, by more than 64-bit products hold)
    const long long item_tiles = (std::min(static_cast<long long>(a.max_pages) * a.cache.page, kMaxPositions) + kTile - 1) / kTile;
    const long long items = static_cast<long long>(a.seqs) * a.cache.heads * ((a.max_tokens * a.group + 2 * kTile - 1) / (2 * kTile));
    a.undivided = item_tiles <= (2 * items >= sms ? 12 : a.max_tokens * a.group > kNarrowRows ? 8 : 4);
    // no more CTAs than the page tables could fill with tiles
    const int ctas = static_cast<int>(std::min<long long>(sms, items * item_tiles));
    // Up to 64 rows: positions as the M operand.  Few rows against many, 60-65 thousand positions of 4
    // sequences, 8 heads of 128: e4m3 16 rows 90 us against 159, 32 rows 100 against 160, 64 rows 155 against
    // 162; bf16 16 rows 155 against 160, 32 rows 156 against 161, 64 rows 165 against 163; 16 short contexts
    // of e4m3 with 20 rows 36.8 against 57.5.
    if (a.max_tokens * a.group <= kNarrowRows) {
        e = launch_tree_narrow(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
        if (e != cudaSuccess || a.undivided) return e;
        return wide_head ? launch_join<true, 128>(a, ctas, s, pdl) : launch_join<true, 64>(a, ctas, s, pdl);
    }
    if (wide_head)
        e = f8 ? launch_wide<true, 128>(a, dev, ctas, rows, tm_k, tm_v, s, pdl) : launch_wide<false, 128>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
    else
        e = f8 ? launch_wide<true, 64>(a, dev, ctas, rows, tm_k, tm_v, s, pdl) : launch_wide<false, 64>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
    if (e != cudaSuccess || a.undivided) return e;
    return wide_head ? launch_join<false, 128>(a, ctas, s, pdl) : launch_join<false, 64>(a, ctas, s, pdl);
}

}  // namespace moe
