// tree_attn_narrow.cu -- tree attention on the tensor cores for up to 64 rows (token, query head of
// the group) of a cache head, by the caller's bound on a sequence's tokens: short chains, small trees
// and single tokens.
//
// Bound: the cache's bytes; 4 * dim flops per position, row and head leave the tensor cores far from
// their limit, so what counts is that nothing else of a tile costs its rows twice: padding 8 or 20
// rows to the 128 lanes of the kernel for many rows (tree_attn.cu) makes every product and every
// exponential 128 wide.  Here the products are the other way round: positions are the M = 128
// operand and rows the N = NT columns (16, 32 or 64),
//
//     S^T = K Q^T [128 positions x NT],  O^T += V^T P^T [128 channels x NT],
//
// K and V^T taken as they lie in the cache (V^T MN-major), Q and the weights P in shared memory.  A
// thread of a softmax warpgroup owns a position, so a tile costs it NT exponentials, and the key and
// value scales of an e4m3 cache are one number per thread.  The row maxima are columns' maxima over
// 128 threads, which is dear, so they are not formed per tile: a tile is weighed against the maxima
// so far, and only when some score lies above its row's by more than 2^8 (a vote of the warpgroup)
// are they formed anew and O rescaled.  The sums stay with the threads until the end of an item.
//
// The two warpgroups take alternate tiles, each with its own maxima, sums and O^T, joined at the
// item's end.  S^T of a warpgroup's next tile is formed while it weighs the present one.  Work list,
// copies, value cleaning and conversion, parts and their join are those of tree_attn.cu.
//
// Measured, 8 cache heads of 128 channels, 60-65 thousand positions of 4 sequences: bf16 with 16 or 32
// rows 156-161 us (6.5-6.7 TB/s of the 6.79 of a copy: the cache's bytes bound it), with 64 rows 169;
// e4m3 with 16 rows 90-97 us (5.5-6.0 TB/s), with 32 rows 100-105, with 64 rows 155: there a tile's
// chain of conversion, weights and products, 1,650 cycles, takes as long as its bytes or longer.
// One token over 300 positions: 8.2 us, a chain of latencies (lengths, page table, K, scores, V).
#include "tree_common.cuh"

namespace moe {
namespace {

constexpr int kProducerWarp = 8, kScoreWarp = 9, kOutWarp = 10, kValueWarp = 11, kAuxWarp = 12;

template <bool F8, int DP, int NT>
struct Lay {
    // bf16: a cleaner (and three idle warps of its warpgroup); F8: two groups of four converters, one
    // for 64 rows, whose softmax needs the registers
    static constexpr int kGroups = F8 && NT < 64 ? 2 : 1, kThreads = kGroups == 2 ? 640 : 512;
    // a thread's registers: the softmax's hold a position's NT scores and NT sums
    static constexpr int kOther = kGroups == 2 ? 48 : 56, kSoft = kGroups == 2 ? 168 : 200;
    static constexpr int kRegs = 256 * kSoft + (kThreads - 256) * kOther;
    static constexpr uint32_t kKSlot = F8 ? 16384 : 128 * DP * 2;
    static constexpr uint32_t kVSlot = 128 * DP * 2;
    static constexpr uint32_t kStage = F8 ? 16384 : 0;
    static constexpr uint32_t kQ = F8 ? 2 * NT * 128 : DP / 64 * NT * 128;
    static constexpr uint32_t kP = 128 * NT * 2;   // weights of a tile: a row of NT per position
    // rings: what fits
    static constexpr int NK = DP == 64 ? 4 : (F8 ? 3 : 2);
    static constexpr int NV = F8 ? 2 : (DP == 64 ? 4 : (NT < 64 ? 3 : 2));
    static constexpr int NS = !F8 ? 0 : (NT < 64 ? 4 : 2);   // even: a slot is one converter group's
    // The converters load a position's scales themselves: two bulk copies a box, next to the codes,
    // cost the producer 800 cycles a tile.
    static constexpr bool kLandScales = false;
    static constexpr int NC = 4, kUsers = 1, kVReaders = F8 ? 4 : 1;
    static constexpr uint32_t oK = 0, oV = oK + NK * kKSlot, oS = oV + NV * kVSlot, oP = oS + NS * kStage,
                              oQ = oP + 2 * kP, oSSc = oQ + kQ, oBar = oSSc;
    static constexpr int bKF = 0, bKE = NK, bVF = 2 * NK, bVE = bVF + NV, bSF = bVE + NV, bSE = bSF + NS, bCF = bSE + NS,
                         bCE = bCF + NC, bS = bCE + NC, bSFree = bS + 2, bP = bSFree + 2, bPV = bP + 2, bQ = bPV + 2,
                         bO = bQ + 1, bFix = bO + 1, bW = bFix + 4, bDrain = bW + kRecords, kBars = bDrain + 1;
    static constexpr uint32_t oMisc = oBar + 8 * kBars + 8;        // TMEM address, abort flag, V tiles issued, tiles copied
    static constexpr uint32_t oBad = (oMisc + 32 + 15) & ~15u;     // uint32 [8 items][2 tiles][4]
    static constexpr uint32_t oScale = oBad + 256;                 // F8: float [NC][ks, vs, log2 of vs][128]
    static constexpr uint32_t oTop = oScale;                       // (not kept)
    static constexpr uint32_t oCs = oScale + (F8 ? NC * 1536 : 0);      // F8: float [NT]: score to log2 units
    static constexpr uint32_t oM = oCs + (F8 ? NT * 4 : 0);    // float [2][NT]: minus a warpgroup's maxima, 0 where there is none
    static constexpr uint32_t oAlpha = oM + 2 * NT * 4;            // float [2][NT]: a rescaling
    static constexpr uint32_t oDelta = oAlpha + 2 * NT * 4;        // float [2][NT]: its logarithm
    static constexpr uint32_t oRed = oDelta + 2 * NT * 4;          // float [2][4][NT]: per warp
    static constexpr uint32_t oMask = oRed + 8 * NT * 4;           // uint64 [NT]: the rows' tree masks
    static constexpr uint32_t oTo = oMask + NT * 8;                // int64 [NT]: the rows' output offsets
    static constexpr uint32_t oWalk = oTo + NT * 8;                // records of walks
    static constexpr uint32_t kSmem = oWalk + kRecords * kRecordBytes;
    static constexpr uint32_t kTmem = 4 * NT < 32 ? 32 : 4 * NT;
    static_assert(kSmem <= 232448, "shared memory");
};

// kind::f8f6f4, A e4m3, B e5m2
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2(int M, int N) { return idesc_e4m3_f32(M, N) | (1u << 10); }

__device__ __forceinline__ void mma_ss_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    tc_mma_bf16(d, a, b, idesc, acc);   // kind::f16; the descriptor names the formats
}

template <int NT>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&x)[NT]) {
    if constexpr (NT == 16) {
        tmem_ld_16_async(addr, x);
    } else {
#pragma unroll
        for (int c = 0; c < NT / 32; ++c) tmem_ld32(addr + 32 * c, reinterpret_cast<uint32_t(&)[32]>(x[32 * c]));
    }
}
template <int NT>
__device__ __forceinline__ void tmem_st_cols(uint32_t addr, const uint32_t (&x)[NT]) {
    if constexpr (NT == 16) {
        tmem_st16(addr, x);
    } else {
#pragma unroll
        for (int c = 0; c < NT / 32; ++c) tmem_st32(addr + 32 * c, reinterpret_cast<const uint32_t(&)[32]>(x[32 * c]));
    }
}

// Sums (or maxima of) v[c] over the warp's lanes: afterwards lane l holds in v[0 .. NT/32) those of
// columns l * NT/32 + i (NT = 16: of column l / 2 in v[0]).  A halving exchange: about NT shuffles in
// all, where a reduction instruction per column took 100 cycles each.  The order is fixed.  N columns
// over lanes FIRST apart and nearer.
template <int N, bool MAX, int FIRST = 16>
__device__ __forceinline__ void warp_columns(float (&v)[N], int lane) {
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int o = FIRST, n = N; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], kept = up ? v[i + n] : v[i];
                    v[i] = join(kept, __shfl_xor_sync(0xFFFFFFFFu, send, o));
                }
            }
        } else {
            v[0] = join(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
        }
    }
}
// The same maxima of x[c] + the lane's own shift; the first exchange goes by x itself, whose registers
// the scores stay in.
template <int NT, bool SHIFT>
__device__ __forceinline__ void warp_maxima(const uint32_t (&x)[NT], float shift, float (&v)[NT / 2], int lane) {
    const bool up = (lane & 16) != 0;
    const float other = SHIFT ? __shfl_xor_sync(0xFFFFFFFFu, shift, 16) : 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) {
        const float kept = __uint_as_float(up ? x[i + NT / 2] : x[i]);
        const float got = __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, up ? x[i] : x[i + NT / 2], 16));
        v[i] = SHIFT ? fmaxf(kept + shift, got + other) : fmaxf(kept, got);
    }
    warp_columns<NT / 2, true, 8>(v, lane);
}
template <int NT, int N>
__device__ __forceinline__ void store_columns(float *to, const float (&v)[N], int lane) {
    if constexpr (NT == 16) {
        if ((lane & 1) == 0) to[lane / 2] = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) to[lane * (NT / 32) + i] = v[i];
    }
}

template <bool F8, int DP, int NT>
__global__ void __launch_bounds__(Lay<F8, DP, NT>::kThreads, 1)
tree_narrow_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ TreeArgs a, int box_rows) {
    using L = Lay<F8, DP, NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    volatile int32_t *const abort_flag = reinterpret_cast<volatile int32_t *>(smem + L::oMisc + 4);
    volatile uint32_t *const v_issued = reinterpret_cast<volatile uint32_t *>(smem + L::oMisc + 8), *const copied = v_issued + 1;
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
            mbar_init(bar(L::bCE + i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::bS + i), 1);
            mbar_init(bar(L::bSFree + i), 4);
            mbar_init(bar(L::bP + i), 4);
            mbar_init(bar(L::bPV + i), 1);
        }
        mbar_init(bar(L::bQ), 8);
        mbar_init(bar(L::bO), 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar(L::bFix + i), 1);
        mbar_init(bar(L::bDrain), 2);
        for (int i = 0; i < kRecords; ++i) mbar_init(bar(L::bW + i), 1);
        *abort_flag = 0;
        *v_issued = copied[0] = copied[1] = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == kScoreWarp) {
        tmem_alloc(base + L::oMisc, L::kTmem);
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
            produce<L, F8, DP, 0, 0>(a, w, &tm_k, &tm_v, smem, box_rows, abort_flag, copied, v_issued, follow);
        } else if (warp == kScoreWarp) {
            // ---------------------------------------------------------------- S^T = K Q^T, tile by tile
            const uint64_t q_desc = desc_kmajor_sw128(base + L::oQ);
            uint32_t c = 0, sc[2] = {0, 0}, items = 0;
            bool ok = true;
            while (ok && walk_follow(a, w, follow, abort_flag)) {
                ok = wait_for(bar(L::bQ), items & 1u, abort_flag, a.err, limit);
                for (int t = 0; ok && t < w.hi - w.lo; ++t, ++c) {
                    const uint32_t slot = c % L::NK, g = t & 1, s_col = tmem + g * NT;
                    // the warpgroup has taken this buffer's previous scores
                    ok = (sc[g] == 0 || wait_for(bar(L::bSFree + g), (sc[g] - 1) & 1u, abort_flag, a.err, limit)) &&
                         wait_for(bar(L::bKF + slot), (c / L::NK) & 1u, abort_flag, a.err, limit);
                    if (!ok) break;
                    ++sc[g];
                    tc_fence_after();
                    const uint64_t k_desc = desc_kmajor_sw128(base + L::oK + slot * L::kKSlot);
                    if (elect_one()) {
                        if (F8) {
#pragma unroll
                            for (int i = 0; i < DP / 32; ++i)
                                tc_mma_f8(s_col, k_desc + 2 * i, q_desc + 2 * i, idesc_e4m3_f32(128, NT), i > 0);
#pragma unroll
                            for (int i = 0; i < DP / 32; ++i)
                                tc_mma_f8(s_col, k_desc + 2 * i, q_desc + NT * 8 + 2 * i, idesc_e4m3_e5m2(128, NT), 1);
                        } else {
#pragma unroll
                            for (int i = 0; i < DP / 16; ++i)   // 64-channel halves
                                tc_mma_bf16(s_col, k_desc + (i / 4) * 1024 + (i % 4) * 2, q_desc + (i / 4) * (NT * 8) + (i % 4) * 2,
                                            idesc_bf16_f32(128, NT), i > 0);
                        }
                        tc_commit(bar(L::bKE + slot));
                        tc_commit(bar(L::bS + g));
                    }
                    __syncwarp();
                }
                ++items;
            }
            // every product is done before the CTA leaves
            if (elect_one()) tc_commit(bar(L::bDrain));
            __syncwarp();
            mbar_wait_drain(bar(L::bDrain), 0, kDrain);
            __syncwarp();
        } else if (warp == kOutWarp) {
            // ---------------------------------------------------------------- O^T += V^T P^T, tile by tile
            // (A warp of its own: a tile's K may come later than the weights of the tile before.)
            uint32_t c = 0, fixes = 0, pc[2] = {0, 0};
            bool ok = true;
            while (ok && walk_follow(a, w, follow, abort_flag)) {
                const int T = w.hi - w.lo;
                for (int t = 0; ok && t < T; ++t, ++c) {
                    const uint32_t slot = c % L::NV, g = t & 1, o_col = tmem + (2 + g) * NT;
                    ok = wait_for(bar(L::bVF + slot), (c / L::NV) & 1u, abort_flag, a.err, limit);
                    if (!F8 && ok && (w.lo + t + 1) * kTile > w.s.ctx) {   // V's cleaner has been over it
                        ok = wait_for(bar(L::bFix + (fixes & 3u)), (fixes >> 2) & 1u, abort_flag, a.err, limit);
                        ++fixes;
                    }
                    // (the first weights of an item come after the previous item's O was read)
                    ok = ok && wait_for(bar(L::bP + g), pc[g] & 1u, abort_flag, a.err, limit);
                    if (!ok) break;
                    ++pc[g];
                    tc_fence_after();
                    const uint64_t v_desc = desc_mn_sw128(base + L::oV + slot * L::kVSlot, DP == 128 ? kTile * 128u : 0u);
                    const uint64_t p_desc = desc_p<NT>(base + L::oP + g * L::kP);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kTile / 16; ++i)   // 16 positions: 2 KB of V's blocks, 2 atoms of P
                            mma_ss_f16(o_col, v_desc + 128 * i, p_desc + (16 * NT * 2 / 16) * i, idesc_vp(NT, F8 ? 0 : 1),
                                       t >= 2 || i > 0);
                        tc_commit(bar(L::bVE + slot));
                        tc_commit(bar(L::bPV + g));
                        if (t == T - 1) tc_commit(bar(L::bO));
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) tc_commit(bar(L::bDrain));
            __syncwarp();
            mbar_wait_drain(bar(L::bDrain), 0, kDrain);
            __syncwarp();
        } else if (warp == kValueWarp) {
            produce<L, F8, DP, 1, 1>(a, w, &tm_k, &tm_v, smem, box_rows, abort_flag, copied, v_issued, follow);
        } else if (warp >= kAuxWarp) {
            if constexpr (F8)
                convert_values<L, DP>(a, w, smem, (warp - kAuxWarp) & 3, (warp - kAuxWarp) >> 2, abort_flag, follow);
            else if (warp == kAuxWarp)   // the other three of its warpgroup are idle
                clean_values<L, DP>(a, w, smem, abort_flag, v_issued, follow);
        }
    } else {
        // ---------------------------------------------------------------- softmax, two warpgroups
        regs_up<L::kSoft>();
        Walk w;
        const int g = warp >> 2, q4 = warp & 3, p = q4 * 32 + lane;   // this thread's position of a tile, and channel of O
        const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t s_addr = tmem + lanes + g * NT, o_addr = tmem + lanes + (2 + g) * NT;
        float *const nm_s = reinterpret_cast<float *>(smem + L::oM) + g * NT;
        float *const alpha_s = reinterpret_cast<float *>(smem + L::oAlpha) + g * NT;
        float *const delta_s = reinterpret_cast<float *>(smem + L::oDelta) + g * NT;
        float *const red_s = reinterpret_cast<float *>(smem + L::oRed) + g * 4 * NT;
        const float *const scale_s = reinterpret_cast<const float *>(smem + L::oScale);
        uint8_t *const p_buf = smem + L::oP + g * L::kP;
        uint32_t sc = 0, tiles = 0;   // this warpgroup's tiles; all tiles
        bool dead = false;            // a wait gave up: only the barriers are kept
        float *const cs_s = reinterpret_cast<float *>(smem + L::oCs);
        uint64_t *const mask_s = reinterpret_cast<uint64_t *>(smem + L::oMask);
        // The next item's queries, 16 bytes a piece, are on their way while an item ends: the lanes of
        // a row are C neighbouring threads.  Rows beyond R are zeros; their columns go nowhere, but
        // their scores have a say in when O is rescaled.
        constexpr int C = DP / 8, PIECES = (NT * C + 255) / 256;
        uint4 queries[PIECES];
        uint64_t next_mask = 0;
        auto fetch = [&](const Walk &v) {
            const int R = v.s.n * G;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int at = static_cast<int>(threadIdx.x) + 256 * i, row = at / C, c = at % C;
                queries[i] = make_uint4(0, 0, 0, 0);
                if (row < R && c * 8 < a.cache.dim)
                    queries[i] = *reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(a.q.ptr) + static_cast<int64_t>(v.s.t0 + row / G) * a.q.token_stride +
                        static_cast<int64_t>(v.hk * G + row % G) * a.q.head_stride + c * 8);
            }
            next_mask = 0;
            const int row = static_cast<int>(threadIdx.x);
            if (row < NT && row < R) {
                next_mask = a.mask != nullptr ? a.mask[v.s.t0 + row / G] : (2ull << (row / G)) - 1ull;
                if (v.s.n < 64) next_mask &= (1ull << v.s.n) - 1ull;
            }
        };
        pdl_wait();
        Walk next;
        bool more = walk_follow(a, next, follow, abort_flag);
        if (more) fetch(next);
        while (true) {
            // the previous item's shared words have been read; everybody leaves together
            if (bar_any(1, 256, dead || *abort_flag != 0) || !more) break;
            w = next;
            const int R = w.s.n * G, T = w.hi - w.lo;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int at = static_cast<int>(threadIdx.x) + 256 * i, row = at / C, c = at % C;
                if (NT * C >= 256 || at < NT * C) {   // whole warps
                    float unscale;
                    store_query<F8, DP>(smem + L::oQ, NT, row, c, queries[i], unscale);
                    if (F8 && c == 0) cs_s[row] = a.scale_log2 * unscale;
                }
            }
            if (threadIdx.x < NT) mask_s[threadIdx.x] = next_mask;
            float m_own = kNone;   // of column p
            bool all_seen = false;
            if (p < NT) nm_s[p] = 0.0f;
            fence_proxy_async_smem();
            warp_arrive(bar(L::bQ));
            named_barrier(4, 256);
            F2 l2[NT / 2];
#pragma unroll
            for (int c = 0; c < NT / 2; ++c) l2[c] = f2(0.0f, 0.0f);
            for (int t = g; t < T; t += 2) {
                const int tt = w.lo + t, pos = tt * kTile + p;
                const bool edge = (tt + 1) * kTile > w.s.ctx;
                const uint32_t no = tiles + t, sb = no % L::NC;
                float ks = 1.0f, vs = 1.0f, lv = 0.0f;   // lv: of the value's scale, in the rows' references
                uint32_t x[NT];
                if (F8 && !dead) dead = !wait_for(bar(L::bCF + sb), (no / L::NC) & 1u, abort_flag, a.err, limit);
                if (!dead) dead = !wait_for(bar(L::bS + g), sc & 1u, abort_flag, a.err, limit);
                tc_fence_after();
                tmem_ld_cols<NT>(s_addr, x);
                if (F8) {
                    ks = scale_s[sb * 384 + p];
                    vs = scale_s[sb * 384 + 128 + p];
                    lv = scale_s[sb * 384 + 256 + p];
                } else {
                    ks = a.scale_log2;
                }
                tmem_wait_ld();
                tc_fence_before();
                if (!dead) {
                    warp_arrive(bar(L::bSFree + g));
                    if (F8) warp_arrive(bar(L::bCE + sb));
                }
                // scores in log2 units above the rows' references so far (above 0 where a row has none);
                // what a row does not see is -inf
                const F2 ks2 = f2(ks, ks);
#pragma unroll
                for (int c = 0; c < NT; c += 4) {
                    const float4 n = *reinterpret_cast<const float4 *>(nm_s + c);
                    F2 s0 = f2(x[c], x[c + 1]), s1 = f2(x[c + 2], x[c + 3]);
                    if (F8) {
                        const float4 k = *reinterpret_cast<const float4 *>(cs_s + c);
                        s0 = f2_fma(f2_mul(s0, ks2), f2(k.x, k.y), f2(n.x, n.y));
                        s1 = f2_fma(f2_mul(s1, ks2), f2(k.z, k.w), f2(n.z, n.w));
                    } else {
                        s0 = f2_fma(s0, ks2, f2(n.x, n.y));
                        s1 = f2_fma(s1, ks2, f2(n.z, n.w));
                    }
                    float s[4];
                    f2_get(s0, s[0], s[1]);
                    f2_get(s1, s[2], s[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[c + i] = __float_as_uint(s[i]);
                }
                if (edge) {
                    const int d = pos - w.s.ctx;   // drafted token; masks have no bits beyond n
                    if (d >= 0) {
#pragma unroll
                        for (int c = 0; c < NT; ++c)
                            if (d >= 64 || !(mask_s[c] >> d & 1ull)) x[c] = __float_as_uint(ninf());
                    }
                }
                // any weight far above its row's largest so far, or a row that had seen nothing?
                bool move = !all_seen;
                float over = ninf();
#pragma unroll
                for (int c = 0; c < NT; c += 2) over = fmaxf(over, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
                move = move || over + lv > kLazy;
                if (bar_any(2 + g, 128, move)) {
                    // the columns' maxima over the 128 positions (NaN left out): over the warp's lanes,
                    // then over the four warps
                    float top[NT / 2];
                    warp_maxima<NT, F8>(x, lv, top, lane);
                    store_columns<NT>(red_s + q4 * NT, top, lane);
                    named_barrier(2 + g, 128);
                    bool unseen = false;
                    if (p < NT) {
                        const float n = nm_s[p];
                        const float here = fmaxf(fmaxf(red_s[p], red_s[NT + p]), fmaxf(red_s[2 * NT + p], red_s[3 * NT + p]));
                        const float mn = fmaxf(m_own, here - n);
                        unseen = mn == kNone;
                        const float n_new = unseen ? 0.0f : -mn;
                        nm_s[p] = n_new;
                        delta_s[p] = n_new - n;
                        alpha_s[p] = ex2(m_own - mn);
                        m_own = mn;
                    }
                    all_seen = !bar_any(2 + g, 128, unseen);
#pragma unroll
                    for (int c = 0; c < NT; c += 4) {
                        const float4 n = *reinterpret_cast<const float4 *>(delta_s + c);
                        float s[4];
                        f2_get(f2_add(f2(x[c], x[c + 1]), f2(n.x, n.y)), s[0], s[1]);
                        f2_get(f2_add(f2(x[c + 2], x[c + 3]), f2(n.z, n.w)), s[2], s[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[c + i] = __float_as_uint(s[i]);
                    }
                    if (t >= 2) {
                        // O so far is complete when the previous product is
                        if (!dead) dead = !wait_for(bar(L::bPV + g), (sc - 1) & 1u, abort_flag, a.err, limit);
                        tc_fence_after();
#pragma unroll
                        for (int c0 = 0; c0 < NT; c0 += 16) {
                            uint32_t o[16];
                            tmem_ld_16_async(o_addr + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                const float2 k = *reinterpret_cast<const float2 *>(alpha_s + c0 + c);
                                l2[(c0 + c) / 2] = f2_mul(l2[(c0 + c) / 2], f2(k.x, k.y));
                                o[c] = __float_as_uint(__uint_as_float(o[c]) * k.x);
                                o[c + 1] = __float_as_uint(__uint_as_float(o[c + 1]) * k.y);
                            }
                            tmem_st16(o_addr + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                // the weights' buffer is free when the previous product has read it
                if (t >= 2 && !dead) dead = !wait_for(bar(L::bPV + g), (sc - 1) & 1u, abort_flag, a.err, limit);
                const F2 vs2 = f2(vs, vs);
#pragma unroll
                for (int c8 = 0; c8 < NT / 8; ++c8) {
                    uint32_t out[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = c8 * 8 + h * 4;
                        float w0, w1, w2, w3;
                        F2 a0 = f2(ex2(__uint_as_float(x[c])), ex2(__uint_as_float(x[c + 1])));
                        F2 a1 = f2(ex2(__uint_as_float(x[c + 2])), ex2(__uint_as_float(x[c + 3])));
                        l2[c / 2] = f2_add(l2[c / 2], a0);
                        l2[c / 2 + 1] = f2_add(l2[c / 2 + 1], a1);
                        if (F8) {
                            a0 = f2_mul(a0, vs2);
                            a1 = f2_mul(a1, vs2);
                        }
                        f2_get(a0, w0, w1);
                        f2_get(a1, w2, w3);
                        out[2 * h] = pack2(w0, w1, F8);
                        out[2 * h + 1] = pack2(w2, w3, F8);
                    }
                    *reinterpret_cast<uint4 *>(p_buf + p_chunk<NT>(p, c8)) = make_uint4(out[0], out[1], out[2], out[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                if (!dead) warp_arrive(bar(L::bP + g));
                ++sc;
            }
            // ------------------------------------------------------------ the item's end
            more = walk_follow(a, next, follow, abort_flag);
            if (more) fetch(next);
            if (!dead) dead = !wait_for(bar(L::bO), static_cast<uint32_t>(w.index) & 1u, abort_flag, a.err, limit);
            tc_fence_after();
            tiles += T;
            float l[NT];
#pragma unroll
            for (int c = 0; c < NT; c += 2) f2_get(l2[c / 2], l[c], l[c + 1]);
            warp_columns<NT, false>(l, lane);
            store_columns<NT>(red_s + q4 * NT, l, lane);
            if (p < NT) nm_s[p] = -m_own;
            named_barrier(4, 256);
            const bool second = T > 1;   // the second warpgroup had a tile
            const float *const m0_s = reinterpret_cast<const float *>(smem + L::oM), *const m1_s = m0_s + NT;
            const float *const red0 = reinterpret_cast<const float *>(smem + L::oRed), *const red1 = red0 + 4 * NT;
            int64_t *const to_s = reinterpret_cast<int64_t *>(smem + L::oTo);
            float *const w0_s = reinterpret_cast<float *>(smem + L::oAlpha), *const w1_s = w0_s + NT;
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.index == 0 ? 0 : 1);
            if (threadIdx.x < NT) {
                const int c = static_cast<int>(threadIdx.x);
                const float ma = -m0_s[c], mb = second ? -m1_s[c] : kNone;
                const float mx = fmaxf(ma, mb), ka = ex2(ma - mx), kb = ex2(mb - mx);
                const float mm = mx == kNone ? ninf() : mx;
                float ll = (red0[c] + red0[NT + c] + red0[2 * NT + c] + red0[3 * NT + c]) * ka;
                if (second) ll += (red1[c] + red1[NT + c] + red1[2 * NT + c] + red1[3 * NT + c]) * kb;
                const bool none = mm == ninf() && ll == 0.0f;
                const float inv = (!w.whole ? 1.0f : (none ? 0.0f : 1.0f / ll)) * (F8 ? 1.0f / kWeightUp : 1.0f);
                w0_s[c] = ka * inv;
                w1_s[c] = second ? kb * inv : 0.0f;
                to_s[c] = static_cast<int64_t>(w.s.t0 + c / G) * a.out.token_stride + static_cast<int64_t>(w.hk * G + c % G) * a.out.head_stride;
                if (c < R) {
                    if (!w.whole)
                        narrow_ml<DP>(a, gridDim.x, slot)[c] = make_float2(mm, ll);
                    else if (a.lse != nullptr)
                        a.lse[static_cast<int64_t>(w.s.t0 + c / G) * a.q.heads + w.hk * G + c % G] =
                            none ? ninf() : (mm + log2f(ll)) * 0.69314718055994531f;
                }
            }
            named_barrier(4, 256);
            // a warpgroup writes half of the rows, a thread one channel of them
            constexpr int H = NT / 2;
            uint32_t oa[H], ob[H];
            if constexpr (H == 8) {
                tmem_ld8(tmem + lanes + 2 * NT + g * H, oa);
                tmem_ld8(tmem + lanes + 3 * NT + g * H, ob);
            } else {
                tmem_ld_cols<H>(tmem + lanes + 2 * NT + g * H, oa);
                tmem_ld_cols<H>(tmem + lanes + 3 * NT + g * H, ob);
            }
            tmem_wait_ld();
            tc_fence_before();
            const uint32_t *const bad = reinterpret_cast<const uint32_t *>(smem + L::oBad) + (w.index & 7) * 8;
            uint32_t any_bad = 0;   // of parts that reach past the context: there the products waited for the words
            if (w.hi * kTile > w.s.ctx) {
#pragma unroll
                for (int i = 0; i < 8; ++i) any_bad |= bad[i];
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int c = g * H + i;
                float o = __uint_as_float(oa[i]) * w0_s[c];
                if (second) o = fmaf(__uint_as_float(ob[i]), w1_s[c], o);
                oa[i] = __float_as_uint(o);
            }
            if (any_bad != 0) {   // non-finite values of drafted tokens, for the rows that see them
#pragma unroll 1
                for (int tt = max(w.lo, w.s.ctx / kTile); tt < w.hi; ++tt)
#pragma unroll 1
                    for (int j = 0; j < kTile; ++j) {
                        if (p >= a.cache.dim || !(bad[(tt & 1) * 4 + j / 32] >> (j & 31) & 1u)) continue;
                        const float v = value_at<F8>(a, w.b, w.hk, tt * kTile + j, p);
                        if (fabsf(v) <= 3.4028234e38f) continue;
                        const int d = tt * kTile + j - w.s.ctx;   // only drafted tokens are marked
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            if (mask_s[g * H + i] >> d & 1ull) oa[i] = __float_as_uint(__uint_as_float(oa[i]) + v);
                    }
            }
            __syncwarp();   // every lane comes here, also those beyond the head's channels
            if (w.whole) {
                // two rows at a time: neighbouring lanes trade, and each stores two channels of one row
                const int odd = lane & 1;
                uint16_t *const out = static_cast<uint16_t *>(a.out.ptr) + (p & ~1);
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float mine = __uint_as_float(odd ? oa[i + 1] : oa[i]);
                    const float other = __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, odd ? oa[i] : oa[i + 1], 1));
                    const int c = g * H + i + odd;
                    if (c < R && p < a.cache.dim)
                        *reinterpret_cast<uint32_t *>(out + to_s[c]) = odd ? pack2(other, mine, false) : pack2(mine, other, false);
                }
            } else if (p < a.cache.dim) {
                float *const po = narrow_out<DP>(a, slot) + p;
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (g * H + i < R) po[(g * H + i) * DP] = __uint_as_float(oa[i]);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducerWarp && *abort_flag != 0) drain_copies<L, F8>(smem, copied);
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

std::mutex g_mu;
bool g_set[64][12];

template <bool F8, int DP, int NT>
cudaError_t launch(const TreeArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                   cudaStream_t s, bool pdl) {
    using L = Lay<F8, DP, NT>;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        bool &set = g_set[dev & 63][(F8 ? 6 : 0) + (DP == 128 ? 3 : 0) + (NT == 16 ? 0 : NT / 32)];
        if (!set) {
            cudaError_t e = cudaFuncSetAttribute(tree_narrow_kernel<F8, DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
            if (e == cudaSuccess) e = check_registers(tree_narrow_kernel<F8, DP, NT>, L::kThreads, L::kRegs);
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
    return cudaLaunchKernelEx(&cfg, tree_narrow_kernel<F8, DP, NT>, tm_k, tm_v, a, rows);
}

template <bool F8, int DP>
cudaError_t by_rows(const TreeArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                    cudaStream_t s, bool pdl) {
    const int R = a.max_tokens * a.group;
    if (R <= 16) return launch<F8, DP, 16>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
    if (R <= 32) return launch<F8, DP, 32>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
    return launch<F8, DP, 64>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
}

}  // namespace

cudaError_t launch_tree_narrow(const TreeArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, cudaStream_t s, bool pdl) {
    const bool f8 = a.cache.dtype == MOE_E4M3;
    if (a.cache.dim <= 64)
        return f8 ? by_rows<true, 64>(a, dev, ctas, rows, tm_k, tm_v, s, pdl) : by_rows<false, 64>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
    return f8 ? by_rows<true, 128>(a, dev, ctas, rows, tm_k, tm_v, s, pdl) : by_rows<false, 128>(a, dev, ctas, rows, tm_k, tm_v, s, pdl);
}

}  // namespace moe
