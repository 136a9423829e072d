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
// (2^-11; a bf16 cache needs bf16 weights, 2^-8), relative to a running power of two.
//
// Every wait is bounded (an abort flag, MOE_ERR_DEVICE_TIMEOUT, then copies and products are
// drained and TMEM is freed).
#include <algorithm>
#include <mutex>

#include "cache_args.cuh"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;                      // rows of an M tile, positions of a K/V tile
constexpr long long kDrain = 400000000ll;       // about 0.2 s
constexpr int kMaxCtas = 256;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kAuxWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;                   // log2 growth of a maximum that O is rescaled for
constexpr float kWeightUp = 128.0f;             // fp16 weights: at most 2^8 * 2^7, flushed below 2^-31

// DP: the head's channels rounded up to 64 or 128.
template <bool F8, int DP>
struct Lay {
    static constexpr int kAuxWarps = F8 ? 4 : 1;   // V converters; the cleaner of V's last tiles
    static constexpr int kThreads = (kAuxWarp + kAuxWarps) * 32;
    static constexpr uint32_t kQTile = F8 ? 2 * 16384 : 128 * DP * 2;
    static constexpr uint32_t kKSlot = F8 ? 16384 : 128 * DP * 2;
    static constexpr uint32_t kVSlot = 128 * DP * 2;
    static constexpr uint32_t kStage = F8 ? 16384 : 0;
    static constexpr int NK = F8 ? 3 : 2, NV = F8 ? 2 : 3, NS = F8 ? 2 : 0;
    static constexpr uint32_t oK = 2 * kQTile, oV = oK + NK * kKSlot, oS = oV + NV * kVSlot;
    static constexpr uint32_t oBar = oS + NS * kStage;
    // barriers: k_full, k_empty, v_full, v_empty, st_full, st_empty, sc_full[2], sc_empty[2],
    // s_full[2], p_ready[2], q_ready, o_full, o_free, v_fix[4], drain
    static constexpr int bKF = 0, bKE = NK, bVF = 2 * NK, bVE = bVF + NV, bSF = bVE + NV, bSE = bSF + NS, bCF = bSE + NS,
                         bCE = bCF + 2, bS = bCE + 2, bP = bS + 2, bQ = bP + 2, bO = bQ + 1, bOF = bO + 1, bFix = bOF + 1,
                         bDrain = bFix + 4, kBars = bDrain + 1;
    static constexpr uint32_t oMisc = oBar + 8 * kBars + 8;        // TMEM address, abort flag, V tiles issued
    static constexpr uint32_t oBad = (oMisc + 16 + 15) & ~15u;     // uint32 [8 items][2 tiles][4]
    static constexpr uint32_t oScale = oBad + 256;                 // F8: float [2][ks, vs][128]
    static constexpr uint32_t oVmax = oScale + (F8 ? 2048 : 0);    // F8: float [2][4]
    static constexpr uint32_t oQs = oVmax + (F8 ? 32 : 0);         // F8: float [2][128], row factors
    static constexpr uint32_t kSmem = oQs + (F8 ? 1024 : 0);
    static_assert(kSmem <= 232448, "shared memory");
};

// ------------------------------------------------------------------ tcgen05 pieces of this kernel
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], 16-bit A and B, fp32 D.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}
// An MN-major operand with the 128-byte swizzle: blocks of 64 16-bit elements (128 bytes) by 8 rows
// of K (1024 bytes), the next 8 rows 1024 bytes on, the next 64 elements `block` bytes on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t block) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
// kind::f16, fp32 D, B MN-major; fmt 0: fp16, 1: bf16
__host__ __device__ constexpr uint32_t idesc_pv(int N, uint32_t fmt) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
// kind::f8f6f4, A e5m2 (format 1), B e4m3 (0), both K-major
__host__ __device__ constexpr uint32_t idesc_e5m2_e4m3(int M, int N) { return idesc_e4m3_f32(M, N) | (1u << 7); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float ninf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool f16) {
    uint32_t r;
    if (f16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Barrier over the 256 softmax threads that also ORs a predicate, so that all of them leave a loop
// together.
__device__ __forceinline__ bool softmax_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// Bounded warp-wide wait until *p has reached v, under mbar_wait's rules.
__device__ __forceinline__ bool wait_count(const volatile uint32_t *p, uint32_t v, volatile int32_t *abort, int32_t *err,
                                           long long limit) {
    const long long t0 = clock64();
    while (!__all_sync(0xFFFFFFFFu, static_cast<int32_t>(*p - v) >= 0)) {
        const bool late = clock64() - t0 > limit;
        if (__any_sync(0xFFFFFFFFu, late || *abort != 0)) {
            if (late) {
                *abort = 1;
                record_error(err, MOE_ERR_DEVICE_TIMEOUT);
            }
            return false;
        }
    }
    __threadfence_block();
    return true;
}

// ------------------------------------------------------------------ the work list
struct Seq {
    int t0, n, ctx, len, tiles, pairs;
    bool bad;
};
__device__ __forceinline__ Seq load_seq(const TreeArgs &a, int b) {
    Seq s;
    s.t0 = a.q_start[b];
    const long long n = static_cast<long long>(a.q_start[b + 1]) - s.t0;
    s.ctx = a.ctx[b];
    const long long len = s.ctx + n;
    s.bad = s.ctx < 0 || n < 0 || n > a.max_tokens || s.t0 < 0 || s.t0 > a.tokens - n ||
            len > static_cast<long long>(a.max_pages) * a.cache.page;
    s.n = s.bad ? 0 : static_cast<int>(n);
    s.len = s.bad ? 0 : static_cast<int>(len);
    s.tiles = (s.len + kTile - 1) / kTile;
    s.pairs = (s.n * a.group + 2 * kTile - 1) / (2 * kTile);
    return s;
}
__device__ __forceinline__ long long seq_work(const TreeArgs &a, const Seq &s) {
    return static_cast<long long>(a.cache.heads) * s.pairs * s.tiles;
}
// The list is cut for at most as many CTAs as it has tiles, so that no range is empty (the join
// reads a part of every CTA between an item's first and last).
__device__ __forceinline__ int used_ctas(long long W, int ctas) { return static_cast<int>(min(W, static_cast<long long>(ctas))); }
// First tile of CTA c's range, and the CTA whose range holds tile x.
__device__ __forceinline__ long long range_lo(long long W, int c, int C) { return W * c / C; }
__device__ __forceinline__ int range_of(long long W, long long x, int C) {
    return static_cast<int>(((x + 1) * C - 1) / W);
}

// A CTA's walk over its range: item by item, the part [lo, hi) of the item's position tiles.
struct Walk {
    Seq s;
    long long at, end, item0;   // next tile of the list, the range's end, the item's first tile
    int b, hk, pair, lo, hi;
    bool whole;                 // the item lies in this CTA alone
    int index;                  // items walked before
};
// The whole warp calls these; the outcome is uniform.
__device__ __forceinline__ void walk_begin(const TreeArgs &a, Walk &w, bool report) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    long long total = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        long long x = 0;
        if (b0 + lane < a.seqs) {
            const Seq s = load_seq(a, b0 + lane);
            if (s.bad && report) record_error(a.err, MOE_ERR_BAD_ID);
            x = seq_work(a, s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        total += x;
    }
    const int C = used_ctas(total, gridDim.x), c = static_cast<int>(blockIdx.x);
    w.at = c < C ? range_lo(total, c, C) : 0;
    w.end = c < C ? range_lo(total, c + 1, C) : 0;
    w.index = -1;
    w.b = 0;
    w.hk = 0;
    w.pair = 0;
    w.item0 = 0;
    if (w.at >= w.end) return;
    long long before = 0;   // tiles of the sequences before
    for (int b0 = 0;; b0 += 32) {
        long long x = 0;
        if (b0 + lane < a.seqs) x = seq_work(a, load_seq(a, b0 + lane));
        long long incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + incl > w.at);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            w.b = b0 + l;
            before += __shfl_sync(0xFFFFFFFFu, incl - x, l);
            break;
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    w.s = load_seq(a, w.b);
    const long long item = (w.at - before) / w.s.tiles;
    w.item0 = before + item * w.s.tiles;
    w.hk = static_cast<int>(item / w.s.pairs);
    w.pair = static_cast<int>(item % w.s.pairs);
}
// Sets the next item's part; false at the end of the range.
__device__ __forceinline__ bool walk_next(const TreeArgs &a, Walk &w) {
    if (w.at >= w.end) return false;
    if (w.index >= 0) {   // step to the item at w.at
        w.item0 += w.s.tiles;
        if (++w.pair == w.s.pairs) {
            w.pair = 0;
            if (++w.hk == a.cache.heads) {
                w.hk = 0;
                do {
                    w.s = load_seq(a, ++w.b);
                } while (w.s.tiles == 0 || w.s.pairs == 0);   // there is work left, so one follows
            }
        }
    }
    ++w.index;
    w.lo = static_cast<int>(w.at - w.item0);
    const long long stop = min(w.end, w.item0 + w.s.tiles);
    w.hi = static_cast<int>(stop - w.item0);
    w.whole = w.lo == 0 && w.hi == w.s.tiles;
    w.at = stop;
    return true;
}

// Partial results: per CTA two slots (its first item, its last), each [2 M tiles][DP / 4][128
// rows][4] fp32 of unnormalised output, then, after all slots, [slot][2][128] (maximum, sum).
template <int DP>
__device__ __forceinline__ float4 *part_out(const TreeArgs &a, int slot, int mt) {
    return reinterpret_cast<float4 *>(a.part) + (static_cast<size_t>(slot) * 2 + mt) * (DP / 4) * kTile;
}
template <int DP>
__device__ __forceinline__ float2 *part_ml(const TreeArgs &a, int ctas, int slot, int mt) {
    return reinterpret_cast<float2 *>(reinterpret_cast<float4 *>(a.part) + static_cast<size_t>(ctas) * 4 * (DP / 4) * kTile) +
           (static_cast<size_t>(slot) * 2 + mt) * kTile;
}

// Element offset of the row of position pos of sequence b, head hk; -1 for a page outside the cache.
__device__ __forceinline__ int64_t row_offset(const TreeArgs &a, int b, int hk, int pos, int &page, int &at) {
    page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / a.cache.page];
    at = pos % a.cache.page;
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.pages)) return -1;
    return page * a.cache.page_stride + at * a.cache.token_stride + hk * a.cache.head_stride;
}

// Which of the 128 positions of tile tt a row sees: bit j of word j / 32.  M: the row's tree mask.
__device__ __forceinline__ void seen_bits(uint64_t M, const Seq &s, int tt, uint32_t (&w)[4]) {
    if (s.n < 64) M &= (1ull << s.n) - 1ull;
    const int base = tt * kTile - s.ctx;   // drafted token of the tile's first position
    uint64_t lo, hi = 0;
    if (base >= 0) {
        lo = base < 64 ? M >> base : 0ull;
    } else {
        const int sh = -base;
        if (sh < 64) {
            lo = M << sh | ((1ull << sh) - 1ull);
            hi = M >> (64 - sh);
        } else {
            lo = ~0ull;
            hi = sh >= 128 ? ~0ull : (M << (sh - 64) | ((1ull << (sh - 64)) - 1ull));
        }
    }
    w[0] = static_cast<uint32_t>(lo);
    w[1] = static_cast<uint32_t>(lo >> 32);
    w[2] = static_cast<uint32_t>(hi);
    w[3] = static_cast<uint32_t>(hi >> 32);
}

__device__ __forceinline__ float f16_of(uint32_t h) {
    float r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return h;
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
    volatile uint32_t *const v_issued = reinterpret_cast<volatile uint32_t *>(smem + L::oMisc + 8);
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const long long limit = a.wait_limit;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NK; ++i) {
            mbar_init(bar(L::bKF + i), 1);
            mbar_init(bar(L::bKE + i), 1);
        }
        for (int i = 0; i < L::NV; ++i) {
            mbar_init(bar(L::bVF + i), F8 ? 4 : 1);
            mbar_init(bar(L::bVE + i), 1);
        }
        for (int i = 0; i < L::NS; ++i) {
            mbar_init(bar(L::bSF + i), 1);
            mbar_init(bar(L::bSE + i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::bCF + i), 4);
            mbar_init(bar(L::bCE + i), 8);
            mbar_init(bar(L::bS + i), 1);
            mbar_init(bar(L::bP + i), 4);
        }
        mbar_init(bar(L::bQ), 8);
        mbar_init(bar(L::bO), 1);
        mbar_init(bar(L::bOF), 8);
        for (int i = 0; i < 4; ++i) mbar_init(bar(L::bFix + i), 1);
        mbar_init(bar(L::bDrain), 1);
        *abort_flag = 0;
        *v_issued = 0;
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
    pdl_wait();
    pdl_trigger();

    Walk w;
    walk_begin(a, w, blockIdx.x == 0 && warp == kMmaWarp);
    const int G = a.group;

    if (warp == kProducerWarp) {
        // ---------------------------------------------------------------- K and V copies
        const int boxes = kTile / box_rows;   // at most 16, one lane each
        uint32_t cnt = 0;
        bool ok = true;
        while (ok && walk_next(a, w)) {
            for (int tt = w.lo; tt < w.hi; ++tt, ++cnt) {
                // the lane's box: its page, read before the waits
                const int pos = tt * kTile + lane * box_rows;
                const bool mine = lane < boxes && pos < w.s.len;
                int page = 0;
                if (mine) {
                    page = a.page_table[static_cast<int64_t>(w.b) * a.max_pages + pos / a.cache.page];
                    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.pages)) {
                        record_error(a.err, MOE_ERR_BAD_ID);
                        page = a.cache.pages;   // beyond the tensor: the copy writes zeros
                    }
                }
                const int row = pos % a.cache.page;
                const uint32_t n_boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
                constexpr uint32_t kRowBytes = F8 ? 128 : DP * 2;
                const uint32_t bytes = n_boxes * box_rows * kRowBytes;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    constexpr int NV = F8 ? L::NS : L::NV;
                    const uint32_t slot = v ? cnt % NV : cnt % L::NK, use = v ? cnt / NV : cnt / L::NK;
                    const uint32_t full = bar((v ? (F8 ? L::bSF : L::bVF) : L::bKF) + slot);
                    const uint32_t empty = bar((v ? (F8 ? L::bSE : L::bVE) : L::bKE) + slot);
                    const uint32_t dst = base + (v ? (F8 ? L::oS + slot * L::kStage : L::oV + slot * L::kVSlot)
                                                   : L::oK + slot * L::kKSlot);
                    if (!warp_wait(empty, (use & 1u) ^ 1u, abort_flag, a.err, limit)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (mine) {
                        const CUtensorMap *tm = v ? &tm_v : &tm_k;
                        const uint32_t d = dst + static_cast<uint32_t>(lane * box_rows) * 128u;
                        tma_load_4d(d, tm, full, 0, row, w.hk, page);
                        if (!F8 && DP == 128) tma_load_4d(d + kTile * 128u, tm, full, 64, row, w.hk, page);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (!F8 && lane == 0) {
                    __threadfence_block();
                    *v_issued = cnt + 1;
                }
            }
        }
        if (*abort_flag != 0) {   // copies nobody waited for must land before the CTA leaves
            constexpr int NV = F8 ? L::NS : L::NV;
            for (uint32_t j = cnt > L::NK ? cnt - L::NK : 0; j <= cnt; ++j)
                mbar_wait_drain(bar(L::bKF + j % L::NK), (j / L::NK) & 1u, j == cnt ? 1000000 : kDrain);
            for (uint32_t j = cnt > NV ? cnt - NV : 0; j < cnt; ++j)
                mbar_wait_drain(bar((F8 ? L::bSF : L::bVF) + j % NV), (j / NV) & 1u, kDrain);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- products
        uint32_t kc = 0, vc = 0, pc[2] = {0, 0}, fixes = 0, items = 0;
        bool ok = true;
        while (ok && walk_next(a, w)) {
            const bool two = w.s.n * G - w.pair * 2 * kTile > kTile;
            const int T = w.hi - w.lo, U = two ? 2 * T : T;
            ok = warp_wait(bar(L::bQ), items & 1u, abort_flag, a.err, limit);
            auto qk = [&](int u) {
                const int g = u & 1;
                const uint32_t slot = kc % L::NK;
                if (!two || g == 0) ok = warp_wait(bar(L::bKF + slot), (kc / L::NK) & 1u, abort_flag, a.err, limit);
                if (!ok) return;
                tc_fence_after();
                const bool last = !two || g == 1;
                if (elect_one()) {
                    const uint32_t q = base + (two ? g : 0) * L::kQTile, k = base + L::oK + slot * L::kKSlot;
                    const uint32_t d = tmem + g * kTile;
                    if (F8) {
#pragma unroll
                        for (int i = 0; i < DP / 32; ++i)
                            tc_mma_f8(d, desc_kmajor_sw128(q + 32u * i), desc_kmajor_sw128(k + 32u * i),
                                      idesc_e4m3_f32(128, 128), i > 0);
#pragma unroll
                        for (int i = 0; i < DP / 32; ++i)
                            tc_mma_f8(d, desc_kmajor_sw128(q + 16384u + 32u * i), desc_kmajor_sw128(k + 32u * i),
                                      idesc_e5m2_e4m3(128, 128), 1);
                    } else {
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            const uint32_t o = (i / 4) * (kTile * 128u) + (i % 4) * 32u;
                            tc_mma_bf16(d, desc_kmajor_sw128(q + o), desc_kmajor_sw128(k + o), idesc_bf16_f32(128, 128),
                                        i > 0);
                        }
                    }
                    if (last) tc_commit(bar(L::bKE + slot));
                    tc_commit(bar(L::bS + g));
                }
                __syncwarp();
                if (last) ++kc;
            };
            for (int u = 0; ok && u < min(2, U); ++u) qk(u);
            for (int u = 0; ok && u < U; ++u) {
                const int g = u & 1, tt = w.lo + (two ? u >> 1 : u);
                const uint32_t slot = vc % L::NV;
                if (!two || g == 0) {
                    ok = warp_wait(bar(L::bVF + slot), (vc / L::NV) & 1u, abort_flag, a.err, limit);
                    if (!F8 && (tt + 1) * kTile > w.s.ctx) {   // V's cleaner has been over it
                        ok = ok && warp_wait(bar(L::bFix + (fixes & 3u)), (fixes >> 2) & 1u, abort_flag, a.err, limit);
                        ++fixes;
                    }
                }
                // O of the previous item has been read
                if (ok && u == 0 && items > 0) ok = warp_wait(bar(L::bOF), (items - 1) & 1u, abort_flag, a.err, limit);
                ok = ok && warp_wait(bar(L::bP + g), pc[g] & 1u, abort_flag, a.err, limit);
                if (!ok) break;
                ++pc[g];
                tc_fence_after();
                const bool last = !two || g == 1;
                if (elect_one()) {
                    const uint32_t v = base + L::oV + slot * L::kVSlot;
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        mma_ts(tmem + 256 + g * DP, tmem + g * kTile + 8 * i, desc_mn_sw128(v + 2048u * i, kTile * 128u),
                               idesc_pv(DP, F8 ? 0 : 1), u >= 2 || i > 0);
                    if (last) tc_commit(bar(L::bVE + slot));
                    if (u == U - 1) tc_commit(bar(L::bO));
                }
                __syncwarp();
                if (last) ++vc;
                if (u + 2 < U) qk(u + 2);
            }
            ++items;
        }
        // every product is done before the CTA leaves
        if (elect_one()) {
            tc_commit(bar(L::bDrain));
            mbar_wait_drain(bar(L::bDrain), 0, kDrain);
        }
        __syncwarp();
    } else if (warp >= kAuxWarp) {
        uint32_t *const bad_all = reinterpret_cast<uint32_t *>(smem + L::oBad);
        const uint32_t full_mask = 0xFFFFFFFFu;
        if constexpr (!F8) {
            // ------------------------------------------------------------ V's cleaner
            // Positions beyond the length become zeros (their weights are 0, what the cache holds
            // there may be anything), and so do non-finite elements of drafted tokens: a row that
            // does not see such a token must not meet it in the product.  Rows that do get it added
            // at the end of the item (bad bits).
            uint32_t cnt = 0, fixes = 0;
            bool ok = true;
            while (ok && walk_next(a, w)) {
                uint32_t *const bad = bad_all + (w.index & 7) * 8;
                if (lane < 8) bad[lane] = 0;
                __syncwarp();
                for (int tt = w.lo; tt < w.hi; ++tt, ++cnt) {
                    if ((tt + 1) * kTile <= w.s.ctx) continue;
                    const uint32_t slot = cnt % L::NV;
                    // only the last tiles are waited for here, so the slot may be some uses behind:
                    // its parity tells this use from the one before once this one was issued
                    if (!wait_count(v_issued, cnt + 1, abort_flag, a.err, limit) ||
                        !warp_wait(bar(L::bVF + slot), (cnt / L::NV) & 1u, abort_flag, a.err, limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t *const v = smem + L::oV + slot * L::kVSlot;
                    constexpr int C = DP / 8;   // 16-byte chunks of a row; 32 / C rows at a time
                    const int c = lane % C;
                    const int first = max(0, w.s.ctx - tt * kTile), stop = min(kTile, w.s.len - tt * kTile);
                    for (int r0 = first / (32 / C) * (32 / C); r0 < kTile; r0 += 32 / C) {
                        const int r = r0 + lane / C;
                        uint4 *const p = reinterpret_cast<uint4 *>(v + (c / 8) * (kTile * 128) + r * 128 + (c % 8) * 16);
                        if (r >= stop) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else if (r >= first) {
                            uint4 x = *p;
                            uint32_t *const q = reinterpret_cast<uint32_t *>(&x);
                            bool hit = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((q[i] & 0x7F80u) == 0x7F80u) {
                                    q[i] &= 0xFFFF0000u;
                                    hit = true;
                                }
                                if ((q[i] & 0x7F800000u) == 0x7F800000u) {
                                    q[i] &= 0x0000FFFFu;
                                    hit = true;
                                }
                            }
                            if (hit) {
                                *p = x;
                                atomicOr(&bad[(tt & 1) * 4 + r / 32], 1u << (r & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __threadfence_block();
                    warp_arrive(bar(L::bFix + (fixes & 3u)));   // at most NV = 3 ahead of the products
                    ++fixes;
                }
            }
        } else {
            // ------------------------------------------------------------ V's converters
            const int cw = warp - kAuxWarp, j = cw * 32 + lane;   // this thread's position of a tile
            float *const scale_s = reinterpret_cast<float *>(smem + L::oScale);
            float *const vmax_s = reinterpret_cast<float *>(smem + L::oVmax);
            uint32_t cnt = 0;
            bool ok = true;
            while (ok && walk_next(a, w)) {
                uint32_t *const bad = bad_all + (w.index & 7) * 8;
                if (lane < 2) bad[lane * 4 + cw] = 0;   // a warp's words are its own
                __syncwarp();
                auto scales = [&](int tt, float &ks, float &vs) {
                    const int pos = tt * kTile + j;
                    ks = vs = 0.0f;
                    if (tt < w.hi && pos < w.s.len) {
                        const int page = a.page_table[static_cast<int64_t>(w.b) * a.max_pages + pos / a.cache.page];
                        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.cache.pages)) {
                            const int64_t o = (static_cast<int64_t>(page) * a.cache.heads + w.hk) * a.cache.page + pos % a.cache.page;
                            ks = __ldg(a.cache.k_scale + o);
                            vs = __ldg(a.cache.v_scale + o);
                        }
                    }
                };
                float ks, vs;
                scales(w.lo, ks, vs);
                for (int tt = w.lo; tt < w.hi; ++tt, ++cnt) {
                    float ks1, vs1;
                    scales(tt + 1, ks1, vs1);   // in flight during this tile
                    const int first = max(0, w.s.ctx - tt * kTile), stop = min(kTile, w.s.len - tt * kTile);
                    const bool drafted = j >= first && j < stop;
                    const bool odd_scale = drafted && !(fabsf(vs) <= 3.4028234e38f);
                    const uint32_t sb = cnt & 1u;
                    if (!(ok = warp_wait(bar(L::bCE + sb), ((cnt >> 1) & 1u) ^ 1u, abort_flag, a.err, limit))) break;
                    scale_s[sb * 256 + j] = ks;
                    scale_s[sb * 256 + 128 + j] = odd_scale ? 0.0f : vs;
                    float mx = fabsf(vs) <= 3.4028234e38f ? fabsf(vs) : 0.0f;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(full_mask, mx, o));
                    if (lane == 0) vmax_s[sb * 4 + cw] = mx;
                    if (odd_scale) atomicOr(&bad[(tt & 1) * 4 + cw], 1u << lane);
                    warp_arrive(bar(L::bCF + sb));
                    const uint32_t ss = cnt % L::NS, slot = cnt % L::NV;
                    if (!(ok = warp_wait(bar(L::bSF + ss), (cnt / L::NS) & 1u, abort_flag, a.err, limit))) break;
                    if (!(ok = warp_wait(bar(L::bVE + slot), ((cnt / L::NV) & 1u) ^ 1u, abort_flag, a.err, limit))) break;
                    const uint8_t *const src = smem + L::oS + ss * L::kStage;
                    uint8_t *const dst = smem + L::oV + slot * L::kVSlot;
                    // a warp converts 32 rows, 4 (8) rows of 128 (64) codes a step: 16 codes per lane
                    constexpr int C = DP / 16, RS = 32 / C;
                    const int c = lane % C;
#pragma unroll 4
                    for (int i = 0; i < 32 / RS; ++i) {
                        const int r = cw * 32 + i * RS + lane / C;
                        uint4 x = *reinterpret_cast<const uint4 *>(src + r * 128 + c * 16);
                        if (r >= first) {   // the tile's part past the context
                            uint32_t *const q = reinterpret_cast<uint32_t *>(&x);
                            if (r >= stop) {
                                x = make_uint4(0, 0, 0, 0);
                            } else {
                                bool hit = false;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        if ((q[k] >> (8 * y) & 0x7Fu) == 0x7Fu) {
                                            q[k] &= ~(0xFFu << (8 * y));
                                            hit = true;
                                        }
                                if (hit) atomicOr(&bad[(tt & 1) * 4 + r / 32], 1u << (r & 31));
                            }
                        }
                        const uint4 lo = make_uint4(e4m3x2_to_f16x2(x.x & 0xFFFFu), e4m3x2_to_f16x2(x.x >> 16),
                                                    e4m3x2_to_f16x2(x.y & 0xFFFFu), e4m3x2_to_f16x2(x.y >> 16));
                        const uint4 hi = make_uint4(e4m3x2_to_f16x2(x.z & 0xFFFFu), e4m3x2_to_f16x2(x.z >> 16),
                                                    e4m3x2_to_f16x2(x.w & 0xFFFFu), e4m3x2_to_f16x2(x.w >> 16));
                        // 64-channel halves; the halves' lanes store their two chunks in opposite
                        // order, so that a step's eight lanes of a row meet eight bank groups
                        uint8_t *const row = dst + (c / 4) * (kTile * 128) + r * 128;
                        const int u = (c % 4) * 2, sw = c / 4;
                        *reinterpret_cast<uint4 *>(row + (((u + sw) ^ (r & 7)) * 16)) = sw ? hi : lo;
                        *reinterpret_cast<uint4 *>(row + (((u + 1 - sw) ^ (r & 7)) * 16)) = sw ? lo : hi;
                    }
                    fence_proxy_async_smem();
                    __threadfence_block();
                    warp_arrive(bar(L::bSE + ss));
                    warp_arrive(bar(L::bVF + slot));
                    ks = ks1;
                    vs = vs1;
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax, two warpgroups
        const int g = warp >> 2, r = (warp & 3) * 32 + lane;   // lane quarter = warp % 4
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + g * kTile, o_addr = tmem + lanes + 256 + g * DP;
        float *const qs = reinterpret_cast<float *>(smem + L::oQs);
        const float *const scale_s = reinterpret_cast<const float *>(smem + L::oScale);
        const volatile float *const vmax_s = reinterpret_cast<const volatile float *>(smem + L::oVmax);
        float4 *const exch = reinterpret_cast<float4 *>(smem);   // [2][128], over Q when Q is done with
        uint32_t sc = 0, scnt = 0;
        bool ok = true;
        while (true) {
            const bool more = walk_next(a, w);
            // the previous item's exchange has been read; everybody leaves together
            if (softmax_any(!ok || *abort_flag != 0) || !more) break;
            const int R = w.s.n * G, row0 = w.pair * 2 * kTile;
            const bool two = R - row0 > kTile;
            const int T = w.hi - w.lo, U = two ? 2 * T : T;
            // Q rows into shared memory: 16-byte chunks (8 channels), zeros beyond the rows
            {
                constexpr int C = DP / 8;
                const int tiles = two ? 2 : 1;
                for (int i = static_cast<int>(threadIdx.x); i < tiles * kTile * C; i += 256) {
                    const int c = i % C, rr = i / C, mt = rr / kTile, lr = rr % kTile;
                    const int row = row0 + rr;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < R && c * 8 < a.cache.dim)
                        x = *reinterpret_cast<const uint4 *>(
                            static_cast<const uint16_t *>(a.q.ptr) + static_cast<int64_t>(w.s.t0 + row / G) * a.q.token_stride +
                            static_cast<int64_t>(w.hk * G + row % G) * a.q.head_stride + c * 8);
                    uint8_t *const q = smem + mt * L::kQTile;
                    if (!F8) {
                        *reinterpret_cast<uint4 *>(q + (c / 8) * (kTile * 128) + lr * 128 + (((c % 8) ^ (lr & 7)) * 16)) = x;
                    } else {
                        // the row's largest exponent over its C lanes (bf16 magnitudes order as integers)
                        const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
                        uint32_t top = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = max(top, max(wd[k] & 0x7FFFu, wd[k] >> 16 & 0x7FFFu));
#pragma unroll
                        for (int o = C / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                        const int e = static_cast<int>(top >> 7);   // biased exponent; 255: not finite
                        // up = 2^(7 - (e - 127)): the largest lands in [128, 256); exponents of the two
                        // factors stay in range by going to at most 2^126
                        const int ub = min(max(127 + 134 - e, 1), 253);
                        const float up = __int_as_float(ub << 23);
                        if (c == 0) qs[mt * 128 + lr] = e == 255 ? __int_as_float(0x7fffffff) : __int_as_float((254 - ub) << 23);
                        uint16_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x0 = bf16_lo(wd[k]) * up, x1 = bf16_hi(wd[k]) * up;
                            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi[k]) : "f"(x1), "f"(x0));
                            const uint32_t h = e4m3x2_to_f16x2(hi[k]);
                            const float r0 = x0 - f16_of(h), r1 = x1 - f16_of(h >> 16);
                            asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo[k]) : "f"(r1), "f"(r0));
                        }
                        uint8_t *const p = q + lr * 128 + (((c / 2) ^ (lr & 7)) * 16) + (c & 1) * 8;
                        *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0] | static_cast<uint32_t>(hi[1]) << 16, hi[2] | static_cast<uint32_t>(hi[3]) << 16);
                        *reinterpret_cast<uint2 *>(p + 16384) = make_uint2(lo[0] | static_cast<uint32_t>(lo[1]) << 16, lo[2] | static_cast<uint32_t>(lo[3]) << 16);
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
            float m = ninf(), l = 0.0f, sigma = 7.888609e-31f;   // 2^-100: below any value scale that counts
            for (int u = g; u < U; u += 2) {
                const int tt = w.lo + (two ? u >> 1 : u);
                const bool edge = (tt + 1) * kTile > w.s.ctx;
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
                if (edge) seen_bits(M, w.s, tt, see);
                const uint32_t tile_no = scnt + (two ? u >> 1 : u), sb = tile_no & 1u;
                const float *const ks = scale_s + sb * 256, *const vs = ks + 128;
                if (F8 && !(ok = warp_wait(bar(L::bCF + sb), (tile_no >> 1) & 1u, abort_flag, a.err, limit))) break;
                if (!(ok = warp_wait(bar(L::bS + g), sc & 1u, abort_flag, a.err, limit))) break;
                ++sc;
                tc_fence_after();
                // the tile's maximum
                float mx = ninf();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32(s_addr + 32 * c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float s = __uint_as_float(x[i]);
                        if (F8) s *= ks[32 * c + i];
                        if (edge && !(see[c] >> i & 1u)) s = ninf();
                        mx = fmaxf(mx, s);
                    }
                }
                mx *= cs;   // cs > 0; -inf stays
                float keep = 1.0f;
                bool move = u < 2 || mx - m > kLazy;
                float sigma_new = sigma;
                if (F8) {
                    const float vm = fmaxf(fmaxf(vmax_s[sb * 4], vmax_s[sb * 4 + 1]), fmaxf(vmax_s[sb * 4 + 2], vmax_s[sb * 4 + 3]));
                    if (vm > sigma) {   // the power of two at or above it
                        sigma_new = __int_as_float(min((__float_as_int(vm) + 0x7fffff) & 0x7f800000, 0x7e800000));
                        move = true;
                    }
                }
                if (__any_sync(0xFFFFFFFFu, move)) {
                    const float mn = fmaxf(m, mx);
                    if (u >= 2) {
                        keep = mn == ninf() ? 1.0f : ex2(m - mn);
                        l *= keep;
                        const float f = F8 ? keep * (sigma / sigma_new) : keep;
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t x[32];
                            tmem_ld32(o_addr + 32 * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            tmem_st32(o_addr + 32 * c, x);
                        }
                    }
                    m = mn;
                    sigma = sigma_new;
                }
                const float ref = m == ninf() ? 0.0f : m;   // nothing seen yet: every weight is 0
                const float unit = F8 ? kWeightUp / sigma : 1.0f;
                float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32], p[16];
                    tmem_ld32(s_addr + 32 * c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float s0 = __uint_as_float(x[2 * i]), s1 = __uint_as_float(x[2 * i + 1]);
                        if (F8) {
                            s0 *= ks[32 * c + 2 * i];
                            s1 *= ks[32 * c + 2 * i + 1];
                        }
                        float p0 = ex2(fmaf(s0, cs, -ref)), p1 = ex2(fmaf(s1, cs, -ref));
                        if (edge) {
                            if (!(see[c] >> (2 * i) & 1u)) p0 = 0.0f;
                            if (!(see[c] >> (2 * i + 1) & 1u)) p1 = 0.0f;
                        }
                        l0 += p0;
                        l1 += p1;
                        if (F8) {
                            p0 *= vs[32 * c + 2 * i] * unit;
                            p1 *= vs[32 * c + 2 * i + 1] * unit;
                        }
                        p[i] = pack2(p0, p1, F8);
                    }
                    tmem_st16(s_addr + 16 * c, p);   // over columns of S already read
                }
                l += l0 + l1;
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(L::bP + g));
                if (F8) warp_arrive_cnt(bar(L::bCE + sb), two ? 1 : 2);
            }
            // ------------------------------------------------------------ the item's end
            ok = ok && warp_wait(bar(L::bO), static_cast<uint32_t>(w.index) & 1u, abort_flag, a.err, limit);
            tc_fence_after();
            scnt += T;
            const float gain = F8 ? sigma / kWeightUp : 1.0f;   // of the accumulator
            float wt[2] = {0.0f, 0.0f}, mm = m, ll = l;
            int c0 = 0, c1 = DP;
            if (!two) {   // both warpgroups hold a part of the same rows: half of the channels each
                exch[g * 128 + r] = make_float4(m, l, gain, 0.0f);
                named_barrier(3, 256);
                const float4 e0 = exch[r], e1 = exch[128 + r];
                mm = fmaxf(e0.x, e1.x);
                const float ref = mm == ninf() ? 0.0f : mm;
                const float k0 = ex2(e0.x - ref), k1 = ex2(e1.x - ref);
                ll = e0.y * k0 + e1.y * k1;
                wt[0] = k0 * e0.z;
                wt[1] = k1 * e1.z;
                c0 = g * (DP / 2);
                c1 = c0 + DP / 2;
            } else {
                wt[g] = gain;
            }
            const bool none = mm == ninf() && ll == 0.0f;
            const float inv = none ? 0.0f : 1.0f / ll;
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.index == 0 ? 0 : 1);
            const uint32_t *const bad = reinterpret_cast<const uint32_t *>(smem + L::oBad) + (w.index & 7) * 8;
            uint32_t any_bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) any_bad |= bad[i];
            const int64_t out_off = static_cast<int64_t>(token) * a.out.token_stride + static_cast<int64_t>(head) * a.out.head_stride;
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
                    for (int tt = max(w.lo, w.s.ctx / kTile); tt < w.hi; ++tt) {
                        uint32_t see[4];
                        seen_bits(M, w.s, tt, see);
                        for (int j = 0; j < kTile; ++j) {
                            if (!(bad[(tt & 1) * 4 + j / 32] >> (j & 31) & 1u) || !(see[j / 32] >> (j & 31) & 1u)) continue;
                            int page, at;
                            const int64_t off = row_offset(a, w.b, w.hk, tt * kTile + j, page, at);
                            if (off < 0) continue;
                            const float vsc = F8 ? a.cache.v_scale[(static_cast<int64_t>(page) * a.cache.heads + w.hk) * a.cache.page + at] : 1.0f;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (c + i >= a.cache.dim) continue;
                                const float x = F8 ? f16_of(e4m3x2_to_f16x2(static_cast<const uint8_t *>(a.cache.v)[off + c + i])) * vsc
                                                   : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.cache.v)[off + c + i]) << 16);
                                if (!(fabsf(x) <= 3.4028234e38f)) o[i] += x;
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
            __syncwarp();
            tc_fence_before();
            warp_arrive(bar(L::bOF));
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
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ joining the parts
// One CTA per 32 rows of a (sequence, cache head): for an item that several CTAs of the first
// kernel shared, out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over its parts in order.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

template <int DP>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a, int ctas) {
    __shared__ long long red[2][kJoinThreads / 32];
    __shared__ float wt[kMaxCtas + 1][kJoinRows];
    const int b = blockIdx.z, hk = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the lengths are no product of the first kernel, which waited for what came before it
    long long before = 0, total = 0;
    for (int i = threadIdx.x; i < a.seqs; i += kJoinThreads) {
        const long long x = seq_work(a, load_seq(a, i));
        total += x;
        if (i < b) before += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
    if (lane == 0) {
        red[0][warp] = before;
        red[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
    for (int i = 0; i < kJoinThreads / 32; ++i) {
        before += red[0][i];
        total += red[1][i];
    }
    const Seq s = load_seq(a, b);
    const int row0 = blockIdx.x * kJoinRows, R = s.n * a.group;
    pdl_wait();
    pdl_trigger();
    if (row0 >= R) return;
    const int pair = row0 / (2 * kTile), mt = row0 / kTile % 2, r0 = row0 % kTile;
    const long long first = before + (static_cast<long long>(hk) * s.pairs + pair) * s.tiles;
    const int C = used_ctas(total, ctas);
    const int ca = range_of(total, first, C), cb = range_of(total, first + s.tiles - 1, C);
    if (ca == cb) return;
    const bool head_slot = range_lo(total, ca, C) == first;   // the item begins its first CTA's range
    auto slot = [&](int c) { return 2 * c + (c == ca && !head_slot ? 1 : 0); };
    const int parts = cb - ca + 1;
    if (warp == 0) {   // a lane per row: the weights of its parts
        const bool live = row0 + lane < R;
        float m = ninf(), l = 0.0f;
        for (int i = 0; i < parts; ++i)
            if (live) m = fmaxf(m, part_ml<DP>(a, ctas, slot(ca + i), mt)[r0 + lane].x);
        const float ref = m == ninf() ? 0.0f : m;
        for (int i = 0; i < parts; ++i) {
            float k = 0.0f;
            if (live) {
                const float2 ml = part_ml<DP>(a, ctas, slot(ca + i), mt)[r0 + lane];
                k = ex2(ml.x - ref);
                l += ml.y * k;
            }
            wt[i][lane] = k;
        }
        const bool none = m == ninf() && l == 0.0f;
        wt[parts][lane] = none ? 0.0f : 1.0f / l;
        if (live && a.lse != nullptr) {
            const int row = row0 + lane;
            a.lse[static_cast<int64_t>(s.t0 + row / a.group) * a.q.heads + hk * a.group + row % a.group] =
                none ? ninf() : (m + log2f(l)) * 0.69314718055994531f;
        }
    }
    __syncthreads();
    // 8 channel quads x 4 rows per warp and step
    for (int i = threadIdx.x; i < kJoinRows * (DP / 4); i += kJoinThreads) {
        const int q8 = i / 32, quad = (q8 % (DP / 32)) * 8 + lane % 8, rr = (q8 / (DP / 32)) * 4 + lane / 8;
        const int row = row0 + rr;
        if (row >= R || quad * 4 >= a.cache.dim) continue;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float4 x = part_out<DP>(a, slot(ca + p), mt)[static_cast<size_t>(quad) * kTile + r0 + rr];
            const float k = wt[p][rr];
            o.x = fmaf(x.x, k, o.x);
            o.y = fmaf(x.y, k, o.y);
            o.z = fmaf(x.z, k, o.z);
            o.w = fmaf(x.w, k, o.w);
        }
        const float inv = wt[parts][rr];
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out.ptr) + static_cast<int64_t>(s.t0 + row / a.group) * a.out.token_stride +
                                   static_cast<int64_t>(hk * a.group + row % a.group) * a.out.head_stride + quad * 4) =
            make_uint2(pack2(o.x * inv, o.y * inv, false), pack2(o.z * inv, o.w * inv, false));
    }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// The cache as a 4-D tensor (channel, row of a page, head, page); boxes of box_rows rows and 128
// bytes.  Channels beyond dim and pages beyond the cache read as zeros.
bool encode(CUtensorMap *map, const moe_kv_cache_t &c, const void *ptr, int box_rows, bool swizzle) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    const uint64_t es = c.dtype == MOE_BF16 ? 2 : 1;
    // a dimension of one element has no step; any valid stride will do
    auto stride = [&](int64_t st, int extent) { return extent == 1 ? 16u * 1024u : static_cast<cuuint64_t>(st) * es; };
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page), static_cast<cuuint64_t>(c.heads),
                          static_cast<cuuint64_t>(c.pages)};
    cuuint64_t strides[3] = {stride(c.token_stride, c.page), stride(c.head_stride, c.heads), stride(c.page_stride, c.pages)};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int box_rows_of(int page) {   // the largest power of two that divides a page, at most a tile
    int b = 8;
    while (b < kTile && page % (2 * b) == 0) b *= 2;
    return b;
}

int dim_padded(int dim) { return dim <= 64 ? 64 : 128; }

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
cudaError_t launch(const TreeArgs &a, int dev, cudaStream_t s, bool pdl) {
    using L = Lay<F8, DP>;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        bool &set = g_dev[dev & 63].set[(F8 ? 2 : 0) + (DP == 128 ? 1 : 0)];
        if (!set) {
            const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<F8, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
            if (e != cudaSuccess) return e;
            set = true;
        }
    }
    const int sms = sm_count(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int rows = box_rows_of(a.cache.page);
    CUtensorMap tm_k, tm_v;
    if (!encode(&tm_k, a.cache, a.cache.k, rows, true) || !encode(&tm_v, a.cache, a.cache.v, rows, !F8))
        return cudaErrorNotSupported;
    // no more CTAs than the page tables could fill with tiles
    const long long most = static_cast<long long>(a.seqs) * a.cache.heads * ((a.max_tokens * a.group + 2 * kTile - 1) / (2 * kTile)) *
                           ((static_cast<long long>(a.max_pages) * a.cache.page + kTile - 1) / kTile);
    const int ctas = static_cast<int>(std::min<long long>(sms, most));
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<F8, DP>, tm_k, tm_v, a, rows);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((a.max_tokens * a.group + kJoinRows - 1) / kJoinRows, a.cache.heads, a.seqs);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<DP>, a, ctas);
}

bool wide16(const moe_heads_t &h) {
    return (reinterpret_cast<uintptr_t>(h.ptr) & 15u) == 0 && h.token_stride % 8 == 0 && h.head_stride % 8 == 0;
}

}  // namespace

bool tree_attn_supports(const moe_kv_cache_t &c, const moe_heads_t &q, const moe_heads_t &out) {
    return q.dtype == MOE_BF16 && out.dtype == MOE_BF16 && (c.dtype == MOE_BF16 || c.dtype == MOE_E4M3) && c.dim <= 128 &&
           c.page % 8 == 0 && wide16(q) && wide16(out);
}

// A workspace serves whichever kernel a call runs on, on any device: room for kMaxCtas CTAs' parts
// is more than most calls touch, so it goes by this device's SMs.
size_t tree_attn_part_bytes(int dim) {
    int dev = 0;
    int sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        const int n = sm_count(dev);
        if (n > 0) sms = n;
    }
    return static_cast<size_t>(sms) * 2 * 2 * kTile * (dim_padded(dim) * sizeof(float) + sizeof(float2));
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t s, bool pdl) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool f8 = a.cache.dtype == MOE_E4M3;
    if (dim_padded(a.cache.dim) == 64) return f8 ? launch<true, 64>(a, dev, s, pdl) : launch<false, 64>(a, dev, s, pdl);
    return f8 ? launch<true, 128>(a, dev, s, pdl) : launch<false, 128>(a, dev, s, pdl);
}

}  // namespace moe
