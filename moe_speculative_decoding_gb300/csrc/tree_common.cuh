// tree_common.cuh -- what the tensor-core attention kernels share: tcgen05 and TMA pieces, the
// work list over (sequence, cache head) items and position tiles, tree masks, and the host's tensor
// maps.
#pragma once

#include <algorithm>
#include <mutex>

#include "cache_args.cuh"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;                      // positions of a K/V tile, lanes of an accumulator
constexpr long long kDrain = 400000000ll;       // about 0.2 s
constexpr int kMaxCtas = 256;
constexpr float kLazy = 8.0f;                   // log2 growth of a maximum that O is rescaled for
constexpr float kWeightUp = 128.0f;             // fp16 weights: at most 2^8 * 2^7, flushed below 2^-31
// e4m3: a row's weight at a position is its exponential times the value's scale, and it is that product's
// largest among what the row sees that its weights are held against (score plus the scale's logarithm,
// in one reference per row).  So neither a scale that a row does not see nor one that it gives no
// weight moves its other weights.  Logarithms are cut to this range: an exponential alone is then
// at most 2^(8 + 90) and the largest product's at least 2^-100, and fp32 sums hold them.
constexpr float kScaleLow = -90.0f, kScaleHigh = 100.0f;   // NaN: the lowest

// ------------------------------------------------------------------ tcgen05, TMA and arithmetic pieces
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
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
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
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Registers of a warpgroup's threads from here on (all its warps call).
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ void f2_get(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
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

// warp_wait with less code: the kernels have many waits, and their code should stay in the
// instruction caches.  (Out of line it cannot be: a function call ends the register shares.)
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int32_t *abort, int32_t *err, long long limit) {
    bool ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    const long long t0 = clock64();
    do {
        const bool late = clock64() - t0 > limit;
        if (__any_sync(0xFFFFFFFFu, late || *abort != 0)) {
            *abort = 1;
            if (late) record_error(err, MOE_ERR_DEVICE_TIMEOUT);
            return false;
        }
        if (!ok) ok = mbar_try_wait(bar, parity);
    } while (!__all_sync(0xFFFFFFFFu, ok));
    return true;
}

// Bounded warp-wide wait until *p has reached v, under mbar_wait's rules.
__device__ __forceinline__ bool wait_count(const volatile uint32_t *p, uint32_t v, volatile int32_t *abort, int32_t *err,
                                           long long limit) {
    if (__all_sync(0xFFFFFFFFu, static_cast<int32_t>(*p - v) >= 0)) return true;
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
            len > static_cast<long long>(a.max_pages) * a.cache.page || len > kMaxPositions;
    s.n = s.bad ? 0 : static_cast<int>(n);
    s.len = s.bad ? 0 : static_cast<int>(len);
    s.tiles = (s.len + kTile - 1) / kTile;
    s.pairs = (s.n * a.group + 2 * kTile - 1) / (2 * kTile);
    return s;
}
// The list is cut by cost, in tiles: an item costs its tiles and, when there are several tiles for
// every CTA, kItemCost more, for its beginning and end (8,000-13,000 cycles against 1,500-4,000 of a
// tile): before that, a CTA with parts of three items took 74,000 cycles where one with the same
// number of tiles of one item took 43,000 (sixteen sequences of 800-4100 positions, 8 heads).
// An item's extra units come first; a CTA whose range holds only such units has nothing to do.
// Those sixteen with chains of 5 over e4m3 codes take 39.7, 37.9, 37.7, 37.6, 39.1 and 41.7 us with 3, 4,
// 5, 6, 10 and 14; eight sequences of 4001-8201 with trees of 64 over bf16 67.2, 66.7, 65.4, 65.2, 66.0
// and 68.1.
constexpr int kItemCost = 6;
struct Work {
    long long tiles, items;
};
__device__ __forceinline__ Work seq_work(const TreeArgs &a, const Seq &s) {
    Work w;
    w.items = s.tiles > 0 ? static_cast<long long>(a.cache.heads) * s.pairs : 0;
    w.tiles = w.items * s.tiles;
    return w;
}
__device__ __forceinline__ int item_cost(const TreeArgs &a, const Work &total, int ctas) {
    return total.tiles > 2ll * ctas && !a.undivided ? kItemCost : 0;
}
// At most as many ranges as units, so that none is empty.
__device__ __forceinline__ int used_ctas(long long W, int ctas) { return static_cast<int>(min(W, static_cast<long long>(ctas))); }
// First unit of CTA c's range, and the CTA whose range holds unit x.
// (In 32 bits where they do: a 64-bit division is some hundred instructions.)
__device__ __forceinline__ long long range_lo(long long W, int c, int C) {
    if (W < (1ll << 23)) return static_cast<uint32_t>(W) * static_cast<uint32_t>(c) / static_cast<uint32_t>(C);
    return W * c / C;
}
__device__ __forceinline__ int range_of(long long W, long long x, int C) {
    if (W < (1ll << 23))
        return static_cast<int>(((static_cast<uint32_t>(x) + 1) * static_cast<uint32_t>(C) - 1) / static_cast<uint32_t>(W));
    return static_cast<int>(((x + 1) * C - 1) / W);
}

// A CTA's walk over its range: item by item, the part [lo, hi) of the item's position tiles.
struct Walk {
    Seq s;
    long long at, end, item0;   // next unit of the list, the range's end, the item's first unit
    int b, hk, pair, lo, hi;
    int extra;                  // units of an item before its tiles
    bool whole;                 // the item lies in this CTA alone
    bool first;                 // the range's first item has not been looked at
    int index;                  // items walked before
};
// The whole warp calls these; the outcome is uniform.
__device__ __forceinline__ void walk_begin(const TreeArgs &a, Walk &w, bool report) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    w.index = -1;
    w.b = w.hk = w.pair = 0;
    w.at = w.end = w.item0 = 0;
    w.extra = 0;
    w.first = true;
    // 32 sequences a step; the last step's stay in registers (all of them, when there is one step)
    Seq mine;
    Work x = {0, 0}, incl = {0, 0}, total = {0, 0};
    auto step = [&](int b0) {
        x.tiles = x.items = 0;
        if (b0 + lane < a.seqs) {
            mine = load_seq(a, b0 + lane);
            x = seq_work(a, mine);
        }
        incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, incl.tiles, o), z = __shfl_up_sync(0xFFFFFFFFu, incl.items, o);
            if (lane >= o) {
                incl.tiles += y;
                incl.items += z;
            }
        }
    };
    mine.bad = false;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        step(b0);
        if (b0 + lane < a.seqs && mine.bad && report) record_error(a.err, MOE_ERR_BAD_ID);
        total.tiles += __shfl_sync(0xFFFFFFFFu, incl.tiles, 31);
        total.items += __shfl_sync(0xFFFFFFFFu, incl.items, 31);
    }
    w.extra = item_cost(a, total, gridDim.x);
    const long long W = total.tiles + w.extra * total.items;
    const int C = used_ctas(W, gridDim.x), c = static_cast<int>(blockIdx.x);
    if (c >= C) return;
    w.at = range_lo(W, c, C);
    w.end = range_lo(W, c + 1, C);
    long long before = 0;   // units of the sequences before
    for (int b0 = 0;; b0 += 32) {
        if (a.seqs > 32) step(b0);
        const long long units = incl.tiles + w.extra * incl.items;
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + units > w.at);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            w.b = b0 + l;
            before += __shfl_sync(0xFFFFFFFFu, units - x.tiles - w.extra * x.items, l);
            w.s.t0 = __shfl_sync(0xFFFFFFFFu, mine.t0, l);
            w.s.n = __shfl_sync(0xFFFFFFFFu, mine.n, l);
            w.s.ctx = __shfl_sync(0xFFFFFFFFu, mine.ctx, l);
            w.s.len = __shfl_sync(0xFFFFFFFFu, mine.len, l);
            w.s.tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, l);
            w.s.pairs = __shfl_sync(0xFFFFFFFFu, mine.pairs, l);
            w.s.bad = false;
            break;
        }
        before += __shfl_sync(0xFFFFFFFFu, units, 31);
    }
    const long long into = w.at - before;
    const int size = w.s.tiles + w.extra;
    const int item = into < (1ll << 31) ? static_cast<int>(static_cast<uint32_t>(into) / static_cast<uint32_t>(size))
                                        : static_cast<int>(into / size);
    w.item0 = before + static_cast<long long>(item) * size;
    w.hk = item / w.s.pairs;
    w.pair = item % w.s.pairs;
    w.first = true;
}
// Sets the next item's part; false at the end of the range.
__device__ __forceinline__ bool walk_next(const TreeArgs &a, Walk &w) {
    while (w.at < w.end) {
        if (!w.first) {   // step to the item at w.at
            w.item0 += w.s.tiles + w.extra;
            if (++w.pair == w.s.pairs) {
                w.pair = 0;
                if (++w.hk == a.cache.heads) {
                    w.hk = 0;
                    do {
                        w.s = load_seq(a, ++w.b);
                    } while (w.s.tiles == 0 || w.s.pairs == 0);   // there are units left, so one follows
                }
            }
        }
        w.first = false;
        const long long tile0 = w.item0 + w.extra, past = tile0 + w.s.tiles, stop = min(w.end, past);
        if (a.undivided) {   // the item is the range's that holds its first tile
            w.lo = w.at > tile0 ? w.s.tiles : 0;
            w.hi = w.s.tiles;
        } else {
            w.lo = static_cast<int>(max(w.at, tile0) - tile0);
            w.hi = static_cast<int>(stop - tile0);
        }
        w.whole = w.lo == 0 && w.hi == w.s.tiles;
        w.at = stop;
        if (w.hi > w.lo) {
            ++w.index;
            return true;
        }
    }
    return false;
}

// The K producer, which runs ahead of all others, walks; the others follow it through a ring of
// records in shared memory (finding an item's place takes a chain of global loads, microseconds
// while the memory is busy).  Every role is less than kRecords items behind: K's ring holds at most
// four tiles, and K of item i + 5 is not copied before item i + 1's queries are in place, that is
// before the softmax has finished item i.
constexpr int kRecords = 8;
constexpr uint32_t kRecordBytes = 104;
static_assert(sizeof(Walk) <= kRecordBytes, "a record holds a walk");
struct Follow {
    uint8_t *ring;      // [kRecords][kRecordBytes]
    uint32_t bars;      // [kRecords]
    uint32_t n;         // records published or taken
};
__device__ __forceinline__ bool walk_lead(const TreeArgs &a, Walk &w, Follow &f) {
    const bool more = walk_next(a, w);
    if ((threadIdx.x & 31) == 0) {
        Walk *const r = reinterpret_cast<Walk *>(f.ring + (f.n % kRecords) * kRecordBytes);
        *r = w;
        if (!more) r->lo = -1;   // the end
    }
    warp_arrive(f.bars + 8u * (f.n % kRecords));
    ++f.n;
    return more;
}
__device__ __forceinline__ bool walk_follow(const TreeArgs &a, Walk &w, Follow &f, volatile int32_t *abort_flag) {
    if (!wait_for(f.bars + 8u * (f.n % kRecords), (f.n / kRecords) & 1u, abort_flag, a.err, a.wait_limit)) return false;
    w = *reinterpret_cast<const Walk *>(f.ring + (f.n % kRecords) * kRecordBytes);
    ++f.n;
    return w.lo >= 0;
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

// The kernel for few rows: [slot][64 rows][DP] fp32, then [slot][64] (maximum, sum).
constexpr int kNarrowRows = 64;
template <int DP>
__device__ __forceinline__ float *narrow_out(const TreeArgs &a, int slot) {
    return static_cast<float *>(a.part) + static_cast<size_t>(slot) * kNarrowRows * DP;
}
template <int DP>
__device__ __forceinline__ float2 *narrow_ml(const TreeArgs &a, int ctas, int slot) {
    return reinterpret_cast<float2 *>(static_cast<float *>(a.part) + static_cast<size_t>(ctas) * 2 * kNarrowRows * DP) +
           static_cast<size_t>(slot) * kNarrowRows;
}

// Division of many numbers below 2^31 by one: with the floor of (2^32 - 1) / d the product's high
// word is the quotient or one less.
struct Divisor {
    uint32_t d, recip;
    __device__ __forceinline__ explicit Divisor(int by) : d(static_cast<uint32_t>(by)), recip(0xFFFFFFFFu / static_cast<uint32_t>(by)) {}
    __device__ __forceinline__ uint32_t quotient(uint32_t x) const {
        const uint32_t q = __umulhi(x, recip);
        return q + (x - q * d >= d ? 1u : 0u);
    }
};

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

// Channel ch of the value at position pos of sequence b, cache head hk, as the cache has it (0 for a
// page outside the cache).
template <bool F8>
__device__ __forceinline__ float value_at(const TreeArgs &a, int b, int hk, int pos, int ch) {
    const moe_kv_cache_t &c = a.cache;
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / c.page], at = pos % c.page;
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(c.pages)) return 0.0f;
    const int64_t off = page * c.page_stride + at * c.token_stride + hk * c.head_stride + ch;
    if (F8)
        return f16_of(e4m3x2_to_f16x2(static_cast<const uint8_t *>(c.v)[off])) *
               c.v_scale[(static_cast<int64_t>(page) * c.heads + hk) * c.page + at];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(c.v)[off]) << 16);
}

// Stores chunk c (8 channels) of a query row into a K-major operand of `rows` rows.  bf16: blocks of
// 64 channels, rows * 128 bytes each.  F8: the row, scaled by a power of two to at most 256, as an
// e4m3 operand and, rows * 128 bytes on, the e5m2 remainder; unscale is the inverse factor (NaN for
// a row that is not finite).  The DP / 8 lanes of a row call together.
template <bool F8, int DP>
__device__ __forceinline__ void store_query(uint8_t *q, int rows, int row, int c, uint4 x, float &unscale) {
    unscale = 1.0f;
    if (!F8) {
        *reinterpret_cast<uint4 *>(q + (c / 8) * (rows * 128) + row * 128 + (((c % 8) ^ (row & 7)) * 16)) = x;
        return;
    }
    // the row's largest exponent (bf16 magnitudes order as integers)
    const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, max(wd[k] & 0x7FFFu, wd[k] >> 16 & 0x7FFFu));
#pragma unroll
    for (int o = DP / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const int e = static_cast<int>(top >> 7);   // biased exponent; 255: not finite
    // up = 2^(7 - (e - 127)): the largest lands in [128, 256); both factors' exponents in range
    const int ub = min(max(261 - e, 1), 253);
    const float up = __int_as_float(ub << 23);
    unscale = e == 255 ? __int_as_float(0x7fffffff) : __int_as_float((254 - ub) << 23);
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x0 = bf16_lo(wd[k]) * up, x1 = bf16_hi(wd[k]) * up;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi[k]) : "f"(x1), "f"(x0));
        const uint32_t h = e4m3x2_to_f16x2(hi[k]);
        const float r0 = x0 - f16_of(h), r1 = x1 - f16_of(h >> 16);
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo[k]) : "f"(r1), "f"(r0));
    }
    uint8_t *const p = q + row * 128 + (((c / 2) ^ (row & 7)) * 16) + (c & 1) * 8;
    *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0] | static_cast<uint32_t>(hi[1]) << 16, hi[2] | static_cast<uint32_t>(hi[3]) << 16);
    *reinterpret_cast<uint2 *>(p + rows * 128) = make_uint2(lo[0] | static_cast<uint32_t>(lo[1]) << 16, lo[2] | static_cast<uint32_t>(lo[3]) << 16);
}

// ------------------------------------------------------------------ roles
// L gives the places in shared memory: oK, oV, oS (V codes landing), oSSc (their scales), oBad,
// oScale, oTop, ring sizes NK, NV, NS, barriers bKF ... at oBar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A producer warp: K (FIRST = 0), V (LAST = 1) or K, then V of each tile, a lane per box of box_rows
// positions.  Boxes beyond the length are not copied.  An e4m3 cache's scales (contiguous over a
// page's rows) land with V's codes where the converters want them there (kLandScales).
template <typename L, bool F8, int DP, int FIRST, int LAST>
__device__ __forceinline__ void produce(const TreeArgs &a, Walk &w, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                        uint8_t *smem, int box_rows, volatile int32_t *abort_flag,
                                        volatile uint32_t *copied, volatile uint32_t *v_issued, Follow f) {
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int boxes = kTile / box_rows;   // of a tile, at most 16
    const moe_kv_cache_t &kc = a.cache;
    constexpr uint32_t NV = F8 ? L::NS : L::NV;
    constexpr int kNone = -2147483647;    // a box beyond the length
    uint32_t cnt = 0, ahead = 0;   // ahead: K of tile cnt is on its way
    bool ok = true;
    while (ok && (FIRST == 0 ? walk_lead(a, w, f) : walk_follow(a, w, f, abort_flag))) {
        const int32_t *const table = a.page_table + static_cast<int64_t>(w.b) * a.max_pages;
        // The places of 32 boxes, a lane each, for 32 / boxes tiles; the next ones are on their way
        // while these are used.
        auto places = [&](int first, int &page, int &row) {
            const int64_t pos = (static_cast<int64_t>(first) * boxes + lane) * box_rows;
            page = kNone;
            row = 0;
            if (pos < w.s.len) {
                page = __ldg(table + static_cast<int>(pos) / kc.page);
                row = static_cast<int>(pos) % kc.page;
            }
        };
        const int per = 32 / boxes;
        int page_now, row_now, page_next, row_next;
        places(w.lo, page_now, row_now);
        places(w.lo + per, page_next, row_next);
        for (int tt = w.lo, k = 0; tt < w.hi; ++tt, ++cnt, ++k) {
            if (k == per) {
                k = 0;
                page_now = page_next;
                row_now = row_next;
                places(tt + per, page_next, row_next);
            }
            int page = __shfl_sync(0xFFFFFFFFu, page_now, (k * boxes + lane) & 31);
            const int row = __shfl_sync(0xFFFFFFFFu, row_now, (k * boxes + lane) & 31);
            const bool mine = lane < boxes && page != kNone;
            const bool good = static_cast<uint32_t>(page) < static_cast<uint32_t>(kc.pages);
            if (mine && !good) {
                record_error(a.err, MOE_ERR_BAD_ID);
                page = kc.pages;   // beyond the tensor: the copy writes zeros
            }
            const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, mine)), n_good = __popc(__ballot_sync(0xFFFFFFFFu, mine && good));
            const uint32_t bytes = n * box_rows * (F8 ? 128u : DP * 2u);
#pragma unroll
            for (int v = FIRST; v <= LAST; ++v) {
                const uint32_t slot = v ? cnt % NV : cnt % L::NK, use = v ? cnt / NV : cnt / L::NK;
                const uint32_t full = bar((v ? (F8 ? L::bSF : L::bVF) : L::bKF) + slot);
                const uint32_t empty = bar((v ? (F8 ? L::bSE : L::bVE) : L::bKE) + slot);
                const uint32_t dst = base + (v ? (F8 ? L::oS + slot * L::kStage : L::oV + slot * L::kVSlot)
                                               : L::oK + slot * L::kKSlot);
                if (!wait_for(empty, (use & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) {
                    ahead = v - FIRST;
                    ok = false;
                    break;
                }
                if (L::kLandScales && v && mine && !good) {   // no scales to copy: zeros
                    float *const sc = reinterpret_cast<float *>(smem + L::oSSc + slot * 1024) + lane * box_rows;
                    for (int i = 0; i < box_rows; ++i) sc[i] = sc[128 + i] = 0.0f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(full, bytes + (L::kLandScales && v ? n_good * box_rows * 8u : 0u));
                __syncwarp();
                if (mine) {
                    const CUtensorMap *tm = v ? tm_v : tm_k;
                    const uint32_t d = dst + static_cast<uint32_t>(lane * box_rows) * 128u;
                    tma_load_4d(d, tm, full, 0, row, w.hk, page);
                    if (!F8 && DP == 128) tma_load_4d(d + kTile * 128u, tm, full, 64, row, w.hk, page);
                    if (L::kLandScales && v && good) {
                        const int64_t o = (static_cast<int64_t>(page) * kc.heads + w.hk) * kc.page + row;
                        const uint32_t sd = base + L::oSSc + slot * 1024 + lane * box_rows * 4u;
                        bulk_load(sd, kc.k_scale + o, box_rows * 4u, full);
                        bulk_load(sd + 512, kc.v_scale + o, box_rows * 4u, full);
                    }
                }
                __syncwarp();
                // for V's cleaner: once a tile is announced, its slot's previous use is over, and the
                // slot's parity tells this use from that one
                if (v == 1 && !F8 && lane == 0) {
                    __threadfence_block();
                    *v_issued = cnt + 1;
                }
            }
            if (!ok) break;
        }
    }
    if (lane == 0) {
        if (FIRST == 0) copied[0] = cnt + ahead;
        if (LAST == 1) copied[1] = cnt;
    }
}

// After an abort copies that nobody waited for must land before the CTA leaves.  One warp calls
// this when all roles have ended: a role may give up after the producers are done.  copied: the
// announced tiles of K and V.
template <typename L, bool F8>
__device__ __forceinline__ void drain_copies(uint8_t *smem, const volatile uint32_t *copied) {
    const uint32_t base = smem_u32(smem), NV = F8 ? L::NS : L::NV, nk = copied[0], nv = copied[1];
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    for (uint32_t j = nk > L::NK ? nk - L::NK : 0; j < nk; ++j)
        mbar_wait_drain(bar(L::bKF + j % L::NK), (j / L::NK) & 1u, kDrain);
    for (uint32_t j = nv > NV ? nv - NV : 0; j < nv; ++j)
        mbar_wait_drain(bar((F8 ? L::bSF : L::bVF) + j % NV), (j / NV) & 1u, kDrain);
}

// bf16: V's cleaner, one warp, over the tiles that reach past the context.  Positions beyond the
// length become zeros (their weights are 0, what the cache holds there may be anything), and so do
// non-finite elements of drafted tokens: a row that does not see such a token must not meet it in
// the product.  Rows that do get it added at the end of the item (bad bits).
template <typename L, int DP>
__device__ __forceinline__ void clean_values(const TreeArgs &a, Walk &w, uint8_t *smem, volatile int32_t *abort_flag,
                                             const volatile uint32_t *v_issued, Follow f) {
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    const int lane = static_cast<int>(threadIdx.x & 31);
    uint32_t cnt = 0, fixes = 0;
    bool ok = true;
    while (ok && walk_follow(a, w, f, abort_flag)) {
        uint32_t *const bad = reinterpret_cast<uint32_t *>(smem + L::oBad) + (w.index & 7) * 8;
        if (lane < 8) bad[lane] = 0;
        __syncwarp();
        for (int tt = w.lo; tt < w.hi; ++tt, ++cnt) {
            if ((tt + 1) * kTile <= w.s.ctx) continue;
            const uint32_t slot = cnt % L::NV;
            // only the last tiles are waited for here, so the slot may be some uses behind: its
            // parity tells this use from the one before once this one was issued
            if (!wait_count(v_issued, cnt + 1, abort_flag, a.err, a.wait_limit) ||
                !wait_for(bar(L::bVF + slot), (cnt / L::NV) & 1u, abort_flag, a.err, a.wait_limit)) {
                ok = false;
                break;
            }
            constexpr int C = DP / 8, ROWS = 32 / C, BATCH = 4;   // 16-byte chunks of a row; rows at a time
            uint8_t *const v = smem + L::oV + slot * L::kVSlot + (lane % C / 8) * (kTile * 128) + (lane % 8) * 16;
            const int first = max(0, w.s.ctx - tt * kTile), stop = min(kTile, w.s.len - tt * kTile);
#pragma unroll 1
            for (int r0 = first + lane / C; r0 < stop; r0 += BATCH * ROWS) {
                uint4 x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (r0 + i * ROWS < stop) x[i] = *reinterpret_cast<const uint4 *>(v + (r0 + i * ROWS) * 128);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = r0 + i * ROWS;
                    uint32_t *const q = reinterpret_cast<uint32_t *>(&x[i]);
                    // bit 15 of a half whose exponent is all ones
                    auto over = [](uint32_t y) { return ((y & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
                    if (r >= stop || (over(q[0]) | over(q[1]) | over(q[2]) | over(q[3])) == 0) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] &= ~((over(q[k]) >> 15) * 0xFFFFu);
                    *reinterpret_cast<uint4 *>(v + r * 128) = x[i];
                    atomicOr(&bad[(tt & 1) * 4 + r / 32], 1u << (r & 31));
                }
            }
#pragma unroll 4
            for (int r = stop + lane / C; r < kTile; r += ROWS) *reinterpret_cast<uint4 *>(v + r * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            warp_arrive(bar(L::bFix + (fixes & 3u)));   // the ring of V keeps this at most NV ahead
            ++fixes;
        }
    }
}

__device__ __forceinline__ float log2_scale(float s) { return fminf(fmaxf(lg2(fabsf(s)), kScaleLow), kScaleHigh); }

// All ones in the bytes of four codes that are not NaN (0x7f, 0xff).
__device__ __forceinline__ uint32_t finite_codes(uint32_t x) {
    const uint32_t nan = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // bit 7 of such a byte
    return ~((nan >> 7) * 0xFFu);
}

// Four codes to fp16, exact.  (Assembling the fp16 bits with integer operations, five or more for four
// codes, made the integer pipe the kernel's bound.)
__device__ __forceinline__ void codes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

// e4m3: V's converters, four warps of 32 positions each: codes to fp16 (exact) in the products'
// layout, the scales into a ring for the softmax: of a position the key's, the value's times
// kWeightUp, and the logarithm of the value's.  The scales come from beside the codes (kLandScales:
// a softmax thread owns a row, and has a bound on the tile's logarithms too, a warp's largest so far
// from each) or are loaded here.  What clean_values does for bf16 is done on the way.
// With two groups of four warps each takes every other tile (of one softmax warpgroup; rings are
// even, so that a slot is one group's).  A tile takes a group 2,000 cycles of its own, 1,150 of them
// the codes' loop, and every second one is its: about what a tile of the cache takes to arrive.
template <typename L, int DP>
__device__ __forceinline__ void convert_values(const TreeArgs &a, Walk &w, uint8_t *smem, int cw, int group,
                                               volatile int32_t *abort_flag, Follow f) {
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    const int lane = static_cast<int>(threadIdx.x & 31), j = cw * 32 + lane;
    float *const scale_s = reinterpret_cast<float *>(smem + L::oScale);
    volatile float *const top_s = reinterpret_cast<volatile float *>(smem + L::oTop);
    const float kMax = 3.4028234e38f;
    // (with a division for each position's page a tile took 300 cycles more)
    const Divisor by_page(a.cache.page);
    auto page_of = [&](uint32_t pos) { return by_page.quotient(pos); };
    uint32_t cnt = 0;
    bool ok = true;
    while (ok && walk_follow(a, w, f, abort_flag)) {
        uint32_t *const bad = reinterpret_cast<uint32_t *>(smem + L::oBad) + (w.index & 7) * 8;
        // a warp's words are its own: with two groups, the tiles of one parity
        const int odd = L::kGroups == 2 ? static_cast<int>((cnt ^ static_cast<uint32_t>(w.lo) ^ static_cast<uint32_t>(group)) & 1u) : 0;
        if (lane < 2 && (L::kGroups == 1 || lane == odd)) bad[lane * 4 + cw] = 0;
        __syncwarp();
        // the largest value scale of the warp's positions so far (formed for each tile anew it cost 4% of
        // 128 rows' time)
        float top = 0.0f, top_log = kScaleLow;
        // without landing scales: this thread's position of the group's tiles, the scales loaded a
        // tile ahead and the page two
        const int32_t *const table = a.page_table + static_cast<int64_t>(w.b) * a.max_pages;
        auto page_at = [&](int tt) {
            const int64_t pos = static_cast<int64_t>(tt) * kTile + j;
            return !L::kLandScales && tt < w.hi && pos < w.s.len ? __ldg(table + page_of(static_cast<uint32_t>(pos))) : -1;
        };
        auto scales_at = [&](int tt, int page, float &ks, float &vs) {
            ks = vs = 0.0f;
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.pages)) return;
            const uint32_t pos = static_cast<uint32_t>(tt * kTile + j);
            const int64_t o = (static_cast<int64_t>(page) * a.cache.heads + w.hk) * a.cache.page +
                              (pos - page_of(pos) * static_cast<uint32_t>(a.cache.page));
            ks = __ldg(a.cache.k_scale + o);
            vs = __ldg(a.cache.v_scale + o);
        };
        const int t0 = w.lo + (L::kGroups == 2 ? static_cast<int>((cnt ^ static_cast<uint32_t>(group)) & 1u) : 0);
        float ks_next = 0.0f, vs_next = 0.0f;
        if (!L::kLandScales) scales_at(t0, page_at(t0), ks_next, vs_next);
        int page_next = page_at(t0 + L::kGroups);
        for (int tt = w.lo; tt < w.hi; ++tt, ++cnt) {
            if (L::kGroups == 2 && (cnt & 1u) != static_cast<uint32_t>(group)) continue;
            const int first = max(0, w.s.ctx - tt * kTile), stop = min(kTile, w.s.len - tt * kTile);
            const uint32_t ss = cnt % L::NS, slot = cnt % L::NV;
            float ks = 0.0f, vs = 0.0f;
            if (L::kLandScales) {
                if (!(ok = wait_for(bar(L::bSF + ss), (cnt / L::NS) & 1u, abort_flag, a.err, a.wait_limit))) break;
                const float *const land = reinterpret_cast<const float *>(smem + L::oSSc + ss * 1024);
                if (j < stop) {
                    ks = land[j];
                    vs = land[128 + j];
                }
            } else {
                ks = ks_next;
                vs = vs_next;
                scales_at(tt + L::kGroups, page_next, ks_next, vs_next);   // in flight during this tile
                page_next = page_at(tt + 2 * L::kGroups);
            }
            const bool odd_scale = j >= first && j < stop && !(fabsf(vs) <= kMax);
            if (odd_scale) vs = 0.0f;
            // The scales have a ring of their own, so that a tile can be weighed before its values are
            // converted (with the V slot's, a tile waited for the product two before it: 4000 cycles
            // for two tiles instead of 2700).
            const uint32_t sb = cnt % L::NC;
            if (!(ok = wait_for(bar(L::bCE + sb), ((cnt / L::NC) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit))) break;
            scale_s[sb * 384 + j] = ks;
            scale_s[sb * 384 + 128 + j] = vs * kWeightUp;
            scale_s[sb * 384 + 256 + j] = log2_scale(vs);
            if (L::kLandScales) {
                if (__any_sync(0xFFFFFFFFu, fabsf(vs) > top)) {
                    top = fmaxf(top, fabsf(vs));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    top_log = log2_scale(top);
                }
                if (lane == 0) top_s[sb * 4 + cw] = top_log;
            }
            if (odd_scale) atomicOr(&bad[(tt & 1) * 4 + cw], 1u << lane);
            warp_arrive(bar(L::bCF + sb));
            if (!L::kLandScales && !(ok = wait_for(bar(L::bSF + ss), (cnt / L::NS) & 1u, abort_flag, a.err, a.wait_limit))) break;
            if (!(ok = wait_for(bar(L::bVE + slot), ((cnt / L::NV) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit))) break;
            uint8_t *const src = smem + L::oS + ss * L::kStage;
            uint8_t *const dst = smem + L::oV + slot * L::kVSlot;
            // 4 (8) rows of 128 (64) codes a step: 16 codes per lane
            constexpr int C = DP / 16, RS = 32 / C, STEPS = 32 / RS;
            const int c = lane % C, row0 = cw * 32 + lane / C;
            if (min(first, stop) < kTile) {   // the tile reaches past the context
#pragma unroll 1
                for (int i = 0; i < STEPS; ++i) {
                    const int r = row0 + i * RS;
                    uint4 *const q = reinterpret_cast<uint4 *>(src + r * 128 + c * 16);
                    if (r >= stop) {
                        *q = make_uint4(0, 0, 0, 0);
                    } else if (r >= first) {
                        const uint4 x = *q;
                        const uint4 keep = make_uint4(finite_codes(x.x), finite_codes(x.y), finite_codes(x.z), finite_codes(x.w));
                        if ((keep.x & keep.y & keep.z & keep.w) != 0xFFFFFFFFu) {
                            atomicOr(&bad[(tt & 1) * 4 + cw], 1u << (r & 31));
                            *q = make_uint4(x.x & keep.x, x.y & keep.y, x.z & keep.z, x.w & keep.w);
                        }
                    }
                }
            }
            // 64-channel halves.  The lanes of the second half take the neighbouring row, so that the
            // eight lanes that store together meet eight bank groups.
            const int rs = row0 ^ (c / 4);
            const uint8_t *const from = src + rs * 128 + c * 16;
            uint8_t *const to = dst + (c / 4) * (kTile * 128) + rs * 128;
            // the row's swizzle; a step of four rows changes its bit 2, a step of eight nothing
            const int o0 = (((c % 4) * 2) ^ (rs & 7)) * 16, o1 = o0 ^ 16;
            // no branch in the loop: the steps' chains of dependent operations overlap
#pragma unroll 4
            for (int i = 0; i < STEPS; ++i) {
                const int flip = RS == 4 ? (i & 1) * 64 : 0;
                const uint4 x = *reinterpret_cast<const uint4 *>(from + i * RS * 128);
                uint4 lo, hi;
                codes_to_f16(x.x, lo.x, lo.y);
                codes_to_f16(x.y, lo.z, lo.w);
                codes_to_f16(x.z, hi.x, hi.y);
                codes_to_f16(x.w, hi.z, hi.w);
                *reinterpret_cast<uint4 *>(to + i * RS * 128 + (o0 ^ flip)) = lo;
                *reinterpret_cast<uint4 *>(to + i * RS * 128 + (o1 ^ flip)) = hi;
            }
            fence_proxy_async_smem();   // (the arrival releases the warp's stores: no other fence)
            warp_arrive(bar(L::bSE + ss));
            warp_arrive(bar(L::bVF + slot));
        }
    }
}

// ------------------------------------------------------------------ host side
// The warpgroups' register shares must fit what a block is launched with: a larger share would be
// waited for without end.
template <typename K>
cudaError_t check_registers(K kernel, int threads, int shares) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    return at.numRegs * threads >= shares ? cudaSuccess : cudaErrorInvalidConfiguration;
}

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
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              // a head's row and no more: 256 bytes where a row has 128 would fetch the next head's too
              c.dim * es > 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int box_rows_of(int page) {   // the largest power of two that divides a page, at most a tile
    int b = 8;
    while (b < kTile && page % (2 * b) == 0) b *= 2;
    return b;
}

int dim_padded(int dim) { return dim <= 64 ? 64 : 128; }

}  // namespace
}  // namespace moe
