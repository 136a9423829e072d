// latent_attn.cu -- attention of drafted tokens over a paged cache of latent rows (absorbed form) on the tensor
// cores (tcgen05 + TMA), bf16.
//
//     s = scale <q, row>,  out = sum_p e^(s_p - lse) latent_p,  lse = ln sum_p e^(s_p)
//
// One cache row of rank + rope channels a position serves all heads, as key and, its first rank channels,
// as value: a tile of the cache is copied once and used twice, for rows (token, head) of one sequence.
//
// Bound: 2 (rank + rope) bytes a position are read once for up to NT rows at a time, against
// 2 (2 rank + rope) flops a row: with rank 512, 242 flops a byte at 128 rows, so up to about that many rows
// the cache's bytes bound it and beyond the products.
//
// Products have the cache as the M operand and the rows as N = NT columns (16, 32 or 64),
//
//     S^T = C Q^T [64 positions x NT],  O^T += C^T P^T [rank channels x NT],
//
// because an accumulator of 128 rows by 512 channels would be all of TMEM, and its queries, 147 KB, most
// of the shared memory.  With 64 rows O^T takes 256 of the 512 columns and Q 74 KB, which leaves
// a ring of eight 16 KB units (64 positions by 128 channels, TMA, 128-byte swizzle) beside three places
// for tiles' rotary channels and then their weights.  A tile is 64 positions, not 128, so that the ring holds two:
// the units of one are held from the scores' product to the output's, and meanwhile the next arrive.
//
// Two softmax warpgroups share a tile, each with half of the rows, its own maxima, sums and vote: the
// columns are weighed against the maxima so far, and only when some score lies above its row's by
// more than 2^8 are these formed anew and O rescaled.  S^T of the next tile is formed while a tile is weighed.
//
// One persistent CTA an SM.  Work is the list of (sequence, block of NT rows) x tiles of positions, cut into
// equal contiguous ranges over the CTAs from the lengths on the device; a range's part of an item
// leaves its unnormalised output, maximum and sum in the workspace, and a second kernel joins the
// parts in order (no atomics: repeats give the same bits).
//
// Measured, rank 512 and 64 rotary channels, 16 heads: 64 sequences of 801-8209 positions, one token each, 66-68 us
// (5.3-5.4 TB/s); two of 100-131 thousand with one token 56, with 4 tokens (64 rows) 65-67 us (4.3 TB/s):
// there the ring, 128 KB, holds a tile's units for its copy's latency under load (3,000 cycles and more) and for the
// tile's scores, weights and product, 6,500 cycles in all, which is what limits the bytes in flight.  Few rows
// take a tile in 3,100 cycles (7.0 TB/s) between a beginning of 10,000 and an end of 6,000 and the join.
// Many rows are bound by shared memory: the products read 4 KB for each of a tile's 36 steps of S^T (32 cycles at
// 128 bytes a cycle) and 6 KB for each of the 16 of O^T, and its copies write 72 KB, together 2,500 cycles;
// a tile of 64 rows takes 2,530 (with 168 registers to a thread a few words spill: 116 bytes stored, 64 loaded by
// the compiler's count).  Four sequences of 4001-8201 with trees of 64 tokens 81-84 us (730 TFLOP/s),
// eight of 4001-16411 with two tokens of 128 heads 70-71 (625).  An item's end costs a CTA 11,000 cycles (its last
// product, sums, and 128 KB of parts at 31 bytes a cycle), the join 6-8 us.  One token over 300 positions: 9.7 us,
// a chain of latencies.
//
// Every wait is bounded (an abort flag, MOE_ERR_DEVICE_TIMEOUT, then copies and products are
// drained and TMEM is freed).
#include "latent_args.cuh"
#include "tree_common.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kPos = 64;                        // positions of a tile
constexpr int kProducerWarp = 8, kScoreWarp = 9, kOutWarp = 11, kThreads = 384;   // two score warps
constexpr uint32_t kUnit = 16384, kRopeTile = 8192;

// What the others need to know of a part of an item: a record of the producer's walk.
struct Item {
    int t0, n, ctx, len;   // the sequence: first token, tokens, cached positions, all positions
    int b, blk, lo, hi;    // its number, the block of rows, the part of its tiles
    int index, whole;      // items before in this CTA; the item lies in this CTA alone
};

template <int NT>
struct Lay {
    // The ring's units and the places for tiles' rotary channels: what fits.  A tile's weights take the
    // place of its rotary channels, which are done with when its scores are formed.
    static constexpr int NU = NT == 64 ? 8 : (NT == 32 ? 10 : 11), NR = 3;
    static_assert(kPos * NT * 2 <= kRopeTile, "the weights of a tile");
    static constexpr uint32_t kQBlock = NT * 128;                    // 64 channels of the queries
    static constexpr uint32_t oU = 0, oR = oU + NU * kUnit, oQ = oR + NR * kRopeTile, oBar = oQ + 9 * kQBlock;
    static constexpr int bUF = 0, bUE = NU, bRF = 2 * NU, bRE = bRF + NR, bS = bRE + NR, bSFree = bS + 2, bP = bSFree + 2,
                         bQ = bP + NR, bSeen = bQ + 1, bO = bSeen + 1, bW = bO + 1, bDrain = bW + kRecords, kBars = bDrain + 1;
    static constexpr uint32_t oMisc = oBar + 8 * kBars;            // TMEM address, abort flag, units, rotary tiles and queries copied
    static constexpr uint32_t oBad = (oMisc + 20 + 15) & ~15u;     // uint32 [2 items][2]: drafted tokens with non-finite latents
    static constexpr uint32_t oM = oBad + 16;                      // float [NT]: minus the rows' maxima, 0 where there is none
    static constexpr uint32_t oAlpha = oM + NT * 4;                // float [NT]: a rescaling; an item's last factors
    static constexpr uint32_t oRed = oAlpha + NT * 4;              // float [2][4][NT / 2]: per warp
    static constexpr uint32_t oMask = oRed + 4 * NT * 4;           // uint64 [NT]: the rows' tree masks
    static constexpr uint32_t oWalk = oMask + NT * 8;              // records of parts
    static constexpr uint32_t kSmem = oWalk + kRecords * sizeof(Item);
    static constexpr uint32_t kTmem = NT == 64 ? 512 : 8 * NT;     // 2 NT of S^T, up to 4 NT of O^T
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// 16 lanes (the quarter's first: an accumulator with M = 64 has 16 rows in each quarter) by 8 N columns:
// of columns 8 i .. 8 i + 7 a thread gets lane / 4's (2 (lane % 4), + 1) in r[4 i], r[4 i + 1], and those of
// the row 8 further in r[4 i + 2], r[4 i + 3].
template <int N>
__device__ __forceinline__ void tmem_ld_16x256(uint32_t addr, uint32_t (&r)[4 * N]) {
    if constexpr (N == 1) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr) : "memory");
    } else {
        static_assert(N == 4, "");
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr) : "memory");
    }
}
// 32 lanes by H columns, a lane's columns in one thread
template <int H>
__device__ __forceinline__ void tmem_ld_rows(uint32_t addr, uint32_t (&x)[H]) {
    if constexpr (H == 8)
        tmem_ld8(addr, x);
    else if constexpr (H == 16)
        tmem_ld_16_async(addr, x);
    else
        tmem_ld32(addr, x);
}
template <int H>
__device__ __forceinline__ void tmem_st_rows(uint32_t addr, const uint32_t (&x)[H]) {
    if constexpr (H == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(x[0]), "r"(x[1]),
                     "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    else if constexpr (H == 16)
        tmem_st16(addr, x);
    else
        tmem_st32(addr, x);
}

// ------------------------------------------------------------------ the work list
// As the list of tree_common.cuh, for one cache head, blocks of NT rows and tiles of kPos positions.
struct Rows {
    int t0, n, ctx, len, tiles, blocks;
    bool bad;
};
__device__ __forceinline__ Rows load_rows(const LatentArgs &a, int nt, int b) {
    Rows s;
    s.t0 = a.q_start[b];
    const long long n = static_cast<long long>(a.q_start[b + 1]) - s.t0;
    s.ctx = a.ctx[b];
    const long long len = s.ctx + n;
    s.bad = s.ctx < 0 || n < 0 || n > a.max_tokens || s.t0 < 0 || s.t0 > a.tokens - n ||
            len > static_cast<long long>(a.max_pages) * a.cache.page || len > kMaxPositions;
    s.n = s.bad ? 0 : static_cast<int>(n);
    s.len = s.bad ? 0 : static_cast<int>(len);
    s.blocks = (s.n * a.heads + nt - 1) / nt;
    s.tiles = s.blocks > 0 ? (s.len + kPos - 1) / kPos : 0;
    return s;
}
// What an item's beginning and end cost, in tiles, when there are several tiles for every CTA.  Sixteen sequences of
// 4001-8201 positions with 64 rows take 47.7, 45.1, 42.8, 41.7 and 41.5 us with 0, 2, 4, 6 and 8; four with 1024
// rows 84.5, 83.1, 81.2, 81.8 and 82.8; 64 of 801-8209 with 16 rows 69.1, 67.1, 67.2, 67.6 and 68.1.
constexpr int kEndCost = 4;
__device__ __forceinline__ int end_cost(const LatentArgs &a, long long tiles, int ctas) {
    return tiles > 2ll * ctas && !a.undivided ? kEndCost : 0;
}

struct Part {
    Rows s;
    long long at, end, item0;   // next unit of the list, the range's end, the item's first unit
    int b, blk, lo, hi;
    int extra;                  // units of an item before its tiles
    int index;                  // items walked before
    bool whole, first;          // the item lies in this CTA alone; the range's first item has not been looked at
};

// The whole warp calls these; the outcome is uniform.
template <int NT>
__device__ __forceinline__ void part_begin(const LatentArgs &a, Part &w, bool report) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    w.index = -1;
    w.b = w.blk = 0;
    w.at = w.end = w.item0 = 0;
    w.extra = 0;
    w.first = true;
    // 32 sequences a step; the last step's stay in registers (all of them, when there is one step)
    Rows mine;
    mine.bad = false;
    long long tiles = 0, items = 0, in_tiles = 0, in_items = 0, all_tiles = 0, all_items = 0;
    auto step = [&](int b0) {
        tiles = items = 0;
        if (b0 + lane < a.seqs) {
            mine = load_rows(a, NT, b0 + lane);
            items = mine.tiles > 0 ? mine.blocks : 0;
            tiles = items * mine.tiles;
        }
        in_tiles = tiles;
        in_items = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, in_tiles, o), z = __shfl_up_sync(0xFFFFFFFFu, in_items, o);
            if (lane >= o) {
                in_tiles += y;
                in_items += z;
            }
        }
    };
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        step(b0);
        if (b0 + lane < a.seqs && mine.bad && report) record_error(a.err, MOE_ERR_BAD_ID);
        all_tiles += __shfl_sync(0xFFFFFFFFu, in_tiles, 31);
        all_items += __shfl_sync(0xFFFFFFFFu, in_items, 31);
    }
    w.extra = end_cost(a, all_tiles, gridDim.x);
    const long long W = all_tiles + w.extra * all_items;
    const int C = used_ctas(W, gridDim.x), c = static_cast<int>(blockIdx.x);
    if (c >= C) return;
    w.at = range_lo(W, c, C);
    w.end = range_lo(W, c + 1, C);
    long long before = 0;   // units of the sequences before
    for (int b0 = 0;; b0 += 32) {
        if (a.seqs > 32) step(b0);
        const long long upto = in_tiles + w.extra * in_items;
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + upto > w.at);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            w.b = b0 + l;
            before += __shfl_sync(0xFFFFFFFFu, upto - tiles - w.extra * items, l);
            w.s.t0 = __shfl_sync(0xFFFFFFFFu, mine.t0, l);
            w.s.n = __shfl_sync(0xFFFFFFFFu, mine.n, l);
            w.s.ctx = __shfl_sync(0xFFFFFFFFu, mine.ctx, l);
            w.s.len = __shfl_sync(0xFFFFFFFFu, mine.len, l);
            w.s.tiles = __shfl_sync(0xFFFFFFFFu, mine.tiles, l);
            w.s.blocks = __shfl_sync(0xFFFFFFFFu, mine.blocks, l);
            w.s.bad = false;
            break;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    const long long into = w.at - before;
    const int size = w.s.tiles + w.extra;
    w.blk = into < (1ll << 31) ? static_cast<int>(static_cast<uint32_t>(into) / static_cast<uint32_t>(size)) : static_cast<int>(into / size);
    w.item0 = before + static_cast<long long>(w.blk) * size;
}
// Sets the next item's part; false at the end of the range.
template <int NT>
__device__ __forceinline__ bool part_next(const LatentArgs &a, Part &w) {
    while (w.at < w.end) {
        if (!w.first) {   // step to the item at w.at
            w.item0 += w.s.tiles + w.extra;
            if (++w.blk == w.s.blocks) {
                w.blk = 0;
                do {
                    w.s = load_rows(a, NT, ++w.b);
                } while (w.s.tiles == 0);   // there are units left, so one follows
            }
        }
        w.first = false;
        const long long tile0 = w.item0 + w.extra, stop = min(w.end, tile0 + w.s.tiles);
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
// The producer walks, the others follow it through a ring of records.  It is at most four items ahead of the
// last: before its next item it waits for a place that the output's product of the tile three before
// frees, and that product's weights came from scores of all tiles up to it.
template <int NT>
__device__ __forceinline__ bool part_lead(const LatentArgs &a, Part &w, Follow &f) {
    const bool more = part_next<NT>(a, w);
    if ((threadIdx.x & 31) == 0) {
        Item *const r = reinterpret_cast<Item *>(f.ring) + f.n % kRecords;
        const Item x = {w.s.t0, w.s.n, w.s.ctx, w.s.len, w.b, w.blk, more ? w.lo : -1, w.hi, w.index, w.whole ? 1 : 0};
        *r = x;
    }
    warp_arrive(f.bars + 8u * (f.n % kRecords));
    ++f.n;
    return more;
}
__device__ __forceinline__ bool part_follow(const LatentArgs &a, Item &w, Follow &f, volatile int32_t *abort_flag) {
    if (!wait_for(f.bars + 8u * (f.n % kRecords), (f.n / kRecords) & 1u, abort_flag, a.err, a.wait_limit)) return false;
    w = reinterpret_cast<const Item *>(f.ring)[f.n % kRecords];
    ++f.n;
    return w.lo >= 0;   // negative: the end
}

// Partial results: per CTA two slots (its first item, its last), each [NT rows][kPitch] fp32 of unnormalised
// output (a constant step: with the rank's own the stores took three times as long), then, after all
// slots, [slot][NT] (maximum, sum).
constexpr int kPitch = 512;
__host__ __device__ constexpr int units_of(int rank) { return (rank + 127) / 128; }
__device__ __forceinline__ float *part_o(const LatentArgs &a, int nt, int slot) {
    return static_cast<float *>(a.part) + static_cast<size_t>(slot) * nt * kPitch;
}
__device__ __forceinline__ float2 *part_s(const LatentArgs &a, int nt, int ctas, int slot) {
    return reinterpret_cast<float2 *>(part_o(a, nt, 2 * ctas)) + static_cast<size_t>(slot) * nt;
}

// ------------------------------------------------------------------ the kernel
template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_r,
                   const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ LatentArgs a, int box_rows, int q_map) {
    using L = Lay<NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::oBar + 8u * i; };
    volatile int32_t *const abort_flag = reinterpret_cast<volatile int32_t *>(smem + L::oMisc + 4);
    volatile uint32_t *const copied = reinterpret_cast<volatile uint32_t *>(smem + L::oMisc + 8);
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const long long limit = a.wait_limit;
    const int U = units_of(a.cache.rank);

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NU; ++i) {
            mbar_init(bar(L::bUF + i), 1);
            mbar_init(bar(L::bUE + i), 1);
        }
        for (int i = 0; i < L::NR; ++i) {
            mbar_init(bar(L::bRF + i), 1);
            mbar_init(bar(L::bRE + i), 1);
            mbar_init(bar(L::bP + i), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::bS + i), 1);
            mbar_init(bar(L::bSFree + i), 8);
        }
        mbar_init(bar(L::bQ), q_map ? 1 : 8);
        mbar_init(bar(L::bSeen), 2);
        mbar_init(bar(L::bO), 1);
        for (int i = 0; i < kRecords; ++i) mbar_init(bar(L::bW + i), 1);
        mbar_init(bar(L::bDrain), 3);
        *abort_flag = 0;
        copied[0] = copied[1] = copied[2] = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_c);
        tma_prefetch_map(&tm_r);
    }
    if (warp == kScoreWarp) {
        tmem_alloc(base + L::oMisc, L::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(smem + L::oMisc), 0);
    Follow follow = {smem + L::oWalk, bar(L::bW), 0};
    pdl_wait();
    pdl_trigger();

    if (warp == kProducerWarp) {
        // -------------------------------------------------------------------- copies
        Part w;
        part_begin<NT>(a, w, blockIdx.x == 0);
        const moe_latent_cache_t &kc = a.cache;
        const int boxes = kPos / box_rows, per = 32 / boxes;   // boxes of a tile, tiles of 32 boxes' places
        constexpr int kOutside = -2147483647;                  // a box beyond the length
        uint32_t uc = 0, rc = 0;                               // units, rotary tiles
        bool ok = true;
        while (ok && part_lead<NT>(a, w, follow)) {
            const int32_t *const table = a.page_table + static_cast<int64_t>(w.b) * a.max_pages;
            // the places of 32 boxes, a lane each; the next ones are on their way while these are used
            auto places = [&](int first, int &page, int &row) {
                const int64_t pos = (static_cast<int64_t>(first) * boxes + lane) * box_rows;
                page = kOutside;
                row = 0;
                if (pos < w.s.len) {
                    page = max(__ldg(table + static_cast<int>(pos) / kc.page), -1);
                    row = static_cast<int>(pos) % kc.page;
                }
            };
            int page_now, row_now, page_next, row_next;
            places(w.lo, page_now, row_now);
            places(w.lo + per, page_next, row_next);
            for (int tt = w.lo, k = 0; ok && tt < w.hi; ++tt, ++k, ++rc) {
                if (k == per) {
                    k = 0;
                    page_now = page_next;
                    row_now = row_next;
                    places(tt + per, page_next, row_next);
                }
                int page = __shfl_sync(0xFFFFFFFFu, page_now, k * boxes + lane % boxes);
                const int row = __shfl_sync(0xFFFFFFFFu, row_now, k * boxes + lane % boxes);
                const bool mine = lane < boxes && page != kOutside;
                if (mine && static_cast<uint32_t>(page) >= static_cast<uint32_t>(kc.pages)) {
                    record_error(a.err, MOE_ERR_BAD_ID);
                    page = kc.pages;   // beyond the tensor: the copy writes zeros
                }
                const uint32_t rs = rc % L::NR;
                if (!(ok = wait_for(bar(L::bRE + rs), ((rc / L::NR) & 1u) ^ 1u, abort_flag, a.err, limit))) break;
                const uint32_t r_dst = base + L::oR + rs * kRopeTile, r_bar = bar(L::bRF + rs);
                const int n = __popc(__ballot_sync(0xFFFFFFFFu, mine));   // the first n boxes
                const uint32_t bytes = static_cast<uint32_t>(n * box_rows) * 128u;
                // Issued by an elected lane from uniform registers, up to E boxes one after the other: by a lane for
                // each box a unit took 450 cycles (64 sequences of 801-8209 positions, pages of 8, 16 and 32: 106.8,
                // 71.9 and 68.3 us against 84, 69.8 and 68.1; unrolled for eight boxes, pages of 16 take 71.5).
                auto issue = [&](auto most) {
                    constexpr int E = decltype(most)::value;
                    int page_e[E], row_e[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        page_e[e] = __shfl_sync(0xFFFFFFFFu, page, e % boxes);
                        row_e[e] = __shfl_sync(0xFFFFFFFFu, row, e % boxes);
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(r_bar, bytes);
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (e < n) tma_load_3d(r_dst + e * box_rows * 128u, &tm_r, r_bar, 0, row_e[e], page_e[e]);
                    }
                    __syncwarp();
                    for (int u = 0; u < U; ++u, ++uc) {
                        const uint32_t slot = uc % L::NU, u_dst = base + L::oU + slot * kUnit, u_bar = bar(L::bUF + slot);
                        if (!wait_for(bar(L::bUE + slot), ((uc / L::NU) & 1u) ^ 1u, abort_flag, a.err, limit)) return false;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(u_bar, 2 * bytes);
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                if (e >= n) continue;
                                tma_load_3d(u_dst + e * box_rows * 128u, &tm_c, u_bar, u * 128, row_e[e], page_e[e]);
                                tma_load_3d(u_dst + 8192u + e * box_rows * 128u, &tm_c, u_bar, u * 128 + 64, row_e[e], page_e[e]);
                            }
                        }
                        __syncwarp();
                    }
                    return true;
                };
                ok = boxes <= 4 ? issue(std::integral_constant<int, 4>()) : issue(std::integral_constant<int, 8>());
                if (!ok) {
                    ++rc;   // the rotary tile's copies are on their way
                    break;
                }
            }
        }
        if (lane == 0) {
            copied[0] = uc;
            copied[1] = rc;
        }
    } else if (warp == kScoreWarp || warp == kScoreWarp + 1) {
        // -------------------------------------------------------------------- S^T = C Q^T
        // Two warps take alternate tiles: the turn of one's loop (waits, fences, the first product's issue) takes
        // as long as ten products, and the other's products go on meanwhile.
        const uint32_t side = static_cast<uint32_t>(warp - kScoreWarp), s_col = tmem + side * NT;
        Item w;
        const uint64_t q_desc = desc_kmajor_sw128(base + L::oQ);
        const int rope_steps = (a.cache.rope + 15) / 16;
        uint32_t c = 0, uc = 0, items = 0;
        bool ok = true;
        while (ok && part_follow(a, w, follow, abort_flag)) {
            ok = wait_for(bar(L::bQ), items & 1u, abort_flag, a.err, limit);
            if (ok) warp_arrive(bar(L::bSeen));
            const int T = __shfl_sync(0xFFFFFFFFu, w.hi - w.lo, 0);
            for (int t = 0; ok && t < T; ++t, ++c) {
                if ((c & 1u) != side) {
                    uc += U;
                    continue;
                }
                const uint32_t rs = c % L::NR;
                // The softmax has taken this buffer's previous scores, tile c - 2's.  So that tile and all before it
                // have landed, the ring's previous uses of this one's places among them, and the parities
                // below tell this use from those.
                ok = (c < 2 || wait_for(bar(L::bSFree + side), ((c >> 1) - 1) & 1u, abort_flag, a.err, limit)) &&
                     wait_for(bar(L::bRF + rs), (c / L::NR) & 1u, abort_flag, a.err, limit);
                if (!ok) break;
                tc_fence_after();
                const uint64_t r_desc = desc_kmajor_sw128(base + L::oR + rs * kRopeTile);
                if (elect_one()) {
                    for (int i = 0; i < rope_steps; ++i)
                        tc_mma_bf16(s_col, r_desc + 2 * i, q_desc + 2 * U * (L::kQBlock / 16) + 2 * i, idesc_bf16_f32(64, NT), i > 0);
                }
                __syncwarp();
                for (int u = 0; u < U;) {
                    // a unit, and those behind it that have landed too
                    uint32_t slot = uc % L::NU;
                    if (!(ok = wait_for(bar(L::bUF + slot), (uc / L::NU) & 1u, abort_flag, a.err, limit))) break;
                    int n = 1;
                    while (u + n < U && __all_sync(0xFFFFFFFFu, mbar_test_wait(bar(L::bUF + (uc + n) % L::NU), ((uc + n) / L::NU) & 1u))) ++n;
                    tc_fence_after();
                    if (elect_one()) {
                        uint64_t qd = q_desc + 2 * u * (L::kQBlock / 16);
                        for (int k = 0; k < n; ++k) {
                            const uint64_t c_desc = desc_kmajor_sw128(base + L::oU + slot * kUnit);
#pragma unroll
                            for (int i = 0; i < 8; ++i)   // two blocks of 64 channels
                                tc_mma_bf16(s_col, c_desc + (i / 4) * 512 + (i % 4) * 2, qd + (i / 4) * (L::kQBlock / 16) + (i % 4) * 2,
                                            idesc_bf16_f32(64, NT), 1);
                            qd += 2 * (L::kQBlock / 16);
                            if (++slot == L::NU) slot = 0;
                        }
                        if (u + n == U) tc_commit(bar(L::bS + side));
                    }
                    __syncwarp();
                    u += n;
                    uc += n;
                }
            }
            ++items;
        }
        // every product is done before the CTA leaves
        if (elect_one()) tc_commit(bar(L::bDrain));
        __syncwarp();
        mbar_wait_drain(bar(L::bDrain), 0, kDrain);
        __syncwarp();
    } else if (warp == kOutWarp) {
        // -------------------------------------------------------------------- O^T += C^T P^T, tile by tile
        Item w;
        uint32_t c = 0, uc = 0;
        bool ok = true;
        while (ok && part_follow(a, w, follow, abort_flag)) {
            const int T = __shfl_sync(0xFFFFFFFFu, w.hi - w.lo, 0);
            for (int t = 0; ok && t < T; ++t, ++c) {
                const uint32_t rs = c % L::NR;
                // the units that the product reads: complete before the scores were
                for (int u = 0; ok && u < U; ++u)
                    ok = wait_for(bar(L::bUF + (uc + u) % L::NU), ((uc + u) / L::NU) & 1u, abort_flag, a.err, limit);
                // (the first weights of an item come after the previous item's O was read)
                ok = ok && wait_for(bar(L::bP + rs), (c / L::NR) & 1u, abort_flag, a.err, limit);
                if (!ok) break;
                tc_fence_after();
                const uint64_t p_desc = desc_p<NT>(base + L::oR + rs * kRopeTile);
                uint32_t slot = uc % L::NU;
                if (elect_one()) {
                    for (int u = 0; u < U; ++u) {
                        const uint64_t c_desc = desc_mn_sw128(base + L::oU + slot * kUnit, 8192u);
#pragma unroll
                        for (int i = 0; i < kPos / 16; ++i)   // 16 positions: 2 KB of a block, 2 atoms of P
                            tc_mma_bf16(tmem + (2 + u) * NT, c_desc + 128 * i, p_desc + (16 * NT * 2 / 16) * i, idesc_vp(NT, 1),
                                        t > 0 || i > 0);
                        tc_commit(bar(L::bUE + slot));
                        if (++slot == L::NU) slot = 0;
                    }
                    tc_commit(bar(L::bRE + rs));
                    if (t == T - 1) tc_commit(bar(L::bO));
                }
                __syncwarp();
                uc += U;
            }
        }
        if (elect_one()) tc_commit(bar(L::bDrain));
        __syncwarp();
        mbar_wait_drain(bar(L::bDrain), 0, kDrain);
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- softmax, two warpgroups
        constexpr int H = NT / 2, G8 = H / 8;   // a warpgroup's rows, in eights
        const int g = warp >> 2, q4 = warp & 3, p = q4 * 32 + lane;
        const int pos0 = q4 * 16 + (lane >> 2), col = (lane & 3) * 2;   // the thread's positions pos0, pos0 + 8 and first row of eight
        const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
        float *const nm_s = reinterpret_cast<float *>(smem + L::oM) + g * H;
        float *const alpha_s = reinterpret_cast<float *>(smem + L::oAlpha) + g * H;
        uint64_t *const mask_s = reinterpret_cast<uint64_t *>(smem + L::oMask) + g * H;
        float *const red_s = reinterpret_cast<float *>(smem + L::oRed) + g * 4 * H;
        uint32_t *const bad_s = reinterpret_cast<uint32_t *>(smem + L::oBad);
        const Divisor by_heads(a.heads);
        const bool even_out = a.out.token_stride == static_cast<int64_t>(a.heads) * a.out.head_stride;
        bool dead = false;   // a wait gave up: only the barriers are kept
        uint32_t c = 0;      // tiles
        Item w = {}, next;
        // An item's queries into shared memory: blocks of 64 channels, [NT rows][128 bytes], the rotary channels'
        // block last.  Rows that are one step apart are copied (q_map): loaded by these threads, 64 rows took
        // 8,000 cycles behind the first tiles' copies.
        uint64_t next_mask = 0;   // of row g * H + p
        auto load_queries = [&](const Item &v) {
            const int R = v.n * a.heads - v.blk * NT;
            // the row's mask goes to shared memory when the present item's are done with
            next_mask = 0;
            if (p < H && g * H + p < R) {
                const uint32_t token = by_heads.quotient(static_cast<uint32_t>(v.blk * NT + g * H + p));
                next_mask = a.mask != nullptr ? a.mask[v.t0 + static_cast<int>(token)] : (2ull << token) - 1ull;
                if (v.n < 64) next_mask &= (1ull << v.n) - 1ull;
            }
            // Both score warps have found the previous item's: with one tile to an item only one of them has formed
            // its scores, and the other's wait by parity would miss a phase that the next one's completion hides.
            if (v.index > 0 && !dead && (!q_map || warp == 0))
                dead = !wait_for(bar(L::bSeen), static_cast<uint32_t>(v.index - 1) & 1u, abort_flag, a.err, limit);
            if (dead) return;
            if (q_map) {   // (rows beyond the block's are another's, or zeros: their columns go nowhere)
                if (warp == 0) {
                    if (elect_one()) {
                        const int row = v.t0 * a.heads + v.blk * NT;
                        mbar_arrive_expect_tx(bar(L::bQ), static_cast<uint32_t>(2 * U + 1) * L::kQBlock);
                        for (int b = 0; b < 2 * U; ++b) tma_load_2d(base + L::oQ + b * L::kQBlock, &tm_q, bar(L::bQ), b * 64, row);
                        tma_load_2d(base + L::oQ + 2 * U * L::kQBlock, &tm_q, bar(L::bQ), a.cache.rank, row);
                        copied[2] = static_cast<uint32_t>(v.index) + 1;
                    }
                    __syncwarp();
                }
                return;
            }
            const int pieces = (2 * U + 1) * NT * 8;
            constexpr int BATCH = 9;
            // 16 bytes a piece; rows beyond the block's repeat its last one, channels beyond are zeros
            const int row0 = v.blk * NT, last = min(R, NT) - 1;
            const uint16_t *const q = static_cast<const uint16_t *>(a.q.ptr) + static_cast<int64_t>(v.t0) * a.q.token_stride;
#pragma unroll 1
            for (int i0 = static_cast<int>(threadIdx.x); i0 < pieces; i0 += BATCH * 256) {
                uint4 x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int at = i0 + i * 256, block = at / (NT * 8), ch = at % 8 * 8;
                    const bool rope = block == 2 * U;
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (at < pieces && (rope ? ch < a.cache.rope : block * 64 + ch < a.cache.rank)) {
                        const uint32_t r = static_cast<uint32_t>(row0 + min(at / 8 % NT, last)), token = by_heads.quotient(r);
                        x[i] = *reinterpret_cast<const uint4 *>(q + static_cast<int64_t>(token) * a.q.token_stride +
                                                                static_cast<int64_t>(r - token * a.heads) * a.q.head_stride +
                                                                (rope ? a.cache.rank : block * 64) + ch);
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int at = i0 + i * 256, block = at / (NT * 8), row = at / 8 % NT, chunk = at % 8;
                    if (at < pieces)
                        *reinterpret_cast<uint4 *>(smem + L::oQ + block * L::kQBlock + row * 128 + ((chunk ^ (row & 7)) * 16)) = x[i];
                }
            }
            fence_proxy_async_smem();
            warp_arrive(bar(L::bQ));
        };
        // The latents as the output's product may have them: positions beyond the length become zeros (their
        // weights are 0, what the ring holds there may be anything), and so do non-finite elements of
        // drafted tokens, which a row that does not see them must not meet.  The scores of the tile are
        // complete, so this changes nothing of them; and where all of them are finite, so are the latents,
        // and are not looked at.  (odd: a warpgroup whose scores are not looks at the whole tile.)
        auto clean = [&](int tt, bool odd) {
            const int first = max(0, w.ctx - tt * kPos), stop = min(kPos, w.len - tt * kPos);
            if (stop < kPos) {
                const int chunk = static_cast<int>(threadIdx.x) & 15, r0 = static_cast<int>(threadIdx.x) >> 4;
                for (int u = 0; u < U; ++u) {
                    uint8_t *const v = smem + L::oU + ((c * U + u) % L::NU) * kUnit + (chunk >> 3) * 8192 + (chunk & 7) * 16;
                    for (int r = stop + r0; r < kPos; r += 16) *reinterpret_cast<uint4 *>(v + r * 128) = make_uint4(0, 0, 0, 0);
                }
            }
            if (!bar_any(2 + g, 128, odd)) return;
            const int chunk = p & 15;
            uint32_t *const bad = bad_s + (w.index & 1) * 2;
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                uint8_t *const v = smem + L::oU + ((c * U + u) % L::NU) * kUnit + (chunk >> 3) * 8192;
#pragma unroll 1
                for (int r = first + (p >> 4); r < stop; r += 8) {
                    uint4 *const q = reinterpret_cast<uint4 *>(v + r * 128 + (((chunk & 7) ^ (r & 7)) * 16));
                    uint4 y = *q;
                    // bit 15 of a half whose exponent is all ones
                    auto over = [](uint32_t z) { return ((z & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
                    if ((over(y.x) | over(y.y) | over(y.z) | over(y.w)) == 0) continue;
                    y.x &= ~((over(y.x) >> 15) * 0xFFFFu);
                    y.y &= ~((over(y.y) >> 15) * 0xFFFFu);
                    y.z &= ~((over(y.z) >> 15) * 0xFFFFu);
                    y.w &= ~((over(y.w) >> 15) * 0xFFFFu);
                    *q = y;
                    const int d = tt * kPos + r - w.ctx;
                    atomicOr(&bad[d >> 5], 1u << (d & 31));
                }
            }
        };
        bool more = part_follow(a, next, follow, abort_flag);
        if (more) load_queries(next);
        while (true) {
            if (threadIdx.x < 2 && more) bad_s[(next.index & 1) * 2 + threadIdx.x] = 0;
            // the previous item's shared words have been read; everybody leaves together
            if (bar_any(1, 256, dead || *abort_flag != 0) || !more) break;
            w = next;
            const int T = w.hi - w.lo;
            const uint32_t *const bad = bad_s + (w.index & 1) * 2;
            float m_own = kNone;   // of row g * H + p
            bool all_seen = false;
            if (p < H) {
                nm_s[p] = 0.0f;
                mask_s[p] = next_mask;
            }
            F2 l2[G8];
#pragma unroll
            for (int i = 0; i < G8; ++i) l2[i] = f2(0.0f, 0.0f);
            named_barrier(2 + g, 128);
            // The first item begins with a pass over nothing, which brings the loop's code into the instruction
            // caches while the first tiles are on their way: after them, behind all CTAs' copies, the first tile's
            // weights took 4,500 cycles, not 600, and the ring stood still meanwhile.
            for (int t = w.index == 0 ? -1 : 0; t < T; ++t) {
                const bool dry = t < 0;
                const int tt = w.lo + t;
                const uint32_t buf = c & 1u, rs = c % L::NR;
                const bool edge = !dry && (tt + 1) * kPos > w.ctx;
                uint32_t x[4 * G8];
                if (!dead && !dry) dead = !wait_for(bar(L::bS + buf), (c >> 1) & 1u, abort_flag, a.err, limit);
                tc_fence_after();
                tmem_ld_16x256<G8>(tmem + lanes + buf * NT + g * H, x);
                tmem_wait_ld();
                tc_fence_before();
                if (!dead && !dry) warp_arrive(bar(L::bSFree + buf));
                bool odd_scores = false;   // of drafted tokens
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 4 * G8; ++i)
                        odd_scores |= tt * kPos + pos0 + (i & 2) * 4 >= w.ctx && !(fabsf(__uint_as_float(x[i])) <= 3.4028234e38f);
                }
                // scores in log2 units above the rows' maxima so far (above 0 where a row has none); what a
                // row does not see is -inf
                const F2 scale2 = f2(a.scale_log2, a.scale_log2);
                float2 ref[G8];
#pragma unroll
                for (int i = 0; i < G8; ++i) {
                    const float2 n = ref[i] = *reinterpret_cast<const float2 *>(nm_s + 8 * i + col);
                    float s[4];
                    f2_get(f2_fma(f2(x[4 * i], x[4 * i + 1]), scale2, f2(n.x, n.y)), s[0], s[1]);
                    f2_get(f2_fma(f2(x[4 * i + 2], x[4 * i + 3]), scale2, f2(n.x, n.y)), s[2], s[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[4 * i + k] = __float_as_uint(s[k]);
                }
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int d = tt * kPos + pos0 + 8 * h - w.ctx;   // drafted token; masks have no bits beyond n
                        if (d < 0) continue;
#pragma unroll
                        for (int i = 0; i < G8; ++i)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                if (d >= 64 || !(mask_s[8 * i + col + k] >> d & 1ull)) x[4 * i + 2 * h + k] = __float_as_uint(ninf());
                    }
                }
                float over = ninf();
#pragma unroll
                for (int i = 0; i < 4 * G8; i += 2) over = fmaxf(over, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                // any score far above its row's largest so far, or a row that had seen nothing?
                if (bar_any(2 + g, 128, !all_seen || over > kLazy)) {
                    // the rows' maxima over the tile (NaN left out): over the warp's positions, then the four warps
                    float top[2 * G8];
#pragma unroll
                    for (int i = 0; i < 2 * G8; ++i) {
                        const int k = 4 * (i / 2) + i % 2;
                        top[i] = fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 2]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
                    }
                    if (lane < 4) {
#pragma unroll
                        for (int i = 0; i < 2 * G8; ++i) red_s[q4 * H + 8 * (i / 2) + col + i % 2] = top[i];
                    }
                    named_barrier(2 + g, 128);
                    bool unseen = false;
                    if (p < H) {
                        const float n = nm_s[p];
                        const float here = fmaxf(fmaxf(red_s[p], red_s[H + p]), fmaxf(red_s[2 * H + p], red_s[3 * H + p]));
                        const float mn = fmaxf(m_own, here - n);
                        unseen = mn == kNone;
                        const float n_new = unseen ? 0.0f : -mn;
                        nm_s[p] = n_new;
                        alpha_s[p] = ex2(m_own - mn);
                        m_own = mn;
                    }
                    all_seen = !bar_any(2 + g, 128, unseen);
#pragma unroll
                    for (int i = 0; i < G8; ++i) {
                        float2 n = *reinterpret_cast<const float2 *>(nm_s + 8 * i + col);
                        n.x -= ref[i].x;
                        n.y -= ref[i].y;
                        const float2 k = *reinterpret_cast<const float2 *>(alpha_s + 8 * i + col);
                        float s[4];
                        f2_get(f2_add(f2(x[4 * i], x[4 * i + 1]), f2(n.x, n.y)), s[0], s[1]);
                        f2_get(f2_add(f2(x[4 * i + 2], x[4 * i + 3]), f2(n.x, n.y)), s[2], s[3]);
                        l2[i] = f2_mul(l2[i], f2(k.x, k.y));
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[4 * i + j] = __float_as_uint(s[j]);
                    }
                    if (t > 0) {
                        // O so far is complete when the previous product is
                        if (!dead) dead = !wait_for(bar(L::bRE + (c - 1) % L::NR), ((c - 1) / L::NR) & 1u, abort_flag, a.err, limit);
                        tc_fence_after();
                        for (int u = 0; u < U; ++u) {
                            uint32_t o[H];
                            tmem_ld_rows<H>(tmem + lanes + (2 + u) * NT + g * H, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < H; i += 4) {
                                const float4 k = *reinterpret_cast<const float4 *>(alpha_s + i);
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * k.x);
                                o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) * k.y);
                                o[i + 2] = __float_as_uint(__uint_as_float(o[i + 2]) * k.z);
                                o[i + 3] = __float_as_uint(__uint_as_float(o[i + 3]) * k.w);
                            }
                            tmem_st_rows<H>(tmem + lanes + (2 + u) * NT + g * H, o);
                        }
                        tmem_wait_st();
                    }
                }
                // (in the place of the rotary channels: the scores are complete)
                uint8_t *const p_buf = smem + L::oR + rs * kRopeTile + col * 2;
#pragma unroll
                for (int i = 0; i < G8; ++i) {
                    float w0 = ex2(__uint_as_float(x[4 * i])), w1 = ex2(__uint_as_float(x[4 * i + 1]));
                    float w2 = ex2(__uint_as_float(x[4 * i + 2])), w3 = ex2(__uint_as_float(x[4 * i + 3]));
                    l2[i] = f2_add(l2[i], f2_add(f2(w0, w1), f2(w2, w3)));
                    if (!dry) {
                        *reinterpret_cast<uint32_t *>(p_buf + p_chunk<NT>(pos0, g * G8 + i)) = pack2(w0, w1, false);
                        *reinterpret_cast<uint32_t *>(p_buf + p_chunk<NT>(pos0 + 8, g * G8 + i)) = pack2(w2, w3, false);
                    }
                }
                if (edge) clean(tt, odd_scores);
                fence_proxy_async_smem();
                tc_fence_before();
                if (dry) {   // as before it
                    m_own = kNone;
                    all_seen = false;
                    if (p < H) nm_s[p] = 0.0f;
#pragma unroll
                    for (int i = 0; i < G8; ++i) l2[i] = f2(0.0f, 0.0f);
                    named_barrier(2 + g, 128);
                    continue;
                }
                if (!dead) warp_arrive(bar(L::bP + rs));
                ++c;
            }
            // ------------------------------------------------------------ the item's end
            // every score of the item is formed: the next one's queries may take the place of these
            more = part_follow(a, next, follow, abort_flag);
            if (more) load_queries(next);
            float l[2 * G8];
#pragma unroll
            for (int i = 0; i < G8; ++i) f2_get(l2[i], l[2 * i], l[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 2 * G8; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
            }
            if (lane < 4) {
#pragma unroll
                for (int i = 0; i < 2 * G8; ++i) red_s[q4 * H + 8 * (i / 2) + col + i % 2] = l[i];
            }
            named_barrier(2 + g, 128);
            const int R = w.n * a.heads - w.blk * NT;   // the block's rows (more, where others follow)
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.index == 0 ? 0 : 1);
            if (p < H) {
                const int r = g * H + p;
                const float mm = m_own == kNone ? ninf() : m_own;
                const float ll = red_s[p] + red_s[H + p] + red_s[2 * H + p] + red_s[3 * H + p];
                const bool none = mm == ninf() && ll == 0.0f;
                alpha_s[p] = !w.whole ? 1.0f : (none ? 0.0f : 1.0f / ll);
                if (r < R) {
                    if (!w.whole) {
                        part_s(a, NT, gridDim.x, slot)[r] = make_float2(mm, ll);
                    } else if (a.lse != nullptr) {
                        const uint32_t row = static_cast<uint32_t>(w.blk * NT + r), token = by_heads.quotient(row);
                        a.lse[static_cast<int64_t>(w.t0 + static_cast<int>(token)) * a.heads + (row - token * a.heads)] =
                            none ? ninf() : (mm + log2f(ll)) * 0.69314718055994531f;
                    }
                }
            }
            named_barrier(2 + g, 128);
            if (!dead) dead = !wait_for(bar(L::bO), static_cast<uint32_t>(w.index) & 1u, abort_flag, a.err, limit);
            tc_fence_after();
            // non-finite latents of drafted tokens (of parts that reach past the context: the products waited
            // for the words there)
            const uint64_t odd_tokens = w.hi * kPos > w.ctx ? *reinterpret_cast<const uint64_t *>(bad) : 0ull;
            for (int u = 0; u < U; ++u) {
                uint32_t o[H];
                tmem_ld_rows<H>(tmem + lanes + (2 + u) * NT + g * H, o);
                tmem_wait_ld();
                const int ch = u * 128 + p;
#pragma unroll
                for (int i = 0; i < H; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha_s[i]);
                if (odd_tokens != 0 && ch < a.cache.rank) {
#pragma unroll 1
                    for (uint64_t left = odd_tokens; left != 0; left &= left - 1) {
                        const int d = __ffsll(static_cast<long long>(left)) - 1, pos = w.ctx + d;
                        const int page = a.page_table[static_cast<int64_t>(w.b) * a.max_pages + pos / a.cache.page];
                        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.pages)) continue;
                        const uint32_t v = static_cast<const uint16_t *>(
                            a.cache.rows)[page * a.cache.page_stride + pos % a.cache.page * a.cache.token_stride + ch];
                        if ((v & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            if (mask_s[i] >> d & 1ull) o[i] = 0x7FFFFFFFu;
                    }
                }
                __syncwarp();
                if (!w.whole) {   // (rows beyond the block's too: they are read by nobody)
                    float *const po = part_o(a, NT, slot) + g * H * kPitch + ch;
#pragma unroll
                    for (int i = 0; i < H; ++i) po[i * kPitch] = __uint_as_float(o[i]);
                    continue;
                }
                // two rows at a time: neighbouring lanes trade, and each stores two channels of one row
                const int odd = lane & 1;
                uint32_t two[H / 2];
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float mine = __uint_as_float(odd ? o[i + 1] : o[i]);
                    const float other = __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, odd ? o[i] : o[i + 1], 1));
                    two[i / 2] = odd ? pack2(other, mine, false) : pack2(mine, other, false);
                }
                if (ch >= a.cache.rank) continue;
                uint16_t *const to = static_cast<uint16_t *>(a.out.ptr) + static_cast<int64_t>(w.t0) * a.out.token_stride + (ch & ~1);
                const int row0 = w.blk * NT + g * H + odd;
                if (even_out && g * H + H <= R) {   // rows one step apart, none beyond
                    uint16_t *at = to + row0 * a.out.head_stride;
#pragma unroll
                    for (int i = 0; i < H; i += 2, at += 2 * a.out.head_stride) *reinterpret_cast<uint32_t *>(at) = two[i / 2];
                } else {
#pragma unroll
                    for (int i = 0; i < H; i += 2) {
                        const uint32_t r = static_cast<uint32_t>(row0 + i), token = by_heads.quotient(r);
                        if (g * H + i + odd < R)
                            *reinterpret_cast<uint32_t *>(to + static_cast<int64_t>(token) * a.out.token_stride +
                                                          static_cast<int64_t>(r - token * a.heads) * a.out.head_stride) = two[i / 2];
                    }
                }
            }
            tc_fence_before();   // the next item's first product follows this warp's arrival on bP
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducerWarp && *abort_flag != 0) {
        // copies that nobody waited for must land before the CTA leaves
        const uint32_t uc = copied[0], rc = copied[1];
        for (uint32_t j = uc > L::NU ? uc - L::NU : 0; j < uc; ++j) mbar_wait_drain(bar(L::bUF + j % L::NU), (j / L::NU) & 1u, kDrain);
        const uint32_t qc = copied[2];   // (of one item at a time)
        if (qc > 0) mbar_wait_drain(bar(L::bQ), (qc - 1) & 1u, kDrain);
        for (uint32_t j = rc > L::NR ? rc - L::NR : 0; j < rc; ++j) mbar_wait_drain(bar(L::bRF + j % L::NR), (j / L::NR) & 1u, kDrain);
    }
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

// ------------------------------------------------------------------ joining the parts
// For an item that several CTAs shared: out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over its parts
// in order.  The parts lie in L2, so what counts is the chain of latencies and how many loads are in
// flight: a warp works by itself, its first parts on their way while it forms the weights, a lane per
// part.  MANY: the CTA's eight warps take every eighth part of 128 channels of a row and add up their
// sums in order; else a warp takes a row, or with few rows half of one.
constexpr int kJoinWarps = 8;

template <bool MANY, int UNITS>   // UNITS: of 128 channels that a warp takes
__global__ void __launch_bounds__(32 * kJoinWarps) latent_join_kernel(const __grid_constant__ LatentArgs a, int nt, int ctas) {
    constexpr int STEP = MANY ? kJoinWarps : 1, AHEAD = MANY ? 8 : 12 / UNITS;
    __shared__ float wt_s[kJoinWarps][kMaxCtas];
    __shared__ float4 sum_s[MANY ? kJoinWarps : 1][32];
    const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the lengths are no product of the first kernel, which waited for what came before it
    const Rows s = load_rows(a, nt, b);
    const int row = MANY ? blockIdx.x : blockIdx.x * kJoinWarps + warp, R = s.n * a.heads;
    if (row >= R) {   // (MANY: the whole CTA)
        pdl_wait();
        return;
    }
    long long sums[4] = {0, 0, 0, 0};   // tiles and items before, in all
    for (int i = lane; i < a.seqs; i += 32) {
        const Rows x = load_rows(a, nt, i);
        const long long items = x.tiles > 0 ? x.blocks : 0, tiles = items * x.tiles;
        sums[2] += tiles;
        sums[3] += items;
        if (i < b) {
            sums[0] += tiles;
            sums[1] += items;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sums[k] += __shfl_xor_sync(0xFFFFFFFFu, sums[k], o);
    }
    const int extra = end_cost(a, sums[2], ctas);
    const long long W = sums[2] + extra * sums[3];
    const int blk = row / nt, r = row % nt;
    const long long item0 = sums[0] + extra * sums[1] + static_cast<long long>(blk) * (s.tiles + extra);
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
    const int parts = cb - ca + 1, i0 = MANY ? warp : 0, ch = blockIdx.z * (UNITS * 128) + lane * 4;
    auto part = [&](int i, int u) { return *reinterpret_cast<const float4 *>(part_o(a, nt, slot(i)) + r * kPitch + u * 128 + ch); };
    float4 x[AHEAD][UNITS];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i0 + i * STEP < parts) {
#pragma unroll
            for (int u = 0; u < UNITS; ++u) x[i][u] = part(i0 + i * STEP, u);
        }
    float m = ninf(), l = 0.0f;
    float *const wt = wt_s[warp];
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, part_s(a, nt, ctas, slot(i))[r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float ref = m == ninf() ? 0.0f : m;
    for (int i = lane; i < parts; i += 32) {
        const float2 y = part_s(a, nt, ctas, slot(i))[r];
        const float k = ex2(y.x - ref);
        l += y.y * k;
        wt[i] = k;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const bool none = m == ninf() && l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l;
    if (a.lse != nullptr && lane == 0 && blockIdx.z == 0 && i0 == 0)
        a.lse[static_cast<int64_t>(s.t0 + row / a.heads) * a.heads + row % a.heads] = none ? ninf() : (m + log2f(l)) * 0.69314718055994531f;
    __syncwarp();
    float4 o[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = i0; p0 < parts; p0 += AHEAD * STEP) {
        if (p0 > i0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (p0 + i * STEP < parts) {
#pragma unroll
                    for (int u = 0; u < UNITS; ++u) x[i][u] = part(p0 + i * STEP, u);
                }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (p0 + i * STEP >= parts) continue;
            const float k = wt[p0 + i * STEP];
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                o[u].x = fmaf(x[i][u].x, k, o[u].x);
                o[u].y = fmaf(x[i][u].y, k, o[u].y);
                o[u].z = fmaf(x[i][u].z, k, o[u].z);
                o[u].w = fmaf(x[i][u].w, k, o[u].w);
            }
        }
    }
    if constexpr (MANY) {
        sum_s[warp][lane] = o[0];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int i = 1; i < kJoinWarps; ++i) {
            const float4 y = sum_s[i][lane];
            o[0].x += y.x;
            o[0].y += y.y;
            o[0].z += y.z;
            o[0].w += y.w;
        }
    }
    uint16_t *const to = static_cast<uint16_t *>(a.out.ptr) + static_cast<int64_t>(s.t0 + row / a.heads) * a.out.token_stride +
                         static_cast<int64_t>(row % a.heads) * a.out.head_stride + ch;
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        if (ch + u * 128 < a.cache.rank)
            *reinterpret_cast<uint2 *>(to + u * 128) =
                make_uint2(pack2(o[u].x * inv, o[u].y * inv, false), pack2(o[u].z * inv, o[u].w * inv, false));
}

// ------------------------------------------------------------------ host side
std::mutex g_mu;
struct Device {
    int sms = 0;
    bool set[3] = {false, false, false};
} g_dev[64];

int sm_count(int dev) {
    std::lock_guard<std::mutex> lock(g_mu);
    Device &d = g_dev[dev & 63];
    if (d.sms == 0) cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    return std::min(d.sms, kMaxCtas);
}

// `channels` of the rows from `first` on as a 3-D tensor (channel, row of a page, page); boxes of box_rows
// rows and 128 bytes.  Channels beyond and pages beyond the cache read as zeros.
bool encode_rows(CUtensorMap *map, const moe_latent_cache_t &c, int first, int channels, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    // a dimension of one element has no step; any valid stride will do
    auto stride = [](int64_t st, int extent) { return extent == 1 ? 16u * 1024u : static_cast<cuuint64_t>(st) * 2; };
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(c.page), static_cast<cuuint64_t>(c.pages)};
    cuuint64_t strides[2] = {stride(c.token_stride, c.page), stride(c.page_stride, c.pages)};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, static_cast<uint16_t *>(c.rows) + first, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as rows (token, head) one step apart, boxes of 64 channels by nt rows; false where they are not.
bool encode_queries(CUtensorMap *map, const LatentArgs &a, int nt) {
    EncodeTiledFn fn = encode_fn();
    const int64_t step = a.heads == 1 ? a.q.token_stride : a.q.head_stride;
    if (fn == nullptr || a.q.token_stride != a.heads * step || step < a.cache.rank + a.cache.rope) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.cache.rank + a.cache.rope), static_cast<cuuint64_t>(a.tokens) * a.heads};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(step) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(nt)};
    cuuint32_t estr[2] = {1, 1};
    return static_cast<int64_t>(a.tokens) * a.heads < (1ll << 31) &&
           fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.q.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch(const LatentArgs &a, int dev, int ctas, int rows, const CUtensorMap &tm_c, const CUtensorMap &tm_r,
                   cudaStream_t s, bool pdl) {
    CUtensorMap tm_q;
    const int q_map = encode_queries(&tm_q, a, NT) ? 1 : 0;
    if (!q_map) tm_q = tm_c;   // not used
    using L = Lay<NT>;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        bool &set = g_dev[dev & 63].set[NT / 32];
        if (!set) {
            const cudaError_t e = cudaFuncSetAttribute(latent_attn_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
            if (e != cudaSuccess) return e;
            set = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_attn_kernel<NT>, tm_c, tm_r, tm_q, a, rows, q_map);
}

template <bool MANY, int UNITS>
cudaError_t launch_join(const LatentArgs &a, int nt, int ctas, cudaStream_t s, bool pdl) {
    const int rows = a.max_tokens * a.heads;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(MANY ? rows : (rows + kJoinWarps - 1) / kJoinWarps, a.seqs, (units_of(a.cache.rank) + UNITS - 1) / UNITS);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_join_kernel<MANY, UNITS>, a, nt, ctas);
}

bool wide16(const moe_heads_t &h) {
    return (reinterpret_cast<uintptr_t>(h.ptr) & 15u) == 0 && h.token_stride % 8 == 0 && h.head_stride % 8 == 0;
}

}  // namespace

bool latent_attn_supports(const moe_latent_cache_t &c, const moe_heads_t &q, const moe_heads_t &out) {
    return q.dtype == MOE_BF16 && out.dtype == MOE_BF16 && c.dtype == MOE_BF16 && c.rope <= 64 && c.page % 8 == 0 && wide16(q) && wide16(out);
}

// For the device that is current when it is asked for: a larger one refuses such a workspace.
size_t latent_attn_part_bytes() {
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        const int n = sm_count(dev);
        if (n > 0) sms = n;
    }
    return static_cast<size_t>(sms) * 2 * 64 * (kPitch * sizeof(float) + sizeof(float2));
}

cudaError_t launch_latent_attn(LatentArgs a, cudaStream_t s, bool pdl) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = sm_count(dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    int box = 8;   // the largest power of two that divides a page, at most a tile
    while (box < kPos && a.cache.page % (2 * box) == 0) box *= 2;
    CUtensorMap tm_c, tm_r;
    if (!encode_rows(&tm_c, a.cache, 0, a.cache.rank, box) || !encode_rows(&tm_r, a.cache, a.cache.rank, a.cache.rope, box))
        return cudaErrorNotSupported;
    // Columns by the rows there can be: two sequences of 100-131 thousand positions with 16 rows each take 56.8 us with
    // 16 columns, 59.4 with 32 and 66.1 with 64; with 32 rows 59.8 and 66.1; 64 of 801-8209 with 16 rows 67.6, 70.6
    // and 79.0.
    const int rows = a.max_tokens * a.heads, nt = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    // (a table may be wider than any sequence is long, by more than 64-bit products hold)
    const long long item_tiles = (std::min(static_cast<long long>(a.max_pages) * a.cache.page, kMaxPositions) + kPos - 1) / kPos;
    const long long items = static_cast<long long>(a.seqs) * ((rows + nt - 1) / nt);
    // Short contexts: an item's few tiles one after the other take less time than another end of an item and the
    // launch that joins the parts, and 2 us less of the host.  Undivided and divided, one token of 16 heads, contexts
    // that fill the table, in us: 4 tiles, 1, 16 and 30 sequences 10.7 and 9.1, 11.0 and 9.5, 11.1 and 11.2 (the host's
    // time decides), 5 tiles 11.8 and 9.3, 12.1 and 9.6, 12.2 and 11.6; 8 tiles, 38, 64 and 75 sequences 16.8 and 14.0,
    // 17.6 and 19.5, 18.4 and 20.9, 9 tiles 18.1 and 16.0, 18.8 and 19.5, 19.6 and 22.0; 12 tiles, 76 and 128 sequences 23.0 and
    // 24.3, 27.7 and 32.1, 16 tiles 28.1 and 27.8, 33.6 and 38.5.  The rule knows the table's width, not the lengths: in a
    // table as wide as one long sequence needs, short ones are divided too.
    a.undivided = item_tiles <= 4 || (4 * items >= sms && item_tiles <= 8) || (2 * items >= sms && item_tiles <= 12);
    // no more CTAs than the page tables could fill with tiles
    const int ctas = static_cast<int>(std::min<long long>(sms, items * item_tiles));
    if (nt == 16)
        e = launch<16>(a, dev, ctas, box, tm_c, tm_r, s, pdl);
    else
        e = nt == 32 ? launch<32>(a, dev, ctas, box, tm_c, tm_r, s, pdl) : launch<64>(a, dev, ctas, box, tm_c, tm_r, s, pdl);
    if (e != cudaSuccess || a.undivided) return e;
    // a CTA for every row's 128 channels, when there are many parts and all those CTAs are resident at once
    const int units = units_of(a.cache.rank);
    if (ctas >= 8 * items && static_cast<int64_t>(a.seqs) * rows * units <= 8ll * sms) return launch_join<true, 1>(a, nt, ctas, s, pdl);
    if (units == 1) return launch_join<false, 1>(a, nt, ctas, s, pdl);
    // Half a row to a warp while the CTAs are few: 1,024 rows of 9.5 parts 37.3 us for the whole call against 39.4, of 2.4 parts
    // 66.7 against 67.6; 2,048 rows of 5.8 parts 72.7 against 70.8, 4,096 of 2.4 85.2 against 82.5.
    if (units == 2 || static_cast<int64_t>(a.seqs) * rows <= 8ll * sms) return launch_join<false, 2>(a, nt, ctas, s, pdl);
    return launch_join<false, 4>(a, nt, ctas, s, pdl);
}

}  // namespace moe
