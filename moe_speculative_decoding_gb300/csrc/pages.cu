// pages.cu -- sequences that share the pages of a cache: fork, reserve with copy on write, acceptance of a
// drafted path with its compaction, free.
//
// A page's holders are counted (refs; 0: free).  Which pages a call hands out goes by their numbers and the
// sequences' order alone, not by the order in which threads run: free pages are found in ascending order and
// requests are met by a prefix sum, so one CTA does the bookkeeping of reserve (counts are 4 bytes a page,
// 32 KB for 8,192 pages a step).  The rows move in a second kernel, in all layers at once, as the bits
// they are: its bound is memory traffic, each row read once and written once.
//
// 24 branches given up, forked and grown by 24 copies of 14 rows in 48 layers of 4 heads of 128 (132 MB): 24 us,
// 15.5 of them the copies; 128 branches in a pool of 40,000 pages, where 10 MB move: 17.6 us, the four kernels'
// chains of loads; 16 sequences' paths of up to 6 rows in 48 layers reserved and accepted: 12 us.
#include <algorithm>

#include "common.cuh"
#include "latent_args.cuh"

namespace moe {
namespace {

constexpr int kBook = 1024;          // threads of the bookkeeping CTA
constexpr int kMine = 8;             // pages a thread looks at in a step
constexpr int kStep = kBook * kMine;

// Lists in the workspace: [4] (copies to make, -, most rows of a copy, -), [seqs][4] (source page, target page, rows, -; of accept: ctx,
// rows to move, pages kept, pages held before; of fork, by target: 1 where its source has no such pages), [pages] free pages in order.
__device__ __forceinline__ int32_t *list_of(const PageArgs &a, int b) { return a.lists + 4 + 4ll * b; }
__device__ __forceinline__ int32_t *order_of(const PageArgs &a) { return a.lists + 4 + 4ll * a.pool.seqs; }
__device__ __forceinline__ int32_t *table_of(const PageArgs &a, int b) { return a.pool.table + static_cast<int64_t>(b) * a.pool.max_pages; }
__device__ __forceinline__ bool in_pool(const PageArgs &a, int page) { return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pool.pages); }

// Pages of n positions (n + page may be more than 31 bits hold).
__device__ __forceinline__ int pages_of(int n, int page) { return n > 0 ? (n - 1) / page + 1 : 0; }

// Sum of v over the threads before this one (32-bit sums hold: requests are at most seqs * max_pages),
// and over all.
__device__ __forceinline__ int before_me(int v, int *tmp, int &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // tmp's last use
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int w = tmp[lane];   // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    return __shfl_sync(0xFFFFFFFFu, w, warp) - tmp[warp] + x - v;
}

// ------------------------------------------------------------------ reserve
// Of a sequence's pages that will be written, one that others hold too is replaced.  The page with rows to keep is
// copied, by each of its holders that asks as long as others are left.  A page behind it (held beyond the length: a
// branch whose length was lowered) has nothing to keep and is replaced whoever else holds it; its
// count, with the copied pages', goes down when all counts have been read.
__global__ void __launch_bounds__(kBook) pages_reserve_kernel(const __grid_constant__ PageArgs a) {
    __shared__ __align__(16) int shared_s[kBook];
    __shared__ int tmp[32], copies_s, rows_s, fail_s;
    pdl_wait();
    pdl_trigger();
    const int b = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const moe_page_pool_t &pool = a.pool;
    const bool in = b < pool.seqs;
    int length = 0, need = 0, held = 0, want = 0, first = 0, rows = 0, at = -1, holders = 0, stop = 0, behind = 0;
    bool bad = false;
    if (in) {
        length = a.length[b];
        need = a.need[b];
        held = pool.held[b];
        const long long end = static_cast<long long>(length) + need;
        bad = need < 0 || length < 0 || held < 0 || held > pool.max_pages || length > static_cast<long long>(held) * pool.page ||
              end > static_cast<long long>(pool.max_pages) * pool.page;
        want = held;
        if (!bad && need > 0) {
            const int pages = static_cast<int>((end + pool.page - 1) / pool.page);
            want = max(held, pages);
            first = length / pool.page;
            rows = length - first * pool.page;
            // the pages that are there and will be written: the one with rows to keep, and those behind
            stop = min(held, pages);
            const int32_t *const row = table_of(a, b);
            int page[2], count[2];   // of the first two at once: mostly there are no more
#pragma unroll
            for (int k = 0; k < 2; ++k) page[k] = first + k < stop ? row[first + k] : 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                bad |= !in_pool(a, page[k]);
                count[k] = first + k < stop && in_pool(a, page[k]) ? pool.refs[page[k]] : 0;
            }
            if (rows > 0) {
                at = page[0];
                holders = count[0];
            } else {
                behind += count[0] > 1;
            }
            behind += count[1] > 1;
#pragma unroll 1
            for (int j = first + 2; j < stop; ++j) {
                const int other = row[j];
                bad |= !in_pool(a, other);
                if (!bad) behind += pool.refs[other] > 1;
            }
        }
        if (bad) {
            record_error(a.err, MOE_ERR_BAD_ID);
            want = held;
        }
    }
    const bool shared = !bad && holders > 1;
    if (bad) behind = 0;
    shared_s[b] = shared ? at : -1;
    if (b == 0) {
        copies_s = rows_s = 0;
        fail_s = kBook;
    }
    __syncthreads();
    // holders before this sequence that take a copy: its own is needed while others are left
    auto sharers = [&](int upto) {
        int n = 0, i = 0;
        for (; i + 4 <= upto; i += 4) {
            const int4 x = *reinterpret_cast<const int4 *>(shared_s + i);
            n += (x.x == at) + (x.y == at) + (x.z == at) + (x.w == at);
        }
        for (; i < upto; ++i) n += shared_s[i] == at;
        return n;
    };
    bool copy = shared && holders - sharers(b) > 1;
    const int extra = want - held + behind + (copy ? 1 : 0);
    int total;
    const int mine = before_me(extra, tmp, total);
    // the lowest free pages, as many as are asked for: the next step's counts are on their way while this
    // one's free pages are numbered
    int found = 0;
    int32_t *const order = order_of(a);
    const bool wide = (reinterpret_cast<uintptr_t>(pool.refs) & 15u) == 0;
    auto counts = [&](int64_t base, int (&x)[kMine]) {
        const int64_t p = base + static_cast<int64_t>(b) * kMine;
        if (wide && p + kMine <= pool.pages) {
            *reinterpret_cast<int4 *>(x) = *reinterpret_cast<const int4 *>(pool.refs + p);
            *reinterpret_cast<int4 *>(x + 4) = *reinterpret_cast<const int4 *>(pool.refs + p + 4);
        } else {
#pragma unroll
            for (int k = 0; k < kMine; ++k) x[k] = p + k < pool.pages ? pool.refs[p + k] : 1;
        }
    };
    alignas(16) int now[kMine], next[kMine];
    if (total > 0) counts(0, now);
    for (int64_t base = 0; found < total && base < pool.pages; base += kStep) {
        counts(base + kStep, next);
        int n = 0, here;
#pragma unroll
        for (int k = 0; k < kMine; ++k) n += now[k] == 0;
        int rank = found + before_me(n, tmp, here);
        const int p = static_cast<int>(base) + b * kMine;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            if (now[k] == 0 && rank < total) order[rank++] = p + k;
            now[k] = next[k];
        }
        found += here;
    }
    bool ok = in && !bad && (extra == 0 || mine + extra <= found);
    if (in && !bad && !ok) atomicMin(&fail_s, b);
    __syncthreads();   // the order is written, the first that goes without is known
    // behind that one a page is the sequence's own only if those before it have given it up
    if (ok && shared && !copy && b > fail_s && holders - sharers(fail_s) > 1) ok = false;
    copy = copy && ok;
    const int grown = ok ? want - held : 0;
    if (in) {
        if (a.got != nullptr) a.got[b] = ok ? 1 : 0;
        if (ok) pool.held[b] = want;
        if (copy) {
            const int page = order[mine];
            table_of(a, b)[first] = page;
            pool.refs[page] = 1;
            int32_t *const e = list_of(a, atomicAdd(&copies_s, 1));   // (in any order: the copies are independent)
            e[0] = at;
            e[1] = page;
            e[2] = rows;
            atomicMax(&rows_s, rows);
        }
        if (ok && behind > 0) {
            int k = mine + (copy ? 1 : 0);
#pragma unroll 1
            for (int j = first + (rows > 0 ? 1 : 0); j < stop; ++j) {
                const int page = table_of(a, b)[j];
                if (pool.refs[page] < 2) continue;
                table_of(a, b)[j] = order[k];
                pool.refs[order[k]] = 1;
                order[k++] = page;
            }
        }
    }
    // the pages behind those held, a warp's sequences one after the other
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, grown > 0); left != 0; left &= left - 1) {
        const int l = __ffs(left) - 1, n = __shfl_sync(0xFFFFFFFFu, grown, l), from = __shfl_sync(0xFFFFFFFFu, held, l);
        const int rank = __shfl_sync(0xFFFFFFFFu, mine + extra - (want - held), l);
        int32_t *const row = table_of(a, warp * 32 + l) + from;
        for (int j = lane; j < n; j += 32) {
            const int page = order[rank + j];
            row[j] = page;
            pool.refs[page] = 1;
        }
    }
    __syncthreads();   // the counts have been read
    if (copy) atomicSub(pool.refs + at, 1);
    if (ok)
#pragma unroll 1
        for (int k = mine + (copy ? 1 : 0); behind > 0; --behind, ++k) atomicSub(pool.refs + order[k], 1);
    if (b == 0) {
        a.lists[0] = copies_s;
        a.lists[2] = rows_s;
    }
}

// ------------------------------------------------------------------ rows
struct Divide {   // of numbers below 2^31, as a product
    uint32_t d, recip;
    __device__ __forceinline__ explicit Divide(uint32_t by) : d(by), recip(0xFFFFFFFFu / by) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
        const uint32_t q = __umulhi(x, recip);
        return q + (x - q * d >= d ? 1u : 0u);
    }
};
__device__ __forceinline__ uint32_t quotient(uint32_t x, uint32_t d, uint32_t recip) {
    const uint32_t q = __umulhi(x, recip);
    return q + (x - q * d >= d ? 1u : 0u);
}

// The first rows of listed pages to others.  An item is up to kUnits units of 16 bytes (4 for scales) of
// one plane of one layer; the CTAs step over the items, whose number the bookkeeping found.
constexpr int kCopy = 256, kUnits = 4 * kCopy;

__global__ void __launch_bounds__(kCopy) pages_copy_kernel(const __grid_constant__ PageArgs a, const __grid_constant__ PageRows p, int row_units) {
    pdl_wait();
    pdl_trigger();
    const int copies = a.lists[0], slices = (a.lists[2] * row_units + kUnits - 1) / kUnits;   // of the copy with most rows
    if (copies == 0) return;
    // (the caller keeps the items below 2^31; with divisions for every item and unit the integer pipe was
    // the bound, 28 us for 66 MB)
    const uint32_t whole = static_cast<uint32_t>(copies * p.layers * p.planes), items = whole * static_cast<uint32_t>(slices);
    const Divide by_whole(whole), by_copies(static_cast<uint32_t>(copies));
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        // (all pages' first slices before their second ones, which copies of few rows do not have)
        const uint32_t slice = by_whole(item), i = item - slice * whole, at = by_copies(i);
        const int layer = static_cast<int>(p.planes == 1 ? at : (p.planes == 2 ? at >> 1 : at >> 2)), which = static_cast<int>(at & (p.planes - 1));
        const int4 e = *reinterpret_cast<const int4 *>(list_of(a, static_cast<int>(i - at * copies)));
        const Plane &pl = p.plane[which];
        const int total = pl.per_row * e.z, u0 = static_cast<int>(slice) * kUnits + static_cast<int>(threadIdx.x);
        if (u0 >= total) continue;
        const uint8_t *const from = static_cast<const uint8_t *>(p.base[layer][which]) + e.x * pl.page_stride;
        uint8_t *const to = static_cast<uint8_t *>(p.base[layer][which]) + e.y * pl.page_stride;
        if (pl.dense && pl.unit == 16) {
            const uint4 *const src = reinterpret_cast<const uint4 *>(from) + u0;
            uint4 *const dst = reinterpret_cast<uint4 *>(to) + u0;
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (u0 + k * kCopy < total) x[k] = src[k * kCopy];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (u0 + k * kCopy < total) dst[k * kCopy] = x[k];
            continue;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int u = u0 + k * kCopy;
            if (u >= total) continue;
            const int r = static_cast<int>(quotient(u, pl.per_row, pl.by_row)), w = u - r * pl.per_row;
            const int sg = static_cast<int>(quotient(w, pl.per_seg, pl.by_seg));
            const int64_t off = r * pl.row_stride + sg * pl.seg_stride + static_cast<int64_t>(w - sg * pl.per_seg) * pl.unit;
            if (pl.unit == 16)
                *reinterpret_cast<uint4 *>(to + off) = *reinterpret_cast<const uint4 *>(from + off);
            else
                *reinterpret_cast<uint32_t *>(to + off) = *reinterpret_cast<const uint32_t *>(from + off);
        }
    }
}

// ------------------------------------------------------------------ accept
// A warp per sequence: checks its path and leaves ctx, the number of rows to move (0 where nothing moves; ctx may be
// overwritten here) and the pages to give up for the rows' kernel.  The counts of holders, which all
// sequences' checks read, go down there: so a page that one sequence gives up is shared for all of this call, and
// nobody moves rows within it while they are read.  Without paths nothing is checked against the counts.
__global__ void __launch_bounds__(256) pages_accept_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    pdl_trigger();
    const int b = static_cast<int>(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const moe_page_pool_t &pool = a.pool;
    if (b >= pool.seqs) return;
    const int ctx = a.ctx[b], count = a.count[b], held = pool.held[b];
    const long long room = static_cast<long long>(held) * pool.page;
    bool bad = held < 0 || held > pool.max_pages || ctx < 0 || ctx > room || count > a.max_path;
    int moves = 0;
    if (!bad && count > 0) {
        const int32_t *const path = a.path != nullptr ? a.path + static_cast<int64_t>(b) * a.max_path : nullptr;
        int last = -1;   // of the 32 before
        for (int i0 = 0; i0 < count; i0 += 32) {
            const int i = i0 + lane, p = i < count ? (path != nullptr ? path[i] : i) : 0;
            int prev = __shfl_up_sync(0xFFFFFFFFu, p, 1);
            if (lane == 0) prev = last;
            bad |= __any_sync(0xFFFFFFFFu, i < count && (p <= prev || static_cast<long long>(ctx) + p >= room));
            if (__any_sync(0xFFFFFFFFu, i < count && p != i)) moves = count;
            last = __shfl_sync(0xFFFFFFFFu, p, 31);
        }
    }
    // The pages that rows leave or go to and those that are given up are pages, and what rows go to nobody else holds.
    if (!bad && count >= 0) {
        const int first = moves > 0 ? ctx / pool.page : pages_of(ctx + count, pool.page), last = moves > 0 ? (ctx + count - 1) / pool.page : -1;
        bool other = false;
        for (int j = first + lane; j < held; j += 32) {
            const int page = table_of(a, b)[j];
            other |= !in_pool(a, page) || (j <= last && pool.refs[page] > 1);
        }
        bad = __any_sync(0xFFFFFFFFu, other);
    }
    if (bad && lane == 0) record_error(a.err, MOE_ERR_BAD_ID);
    const bool act = !bad && count >= 0;
    const int after = act ? ctx + count : ctx;
    const int left = pages_of(after, pool.page);   // at most held
    if (lane == 0) {
        int32_t *const e = list_of(a, b);
        e[0] = ctx;
        e[1] = act ? moves : 0;
        e[2] = left;
        e[3] = act ? held : left;
        if (a.after != nullptr) a.after[b] = after;
        if (act) pool.held[b] = left;
    }
    if (!act || a.path != nullptr) return;
    const int32_t *const table = table_of(a, b);
    for (int j = left + lane; j < held; j += 32) atomicSub(pool.refs + table[j], 1);
}

// A thread takes one column of a row (16 bytes, 4 of scales) through all of a sequence's moves in order: the
// path ascends, so target i is at or before source i and before every later one, and no row is written
// before it was read.  Eight rows' loads are in flight together.
__global__ void __launch_bounds__(kMove) pages_move_kernel(const __grid_constant__ PageArgs a, const __grid_constant__ PageRows p, int columns, int slices, int settle) {
    __shared__ int source_s[MOE_MAX_TREE_TOKENS][2], target_s[MOE_MAX_TREE_TOKENS][2];   // page, row
    pdl_wait();
    pdl_trigger();
    const uint32_t seqs = static_cast<uint32_t>(a.pool.seqs), whole = seqs * static_cast<uint32_t>(p.layers);
    const uint32_t items = whole * static_cast<uint32_t>(slices);   // (the caller keeps them below 2^31)
    if (settle) {
        for (int b = static_cast<int>(blockIdx.x); b < a.pool.seqs; b += static_cast<int>(gridDim.x)) {
            const int4 e = *reinterpret_cast<const int4 *>(list_of(a, b));
            const int32_t *const table = table_of(a, b);
            for (int j = e.z + static_cast<int>(threadIdx.x); j < e.w; j += kMove) atomicSub(a.pool.refs + table[j], 1);
        }
        if (items == 0) return;
    }
    const Divide by_whole(whole), by_seqs(seqs);
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t slice = by_whole(item), i = item - slice * whole, layer = by_seqs(i);
        const int b = static_cast<int>(i - layer * seqs);
        int column = static_cast<int>(slice) * kMove + static_cast<int>(threadIdx.x);
        const int32_t *const e = list_of(a, b);
        const int ctx = e[0], count = e[1];
        if (count == 0) continue;
        const int32_t *const path = a.path + static_cast<int64_t>(b) * a.max_path;
        __syncthreads();   // the previous item's places
        {
            const int i = static_cast<int>(threadIdx.x) & 63;
            if (i < count) {
                const int pos = ctx + (threadIdx.x < 64 ? path[i] : i), k = pos / a.pool.page;
                const int page = table_of(a, b)[k];
                int(&to)[2] = threadIdx.x < 64 ? source_s[i] : target_s[i];
                to[0] = page;
                to[1] = pos - k * a.pool.page;
            }
        }
        __syncthreads();
        if (column >= columns) continue;
        int which = 0;
        while (column >= p.plane[which].per_row) column -= p.plane[which++].per_row;
        const Plane &pl = p.plane[which];
        const int unit = pl.unit, seg = static_cast<int>(quotient(column, pl.per_seg, pl.by_seg));
        uint8_t *const base = static_cast<uint8_t *>(p.base[layer][which]) + seg * pl.seg_stride + static_cast<int64_t>(column - seg * pl.per_seg) * unit;
        auto at = [&](const int (&x)[2]) { return base + x[0] * pl.page_stride + x[1] * pl.row_stride; };
        constexpr int AHEAD = 8;
        for (int i0 = 0; i0 < count; i0 += AHEAD) {
            uint4 x[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int i = i0 + k;
                if (i >= count) continue;
                if (unit == 16)
                    x[k] = *reinterpret_cast<const uint4 *>(at(source_s[i]));
                else
                    x[k].x = *reinterpret_cast<const uint32_t *>(at(source_s[i]));
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int i = i0 + k;
                if (i >= count) continue;
                if (unit == 16)
                    *reinterpret_cast<uint4 *>(at(target_s[i])) = x[k];
                else
                    *reinterpret_cast<uint32_t *>(at(target_s[i])) = x[k].x;
            }
        }
    }
}

// ------------------------------------------------------------------ fork, free
// Every CTA checks all pairs (a thread each) and copies the page numbers of some, a warp to a pair, once it has
// looked at all of them (with several CTAs the target's list entry says whether they were pages); the last CTA
// to be done writes what the checks read, the lengths and the numbers of pages held.
__global__ void __launch_bounds__(kBook) pages_fork_kernel(const __grid_constant__ PageArgs a) {
    __shared__ __align__(16) int dst_s[kBook];
    __shared__ int src_s[kBook], pages_s[kBook], last_s;
    pdl_wait();
    pdl_trigger();
    const int i = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const moe_page_pool_t &pool = a.pool;
    const bool in = i < a.items;
    int src = 0, dst = -1, length = 0;
    bool ok = in;
    if (in) {
        src = a.src[i];
        dst = a.ids[i];
        ok = static_cast<uint32_t>(src) < static_cast<uint32_t>(pool.seqs) && static_cast<uint32_t>(dst) < static_cast<uint32_t>(pool.seqs) && src != dst;
        if (ok) {
            length = a.length_out[src];
            const int held = pool.held[src];
            ok = pool.held[dst] == 0 && held >= 0 && held <= pool.max_pages && length >= 0 && length <= static_cast<long long>(held) * pool.page;
        }
    }
    dst_s[i] = dst;
    src_s[i] = src;
    __syncthreads();
    int same = 0, k = 0;   // pairs before this one with its target
    for (; k + 4 <= i && ok; k += 4) {
        const int4 x = *reinterpret_cast<const int4 *>(dst_s + k);
        same += (x.x == dst) + (x.y == dst) + (x.z == dst) + (x.w == dst);
    }
    for (; k < i && ok; ++k) same += dst_s[k] == dst;
    ok = ok && same == 0;
    if (in && !ok) record_error(a.err, MOE_ERR_BAD_ID);
    const int pages = ok ? pages_of(length, pool.page) : 0;
    pages_s[i] = pages;
    __syncthreads();
    for (int p = blockIdx.x * 32 + warp; p < a.items; p += gridDim.x * 32) {
        const int n = pages_s[p];
        if (n == 0) continue;
        const int32_t *const from = table_of(a, src_s[p]);
        int32_t *const to = table_of(a, dst_s[p]);
        constexpr int MINE = 4;   // a lane's first page numbers stay in registers
        int first[MINE];
        bool out = false;
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            first[k] = lane + 32 * k < n ? from[lane + 32 * k] : 0;
            out |= !in_pool(a, first[k]);
        }
        for (int j = lane + 32 * MINE; j < n; j += 32) out |= !in_pool(a, from[j]);
        out = __any_sync(0xFFFFFFFFu, out);
        if (lane == 0) {
            if (gridDim.x > 1) list_of(a, dst_s[p])[0] = out ? 1 : 0;
            if (out) {
                pages_s[p] = -1;
                record_error(a.err, MOE_ERR_BAD_ID);
            }
        }
        if (out) continue;
        auto take = [&](int j, int page) {
            to[j] = page;
            atomicAdd(pool.refs + page, 1);
        };
#pragma unroll
        for (int k = 0; k < MINE; ++k)
            if (lane + 32 * k < n) take(lane + 32 * k, first[k]);
        for (int j = lane + 32 * MINE; j < n; j += 32) take(j, from[j]);
    }
    __syncthreads();
    if (gridDim.x > 1) {
        if (i == 0) last_s = atom_add_acq_rel_gpu(a.forked, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!last_s) return;
        if (i == 0) *a.forked = 0;   // for the next call
    }
    const bool bad = gridDim.x > 1 ? ok && pages > 0 && list_of(a, dst)[0] != 0 : pages_s[i] < 0;
    if (ok && !bad) {
        pool.held[dst] = pages;
        a.length_out[dst] = length;
    }
}

__global__ void __launch_bounds__(256) pages_free_kernel(const __grid_constant__ PageArgs a) {
    pdl_wait();
    pdl_trigger();
    const int i = static_cast<int>(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (i >= a.items) return;
    const int b = a.ids[i];
    if (b < 0) return;
    if (b >= a.pool.seqs) {
        if (lane == 0) record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    // Of several warps that name the sequence one finds its pages below; here any may find them or none left.
    int held = *const_cast<volatile int32_t *>(a.pool.held + b);
    held = __shfl_sync(0xFFFFFFFFu, held, 0);
    const int32_t *const table = table_of(a, b);
    constexpr int MINE = 4;   // a lane's first page numbers stay in registers
    int first[MINE];
    bool bad = held < 0 || held > a.pool.max_pages;
    if (!bad) {
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            first[k] = lane + 32 * k < held ? table[lane + 32 * k] : 0;
            bad |= !in_pool(a, first[k]);
        }
        for (int j = lane + 32 * MINE; j < held; j += 32) bad |= !in_pool(a, table[j]);
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
        if (lane == 0) record_error(a.err, MOE_ERR_BAD_ID);
        return;
    }
    if (lane == 0) {
        if (held > 0) held = atomicExch(a.pool.held + b, 0);
        if (a.length_out != nullptr) a.length_out[b] = 0;
    }
    held = __shfl_sync(0xFFFFFFFFu, held, 0);
#pragma unroll
    for (int k = 0; k < MINE; ++k)
        if (lane + 32 * k < held) atomicSub(a.pool.refs + first[k], 1);
    for (int j = lane + 32 * MINE; j < held; j += 32) atomicSub(a.pool.refs + table[j], 1);
}

template <typename K, typename... Args>
cudaError_t launch(K kernel, unsigned grid, unsigned threads, cudaStream_t s, bool pdl, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int64_t kSms = 152;

}  // namespace

size_t pages_list_bytes(const moe_page_pool_t &pool) { return 16 + 16 * static_cast<size_t>(pool.seqs) + 4 * static_cast<size_t>(pool.pages); }

cudaError_t launch_pages_reserve(const PageArgs &a, const PageRows *rows, int launches, cudaStream_t s, bool pdl) {
    cudaError_t e = launch(pages_reserve_kernel, 1, kBook, s, pdl, a);
    for (int i = 0; i < launches && e == cudaSuccess; ++i) {
        int most = 1;   // units of a row in a plane
        for (int k = 0; k < rows[i].planes; ++k) most = std::max(most, rows[i].plane[k].per_row);
        const int64_t slices = (static_cast<int64_t>(most) * a.pool.page + kUnits - 1) / kUnits;
        const int64_t items = static_cast<int64_t>(a.pool.seqs) * rows[i].layers * rows[i].planes * slices;
        e = launch(pages_copy_kernel, static_cast<unsigned>(std::min<int64_t>(items, kSms * 8)), kCopy, s, pdl, a, rows[i], most);
    }
    return e;
}

cudaError_t launch_pages_accept(const PageArgs &a, const PageRows *rows, int launches, cudaStream_t s, bool pdl) {
    cudaError_t e = launch(pages_accept_kernel, (static_cast<unsigned>(a.pool.seqs) + 7) / 8, 256, s, pdl, a);
    if (a.path == nullptr) return e;   // nothing moves
    // the first launch gives the pages up; without caches it does nothing else
    static const PageRows none = {};
    for (int i = 0; i < std::max(launches, 1) && e == cudaSuccess; ++i) {
        const PageRows &r = launches > 0 ? rows[i] : none;
        const int slices = move_slices(r);
        const int64_t items = std::max<int64_t>(static_cast<int64_t>(a.pool.seqs) * r.layers * slices, a.pool.seqs);
        e = launch(pages_move_kernel, static_cast<unsigned>(std::min<int64_t>(items, kSms * 16)), kMove, s, pdl, a, r, move_columns(r), slices, i == 0 ? 1 : 0);
    }
    return e;
}

cudaError_t launch_pages_fork(const PageArgs &a, cudaStream_t s, bool pdl) {
    return launch(pages_fork_kernel, static_cast<unsigned>(std::min((a.items + 31) / 32, 32)), kBook, s, pdl, a);
}

cudaError_t launch_pages_free(const PageArgs &a, cudaStream_t s, bool pdl) {
    return launch(pages_free_kernel, (static_cast<unsigned>(a.items) + 7) / 8, 256, s, pdl, a);
}

}  // namespace moe
