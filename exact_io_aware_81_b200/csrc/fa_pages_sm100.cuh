// fa_pages_sm100.cuh -- the pages of a KV cache: handing out, sharing, giving back,
// compacting and copying them.
//
// State, all in device memory and owned by the caller: block_table (S, max_pages), seqlens
// (S) and refcount (num_pages), the number of table entries that name a page.  A slot of
// length L holds ceil(L / page_size) pages; a page with refcount 0 is free.  Every result is
// a function of the state and the arguments alone: the free pages handed out are the lowest,
// slot by slot in ascending order, so no order of atomics or blocks shows in it.
//
//   fork     dst takes over the first `length` tokens of src: its row copies src's entries and
//            their refcounts go up by one.  No page data moves; a shared page that is only
//            partly filled is split when somebody extends it.
//   free     cuts a slot to `keep` tokens: refcounts of the pages behind them go down.
//   reserve  lengthens slots by `add` tokens: pages for them, plus a private copy of a last
//            page that is partly filled and shared (refcount > 1), reported in `copies`.
//            Exclusive sums over the slots give every slot its place in the list of free
//            pages, which is the compaction of {i : refcount[i] = 0} by ranks.  All or nothing.
//   compact  n = number of live pages; the k-th live page >= n moves into the k-th free page
//            < n (their numbers agree, since both count n minus the live pages < n).
//   copy     moves the data of (source, destination) pairs in the K and V pools.
//
// Bounds.  The bookkeeping touches kilobytes and is bound by latency: fork and free run one
// CTA per slot; reserve and compact need sums over all slots or pages and run as one CTA of
// 1024 threads (16 bytes of refcounts per thread and step), so each is one launch with no
// grid-wide step.  The copy is bound by HBM: 16-byte loads, kCopyUnroll in flight per thread,
// both ways past the caches' regular replacement (504 pages of 128 KB in two pools, 264 MB
// there and back: 44 us = 6.0 TB/s; four loads without the hints 48).
#pragma once

#include <cstdint>

#include "fa.h"
#include "fa_common.cuh"

namespace fa {

struct PageTables {
    int *block_table;  // (S, max_pages)
    int *seqlens;      // (S)
    int *refcount;     // (num_pages)
    int S, max_pages, num_pages, page_size;

    __device__ __forceinline__ int length(int s) const { return read_at(seqlens, s, S); }
    __device__ __forceinline__ void set_length(int s, int n) const { write_at(seqlens, s, S, n); }
    __device__ __forceinline__ int page(int s, int j) const
    {
        return read_at(block_table, (long long)s * max_pages + j, (long long)S * max_pages);
    }
    __device__ __forceinline__ void set_page(int s, int j, int pg) const
    {
        write_at(block_table, (long long)s * max_pages + j, (long long)S * max_pages, pg);
    }
    __device__ __forceinline__ void set_count(int pg, int n) const { write_at(refcount, pg, num_pages, n); }
    // adds to a page's count and returns what it was
    __device__ __forceinline__ int count(int pg, int by) const
    {
        return in_bounds(pg, num_pages) ? atomicAdd(refcount + pg, by) : 0;
    }
};

namespace pages {

constexpr int kSlotThreads = 128;  // fork, free: one CTA per listed slot
constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;     // 16-byte loads in flight per thread
constexpr int kPieceBytes = 16 * kCopyThreads * kCopyUnroll;  // one CTA's share of a page

__device__ __forceinline__ int pages_of(int len, int page_size) { return (len + page_size - 1) / page_size; }

// Is `len` a length that a slot can have?
__device__ __forceinline__ bool len_ok(const PageTables &t, int len)
{
    return len >= 0 && (long long)len <= (long long)t.page_size * t.max_pages;
}

// Exclusive prefix sum over the CTA (kPlanThreads); `total` is the sum over all threads.  A warp
// counts for `most` at most: where no prefix passes `most` that changes nothing, and prefixes
// that pass it stay above it, whatever the true sum, while 32 warps cannot overflow an int.
__device__ __forceinline__ int block_scan(int v, int &total, int *warp_sums, int most = 0x7fffffff)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // warp_sums of the previous call has been read
    if (lane == 31) warp_sums[warp] = min(x, most);
    __syncthreads();
    int w = warp_sums[lane];  // kPlanThreads / 32 = 32 warps
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int base = __shfl_sync(0xffffffffu, w, warp) - warp_sums[warp];
    return base + x - v;
}

// Four refcounts from `i` on; entries past the end read as `past`.
__device__ __forceinline__ int4 load4(const int *ref, int i, int n, int past)
{
    int4 r = make_int4(past, past, past, past);
    if (i + 3 < n && (reinterpret_cast<uintptr_t>(ref) & 15) == 0)
        return in_bounds(i, n) ? *reinterpret_cast<const int4 *>(ref + i) : r;
    if (i < n) r.x = read_at(ref, i, n);
    if (i + 1 < n) r.y = read_at(ref, i + 1, n);
    if (i + 2 < n) r.z = read_at(ref, i + 2, n);
    if (i + 3 < n) r.w = read_at(ref, i + 3, n);
    return r;
}

}  // namespace pages

struct ForkParams {
    PageTables t;
    const int *src, *dst, *lengths;  // (n); lengths may be null: all of src
    int n;
};

// One CTA per pair.  A pair is refused, and reported, when a slot is out of range, dst is not
// empty, dst is also a source or the destination of an earlier pair, or the length is not one
// of src's.  A destination is never a source, so what the CTAs read no CTA writes.
__global__ void __launch_bounds__(pages::kSlotThreads) fa_pages_fork_kernel(const ForkParams p)
{
    using namespace pages;
    const int i = blockIdx.x;
    const int s = read_at(p.src, i, p.n), d = read_at(p.dst, i, p.n);
    bool bad = s < 0 || s >= p.t.S || d < 0 || d >= p.t.S;
    for (int j = threadIdx.x; j < p.n; j += kSlotThreads) {
        const int e = read_at(p.dst, j, p.n);
        bad |= e == s || (j < i && e == d);
    }
    int len = 0;
    if (!bad) {
        len = p.t.length(s);
        bad = !len_ok(p.t, len) || p.t.length(d) != 0;
        if (!bad && p.lengths) {
            const int want = read_at(p.lengths, i, p.n);
            bad = want < 0 || want > len;
            len = want;
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) raise_error(kErrSlot);
        return;
    }
    const int np = pages_of(len, p.t.page_size);
    for (int j = threadIdx.x; j < np; j += kSlotThreads) {
        const int pg = p.t.page(s, j);
        p.t.set_page(d, j, pg);
        if (pg >= 0 && pg < p.t.num_pages) p.t.count(pg, 1);
        else raise_error(kErrPageRange);
    }
    if (threadIdx.x == 0) p.t.set_length(d, len);
}

struct FreeParams {
    PageTables t;
    const int *slots, *keep;  // (n); keep may be null: nothing is kept
    int n;
};

// One CTA per listed slot; a slot listed a second time is refused and reported.
__global__ void __launch_bounds__(pages::kSlotThreads) fa_pages_free_kernel(const FreeParams p)
{
    using namespace pages;
    const int i = blockIdx.x;
    const int s = read_at(p.slots, i, p.n);
    bool bad = s < 0 || s >= p.t.S;
    for (int j = threadIdx.x; j < i; j += kSlotThreads) bad |= read_at(p.slots, j, p.n) == s;
    // every thread agrees on `bad` before the length is read: an earlier CTA of the same slot
    // may be writing it
    bool refused = __syncthreads_or(bad);
    int len = 0, keep = 0;
    if (!refused) {
        len = p.t.length(s);
        if (p.keep) keep = read_at(p.keep, i, p.n);
        refused = !len_ok(p.t, len) || keep < 0 || keep > len;
    }
    __syncthreads();  // the length is read by all before it changes
    if (refused) {
        if (threadIdx.x == 0) raise_error(kErrSlot);
        return;
    }
    const int end = pages_of(len, p.t.page_size);
    for (int j = pages_of(keep, p.t.page_size) + threadIdx.x; j < end; j += kSlotThreads) {
        const int pg = p.t.page(s, j);
        p.t.set_page(s, j, -1);
        if (pg < 0 || pg >= p.t.num_pages) {
            raise_error(kErrPageRange);
        } else if (p.t.count(pg, -1) <= 0) {  // the page was not held
            p.t.count(pg, 1);
            raise_error(kErrSlot);
        }
    }
    if (threadIdx.x == 0) p.t.set_length(s, keep);
}

struct ReserveParams {
    PageTables t;
    const int *add;   // (S)
    int *copies;      // (S, 2)
    int *status;      // (1) or null: what became of the call
    int *first;       // workspace (S): place of a slot's pages in free_ids
    int *free_ids;    // workspace (num_pages)
};

namespace pages {

// What slot s needs: `begin`, the first table entry that gets a new page, `end`, one past the
// last, and the shared page that is split (or -1).
struct Need {
    int len, begin, end, split;
};

__device__ __forceinline__ Need need_of(const ReserveParams &p, int s, bool &bad)
{
    Need n;
    const int add = read_at(p.add, s, p.t.S);
    n.len = p.t.length(s);
    n.begin = n.end = 0;
    n.split = -1;
    if (add == 0) return n;
    if (add < 0 || !len_ok(p.t, n.len) || (long long)n.len + add > (long long)p.t.page_size * p.t.max_pages) {
        bad = true;
        return n;
    }
    n.begin = pages_of(n.len, p.t.page_size);
    n.end = pages_of(n.len + add, p.t.page_size);
    if (n.len % p.t.page_size) {
        const int last = p.t.page(s, n.begin - 1);
        if (last < 0 || last >= p.t.num_pages) {
            bad = true;
        } else if (read_at(p.t.refcount, last, p.t.num_pages) > 1) {
            n.split = last;
            --n.begin;
        }
    }
    return n;
}

}  // namespace pages

__global__ void __launch_bounds__(pages::kPlanThreads, 1) fa_pages_reserve_kernel(const ReserveParams p)
{
    using namespace pages;
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31;

    // places of the slots in the list of free pages
    int total = 0;
    bool bad = false;
    for (int s0 = 0; s0 < p.t.S; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int want = 0;
        if (s < p.t.S) {
            const Need n = need_of(p, s, bad);
            // more than the pool has ends the call whatever the excess (and 1024 such
            // terms stay below 2^31: num_pages < 2^21 - 1)
            want = min(n.end - n.begin, p.t.num_pages + 1);
        }
        int sum;
        const int at = block_scan(want, sum, warp_sums);
        if (s < p.t.S) write_at(p.first, s, p.t.S, total + at);
        if (sum > p.t.num_pages - total) {
            total = p.t.num_pages + 1;
            break;
        }
        total += sum;
    }
    bad = __syncthreads_or(bad);

    // the lowest `total` free pages
    int found = 0;
    if (!bad && total <= p.t.num_pages) {
        int4 next = load4(p.t.refcount, 4 * tid, p.t.num_pages, 1);
        for (int i0 = 0; i0 < p.t.num_pages && found < total; i0 += 4 * kPlanThreads) {
            const int i = i0 + 4 * tid;
            const int4 r = next;
            next = load4(p.t.refcount, i + 4 * kPlanThreads, p.t.num_pages, 1);  // in flight over the scan
            const int f0 = r.x <= 0, f1 = r.y <= 0, f2 = r.z <= 0, f3 = r.w <= 0;
            int sum;
            int at = found + block_scan(f0 + f1 + f2 + f3, sum, warp_sums);
            if (f0 && at < total) write_at(p.free_ids, at, p.t.num_pages, i);
            at += f0;
            if (f1 && at < total) write_at(p.free_ids, at, p.t.num_pages, i + 1);
            at += f1;
            if (f2 && at < total) write_at(p.free_ids, at, p.t.num_pages, i + 2);
            at += f2;
            if (f3 && at < total) write_at(p.free_ids, at, p.t.num_pages, i + 3);
            found += sum;
        }
    }
    if (bad || found < total) {
        if (tid == 0) {
            if (bad || !p.status) raise_error(bad ? kErrSlot : kErrNoPages);
            if (p.status) *p.status = bad ? FA_ERR_DEVICE_ARG : FA_ERR_NO_PAGES;
        }
        for (int s = tid; s < 2 * p.t.S; s += kPlanThreads) write_at(p.copies, s, 2LL * p.t.S, -1);
        return;
    }
    if (p.status && tid == 0) *p.status = FA_OK;
    __syncthreads();  // free_ids is complete

    // The sums decided on the refcounts at the start of the call, and this pass lowers some of
    // them as it goes, so it takes the splits from the places instead: a slot splits its last
    // page exactly if it was given one page more than its growth.
    for (int s0 = 0; s0 < p.t.S; s0 += kPlanThreads) {
        const int s = s0 + tid;
        Need n{0, 0, 0, -1};
        int at = 0, add = 0;
        if (s < p.t.S) {
            add = read_at(p.add, s, p.t.S);
            at = read_at(p.first, s, p.t.S);
            if (add > 0) {
                n.len = p.t.length(s);
                n.begin = pages_of(n.len, p.t.page_size);
                n.end = pages_of(n.len + add, p.t.page_size);
                const int next = s + 1 < p.t.S ? read_at(p.first, s + 1, p.t.S) : total;
                if (next - at > n.end - n.begin) {
                    --n.begin;
                    n.split = p.t.page(s, n.begin);
                }
            }
        }
        const int want = n.end - n.begin;
        // short growth by the lane itself, longer growth by the whole warp
        constexpr int kOwn = 2;
        int split_to = -1;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            if (k < want && (want <= kOwn || k == 0)) {
                const int id = read_at(p.free_ids, at + k, p.t.num_pages);
                p.t.set_page(s, n.begin + k, id);
                p.t.set_count(id, 1);
                if (k == 0) split_to = id;
            }
        }
        unsigned more = __ballot_sync(0xffffffffu, want > kOwn);
        while (more) {
            const int l = __ffs(more) - 1;
            more &= more - 1;
            const int ls = __shfl_sync(0xffffffffu, s, l), la = __shfl_sync(0xffffffffu, at, l);
            const int lb = __shfl_sync(0xffffffffu, n.begin, l), lw = __shfl_sync(0xffffffffu, want, l);
            for (int k = 1 + lane; k < lw; k += 32) {
                const int id = read_at(p.free_ids, la + k, p.t.num_pages);
                p.t.set_page(ls, lb + k, id);
                p.t.set_count(id, 1);
            }
        }
        if (s < p.t.S) {
            if (add > 0) p.t.set_length(s, n.len + add);
            if (n.split >= 0) p.t.count(n.split, -1);
            write_at(p.copies, 2 * s, 2LL * p.t.S, n.split);
            write_at(p.copies, 2 * s + 1, 2LL * p.t.S, n.split >= 0 ? split_to : -1);
        }
    }
}

struct CompactParams {
    PageTables t;
    int *copies;   // (num_pages / 2, 2)
    int *rank;     // workspace (num_pages): line of `copies` of a page that moves
    int *holes;    // workspace (num_pages)
    int *n_live;   // workspace (1)
};

__global__ void __launch_bounds__(pages::kPlanThreads, 1) fa_pages_compact_kernel(const CompactParams p)
{
    using namespace pages;
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, N = p.t.num_pages;
    int mine = 0;
#pragma unroll 4
    for (int i = 4 * tid; i < N; i += 4 * kPlanThreads) {
        const int4 r = load4(p.t.refcount, i, N, 0);
        mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
    int n_live;
    block_scan(mine, n_live, warp_sums);
    if (tid == 0) *p.n_live = n_live;

    int holes = 0;
    int4 next = load4(p.t.refcount, 4 * tid, n_live, 1);
    for (int i0 = 0; i0 < n_live; i0 += 4 * kPlanThreads) {
        const int i = i0 + 4 * tid;
        const int4 r = next;
        next = load4(p.t.refcount, i + 4 * kPlanThreads, n_live, 1);  // in flight over the scan
        const int f0 = r.x <= 0, f1 = r.y <= 0, f2 = r.z <= 0, f3 = r.w <= 0;
        int sum;
        int at = holes + block_scan(f0 + f1 + f2 + f3, sum, warp_sums);
        if (f0) write_at(p.holes, at++, N, i);
        if (f1) write_at(p.holes, at++, N, i + 1);
        if (f2) write_at(p.holes, at++, N, i + 2);
        if (f3) write_at(p.holes, at++, N, i + 3);
        holes += sum;
    }
    __syncthreads();  // the list of holes is complete

    // movers: the live pages from n_live on (their number is `holes`)
    int moved = 0;
    next = load4(p.t.refcount, (n_live & ~3) + 4 * tid, N, 0);
    for (int i0 = n_live & ~3; i0 < N && moved < holes; i0 += 4 * kPlanThreads) {
        const int i = i0 + 4 * tid;
        const int ref[4] = {next.x, next.y, next.z, next.w};
        next = load4(p.t.refcount, i + 4 * kPlanThreads, N, 0);
        int c = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c += ref[k] > 0 && i + k >= n_live;
        int sum;
        int at = moved + block_scan(c, sum, warp_sums);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (ref[k] > 0 && i + k >= n_live) {
                const int to = read_at(p.holes, at, N);
                write_at(p.copies, 2 * at, N, i + k);
                write_at(p.copies, 2 * at + 1, N, to);
                write_at(p.rank, i + k, N, at);
                p.t.set_count(to, ref[k]);
                p.t.set_count(i + k, 0);
                ++at;
            }
        }
        moved += sum;
    }
    for (int k = moved + tid; k < N / 2; k += kPlanThreads) {
        write_at(p.copies, 2 * k, N, -1);
        write_at(p.copies, 2 * k + 1, N, -1);
    }
}

// The tables follow the pages: one CTA per slot.
__global__ void __launch_bounds__(pages::kSlotThreads) fa_pages_remap_kernel(const CompactParams p)
{
    using namespace pages;
    const int s = blockIdx.x;
    const int n_live = *p.n_live;
    const int len = p.t.length(s);
    if (!len_ok(p.t, len)) {
        if (threadIdx.x == 0) raise_error(kErrSlot);
        return;
    }
    const int N = p.t.num_pages, end = pages_of(len, p.t.page_size);
    for (int j = threadIdx.x; j < end; j += kSlotThreads) {
        const int pg = p.t.page(s, j);
        if (pg < 0 || pg >= p.t.num_pages) {
            raise_error(kErrPageRange);
        } else if (pg >= n_live) {
            // a page that did not move has no rank (it was not live): its line names another
            const int k = read_at(p.rank, pg, N);
            if (k >= 0 && k < N / 2 && read_at(p.copies, 2 * k, N) == pg) p.t.set_page(s, j, read_at(p.copies, 2 * k + 1, N));
            else raise_error(kErrSlot);
        }
    }
}

struct PageCopyParams {
    uint4 *k, *v;          // the pools; v may be null
    const int *copies;     // (n, 2): source, destination; an entry below 0 is skipped
    int n, num_pages;
    long long page_vecs;   // 16-byte pieces of a page
    int pieces;            // ceil(page bytes / kPieceBytes)
};

__global__ void __launch_bounds__(pages::kCopyThreads) fa_pages_copy_kernel(const PageCopyParams p)
{
    using namespace pages;
    const int per = p.pieces * (p.v ? 2 : 1);
    const long long items = (long long)p.n * per;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const long long e = item / per;
        const int c = (int)(item - e * per);
        const int2 pair = make_int2(read_at(p.copies, 2 * e, 2LL * p.n), read_at(p.copies, 2 * e + 1, 2LL * p.n));
        if (pair.x < 0 && pair.y < 0) continue;
        if (pair.x < 0 || pair.y < 0 || pair.x >= p.num_pages || pair.y >= p.num_pages) {
            if (threadIdx.x == 0) raise_error(kErrPageRange);
            continue;
        }
        uint4 *pool = c < p.pieces ? p.k : p.v;
        const long long size = p.num_pages * p.page_vecs;
        const long long at = (long long)(c < p.pieces ? c : c - p.pieces) * (kCopyThreads * kCopyUnroll) + threadIdx.x;
        const long long src = pair.x * p.page_vecs + at, dst = pair.y * p.page_vecs + at;
        uint4 x[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (at + u * kCopyThreads < p.page_vecs && in_bounds(src + u * kCopyThreads, size))
                x[u] = __ldcs(pool + src + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (at + u * kCopyThreads < p.page_vecs && in_bounds(dst + u * kCopyThreads, size))
                __stcs(pool + dst + u * kCopyThreads, x[u]);
    }
}

}  // namespace fa
