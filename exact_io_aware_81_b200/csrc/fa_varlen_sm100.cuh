// fa_varlen_sm100.cuh -- exact attention forward over packed sequences of different lengths, and
// over packed queries of a paged cache.
//
// Method, tiles, tensor-memory layout, warp roles and softmax are those of fa_prefill_sm100.cuh;
// what differs is where the work comes from:
//   Tiles.  A Q tile holds tile_tokens = 128 / pack tokens of the `pack` query heads that share
//     a K/V head (row = token * pack + head; the TMA box of a (d, heads, tokens) map lays them
//     out so).  A unit is two such tiles, consecutive tokens, of one K/V head: every K/V tile
//     staged serves 256 rows whatever the grouping, and a sequence of a few tokens fills few
//     tiles (one token of four heads: 4 rows of one tile, where a tile per head would be four).
//   Twins (SHORT variant).  Where a sequence has tokens for one tile only, both tiles hold those
//     tokens and take alternate key tiles; tile 0's warps join the two partial softmaxes from
//     tensor memory, as key blocks are joined anywhere (rescale to the larger maximum).  The
//     second tile would otherwise idle, and nothing would run beside the first tile's S ->
//     softmax -> P V chain.
//   Order.  The lengths are known on the device only.  fa_varlen_plan_kernel lists the jobs (the
//     tokens of two tiles of one sequence) by falling number of steps: a counting sort over
//     kBins classes, whose order within a class is left open (it decides which CTA computes
//     what, never a result).  The attention kernel's CTAs draw units (job x head slot) from a
//     counter, longest first, so that they end together.  Only the producer warp draws; it hands
//     each unit to the other roles through a ring of records in shared memory.  A call whose
//     units fit one wave of CTAs goes without a plan, each CTA finding its own (8 prompts of up
//     to 64 tokens: 10.3 instead of 12.4 us).
//   Rounding.  Scores, maxima, sums and the accumulators are 32 bits.  The weights are rounded to
//     bf16, half a step of 2^-8 each, because the matrix instruction takes both operands in one
//     type and V is bf16; the normaliser takes the rounding of a tile's largest weight back (see
//     `lo`).  O is rounded once, to its type.  In relative norm the outputs are 0.0017-0.0023 from
//     the 64-bit form; weights of 32 bits leave 0.0015-0.0017, the rounding of a bf16 O alone.
//   Bits.  A unit's tiles, and with them the order of its sums, come from the lengths and the
//     variant alone.  LONG and SHORT order them differently, so a sequence's last bits can change
//     with what chooses the variant: the other lengths, the heads, and the size of the pool.
//   Isolation.  A key tile that passes its sequence's end holds other rows (the next sequence's,
//     or whatever a page has there): their scores are masked, and their V rows are cleared in
//     shared memory before P V, since 0 * NaN would reach the output.
//   Rows without a key (more causal queries than keys, or no keys) end with l = 0 and are written
//     as O = 0, LSE = -inf; the running maximum starts at a finite floor, so nothing is NaN.
//   Pages.  The producer's lanes look up the pages of a key tile's copies two tiles ahead and
//     issue a copy each.
// Bound: the softmax warps' latencies (a step, one key tile for both Q tiles, takes 1.75 us at
// d = 64 and 128 alike; on 9 long sequences XU 46%, FMA 40%, tensor pipe 65% busy, with a window at
// d = 64 25%, 25% and 18%), and 3-4 us at each unit's boundary.  Measured on B200, 32 + 8 heads,
// d = 128, causal, replayed graphs, with the clock: 9 sequences of 500 to 8192 tokens 1.14-1.33 ms
// (1.05-1.23 PFLOP/s), and four of 8192 1.91-2.03 ms, where the dense kernel takes 1.91-2.00; 16
// prompts of 16 to 2048 tokens 96-106 us, up to 125 under the power cap; 12 chunks of 1 to 512 tokens
// over paged contexts of up to 8192 tokens 131-137 us.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "fa_common.cuh"
#include "fa_pages_sm100.cuh"
#include "fa_prefill_sm100.cuh"
#include "ptx_sm100.cuh"

namespace fa {

// ------------------------------------------------------------------------- the plan
//
// Bound: latency.  One CTA: sums of the tile counts over the sequences, then one thread per
// job (the sequence by bisection of the sums), two passes.  It releases the attention kernel's
// launch at once (programmatic dependent launch), whose set-up then overlaps it.

struct VarlenPlanParams {
    const int *cu_q;     // (B + 1)
    const int *cu_k;     // (B + 1), or
    const int *seqlens;  // (B): key counts of a paged cache (k rows then start at 0)
    int4 *plan;          // (2 * max_jobs)
    int *head;           // [0] number of jobs, [1] counter
    int B, Tq, Tk;       // Tk: rows of k, or the most keys the block table holds
    int rows;            // query tokens of a job: two tiles'
    int causal, window;
    int twins;           // the attention kernel's SHORT variant follows
    int max_jobs;        // Tq / rows + B
};

namespace varlen {

constexpr int kThreads = 1024;
constexpr int kMaxSeqs = 4096;
constexpr int kBins = 1024;

struct Seq {
    int q0, nq, k0, nk;
};

// Sequence b, forced into the tensors; `bad` when that changed it.
__device__ __forceinline__ Seq sequence(const VarlenPlanParams &p, int b, bool &bad)
{
    Seq s;
    const int q0 = read_at(p.cu_q, b, p.B + 1), q1 = read_at(p.cu_q, b + 1, p.B + 1);
    s.q0 = min(max(q0, 0), p.Tq);
    s.nq = min(max(q1, s.q0), p.Tq) - s.q0;
    bad |= s.q0 != q0 || s.q0 + s.nq != q1;
    if (p.seqlens) {
        const int n = read_at(p.seqlens, b, p.B);
        s.k0 = 0;
        s.nk = min(max(n, 0), p.Tk);
        bad |= s.nk != n;
    } else {
        const int k0 = read_at(p.cu_k, b, p.B + 1), k1 = read_at(p.cu_k, b + 1, p.B + 1);
        s.k0 = min(max(k0, 0), p.Tk);
        s.nk = min(max(k1, s.k0), p.Tk) - s.k0;
        bad |= s.k0 != k0 || s.k0 + s.nk != k1;
    }
    return s;
}

// Cost of the unit with the tokens [r, r + rows) of a sequence, in steps of two tiles.
__device__ __forceinline__ int cost_of(const VarlenPlanParams &p, const Seq &s, int r)
{
    int lo = 0, hi = (s.nk + 127) / 128;
    if (p.causal) {
        const int delta = s.nk - s.nq;
        const int last = min(r + p.rows, s.nq) - 1 + delta;  // last key of the last row
        hi = min(hi, max(0, last) / 128 + 1);
        if (p.window > 0) lo = max(0, r + delta - p.window + 1) / 128;
    }
    const int n = max(1, hi - lo);
    // twins take two key tiles a step, and half as long again as two tiles with one
    return p.twins && r + p.rows / 2 >= s.nq ? (3 * n + 3) / 4 : n;
}

}  // namespace varlen

__global__ void __launch_bounds__(varlen::kThreads, 1) fa_varlen_plan_kernel(const VarlenPlanParams p)
{
    using namespace varlen;
    __shared__ int first[kMaxSeqs + 1];  // jobs of the sequences before each
    __shared__ int bins[kBins];
    __shared__ int warp_sums[32];
    __shared__ int top;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) top = 1;
    for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;

    // Sequences that overlap (cu_q that does not ascend) can ask for more jobs than the plan holds,
    // and than an int does: counts, sums and `first` stop at one job more than that.
    const int most = p.max_jobs + 1;  // (2^26 / 8 + 4096 at most: 32 of them stay below 2^29)
    bool bad = false;
    int n_jobs = 0, longest = 1;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B) {
            const Seq s = sequence(p, b, bad);
            n = min((s.nq + p.rows - 1) / p.rows, most);
            longest = max(longest, (s.nk + 127) / 128);
        }
        int sum;
        const int at = pages::block_scan(n, sum, warp_sums, most);
        if (b < p.B) first[b] = min(n_jobs + at, most);
        n_jobs = min(n_jobs + sum, most);
    }
    if (tid == 0) first[p.B] = n_jobs;
    if (n_jobs > p.max_jobs) {
        bad = true;
        n_jobs = p.max_jobs;
    }
    if (bad) raise_error(kErrCuSeqlens);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((tid & 31) == 0) atomicMax(&top, longest);
    __syncthreads();
    longest = top;

    // the class of a job, falling with its cost, and the job itself
    auto job_of = [&](int j, Seq &s, int &b, int &r) -> int {
        int lo = 0, hi = p.B;  // the last b with first[b] <= j
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= j) lo = mid;
            else hi = mid;
        }
        bool ignore = false;
        b = lo;
        s = sequence(p, b, ignore);
        r = (j - first[b]) * p.rows;
        const int cost = min(cost_of(p, s, r), longest);
        return (int)((long long)(longest - cost) * (kBins - 1) / longest);
    };
    Seq s;
    int b, r;
    for (int j = tid; j < n_jobs; j += kThreads) atomicAdd(&bins[job_of(j, s, b, r)], 1);
    __syncthreads();
    int sum;
    const int at = pages::block_scan(bins[tid], sum, warp_sums);  // kBins == kThreads
    bins[tid] = at;
    __syncthreads();
    for (int j = tid; j < n_jobs; j += kThreads) {
        const int bin = job_of(j, s, b, r);
        const int to = atomicAdd(&bins[bin], 1);
        write_at(p.plan, 2 * to, 2LL * p.max_jobs, make_int4(s.q0, s.nq, s.k0, s.nk));
        write_at(p.plan, 2 * to + 1, 2LL * p.max_jobs, make_int4(r, b, 0, 0));
    }
    if (tid == 0) {
        p.head[0] = n_jobs;
        p.head[1] = 0;
    }
}

static_assert(varlen::kThreads == pages::kPlanThreads && varlen::kBins == varlen::kThreads, "one scan, one bin a thread");

// ---------------------------------------------------------------------- the attention

struct VarlenParams {
    CUtensorMap tm_q;  // (d, Hq, Tq) bf16, box (64, pack, tile_tokens), 128B swizzle
    CUtensorMap tm_k;  // (d, Tk, Hkv), box (64, 128, 1); paged: (d, page_size, num_pages * Hkv), box (64, box_rows, 1)
    CUtensorMap tm_v;
    CUtensorMap tm_o;  // (d, Hq, Tq) bf16 output, box (64, pack, 32 / pack): one warp's rows
    void *o;           // (Tq, Hq, d)
    float *lse;        // (Hq, Tq)
    const int4 *plan;  // two per job: {q row of the sequence, Nq, k row, Nk}, {first token, sequence, -, -};
                       // null: as many CTAs as units at most, each finds its own
    int *plan_head;    // [0] number of jobs, [1] units handed out so far
    int Tq, Hq, Hkv, R;
    int causal, window;
    int pack;          // query heads of one K/V head in a tile: row = token * pack + head
    int tile_tokens;   // 128 / pack
    int slots;         // head slots: Hq / pack
    float scale_log2;  // scale * log2(e)
    unsigned long long wait_limit_ns;
    // paged only
    const int *block_table;  // (B, max_pages)
    int B, page_size, max_pages, num_pages;
    int box_rows;            // rows per copy: a power of two <= 128 that divides page_size
    VarlenPlanParams jobs;   // without a plan: what the jobs are made from
};

namespace varlen {

using prefill::BM;
using prefill::BN;
using prefill::kChunkBytes;
using prefill::kLazyThreshold;
using prefill::kLn2;
using prefill::kRegsHigh;
using prefill::kRegsLow;

constexpr int kAttnThreads = prefill::kThreads;
constexpr float kFloor = -3.0e38f;  // start of the running maximum (log2 units): below any score

// A unit as the producer hands it to the other roles.  Tile s visits key tiles a[s], a[s] +
// stride, ... below n[s]: stride 1, or 2 for twins.  a[1] = n[1]: tile 1 has no tokens and no
// twin's share.
constexpr int kRecords = 4;
struct Record {
    int valid, q_row, nq, nk, head, r[2], a[2], n[2], stride;
};

template <int D, bool SHORT>
struct Cfg {
    static constexpr int kTileBytes = 128 * D * 2;
    // Two sets of the unit's two Q tiles, so that the next unit's Q is loaded while one runs.  SHORT:
    // one set, and the room for more key tiles in flight -- units are few and long there, and every
    // K/V tile is read by one CTA only, straight from HBM: with two sets and 3 stages twins took 3.1
    // us a pair of key tiles instead of 2.7, 12 paged chunks 164 us instead of 132.
    static constexpr int kSets = SHORT ? 1 : 2;
    static constexpr int kStages = (D == 128) ? (SHORT ? 5 : 3) : (SHORT ? 12 : 8);
    static constexpr int kQOff = 0;
    static constexpr int kKVOff = 2 * kSets * kTileBytes;
    static constexpr int kBarOff = kKVOff + kStages * kTileBytes;
    // barriers: kv_full[S], kv_empty[S], q_full[2][2], q_empty[2][2], s_full[2], p_ready[2],
    //           o_done[2], o_free[2], teardown, rec_full[kRecords], joined
    static constexpr int kNumBars = 2 * kStages + 18 + kRecords;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kRecOff = kMiscOff + 16;
    static constexpr int kSmemBytes = kRecOff + kRecords * (int)sizeof(Record) + 1024;  // + alignment slack
};

struct Unit {
    int b, g, h0, q_row, k_row, nq, nk, r0, a0, a1, n0, n1;
    bool twin;
};

// The unit of head slot `slot` and the plan's entry (x, y).  A tile whose tokens see no key at
// all reads one key tile, wholly masked.
template <bool WINDOW, bool SHORT>
__device__ __forceinline__ void make_unit(const VarlenParams &p, const int4 &x, const int4 &y, int slot, Unit &w)
{
    w.q_row = x.x;
    w.nq = x.y;
    w.k_row = x.z;
    w.nk = x.w;
    w.r0 = y.x;
    w.b = y.y;
    w.h0 = slot * p.pack;
    w.g = w.h0 / p.R;
    const int r1 = w.r0 + p.tile_tokens;
    const int nkt = max(1, (w.nk + BN - 1) / BN);
    w.a0 = w.a1 = 0;
    w.n0 = w.n1 = nkt;
    if (p.causal) {
        const int delta = w.nk - w.nq;
        // the last token of a tile sees keys up to its own position
        w.n0 = min(nkt, max(0, min(r1, w.nq) - 1 + delta) / BN + 1);
        w.n1 = min(nkt, max(0, min(r1 + p.tile_tokens, w.nq) - 1 + delta) / BN + 1);
        if (WINDOW) {
            w.a0 = min(w.n0 - 1, max(0, w.r0 + delta - p.window + 1) / BN);
            w.a1 = min(w.n1 - 1, max(0, r1 + delta - p.window + 1) / BN);
        }
    }
    w.twin = false;
    if (r1 >= w.nq) {
        w.twin = SHORT && w.n0 - w.a0 >= 2;
        w.n1 = w.n0;
        w.a1 = w.twin ? w.a0 + 1 : w.n0;
    }
}

// Job number `job` in order of the sequences, for a call without a plan; false behind the last.
// Whole warp, 32 sequences a step.  Lengths out of range are reported by CTA 0.
__device__ __forceinline__ bool find_job(const VarlenPlanParams &m, int job, int4 &x, int4 &y)
{
    const int lane = threadIdx.x & 31;
    bool found = false, bad = false;
    int base = 0;
    for (int b0 = 0; b0 < m.B; b0 += 32) {
        Seq s{0, 0, 0, 0};
        if (b0 + lane < m.B) s = sequence(m, b0 + lane, bad);
        const int n = (s.nq + m.rows - 1) / m.rows;
        int upto = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + upto > job);
        if (!found && hit) {
            const int l = __ffs(hit) - 1;
            x = make_int4(__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.nq, l),
                          __shfl_sync(0xffffffffu, s.k0, l), __shfl_sync(0xffffffffu, s.nk, l));
            y = make_int4((job - base - __shfl_sync(0xffffffffu, upto - n, l)) * m.rows, b0 + l, 0, 0);
            found = true;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (__any_sync(0xffffffffu, bad) && blockIdx.x == 0 && lane == 0) raise_error(kErrCuSeqlens);
    return found;
}

// Clear rows [first, 128) of a V tile (all slabs; the swizzle permutes within a row).  Whole warp.
template <int D>
__device__ __forceinline__ void clear_v_rows(uint8_t *tile, int first, int lane)
{
    const int n = (BN - first) * 8;  // 16-byte chunks of one slab
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(tile + c * kChunkBytes + first * 128);
        for (int i = lane; i < n; i += 32) at[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    ptx::fence_proxy_async_smem();  // the tensor core reads these through the async proxy
    __syncwarp();
}

// A value that all lanes hold, as one the compiler knows to be the same in all of them: the
// MMA warp's loop bounds, and all that follows from them, then stay in uniform registers (from
// plain loads of the record they took vector registers, 190 bytes of spills in that warp).
__device__ __forceinline__ int warp_uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace varlen

// One persistent CTA per SM; roles by warp as in the prefill kernel (0-3 and 4-7 softmax of tiles
// 0 and 1, 8 producer, 9 MMA, 10-11 idle).  SHORT: the variant for calls with few tokens per
// sequence in few units (see launch), with twins, late draws and one set of Q slots; all that costs
// calls without twins 10% (measured on B200: four sequences of 8192 tokens 2.12 against 1.93 ms), so
// calls of long sequences get a kernel that has none of it.
template <int D, bool OUT_F32, bool WINDOW, bool PAGED, bool SHORT>
__global__ void __launch_bounds__(varlen::kAttnThreads, 1) fa_varlen_kernel(const __grid_constant__ VarlenParams p)
{
    using namespace varlen;
    using C = Cfg<D, SHORT>;
    constexpr int kBoxes = D / 64;  // 128-byte column boxes per tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *kv_full = bars;
    uint64_t *kv_empty = bars + C::kStages;
    uint64_t *q_full = bars + 2 * C::kStages;  // [set * 2 + tile]
    uint64_t *q_empty = q_full + 4;            // [set * 2 + tile]
    uint64_t *s_full = q_full + 8;
    uint64_t *p_ready = q_full + 10;
    uint64_t *o_done = q_full + 12;
    uint64_t *o_free = q_full + 14;
    uint64_t *teardown = q_full + 16;
    uint64_t *rec_full = q_full + 17;          // [kRecords]: a unit's record written
    uint64_t *joined = q_full + 17 + kRecords; // twins: tile 1's softmax state is in its Q slot
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
    int *stop_flag = reinterpret_cast<int *>(smem + C::kMiscOff + 4);
    volatile Record *records = reinterpret_cast<volatile Record *>(smem + C::kRecOff);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(&kv_full[i], 1);
            ptx::mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(&q_full[i], 1);
            // a Q slot is free again once its last S MMA is done (MMA commit) and the epilogue,
            // which stages O through it, has stored it (one arrive per softmax warp)
            ptx::mbar_init(&q_empty[i], 5);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&s_full[s], 1);
            ptx::mbar_init(&p_ready[s], 128);
            ptx::mbar_init(&o_done[s], 1);
            ptx::mbar_init(&o_free[s], 128);
        }
        for (int i = 0; i < kRecords; ++i) ptx::mbar_init(&rec_full[i], 1);
        ptx::mbar_init(teardown, 1);
        ptx::mbar_init(joined, 128);
        *stop_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 9) {
        ptx::tmem_alloc(tmem_holder, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        ptx::tma_prefetch_desc(&p.tm_q);
        ptx::tma_prefetch_desc(&p.tm_k);
        ptx::tma_prefetch_desc(&p.tm_v);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const StopFlag sf{stop_flag, p.wait_limit_ns};
    // Q slot of tile s of unit number i, and the parity of the phase in which it is filled
    auto q_index = [](uint32_t i, int s) { return C::kSets == 2 ? 2 * (int)(i & 1u) + s : s; };
    auto q_parity = [](uint32_t i) { return C::kSets == 2 ? (i >> 1) & 1u : i & 1u; };
    // unit number i of this CTA's order has a record (false at the end)
    auto have_record = [&](uint32_t i) -> bool {
        if (!wait_warp(&rec_full[i % kRecords], (i / kRecords) & 1u, sf)) return false;
        return __any_sync(0xffffffffu, records[i % kRecords].valid);
    };

    const uint32_t q_saddr0 = ptx::smem_addr(smem + C::kQOff);
    const uint32_t kv_saddr0 = ptx::smem_addr(smem + C::kKVOff);

    if (warp == 8) {
        // ------------------------------------------------------------ TMA producer
        // The whole warp runs the loop (every value is warp-uniform); one elected lane issues
        // the copies (paged K and V: a lane per box).
        ptx::regs_decrease<kRegsLow>();
        const bool leader = ptx::elect_one();
        const int leader_lane = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
        uint32_t kv_it = 0;
        uint32_t q_fills[4] = {0u, 0u, 0u, 0u};
        bool ok = true;
        // Q tiles of unit number i are loaded one unit ahead, whenever their slot is free, between
        // K/V loads; only at the end of a unit does the warp block on them.
        // A tile has tile_tokens * pack rows (the last of 128 stay as they are when pack does not
        // divide 128; their results are not stored).
        auto issue_q = [&](const Unit &uw, uint32_t i, int s) {
            const int qi = q_index(i, s);
            ++q_fills[qi];
            if (leader) {
                uint8_t *dst = smem + C::kQOff + qi * C::kTileBytes;
                const int row = uw.q_row + uw.r0 + (s && !uw.twin ? p.tile_tokens : 0);
                ptx::mbar_arrive_expect_tx(&q_full[qi], kBoxes * 128 * p.pack * p.tile_tokens);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c)
                    ptx::tma_load_4d(dst + c * kChunkBytes, &p.tm_q, &q_full[qi], 64 * c, uw.h0, row, 0);
            }
            __syncwarp();
        };
        auto q_slot = [&](uint32_t i, int s) { return &q_empty[q_index(i, s)]; };
        auto q_free_parity = [&](uint32_t i) { return q_parity(i) ^ 1u; };

        // Unit 0 is the CTA's own number, the others come from the counter.  With many units per
        // CTA the number of unit i + 1 is known when unit i starts and that of i + 2 is asked for
        // then, so neither the counter's nor the plan's latency holds up the K/V stream.  With few
        // (`late`), a number drawn early is a long unit dealt out blindly: unit i + 1 is then drawn
        // four key tiles before unit i's last, one step of its way per tile.
        const bool alone = SHORT && p.plan == nullptr;  // one unit per CTA, found without a plan
        if (!alone) asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is complete
        const int n_units = alone ? 0 : __ldcg(&p.plan_head[0]) * p.slots;
        const bool late = SHORT && n_units < 4 * (int)gridDim.x;
        auto draw = [&]() { return leader ? (int)gridDim.x + atomicAdd(&p.plan_head[1], 1) : 0; };
        auto read_plan = [&](int job, int4 &x, int4 &y) {
            if (!in_bounds(job, p.jobs.max_jobs)) return;
            x = __ldcg(p.plan + 2 * job);
            y = __ldcg(p.plan + 2 * job + 1);
        };
        // A record's slot is reused four units later: Q(i) was issued, so unit i - 2 has released
        // its Q slots, and every role is done with unit i - 3, whose slot unit i + 1 takes.
        auto publish = [&](uint32_t i, bool valid, const Unit &uw) {
            if (leader) {
                volatile Record &r = records[i % kRecords];
                r.valid = valid ? 1 : 0;
                if (valid) {
                    r.q_row = uw.q_row;
                    r.nq = uw.nq;
                    r.nk = uw.nk;
                    r.head = uw.h0;
                    r.r[0] = uw.r0;
                    r.r[1] = uw.r0 + (uw.twin ? 0 : p.tile_tokens);
                    r.a[0] = uw.a0;
                    r.a[1] = uw.a1;
                    r.n[0] = uw.n0;
                    r.n[1] = uw.n1;
                    r.stride = uw.twin ? 2 : 1;
                }
                ptx::mbar_arrive(&rec_full[i % kRecords]);
            }
            __syncwarp();
        };
        // Pages: lane l looks up the page of copy l of a key tile (box_rows keys).  Keys past the
        // end, and pages outside the pool (reported), read the plane behind the last, which the
        // copy engine fills with zeros.
        const int boxes = PAGED ? BN / p.box_rows : 1;
        constexpr int kNoPage = -0x40000000;
        auto page_of = [&](const Unit &uw, int j) -> int {
            const int pos = BN * j + lane * p.box_rows;
            if (lane >= boxes || j >= uw.n1 || pos >= uw.nk) return kNoPage;
            const long long at = (long long)uw.b * p.max_pages + pos / p.page_size;
            return in_bounds(at, (long long)p.B * p.max_pages) ? p.block_table[at] : kNoPage;
        };
        auto load_tile = [&](const CUtensorMap *map, const Unit &uw, int j, int page) -> bool {
            const uint32_t st = kv_it % C::kStages;
            const uint32_t ph = (kv_it / C::kStages) & 1u;
            if (!wait_warp(&kv_empty[st], ph ^ 1u, sf)) return false;
            uint8_t *dst = smem + C::kKVOff + st * C::kTileBytes;
            if (leader) {
                ptx::mbar_arrive_expect_tx(&kv_full[st], C::kTileBytes);
                if (!PAGED) {
#pragma unroll
                    for (int c = 0; c < kBoxes; ++c)
                        ptx::tma_load_4d(dst + c * kChunkBytes, map, &kv_full[st], 64 * c, uw.k_row + BN * j, uw.g, 0);
                }
            }
            __syncwarp();
            if (PAGED) {
                if (lane < boxes) {
                    int plane = p.num_pages * p.Hkv;
                    if (page >= 0 && page < p.num_pages) plane = page * p.Hkv + uw.g;
                    else if (page != kNoPage) raise_error(kErrPageRange);
                    const int pos = BN * j + lane * p.box_rows;
#pragma unroll
                    for (int c = 0; c < kBoxes; ++c)
                        ptx::tma_load_3d(dst + c * kChunkBytes + lane * p.box_rows * 128, map, &kv_full[st], 64 * c,
                                         pos % p.page_size, plane);
                }
                __syncwarp();
            }
            ++kv_it;
            return true;
        };

        Unit w, wn;
        int slot = 0, u = (int)blockIdx.x;
        int next_raw = late ? 0 : draw();
        uint32_t i = 0;
        const int job0 = u / p.slots;
        slot = u - job0 * p.slots;
        int4 x0 = make_int4(0, 0, 0, 0), y0 = x0;
        bool have;
        if (alone) {
            have = find_job(p.jobs, job0, x0, y0);
        } else if ((have = u < n_units)) {
            read_plan(job0, x0, y0);
        }
        if (have) make_unit<WINDOW, SHORT>(p, x0, y0, slot, w);
        publish(0, have, w);
        for (int s = 0; ok && have && s < 2; ++s) {
            if (!wait_warp(q_slot(0, s), q_free_parity(0), sf)) ok = false;
            else issue_q(w, 0, s);
        }
        // pages of the even and odd key tiles (counted from a0) next to be loaded
        int page0 = PAGED && have ? page_of(w, w.a0) : 0, page1 = PAGED && have ? page_of(w, w.a0 + 1) : 0;
        int page0_n = 0, page1_n = 0;
        for (; ok && have; ++i) {
            bool have_n = false;
            int4 px = make_int4(0, 0, 0, 0), py = px;  // the next unit's plan entry, in flight
            int q_next = alone ? 2 : 0;                // look-ahead Q tiles already issued
            enum { kAsk, kLookUp, kTell, kTold } step = alone ? kTell : late ? kAsk : kLookUp;
            auto ask = [&]() {
                next_raw = draw();
                step = kLookUp;
            };
            auto look_up = [&]() {
                u = __shfl_sync(0xffffffffu, next_raw, leader_lane);
                have_n = u < n_units;
                if (have_n) {
                    const int job = u / p.slots;
                    slot = u - job * p.slots;
                    read_plan(job, px, py);
                    if (!late) next_raw = draw();
                } else {
                    q_next = 2;
                }
                step = kTell;
            };
            auto tell = [&]() {
                if (have_n) {
                    make_unit<WINDOW, SHORT>(p, px, py, slot, wn);
                    if (PAGED) {
                        page0_n = page_of(wn, wn.a0);
                        page1_n = page_of(wn, wn.a0 + 1);
                    }
                }
                publish(i + 1, have_n, wn);
                step = kTold;
            };
            if (step == kLookUp) look_up();
            // K and V of key tile after key tile; twins: K, K, V, V of a pair of key tiles, the
            // order in which their S and P V MMAs release the ring's stages.
            const int tiles = w.n1 - w.a0;
            for (int e = 0; e < 2 * tiles; ++e) {
                int t = e >> 1, v = e & 1;
                if (SHORT && w.twin && (e | 3) < 2 * tiles) {
                    t = 2 * (e >> 2) + (e & 1);
                    v = (e >> 1) & 1;
                }
                if (!load_tile(v ? &p.tm_v : &p.tm_k, w, w.a0 + t, (t & 1) ? page1 : page0)) { ok = false; break; }
                if (PAGED && v) {
                    const int pg = page_of(w, w.a0 + t + 2);
                    if (t & 1) page1 = pg;
                    else page0 = pg;
                }
                if (v) {
                    if (step == kTell) tell();
                    else if (SHORT && step == kLookUp) look_up();
                    else if (SHORT && step == kAsk && tiles - t <= 4) ask();
                }
                // (With one set the slot is this unit's own: it is not free before the unit's end, and
                // this look, a try_wait, would suspend the warp and with it K and V.  Of two sets the
                // other is free within a tile or so; a plain probe there cost LONG 1%.)
                while (C::kSets == 2 && step == kTold && q_next < 2 &&
                       __all_sync(0xffffffffu, ptx::mbar_test(q_slot(i + 1, q_next), q_free_parity(i + 1)))) {
                    issue_q(wn, i + 1, q_next);
                    ++q_next;
                }
            }
            if (SHORT) {
                if (step == kAsk) ask();
                if (step == kLookUp) look_up();
                if (step == kTell) tell();
            }
            for (; ok && q_next < 2; ++q_next) {
                if (!wait_warp(q_slot(i + 1, q_next), q_free_parity(i + 1), sf)) ok = false;
                else issue_q(wn, i + 1, q_next);
            }
            have = have_n;
            w = wn;
            page0 = page0_n;
            page1 = page1_n;
        }
        // Let every copy this warp started land before the CTA can exit.
        if (leader) {
            for (uint32_t st = 0; st < (uint32_t)C::kStages && st < kv_it; ++st) {
                const uint32_t last = kv_it - 1 - ((kv_it - 1 - st) % C::kStages);
                prefill::drain_wait(&kv_full[st], (last / C::kStages) & 1u, p.wait_limit_ns);
            }
            for (int qi = 0; qi < 4; ++qi)
                if (q_fills[qi] > 0) prefill::drain_wait(&q_full[qi], (q_fills[qi] - 1) & 1u, p.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp == 9) {
        // --------------------------------------------------------------- MMA issuer
        ptx::regs_decrease<kRegsLow>();
        const bool leader = ptx::elect_one();
        uint32_t kv_it = 0, units = 0;
        uint32_t p_ph[2] = {0u, 0u};
        bool ok = true;
        // The P V of tile 1's last key tile is carried into the next unit's first iteration, after
        // that unit's first S0 MMA, so the S0 / PV1 / S1 / PV0 ping-pong runs on across units.
        bool pend = false, pend_acc = false, pend_free = false;
        uint32_t pend_v = 0, pend_free_par = 0;
        auto stage_addr = [&](uint32_t st) { return kv_saddr0 + st * C::kTileBytes; };
        // P V of Q tile s with the V tile in ring stage v_stage
        auto issue_pv_of = [&](int s, uint32_t v_stage, bool acc, bool need_free, uint32_t fpar) -> bool {
            if (!wait_warp(&p_ready[s], p_ph[s], sf)) return false;
            p_ph[s] ^= 1u;
            if (need_free && !wait_warp(&o_free[s], fpar, sf)) return false;
            ptx::tc_fence_after();
            if (leader) prefill::issue_pv<D, 0, 8>(tmem + 256 + 128 * s, tmem + 128 * s, stage_addr(v_stage), acc);
            __syncwarp();
            return true;
        };
        auto issue_pv1 = [&](uint32_t v_stage, bool acc, bool need_free, uint32_t fpar, bool last) -> bool {
            if (!issue_pv_of(1, v_stage, acc, need_free, fpar)) return false;
            if (leader) {
                ptx::mma_commit(&kv_empty[v_stage]);
                if (last) ptx::mma_commit(&o_done[1]);
            }
            __syncwarp();
            return true;
        };
        while (ok && have_record(units)) {
            const volatile Record &r = records[units % kRecords];
            const int nk = warp_uniform(r.nk);
            const int n0 = warp_uniform(r.n[0]), n1 = warp_uniform(r.n[1]);
            const int a0 = WINDOW ? warp_uniform(r.a[0]) : 0, a1 = warp_uniform(r.a[1]);
            const bool twin = SHORT && warp_uniform(r.stride) == 2;
            const uint32_t free_par = (units & 1u) ^ 1u;  // first unit passes at once
            const uint32_t q_par = q_parity(units);
            uint64_t *qf = q_full + q_index(units, 0);
            uint64_t *qe = q_empty + q_index(units, 0);
            const uint32_t q_saddr = q_saddr0 + q_index(units, 0) * C::kTileBytes;
            if (!wait_warp(&qf[0], q_par, sf) || !wait_warp(&qf[1], q_par, sf)) break;
            ptx::tc_fence_after();
            // wait for ring entry `it`; a V tile that passes the last key is cleared behind it
            auto arrived = [&](uint32_t it) -> bool {
                if (!wait_warp(&kv_full[it % C::kStages], (it / C::kStages) & 1u, sf)) return false;
                ptx::tc_fence_after();
                return true;
            };
            auto v_arrived = [&](uint32_t it, int j) -> bool {
                if (!wait_warp(&kv_full[it % C::kStages], (it / C::kStages) & 1u, sf)) return false;
                if (BN * j + BN > nk)
                    clear_v_rows<D>(smem + C::kKVOff + (it % C::kStages) * C::kTileBytes, max(0, nk - BN * j), lane);
                return true;
            };
            uint32_t prev_v = 0;
            if (!twin) {
                // Key tile j feeds S0 / P V0 when a0 <= j < n0 and S1 / P V1 when a1 <= j < n1
                // (a1 = n1: tile 1 has no tokens).
                for (int j = a0; j < n1; ++j) {
                    const uint32_t ks = kv_it % C::kStages, vs = (kv_it + 1) % C::kStages;
                    if (!arrived(kv_it)) { ok = false; break; }
                    if (j < n0) {
                        if (leader) {
                            prefill::issue_qk<D>(tmem + 0, q_saddr, stage_addr(ks));
                            ptx::mma_commit(&s_full[0]);
                            if (j == n0 - 1) ptx::mma_commit(&qe[0]);
                        }
                        __syncwarp();
                    }
                    if (j > a1) {
                        if (!issue_pv1(prev_v, j - 1 > a1, j - 1 == a1, free_par, false)) { ok = false; break; }
                    } else if (pend) {
                        if (!issue_pv1(pend_v, pend_acc, pend_free, pend_free_par, true)) { ok = false; break; }
                        pend = false;
                    }
                    if (leader) {
                        if (j >= a1) {
                            prefill::issue_qk<D>(tmem + 128, q_saddr + C::kTileBytes, stage_addr(ks));
                            ptx::mma_commit(&s_full[1]);
                        }
                        ptx::mma_commit(&kv_empty[ks]);
                        if (j == n1 - 1) ptx::mma_commit(&qe[1]);
                    }
                    __syncwarp();
                    if (!v_arrived(kv_it + 1, j)) { ok = false; break; }
                    if (j < n0) {
                        if (!issue_pv_of(0, vs, j > a0, j == a0, free_par)) { ok = false; break; }
                        if (leader && j == n0 - 1) ptx::mma_commit(&o_done[0]);
                        __syncwarp();
                    }
                    if (j < a1) {  // a V tile that Q tile 1 never reads
                        if (leader) ptx::mma_commit(&kv_empty[vs]);
                        __syncwarp();
                    }
                    prev_v = vs;
                    kv_it += 2;
                }
                if (!ok) break;
                pend = a1 < n1;
                if (!pend) {
                    // Tile 1's accumulator is passed on unused -- but not before every softmax warp of
                    // tile 1 has seen the last unit's o_done: two phases on, a parity wait for it
                    // would not end.
                    if (!wait_warp(&o_free[1], free_par, sf)) break;
                    if (leader) ptx::mma_commit(&o_done[1]);
                    __syncwarp();
                }
                pend_acc = n1 - 1 > a1;
                pend_free = n1 - 1 == a1;
            } else {
                // Twins: key tiles a0, a0 + 2, ... feed tile 0 and a0 + 1, ... tile 1.  Ring
                // entries of a pair: K, K, V, V; of a last single tile: K, V.
                const int tiles = n0 - a0;
                for (int t = 0; t < tiles; t += 2) {
                    const bool two = t + 1 < tiles;
                    const uint32_t ka = kv_it, kb = kv_it + 1, va = kv_it + (two ? 2 : 1), vb = kv_it + 3;
                    if (!arrived(ka)) { ok = false; break; }
                    if (leader) {
                        prefill::issue_qk<D>(tmem + 0, q_saddr, stage_addr(ka % C::kStages));
                        ptx::mma_commit(&s_full[0]);
                        ptx::mma_commit(&kv_empty[ka % C::kStages]);
                        if (t + 2 >= tiles) ptx::mma_commit(&qe[0]);
                    }
                    __syncwarp();
                    if (t > 0) {
                        if (!issue_pv1(prev_v, t > 2, t == 2, free_par, !two)) { ok = false; break; }
                    } else if (pend) {
                        if (!issue_pv1(pend_v, pend_acc, pend_free, pend_free_par, true)) { ok = false; break; }
                        pend = false;
                    }
                    if (two) {
                        if (!arrived(kb)) { ok = false; break; }
                        if (leader) {
                            prefill::issue_qk<D>(tmem + 128, q_saddr + C::kTileBytes, stage_addr(kb % C::kStages));
                            ptx::mma_commit(&s_full[1]);
                            ptx::mma_commit(&kv_empty[kb % C::kStages]);
                            if (t + 3 >= tiles) ptx::mma_commit(&qe[1]);
                        }
                        __syncwarp();
                    }
                    if (!v_arrived(va, a0 + t) || !issue_pv_of(0, va % C::kStages, t > 0, t == 0, free_par)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        ptx::mma_commit(&kv_empty[va % C::kStages]);
                        if (t + 2 >= tiles) ptx::mma_commit(&o_done[0]);
                    }
                    __syncwarp();
                    if (two) {
                        if (!v_arrived(vb, a0 + t + 1)) { ok = false; break; }
                        prev_v = vb % C::kStages;
                    }
                    kv_it += two ? 4 : 2;
                }
                if (!ok) break;
                pend = (tiles & 1) == 0;  // of an odd number, tile 1's last P V is issued above
                pend_acc = tiles > 2;
                pend_free = tiles == 2;
            }
            pend_v = prev_v;
            pend_free_par = free_par;
            if (SHORT && pend) {  // not carried: the next unit's Q waits for this unit's end
                if (!issue_pv1(pend_v, pend_acc, pend_free, pend_free_par, true)) { ok = false; break; }
                pend = false;
            }
            ++units;
        }
        if (ok && pend) issue_pv1(pend_v, pend_acc, pend_free, pend_free_par, true);
        // Every MMA and commit issued above completes before the CTA can exit.
        if (leader) {
            ptx::mma_commit(teardown);
            prefill::drain_wait(teardown, 0, p.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax warps
        ptx::regs_increase<kRegsHigh>();
        const int s = warp >> 2;              // which Q tile of the unit
        const int tid = threadIdx.x & 127;    // row inside the tile = TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + 128u * s;         // S_s, and P_s over it
        const uint32_t tO = tmem + lane_base + 256u + 128u * s;  // O_s
        const float sl2 = p.scale_log2;
        uint32_t s_ph = 0, units = 0, joins = 0;
        for (; have_record(units); ++units) {
            // What the key loop needs is read from the record here, what the epilogue needs there
            // (the record stays in place until this unit's last role is done), so that it takes no
            // registers in between.
            const volatile Record &rec = records[units % kRecords];
            const int n = rec.n[s], stride = SHORT ? rec.stride : 1;
            int lim, first = 0;
            {
                const int nk = rec.nk;
                const int diag = rec.r[s] + tid / p.pack + (nk - rec.nq);  // last key of a causal row
                lim = p.causal ? min(diag, nk - 1) : nk - 1;
                if (WINDOW) first = diag - p.window + 1;
            }
            // l: sum of the fp32 weights (gives the LSE).  lo: normaliser of O, the same sum
            // corrected, tile by tile, by the bf16 rounding of the tile's largest weight --
            // the rounding the P V product actually saw.  For a row dominated by one key
            // this makes O exactly that key's value row, as it should be.
            float m = kFloor, l = 0.f, lo = 0.f;
            bool ok = true, fresh = true;
            for (int j = rec.a[s]; j < n; j += stride) {
                if (!wait_warp(&s_full[s], s_ph, sf)) { ok = false; break; }
                s_ph ^= 1u;
                ptx::tc_fence_after();
                uint32_t x[128];
                const int kbase = BN * j;
                float alpha = 1.f;
                bool rescale = false;
                // Scores of this tile, masked past the row's last visible key; the tile maximum;
                // lazy update of the reference maximum m (moved only when the new one exceeds it
                // by more than kLazyThreshold, which then rescales O).
                ptx::tmem_ld32(tS + 0, &x[0]);
                ptx::tmem_ld32(tS + 32, &x[32]);
                ptx::tmem_ld32(tS + 64, &x[64]);
                ptx::tmem_ld32(tS + 96, &x[96]);
                ptx::tmem_wait_ld();
                prefill::mask_cols<0, 128>(x, kbase, lim);
                if (WINDOW) prefill::mask_cols_below<0, 128>(x, kbase, first);
                const float mx = fmaxf(prefill::row_max64<0>(x), prefill::row_max64<64>(x)) * sl2;
                if (fresh) {
                    m = fmaxf(mx, kFloor);  // O is not written yet: the first P V overwrites it
                    fresh = false;
                } else if (mx - m > kLazyThreshold) {
                    alpha = ptx::ex2(m - mx);
                    m = mx;
                    rescale = true;
                }
                const float sum = prefill::exp2_pack<64, 0, 0>(x, sl2, m) + prefill::exp2_pack<64, 64, 32>(x, sl2, m);
                ptx::tmem_st32(tS + 0, &x[0]);
                ptx::tmem_st32(tS + 32, &x[32]);
                // Rare (lazy) rescale of the partial output, before any P V of this tile is issued
                // (P V of the previous tile is complete: the commit that signalled this S tile
                // covers it); warp-uniform because TMEM accesses are collective.
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        ptx::tmem_ld32(tO + 32 * c, ov);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        ptx::tmem_st32(tO + 32 * c, ov);
                    }
                }
                ptx::tmem_wait_st();
                const float p_top = ptx::ex2(mx - m);  // the tile's largest weight (0 if masked)
                const float p_top_bf = __uint_as_float(ptx::pack_bf16x2(p_top, 0.f) << 16);
                l = l * alpha + sum;
                lo = lo * alpha + sum + (p_top_bf - p_top);
                ptx::tc_fence_before();
                ptx::mbar_arrive(&p_ready[s]);
            }
            if (!ok) break;
            // ------------------------------------------------------------- epilogue
            // O_s / lo leaves TMEM as soon as it is read (o_free lets the next unit's first P V
            // overwrite it).  bf16 output is staged, 128-byte swizzled, in this unit's Q slot -- no
            // MMA reads it any more -- and each warp writes its own 32 rows, then hands its part of
            // the slot back to the producer, so no warp waits for another.
            if (!wait_warp(&o_done[s], units & 1u, sf)) break;
            ptx::tc_fence_after();
            const int qi = q_index(units, s);
            uint8_t *stage = smem + C::kQOff + qi * C::kTileBytes;
            const bool twin = SHORT && rec.stride == 2;
            float f0 = 1.f, f1 = 0.f;  // twins: factors of the two partial outputs
            if (s == 1) {
                if (twin) {
                    // tile 0's warps finish the unit: they read this state and O_1, then release
                    // O_1 and this Q slot
                    float *state = reinterpret_cast<float *>(stage);
                    state[tid] = m;
                    state[128 + tid] = l;
                    state[256 + tid] = lo;
                    ptx::fence_proxy_async_smem();  // before the copy engine refills the slot
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(joined);
                    continue;
                }
                if (rec.a[1] == rec.n[1]) {  // no tokens in this tile
                    ptx::mbar_arrive(&o_free[1]);
                    if (lane == 0) ptx::mbar_arrive(&q_empty[qi]);
                    continue;
                }
            } else if (twin) {
                if (!wait_warp(joined, joins & 1u, sf) || !wait_warp(&o_done[1], units & 1u, sf)) break;
                ++joins;
                ptx::tc_fence_after();
                const float *state = reinterpret_cast<const float *>(stage + C::kTileBytes);
                const float m1 = state[tid], l1 = state[128 + tid], lo1 = state[256 + tid];
                const float top = fmaxf(m, m1);
                f0 = ptx::ex2(m - top);
                f1 = ptx::ex2(m1 - top);
                m = top;
                l = l * f0 + l1 * f1;
                lo = lo * f0 + lo1 * f1;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&q_empty[qi + 1]);
            }
            const int nq = rec.nq, q_row = rec.q_row, r0 = rec.r[s], head = rec.head;
            const int row = r0 + tid / p.pack, h = head + tid % p.pack;
            const bool valid = row < nq && tid < p.pack * p.tile_tokens;
            const bool none = l == 0.f;  // the row sees no key
            const float inv_l = none ? 0.f : 1.f / lo;
            const int wr = 32 * (warp & 3);  // this warp's rows of the tile
            const long long ooff = ((q_row + (long long)row) * p.Hq + h) * D;
            const bool store = valid && in_bounds(ooff + D - 1, (long long)p.Hq * p.Tq * D);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t ov[64];
                ptx::tmem_ld32(tO + 64 * c, &ov[0]);
                ptx::tmem_ld32(tO + 64 * c + 32, &ov[32]);
                ptx::tmem_wait_ld();
                if (twin) {  // (s = 0: O_1 is 128 columns on)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t o1[32];
                        ptx::tmem_ld32(tO + 128 + 64 * c + 32 * q, o1);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[32 * q + e] = __float_as_uint(__uint_as_float(ov[32 * q + e]) * f0 + __uint_as_float(o1[e]) * f1);
                    }
                }
                if (c == D / 64 - 1) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&o_free[s]);
                    if (twin) ptx::mbar_arrive(&o_free[1]);
                }
                if (__any_sync(0xffffffffu, none)) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) ov[e] = none ? 0u : ov[e];
                }
                if (OUT_F32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.o) + ooff + 64 * c);
                    if (store) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            dst[e] = make_float4(__uint_as_float(ov[4 * e]) * inv_l, __uint_as_float(ov[4 * e + 1]) * inv_l,
                                                 __uint_as_float(ov[4 * e + 2]) * inv_l, __uint_as_float(ov[4 * e + 3]) * inv_l);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t *src = &ov[8 * e];
                        uint4 v4;
                        v4.x = ptx::pack_bf16x2(__uint_as_float(src[0]) * inv_l, __uint_as_float(src[1]) * inv_l);
                        v4.y = ptx::pack_bf16x2(__uint_as_float(src[2]) * inv_l, __uint_as_float(src[3]) * inv_l);
                        v4.z = ptx::pack_bf16x2(__uint_as_float(src[4]) * inv_l, __uint_as_float(src[5]) * inv_l);
                        v4.w = ptx::pack_bf16x2(__uint_as_float(src[6]) * inv_l, __uint_as_float(src[7]) * inv_l);
                        *reinterpret_cast<uint4 *>(stage + c * kChunkBytes + tid * 128 + ((e ^ (tid & 7)) << 4)) = v4;
                    }
                }
            }
            if (!OUT_F32) {
                // One TMA box holds the warp's 32 rows if they are whole tokens and all of this
                // sequence; otherwise the warp copies the rows that exist from the stage.
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (32 % p.pack == 0 && r0 + (wr + 32) / p.pack <= nq) {
                    if (lane == 0 && in_bounds(head, p.Hq)) {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            ptx::tma_store_4d(&p.tm_o, stage + c * kChunkBytes + wr * 128, 64 * c, head,
                                              q_row + r0 + wr / p.pack, 0);
                        ptx::bulk_commit_group();
                        ptx::bulk_wait_group_read0();
                    }
                } else {
                    for (int i = lane; i < 32 * (D / 8); i += 32) {
                        const int t = wr + i / (D / 8), e = i % (D / 8);
                        const int token = t / p.pack;
                        if (t >= p.pack * p.tile_tokens || r0 + token >= nq) break;  // (rows ascend with i)
                        const long long at = ((q_row + (long long)r0 + token) * p.Hq + head + t - token * p.pack) * D + 8 * e;
                        if (in_bounds(at + 7, (long long)p.Hq * p.Tq * D))
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + at) =
                                *reinterpret_cast<const uint4 *>(stage + (e >> 3) * kChunkBytes + t * 128 +
                                                                 (((e & 7) ^ (t & 7)) << 4));
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) ptx::mbar_arrive(&q_empty[qi]);
            const long long lrow = (long long)h * p.Tq + q_row + row;
            if (valid && in_bounds(lrow, (long long)p.Hq * p.Tq)) p.lse[lrow] = none ? -INFINITY : (m + ptx::lg2(l)) * kLn2;
        }
        if (!OUT_F32 && lane == 0) ptx::bulk_wait_group0();  // stores complete before exit
    } else {
        ptx::regs_decrease<kRegsLow>();
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace fa
