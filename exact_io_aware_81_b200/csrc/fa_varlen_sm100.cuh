// fa_varlen_sm100.cuh -- the order of work for attention over packed sequences.
//
// The lengths are known on the device only.  A job is one row tile (128 query rows, or 256
// where a unit of the attention kernel is a pair of row tiles) of one sequence; its cost is
// the number of key tiles that its last row sees.  The plan lists all jobs in order of falling
// cost (longest first), so that the attention kernel's CTAs, which draw units from a counter,
// end together: a counting sort over kBins classes of cost, whose order within a class is left
// open (it decides which CTA computes what, never a result).
//
// Bound: latency.  One CTA: sums of the tile counts over the sequences, then one thread per
// job (the sequence by bisection of the sums), two passes.  It releases the attention kernel's
// launch at once (programmatic dependent launch), whose set-up then overlaps it.
#pragma once

#include <cstdint>

#include "fa_common.cuh"
#include "fa_pages_sm100.cuh"

namespace fa {

struct VarlenPlanParams {
    const int *cu_q;     // (B + 1)
    const int *cu_k;     // (B + 1), or
    const int *seqlens;  // (B): key counts of a paged cache (k rows then start at 0)
    int4 *plan;          // (2 * max_jobs)
    int *head;           // [0] number of jobs, [1] counter
    int B, Tq, Tk;       // Tk: rows of k, or the most keys the block table holds
    int rows;            // query rows of a job: 128 or 256
    int causal, window;
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
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
    s.q0 = min(max(q0, 0), p.Tq);
    s.nq = min(max(q1, s.q0), p.Tq) - s.q0;
    bad |= s.q0 != q0 || s.q0 + s.nq != q1;
    if (p.seqlens) {
        const int n = p.seqlens[b];
        s.k0 = 0;
        s.nk = min(max(n, 0), p.Tk);
        bad |= s.nk != n;
    } else {
        const int k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
        s.k0 = min(max(k0, 0), p.Tk);
        s.nk = min(max(k1, s.k0), p.Tk) - s.k0;
        bad |= s.k0 != k0 || s.k0 + s.nk != k1;
    }
    return s;
}

// Key tiles that the rows [r, r + rows) of a sequence read.
__device__ __forceinline__ int cost_of(const VarlenPlanParams &p, const Seq &s, int r)
{
    int lo = 0, hi = (s.nk + 127) / 128;
    if (p.causal) {
        const int delta = s.nk - s.nq;
        const int last = min(r + p.rows, s.nq) - 1 + delta;  // last key of the last row
        hi = min(hi, max(0, last) / 128 + 1);
        if (p.window > 0) lo = max(0, r + delta - p.window + 1) / 128;
    }
    return max(1, hi - lo);
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

    bool bad = false;
    int n_jobs = 0, longest = 1;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B) {
            const Seq s = sequence(p, b, bad);
            n = (s.nq + p.rows - 1) / p.rows;
            longest = max(longest, (s.nk + 127) / 128);
        }
        int sum;
        const int at = pages::block_scan(n, sum, warp_sums);
        if (b < p.B) first[b] = n_jobs + at;
        n_jobs += sum;
    }
    if (tid == 0) first[p.B] = n_jobs;
    // sequences that overlap could ask for more jobs than the plan holds
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
        p.plan[2 * to] = make_int4(s.q0, s.nq, s.k0, s.nk);
        p.plan[2 * to + 1] = make_int4(r, b, 0, 0);
    }
    if (tid == 0) {
        p.head[0] = n_jobs;
        p.head[1] = 0;
    }
}

static_assert(varlen::kThreads == pages::kPlanThreads && varlen::kBins == varlen::kThreads, "one scan, one bin a thread");

}  // namespace fa
