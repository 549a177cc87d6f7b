// page_plan.cuh -- what the planning kernels of the page calls share: one cluster of 8 CTAs of 1024 threads
// scans the refcounts and finds free pages in the order of their numbers.
#pragma once

#include <cooperative_groups.h>

#include "smla_internal.cuh"

namespace cg = cooperative_groups;

namespace smla {

namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanShared {
    int warp[2][kPlanWarps];    // a scan's sums by warp; two sets in turn
    int part;                   // this CTA's total and status bits, read by the other CTAs
    unsigned bits;
};

// Exclusive sum over the CTA's threads in thread order; *total gets the sum. `turn`
// alternates from scan to scan (one barrier a scan: the sums of the last but one are read).
__device__ __forceinline__ int cta_scan(int v, PlanShared& sh, int& turn, int* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh.warp[turn][warp] = x;
    __syncthreads();
    static_assert(kPlanWarps == 32, "a lane for each warp's sum");
    int y = sh.warp[turn][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) y += z;
    }
    turn ^= 1;
    *total = __shfl_sync(0xffffffffu, y, 31);
    const int before = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
    return (warp ? before : 0) + x - v;
}

// This CTA's share of the pages: [lo, hi), lo a multiple of 4.
__device__ __forceinline__ void page_slice(int num_pages, int rank, int& lo, int& hi) {
    const int per = ((num_pages + kPlanCtas - 1) / kPlanCtas + 3) / 4 * 4;
    const int64_t a = int64_t(per) * rank, b = a + per;
    lo = int(a < num_pages ? a : num_pages);
    hi = int(b < num_pages ? b : num_pages);
}

// refcount[i .. i+3]; -1 past the end.
__device__ __forceinline__ int4 load4(const int32_t* rc, int i, int hi) {
    if (i + 4 <= hi) return __ldcg(reinterpret_cast<const int4*>(rc + i));
    int4 v = make_int4(-1, -1, -1, -1);
    if (i < hi) v.x = __ldcg(rc + i);
    if (i + 1 < hi) v.y = __ldcg(rc + i + 1);
    if (i + 2 < hi) v.z = __ldcg(rc + i + 2);
    return v;
}

// Pages i of [lo, hi) with pred(i, refcount) (refcount -1 never counts).
template <class Pred>
__device__ int count_pages(const int32_t* rc, int lo, int hi, PlanShared& sh, int& turn, Pred pred) {
    int n = 0;
#pragma unroll 4
    for (int i = lo + 4 * int(threadIdx.x); i < hi; i += 4 * kPlanThreads) {
        const int4 v = load4(rc, i, hi);
        n += int(pred(i, v.x)) + int(pred(i + 1, v.y)) + int(pred(i + 2, v.z)) + int(pred(i + 3, v.w));
    }
    int total;
    cta_scan(n, sh, turn, &total);
    return total;
}

// out(rank, i) for the pages i of [lo, hi) with pred(i, refcount), in order,
// ranks from `rank` on, until `limit`.
template <class Pred, class Out>
__device__ void emit_pages(const int32_t* rc, int lo, int hi, int rank, int limit, PlanShared& sh, int& turn,
                           Pred pred, Out out) {
    for (int base = lo; base < hi && rank < limit; base += 4 * kPlanThreads) {
        const int i = base + 4 * int(threadIdx.x);
        const int4 v = load4(rc, i, hi);
        const bool p0 = pred(i, v.x), p1 = pred(i + 1, v.y), p2 = pred(i + 2, v.z), p3 = pred(i + 3, v.w);
        int total;
        int r = rank + cta_scan(int(p0) + int(p1) + int(p2) + int(p3), sh, turn, &total);
        if (p0) { if (r < limit) out(r, i); ++r; }
        if (p1) { if (r < limit) out(r, i + 1); ++r; }
        if (p2) { if (r < limit) out(r, i + 2); ++r; }
        if (p3) { if (r < limit) out(r, i + 3); ++r; }
        rank += total;
    }
}

// The CTAs' totals: their sum, the sum over those before this one; and all status bits.
__device__ __forceinline__ void join(cg::cluster_group& cl, PlanShared& sh, int& before, int& all, unsigned& bits) {
    int part[kPlanCtas];
    unsigned b[kPlanCtas];
#pragma unroll
    for (unsigned r = 0; r < kPlanCtas; ++r) {
        part[r] = cl.map_shared_rank(&sh, r)->part;
        b[r] = cl.map_shared_rank(&sh, r)->bits;
    }
    before = 0;
    all = 0;
    bits = 0;
#pragma unroll
    for (unsigned r = 0; r < kPlanCtas; ++r) {
        if (r < cl.block_rank()) before += part[r];
        all += part[r];
        bits |= b[r];
    }
}

// Exclusive sums of need(i), i < n, saturated at `most`; each(i, need, sum before). Returns the sum.
template <class Need, class Each>
__device__ int scan_needs(int n, int most, PlanShared& sh, int& turn, Need need, Each each) {
    int64_t sum = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + int(threadIdx.x);
        // (a row's need is below 2^20 here or the call is short of pages anyway: see callers)
        const int v = i < n ? need(i) : 0;
        int total;
        const int64_t at = sum + cta_scan(v, sh, turn, &total);
        if (i < n) each(i, v, int(at < most ? at : most));
        sum += total;
        if (sum > most) sum = most;
    }
    return int(sum);
}

__device__ __forceinline__ bool is_free(int, int rc) { return rc == 0; }

// A length as pages, clamped to the table.
__device__ __forceinline__ int clamp_len(int len, int64_t limit, unsigned& bits) {
    if (len >= 0 && len <= limit) return len;
    bits |= 1u << SMLA_ERR_INDEX;
    return len < 0 ? 0 : int(limit);
}

// All bits of the CTA's threads.
__device__ __forceinline__ unsigned cta_bits(unsigned bits) {
    const bool index = __syncthreads_or(bits & (1u << SMLA_ERR_INDEX)) != 0;
    const bool count = __syncthreads_or(bits & (1u << SMLA_ERR_REFCOUNT)) != 0;
    return (index ? 1u << SMLA_ERR_INDEX : 0u) | (count ? 1u << SMLA_ERR_REFCOUNT : 0u);
}

// Free pages for the rows i < B, need_of[i] each (written by the cluster before this call), rows in order,
// pages in the order of their numbers: row i gets pages[first[i]] and on, whose refcounts become 1. All or
// nothing. Writes the status word with `bits` (of any thread; one with SMLA_ERR_REFCOUNT grants nothing) and
// SMLA_ERR_PAGES where there are too few; returns whether the pages were granted.
__device__ bool grant_pages(const CacheView& c, int B, const int32_t* need_of, int32_t* first, int32_t* pages,
                            unsigned bits, PlanShared& sh, int& turn, cg::cluster_group& cl, unsigned* status) {
    const int rank = int(cl.block_rank());
    int lo, hi;
    page_slice(c.num_pages, rank, lo, hi);
    const int mine = count_pages(c.refcount, lo, hi, sh, turn, is_free);
    bits = cta_bits(bits);
    if (threadIdx.x == 0) { sh.part = mine; sh.bits = bits; }
    cl.sync();
    int before, have;
    join(cl, sh, before, have, bits);
    // A sum of 1024 needs, each cut at 2^20, fits 32 bits; a row that needs more than
    // 2^20 pages is counted as 2^20 in the first pass only if that many are not there
    const int cap = have < (1 << 20) ? have + 1 : (1 << 20);
    int64_t big = 0;
    const int want = scan_needs(B, have + 1, sh, turn,
                                [&](int i) {
                                    const int v = __ldcg(need_of + i);
                                    if (v > cap) big = 1;
                                    return v < cap ? v : cap;
                                },
                                [&](int i, int, int at) { if (rank == 0) first[i] = at; });
    const bool huge = __syncthreads_or(int(big)) != 0 && have >= (1 << 20);
    // (rows of more than 2^20 pages, in a pool that has as many: summed one by one)
    int need = want;
    if (huge) {
        int64_t sum = 0;
        for (int i = 0; i < B; ++i) {
            if (rank == 0 && threadIdx.x == 0) first[i] = int(sum < have ? sum : have);
            sum += __ldcg(need_of + i);
        }
        need = int(sum < int64_t(have) + 1 ? sum : int64_t(have) + 1);
    }
    const bool enough = need <= have, ok = enough && !(bits & (1u << SMLA_ERR_REFCOUNT));
    if (ok)
        emit_pages(c.refcount, lo, hi, before, need, sh, turn, is_free, [&](int r, int i) {
            pages[r] = i;
            c.refcount[i] = 1;
        });
    if (rank == 0 && threadIdx.x == 0) *status = bits | (enough ? 0u : 1u << SMLA_ERR_PAGES);
    cl.sync();                                  // offsets and pages are written; parts are read
    return ok;
}

}  // namespace

}  // namespace smla
