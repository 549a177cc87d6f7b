// k_cache_pages.cu -- pages of the cache: allocating, forking, giving back,
// compacting and copying them.
//
// Each call plans with one kernel of a single cluster (8 CTAs of 1024 threads:
// its barrier and distributed shared memory join the parts of a scan over the
// refcounts without another launch) and then copies with one kernel on the
// whole GPU, which reads the plan's lists and their length on the device.
// Free pages are found in the order of their numbers, so the result of every
// call is fixed by its inputs. Integer atomics only.
//
// Bound: the copies by HBM (each moved byte read once and written once); the
// plan by latency.
#include <cooperative_groups.h>

#include "smla_internal.cuh"

namespace cg = cooperative_groups;

namespace smla {

namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                   // 16-byte pieces a thread has in flight
constexpr int kCopyChunk = kCopyThreads * kCopyVecs * 16;      // 16 KB

struct PlanShared {
    long long warp[kPlanWarps];
    long long part[4];          // this CTA's totals, read by the other CTAs
};

// Exclusive sum over the CTA's threads in thread order; *total gets the sum.
__device__ __forceinline__ long long cta_scan(long long v, PlanShared& sh, long long* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                                           // the last scan's sums are read
    if (lane == 31) sh.warp[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const long long t = sh.warp[w];
        if (w < warp) before += t;
        all += t;
    }
    *total = all;
    return before + x - v;
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
__device__ long long count_pages(const int32_t* rc, int lo, int hi, PlanShared& sh, Pred pred) {
    int n = 0;
    for (int i = lo + 4 * int(threadIdx.x); i < hi; i += 4 * kPlanThreads) {
        const int4 v = load4(rc, i, hi);
        n += int(pred(i, v.x)) + int(pred(i + 1, v.y)) + int(pred(i + 2, v.z)) + int(pred(i + 3, v.w));
    }
    long long total;
    cta_scan(n, sh, &total);
    return total;
}

// out(rank, i) for the pages i of [lo, hi) with pred(i, refcount), in order,
// ranks from `rank` on, until `limit`.
template <class Pred, class Out>
__device__ void emit_pages(const int32_t* rc, int lo, int hi, long long rank, long long limit,
                           PlanShared& sh, Pred pred, Out out) {
    for (int base = lo; base < hi && rank < limit; base += 4 * kPlanThreads) {
        const int i = base + 4 * int(threadIdx.x);
        const int4 v = load4(rc, i, hi);
        const bool p0 = pred(i, v.x), p1 = pred(i + 1, v.y), p2 = pred(i + 2, v.z), p3 = pred(i + 3, v.w);
        long long total;
        long long r = rank + cta_scan(int(p0) + int(p1) + int(p2) + int(p3), sh, &total);
        if (p0) { if (r < limit) out(r, i); ++r; }
        if (p1) { if (r < limit) out(r, i + 1); ++r; }
        if (p2) { if (r < limit) out(r, i + 2); ++r; }
        if (p3) { if (r < limit) out(r, i + 3); ++r; }
        rank += total;
    }
}

// Sum of part[k] over the CTAs, and over those before this one.
__device__ __forceinline__ void join(cg::cluster_group& cl, PlanShared& sh, int k, long long& before,
                                     long long& all) {
    before = 0;
    all = 0;
    for (unsigned r = 0; r < kPlanCtas; ++r) {
        const long long t = cl.map_shared_rank(&sh, r)->part[k];
        if (r < cl.block_rank()) before += t;
        all += t;
    }
}

// Exclusive sums of need[0..n) into off (written by CTA 0 only); returns the sum.
__device__ long long scan_needs(const int32_t* need, int n, int32_t* off, PlanShared& sh) {
    long long sum = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + int(threadIdx.x);
        long long total;
        const long long at = sum + cta_scan(i < n ? __ldcg(need + i) : 0, sh, &total);
        // offsets past 2^31 belong to a call that has too few pages: never used
        if (off && i < n) off[i] = int32_t(at < INT32_MAX ? at : INT32_MAX);
        sum += total;
    }
    return sum;
}

__device__ __forceinline__ bool is_free(int, int rc) { return rc == 0; }

// A length as pages, clamped to the table.
__device__ __forceinline__ int clamp_len(int len, int64_t limit, unsigned* status) {
    if (len >= 0 && len <= limit) return len;
    flag_status(status, SMLA_ERR_INDEX);
    return len < 0 ? 0 : int(limit);
}

// Copies 16 KB pieces of the pages in pairs (src[k], dst[k]), k < m, over the grid.
__device__ void copy_pairs(const CacheView& c, const int32_t* src, const int32_t* dst, int m,
                           unsigned* status) {
    const int64_t page_bytes = int64_t(kD) << c.page_shift;
    const int chunks = int((page_bytes + kCopyChunk - 1) / kCopyChunk);
    const int nscale = 1 << (c.page_shift - c.block_shift);
    for (int64_t w = blockIdx.x; w < int64_t(m) * chunks; w += gridDim.x) {
        const int k = int(w / chunks), ch = int(w % chunks);
        const int a = __ldg(src + k), b = __ldg(dst + k);
        if (a < 0 || a >= c.num_pages || b < 0 || b >= c.num_pages) {
            if (threadIdx.x == 0) flag_status(status, SMLA_ERR_INDEX);
            continue;
        }
        const uint4* from = reinterpret_cast<const uint4*>(c.pages + a * page_bytes) + ch * (kCopyChunk / 16);
        uint4* to = reinterpret_cast<uint4*>(c.pages + b * page_bytes) + ch * (kCopyChunk / 16);
        const int n = int((page_bytes - int64_t(ch) * kCopyChunk) / 16);
        uint4 v[kCopyVecs];
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i) {
            const int x = i * kCopyThreads + threadIdx.x;
            if (x < n) v[i] = __ldcs(from + x);
        }
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i) {
            const int x = i * kCopyThreads + threadIdx.x;
            if (x < n) __stcs(to + x, v[i]);
        }
        if (ch == 0 && threadIdx.x < nscale)
            c.scales[int64_t(b) * nscale + threadIdx.x] = c.scales[int64_t(a) * nscale + threadIdx.x];
    }
}

}  // namespace

// Every entry table[b, j] = -1 with j < ceil(lens[b] / page_size) gets a free page.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
alloc_kernel(const CacheView c, int32_t* __restrict__ table, const int32_t* __restrict__ lens, int B,
             int max_pages, const PageScratch w, unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = int(cl.block_rank()), lane = threadIdx.x & 31;
    const int gw = rank * kPlanWarps + (threadIdx.x >> 5);
    const int64_t limit = int64_t(max_pages) << c.page_shift;
    const int round = (1 << c.page_shift) - 1;
    for (int b = gw; b < B; b += kPlanCtas * kPlanWarps) {
        const int len = clamp_len(__ldg(lens + b), limit, status);
        const int np = int((int64_t(len) + round) >> c.page_shift);
        int n = 0;
        for (int j = lane; j < np; j += 32) n += table[int64_t(b) * max_pages + j] == -1;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) w.need[b] = n;
    }
    int lo, hi;
    page_slice(c.num_pages, rank, lo, hi);
    const long long mine = count_pages(c.refcount, lo, hi, sh, is_free);
    if (threadIdx.x == 0) sh.part[0] = mine;
    cl.sync();
    long long before, have;
    join(cl, sh, 0, before, have);
    const long long want = scan_needs(w.need, B, rank == 0 ? w.src : nullptr, sh);
    const bool ok = want <= have;
    if (ok)
        emit_pages(c.refcount, lo, hi, before, want, sh, is_free, [&](long long r, int i) {
            w.dst[r] = i;
            c.refcount[i] = 1;
        });
    else if (rank == 0 && threadIdx.x == 0)
        flag_status(status, SMLA_ERR_PAGES);
    cl.sync();                                  // offsets and pages are written; part[] is read
    if (!ok) return;
    for (int b = gw; b < B; b += kPlanCtas * kPlanWarps) {
        const int len = min(max(__ldg(lens + b), 0), int(limit));
        const int np = int((int64_t(len) + round) >> c.page_shift);
        int at = __ldcg(w.src + b);
        for (int j0 = 0; j0 < np; j0 += 32) {
            int32_t* e = table + int64_t(b) * max_pages + j0 + lane;
            const bool empty = j0 + lane < np && *e == -1;
            const unsigned m = __ballot_sync(0xffffffffu, empty);
            if (empty) *e = __ldcg(w.dst + at + __popc(m & ((1u << lane) - 1)));
            at += __popc(m);
        }
    }
}

// Plan of a fork: w.need[i] = 1 where child i needs a copy of its parent's
// last page, w.src / w.dst the pages to copy, w.map[i] the number of child i's
// copy, w.count[0] their number (-1: too few free pages), w.count[1] = 0.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
fork_plan_kernel(const CacheView c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                 const int32_t* __restrict__ parents, int B, int n, int max_pages, const PageScratch w,
                 unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = int(cl.block_rank());
    const int64_t limit = int64_t(max_pages) << c.page_shift;
    const int gt = rank * kPlanThreads + threadIdx.x;
    // the page that child i copies, or -1
    auto tail_of = [&](int i, unsigned* st) {
        const int p = __ldg(parents + i);
        if (p < 0 || p >= B) { if (st) flag_status(st, SMLA_ERR_INDEX); return -1; }
        int len = __ldg(lens + p);
        if (len < 0 || len > limit) {
            if (st) flag_status(st, SMLA_ERR_INDEX);
            len = len < 0 ? 0 : int(limit);
        }
        if ((len & ((1 << c.page_shift) - 1)) == 0) return -1;
        const int e = __ldg(table + int64_t(p) * max_pages + (len >> c.page_shift));
        if (e < 0 || e >= c.num_pages) { if (st) flag_status(st, SMLA_ERR_INDEX); return -1; }
        if (__ldcg(c.refcount + e) <= 0) { if (st) flag_status(st, SMLA_ERR_REFCOUNT); return -1; }
        return e;
    };
    for (int i = gt; i < n; i += kPlanCtas * kPlanThreads) w.need[i] = tail_of(i, status) >= 0 ? 1 : 0;
    int lo, hi;
    page_slice(c.num_pages, rank, lo, hi);
    const long long mine = count_pages(c.refcount, lo, hi, sh, is_free);
    if (threadIdx.x == 0) sh.part[0] = mine;
    cl.sync();
    long long before, have;
    join(cl, sh, 0, before, have);
    const long long want = scan_needs(w.need, n, nullptr, sh);
    const bool ok = want <= have;
    if (ok) emit_pages(c.refcount, lo, hi, before, want, sh, is_free,
                       [&](long long r, int i) { w.dst[r] = i; });
    if (ok && rank == 0) {
        long long sum = 0;
        for (int base = 0; base < n; base += kPlanThreads) {
            const int i = base + int(threadIdx.x);
            const int need = i < n ? __ldcg(w.need + i) : 0;
            long long total;
            const long long at = sum + cta_scan(need, sh, &total);
            if (need) w.src[at] = tail_of(i, nullptr);
            if (i < n) w.need[i] = need ? int(at) : -1;      // its place in the lists
            sum += total;
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        w.count[0] = ok ? int(want) : -1;
        w.count[1] = 0;
        if (!ok) flag_status(status, SMLA_ERR_PAGES);
    }
    cl.sync();                                  // no CTA leaves while another reads its part[]
}

// The children's table rows, the shared pages' counts and the copies.
__global__ void __launch_bounds__(kCopyThreads)
fork_kernel(const CacheView c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
            const int32_t* __restrict__ parents, int32_t* __restrict__ child, int B, int n, int max_pages,
            const PageScratch w, unsigned* status) {
    const int m = w.count[0];
    const int64_t limit = int64_t(max_pages) << c.page_shift;
    const int64_t threads = int64_t(gridDim.x) * kCopyThreads;
    for (int64_t x = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x; x < int64_t(n) * max_pages; x += threads) {
        const int i = int(x / max_pages), j = int(x - int64_t(i) * max_pages);
        const int p = __ldg(parents + i);
        int e = -1;
        if (m >= 0 && p >= 0 && p < B) {
            const int len = min(int64_t(max(__ldg(lens + p), 0)), limit);
            const int full = len >> c.page_shift;
            if (j < full) {
                e = __ldg(table + int64_t(p) * max_pages + j);
                if (e < 0 || e >= c.num_pages) {
                    flag_status(status, SMLA_ERR_INDEX);
                    e = -1;
                } else if (__ldcg(c.refcount + e) <= 0) {    // counts of owned pages only rise here
                    flag_status(status, SMLA_ERR_REFCOUNT);
                    e = -1;
                } else {
                    atomicAdd(c.refcount + e, 1);
                }
            } else if (j == full) {
                const int k = __ldg(w.need + i);
                if (k >= 0) e = __ldg(w.dst + k);
            }
        }
        child[x] = e;
    }
    if (m > 0) copy_pairs(c, w.src, w.dst, m, status);
    // the new pages are counted by the last CTA, when no other looks at counts any more
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(w.count + 1, 1) == int(gridDim.x) - 1;
    }
    __syncthreads();
    if (last)
        for (int k = threadIdx.x; k < m; k += kCopyThreads) c.refcount[__ldg(w.dst + k)] = 1;
}

__global__ void __launch_bounds__(256)
free_kernel(const CacheView c, int32_t* __restrict__ table, const int32_t* __restrict__ rows, int B, int n,
            int max_pages, unsigned* status) {
    const int64_t threads = int64_t(gridDim.x) * blockDim.x;
    for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < int64_t(n) * max_pages; x += threads) {
        const int i = int(x / max_pages), j = int(x - int64_t(i) * max_pages);
        const int b = rows ? __ldg(rows + i) : i;
        if (b < 0 || b >= B) { flag_status(status, SMLA_ERR_INDEX); continue; }
        int32_t* at = table + int64_t(b) * max_pages + j;
        if (__ldcg(at) == -1) continue;
        const int e = atomicExch(at, -1);                  // a row listed twice is given back once
        if (e == -1) continue;
        if (e < 0 || e >= c.num_pages) { flag_status(status, SMLA_ERR_INDEX); continue; }
        if (atomicSub(c.refcount + e, 1) <= 0) {
            atomicAdd(c.refcount + e, 1);
            flag_status(status, SMLA_ERR_REFCOUNT);
        }
    }
}

// Plan of a compaction: count[0] moves src[k] -> dst[k], count[1] live pages,
// map[src[k]] = dst[k].
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
compact_plan_kernel(const CacheView c, const PageScratch w) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = int(cl.block_rank());
    int lo, hi;
    page_slice(c.num_pages, rank, lo, hi);
    const long long mine = count_pages(c.refcount, lo, hi, sh, [](int, int rc) { return rc > 0; });
    if (threadIdx.x == 0) sh.part[0] = mine;
    cl.sync();
    long long before, live;
    join(cl, sh, 0, before, live);
    auto hole = [&](int i, int rc) { return rc == 0 && i < live; };
    auto high = [&](int i, int rc) { return rc > 0 && i >= live; };
    const long long holes = count_pages(c.refcount, lo, hi, sh, hole);
    const long long highs = count_pages(c.refcount, lo, hi, sh, high);
    if (threadIdx.x == 0) { sh.part[1] = holes; sh.part[2] = highs; }
    cl.sync();
    long long hole0, high0, m, m2;
    join(cl, sh, 1, hole0, m);
    join(cl, sh, 2, high0, m2);
    if (m2 < m) m = m2;       // equal, unless a count is negative
    emit_pages(c.refcount, lo, hi, hole0, m, sh, hole, [&](long long r, int i) { w.dst[r] = i; });
    emit_pages(c.refcount, lo, hi, high0, m, sh, high, [&](long long r, int i) { w.src[r] = i; });
    if (rank == 0 && threadIdx.x == 0) { w.count[0] = int(m); w.count[1] = int(live); }
    cl.sync();
    for (int k = rank * kPlanThreads + threadIdx.x; k < m; k += kPlanCtas * kPlanThreads)
        w.map[__ldcg(w.src + k)] = __ldcg(w.dst + k);
}

__global__ void __launch_bounds__(kCopyThreads)
compact_kernel(const CacheView c, const int32_t* __restrict__ table, int32_t* __restrict__ new_table,
               int32_t* __restrict__ new_refcount, int B, int max_pages, const PageScratch w,
               unsigned* status) {
    const int m = w.count[0], live = w.count[1];
    const int64_t first = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x;
    const int64_t threads = int64_t(gridDim.x) * kCopyThreads;
    for (int64_t x = first; x < int64_t(B) * max_pages; x += threads) {
        int e = __ldg(table + x);
        if (e != -1) {
            if (e < 0 || e >= c.num_pages) {
                flag_status(status, SMLA_ERR_INDEX);
                e = -1;
            } else if (__ldg(c.refcount + e) <= 0) {
                flag_status(status, SMLA_ERR_REFCOUNT);
                e = -1;
            } else if (e >= live) {
                e = __ldg(w.map + e);
            }
        }
        new_table[x] = e;
    }
    for (int64_t i = first; i < c.num_pages; i += threads) {
        const int rc = __ldg(c.refcount + i);
        if (i >= live) new_refcount[i] = 0;
        else if (rc != 0) new_refcount[i] = rc;             // a hole's count comes with its page, below
    }
    for (int64_t k = first; k < m; k += threads)
        new_refcount[__ldg(w.dst + k)] = __ldg(c.refcount + __ldg(w.src + k));
    copy_pairs(c, w.src, w.dst, m, status);
}

// count[0] = n if all dst differ from each other and from every src, else 0.
// map[] (zeroed) marks the dst pages.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
copy_check_kernel(const CacheView c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                  const PageScratch w, unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int first = int(cl.block_rank()) * kPlanThreads + threadIdx.x;
    bool twice = false;
    for (int k = first; k < n; k += kPlanCtas * kPlanThreads) {
        const int a = __ldg(src + k), b = __ldg(dst + k);
        if (a >= 0 && a < c.num_pages && b >= 0 && b < c.num_pages) twice |= atomicExch(w.map + b, 1) != 0;
    }
    cl.sync();
    for (int k = first; k < n; k += kPlanCtas * kPlanThreads) {
        const int a = __ldg(src + k), b = __ldg(dst + k);
        if (a >= 0 && a < c.num_pages && b >= 0 && b < c.num_pages) twice |= __ldcg(w.map + a) != 0;
    }
    twice = __syncthreads_or(twice) != 0;
    if (threadIdx.x == 0) sh.part[0] = twice;
    cl.sync();
    long long before, all;
    join(cl, sh, 0, before, all);
    if (cl.block_rank() == 0 && threadIdx.x == 0) {
        w.count[0] = all ? 0 : n;
        if (all) flag_status(status, SMLA_ERR_OVERLAP);
    }
    cl.sync();
}

__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const CacheView c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            const PageScratch w, unsigned* status) {
    copy_pairs(c, src, dst, w.count[0], status);
}

namespace {

// CTAs of the copying kernels: what the GPU holds at once (8 of 256 threads
// per SM), or fewer where the call cannot have more work.
int copy_grid(int64_t most) {
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t g = 8 * int64_t(sms);
    return int(most < 1 ? 1 : most < g ? most : g);
}

int64_t page_chunks(const CacheView& c) {
    return ((int64_t(kD) << c.page_shift) + kCopyChunk - 1) / kCopyChunk;
}

int64_t blocks_for(int64_t n, int threads) { return (n + threads - 1) / threads; }

}  // namespace

cudaError_t launch_cache_alloc(const CacheView& c, int32_t* table, const int32_t* lens, int B,
                               int max_pages, const PageScratch& w, unsigned* status, cudaStream_t s) {
    alloc_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, table, lens, B, max_pages, w, status);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheView& c, const int32_t* table, const int32_t* lens,
                              const int32_t* parents, int32_t* child_table, int B, int n,
                              int max_pages, const PageScratch& w, unsigned* status, cudaStream_t s) {
    fork_plan_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, table, lens, parents, B, n, max_pages, w, status);
    const int64_t most = n * page_chunks(c) + blocks_for(int64_t(n) * max_pages, kCopyThreads);
    fork_kernel<<<copy_grid(most), kCopyThreads, 0, s>>>(c, table, lens, parents, child_table, B, n, max_pages,
                                                         w, status);
    note_launch(2);
    return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheView& c, int32_t* table, const int32_t* rows, int B, int n,
                              int max_pages, unsigned* status, cudaStream_t s) {
    const int grid = copy_grid(blocks_for(int64_t(n) * max_pages, 256));
    free_kernel<<<grid, 256, 0, s>>>(c, table, rows, B, n, max_pages, status);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheView& c, const int32_t* table, int32_t* new_table,
                                 int32_t* new_refcount, int B, int max_pages, const PageScratch& w,
                                 unsigned* status, cudaStream_t s) {
    compact_plan_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, w);
    const int64_t most = c.num_pages / 2 * page_chunks(c) + 1;
    compact_kernel<<<copy_grid(most), kCopyThreads, 0, s>>>(c, table, new_table, new_refcount, B, max_pages, w,
                                                            status);
    note_launch(2);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy(const CacheView& c, const int32_t* src, const int32_t* dst, int n,
                              const PageScratch& w, unsigned* status, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(w.map, 0, size_t(c.num_pages) * 4, s);
    if (e != cudaSuccess) return e;
    copy_check_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, src, dst, n, w, status);
    copy_kernel<<<copy_grid(n * page_chunks(c)), kCopyThreads, 0, s>>>(c, src, dst, w, status);
    note_launch(2);
    return cudaGetLastError();
}

}  // namespace smla
