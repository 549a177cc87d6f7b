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
// plan by latency (a cluster's launch, two passes over its share of the counts and
// two cluster barriers: 5 to 9 us). Compaction of 40000 pages of 32 KB, 9900 of them live and
// 7400 of these moved: 83 us, of which the copies take 69; 5.9 TB/s over all. Fork of 1024 children, each with
// a page to copy, after a free of as many: 26 us; of 32: 13 us. Reordering of 1024 beams (their weights too) in that
// pool: 17 us with a copy of the counts before it (plan 4.5, moves 8.5), where fork and free copy every beam's last
// page; of 32: 10.
#include "page_plan.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr int kFreeEach = 4;                                   // entries of a thread of a small free
constexpr int kFreeFew = kPlanCtas * kPlanThreads * kFreeEach;
constexpr int kCopyThreads = 256;
constexpr int kEntryThreads = kCopyThreads - 32;               // all but the copying warp
constexpr int kCopySlots = 6, kCopyLag = 3;
constexpr int kCopyBytes = 32768;                              // of a slot
constexpr int kCopySmem = kCopySlots * kCopyBytes;
constexpr uint64_t kCopyWaitNs = 2000000000u;
constexpr int kReorderThreads = 1024;
constexpr int kReorderRows = 4096;                             // rows of a plan in shared memory
constexpr int kReorderFresh = 1 << 30;                         // (a call has at most 2^24 copies)

struct CopyShared {
    uint64_t full[kCopySlots];
    int to[kCopySlots][kCopyBytes / (16 * kD)];
};

// Copies the pages in pairs (src(k), dst(k)), k < m, over the grid: warp 0 moves the rows, 32 KB of a
// page or several small pages at a time, by bulk copies through a ring of six slots in shared
// memory (three loads and three stores in flight: no register holds a byte, and one CTA an SM
// keeps HBM busy), the other warps the scales.
template <class Src, class Dst>
__device__ void copy_pairs(const CacheView& c, uint8_t* ring, CopyShared& sh, Src src, Dst dst, int m,
                           unsigned* status) {
    const int nscale = 1 << (c.page_shift - c.block_shift);
    if (threadIdx.x >= 32) {
        const int64_t each = blockDim.x - 32, threads = int64_t(gridDim.x) * each;
        for (int64_t x = int64_t(blockIdx.x) * each + threadIdx.x - 32; x < int64_t(m) * nscale; x += threads) {
            const int k = int(x / nscale), i = int(x - int64_t(k) * nscale), a = src(k), b = dst(k);
            if (a >= 0 && a < c.num_pages && b >= 0 && b < c.num_pages)
                c.scales[int64_t(b) * nscale + i] = c.scales[int64_t(a) * nscale + i];
        }
        return;
    }
    const int lane = threadIdx.x;
    const int64_t page_bytes = int64_t(kD) << c.page_shift;
    const int piece = int(page_bytes < kCopyBytes ? page_bytes : kCopyBytes);
    const int per = kCopyBytes / piece;                        // pages of a slot: a lane each
    const int parts = int(page_bytes / piece);                 // slots of a page, a power of two
    const int shift = __ffs(parts) - 1;
    const int64_t units = per > 1 ? (int64_t(m) + per - 1) / per : int64_t(m) * parts;
    const int mine = units > blockIdx.x ? int((units - blockIdx.x - 1) / gridDim.x) + 1 : 0;
    if (lane == 0) {
        for (int i = 0; i < kCopySlots; ++i) mbar_init(&sh.full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    int a1, b1;                                  // the lane's pair in the next unit, read ahead
    auto look = [&](int i) {
        const int64_t u = blockIdx.x + int64_t(i) * gridDim.x, k = per > 1 ? u * per + lane : u >> shift;
        a1 = b1 = -1;
        if (i >= mine || lane >= per || k >= m) return;
        a1 = src(int(k));
        b1 = dst(int(k));
        if (a1 < 0 || a1 >= c.num_pages || b1 < 0 || b1 >= c.num_pages) {
            flag_status(status, SMLA_ERR_INDEX);
            a1 = b1 = -1;
        }
    };
    auto at = [&](int page, int i) {
        return c.pages + page * page_bytes + ((blockIdx.x + int64_t(i) * gridDim.x) & (parts - 1)) * kCopyBytes;
    };
    look(0);
#pragma unroll 1
    for (int i = 0; i < mine + kCopyLag; ++i) {
        if (i < mine) {
            const int slot = i % kCopySlots, a = a1;
            // the slot's store (each lane's own, six units before) has read it
            if (i >= kCopySlots) bulk_wait_read<kCopySlots - kCopyLag - 1>();
            const int lanes = __popc(__ballot_sync(0xffffffffu, a >= 0));
            if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], uint32_t(lanes) * piece);
            __syncwarp();
            if (a >= 0) bulk_load(ring + slot * kCopyBytes + lane * piece, at(a, i), piece, &sh.full[slot]);
            if (lane < per) sh.to[slot][lane] = b1;
            look(i + 1);
        }
        if (i >= kCopyLag) {
            const int j = i - kCopyLag, slot = j % kCopySlots;
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[slot], uint32_t(j / kCopySlots) & 1u, kCopyWaitNs))) {
                flag_status(status, SMLA_ERR_TIMEOUT);
                for (int k = j; k <= i && k < mine; ++k)       // loads already issued land before the CTA exits
                    mbar_wait(&sh.full[k % kCopySlots], uint32_t(k / kCopySlots) & 1u, kCopyWaitNs / 8);
                break;
            }
            const int b = lane < per ? sh.to[slot][lane] : -1;
            if (b >= 0) bulk_store(at(b, j), ring + slot * kCopyBytes + lane * piece, piece);
            bulk_commit();
        }
    }
    bulk_wait_all();
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
    unsigned bits = 0;
    int turn = 0;
    for (int b = gw; b < B; b += kPlanCtas * kPlanWarps) {
        const int len = clamp_len(__ldg(lens + b), limit, bits);
        const int np = int((int64_t(len) + round) >> c.page_shift);
        int n = 0;
        for (int j = lane; j < np; j += 32) n += table[int64_t(b) * max_pages + j] == -1;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) w.need[b] = n;
    }
    const bool ok = grant_pages(c, B, w.need, w.src, w.dst, bits, sh, turn, cl, status);
    if (!ok) return;
    for (int b = gw; b < B; b += kPlanCtas * kPlanWarps) {
        const int len = int(min(int64_t(max(__ldg(lens + b), 0)), limit));
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

// Plan of a fork: w.src / w.dst the pages to copy, w.need[i] the place of child i's
// copy in them (-1: none), w.count[0] their number (-1: too few free pages), w.count[1] = 0.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
fork_plan_kernel(const CacheView c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                 const int32_t* __restrict__ parents, int B, int n, int max_pages, const PageScratch w,
                 unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    grid_dep_launch();                          // the copying kernel's blocks wait for this one's end
    const int rank = int(cl.block_rank());
    const int64_t limit = int64_t(max_pages) << c.page_shift;
    unsigned bits = 0;
    int turn = 0;
    // w.tail[i]: the page that child i copies, or -1
    for (int i = rank * kPlanThreads + threadIdx.x; i < n; i += kPlanCtas * kPlanThreads) {
        int e = -1;
        const int p = __ldg(parents + i);
        if (p < 0 || p >= B) {
            bits |= 1u << SMLA_ERR_INDEX;
        } else {
            const int len = clamp_len(__ldg(lens + p), limit, bits);
            if (len & ((1 << c.page_shift) - 1)) {
                e = __ldg(table + int64_t(p) * max_pages + (len >> c.page_shift));
                if (e < 0 || e >= c.num_pages) {
                    bits |= 1u << SMLA_ERR_INDEX;
                    e = -1;
                } else if (__ldcg(c.refcount + e) <= 0) {
                    bits |= 1u << SMLA_ERR_REFCOUNT;
                    e = -1;
                }
            }
        }
        w.tail[i] = e;
    }
    int lo, hi;
    page_slice(c.num_pages, rank, lo, hi);
    const int mine = count_pages(c.refcount, lo, hi, sh, turn, is_free);
    const bool index = __syncthreads_or(bits & (1u << SMLA_ERR_INDEX)) != 0;
    const bool count = __syncthreads_or(bits & (1u << SMLA_ERR_REFCOUNT)) != 0;
    if (threadIdx.x == 0) {
        sh.part = mine;
        sh.bits = (index ? 1u << SMLA_ERR_INDEX : 0u) | (count ? 1u << SMLA_ERR_REFCOUNT : 0u);
    }
    cl.sync();
    int before, have;
    join(cl, sh, before, have, bits);
    const int want = scan_needs(n, INT32_MAX, sh, turn,
                                [&](int i) { return __ldcg(w.tail + i) >= 0 ? 1 : 0; },
                                [&](int i, int need, int at) {
                                    if (rank != 0) return;
                                    w.need[i] = need ? at : -1;
                                    if (need) w.src[at] = __ldcg(w.tail + i);
                                });
    const bool ok = want <= have;
    if (ok) emit_pages(c.refcount, lo, hi, before, want, sh, turn, is_free, [&](int r, int i) { w.dst[r] = i; });
    if (rank == 0 && threadIdx.x == 0) {
        w.count[0] = ok ? want : -1;
        w.count[1] = 0;
        *status = bits | (ok ? 0u : 1u << SMLA_ERR_PAGES);
    }
    cl.sync();                                  // no CTA leaves while another reads its part
}

// The children's table rows, the shared pages' counts and the copies.
__global__ void __launch_bounds__(kCopyThreads)
fork_kernel(const CacheView c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
            const int32_t* __restrict__ parents, int32_t* __restrict__ child, int B, int n, int max_pages,
            const PageScratch w, unsigned* status) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ CopyShared sh;
    grid_dep_wait();
    const int m = __ldcg(w.count);
    const int64_t limit = int64_t(max_pages) << c.page_shift;
    const int64_t threads = int64_t(gridDim.x) * kEntryThreads;
    const int64_t first = int64_t(blockIdx.x) * kEntryThreads + threadIdx.x - 32;
    for (int64_t x = threadIdx.x < 32 ? int64_t(n) * max_pages : first; x < int64_t(n) * max_pages; x += threads) {
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
                const int k = __ldcg(w.need + i);
                if (k >= 0) e = __ldcg(w.dst + k);
            }
        }
        child[x] = e;
    }
    if (m > 0)
        copy_pairs(c, ring, sh, [&](int k) { return __ldcg(w.src + k); }, [&](int k) { return __ldcg(w.dst + k); }, m,
                   status);
    // the new pages are counted by the last CTA, when no other looks at counts any more
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(w.count + 1, 1) == int(gridDim.x) - 1;
    }
    __syncthreads();
    if (last)
        for (int k = threadIdx.x; k < m; k += kCopyThreads) c.refcount[__ldcg(w.dst + k)] = 1;
}

// Gives back an entry taken out of the table (-1: none).
__device__ __forceinline__ void give_back(const CacheView& c, int e, unsigned& bits) {
    if (e == -1) return;
    if (e < 0 || e >= c.num_pages) { bits |= 1u << SMLA_ERR_INDEX; return; }
    if (atomicSub(c.refcount + e, 1) <= 0) {
        atomicAdd(c.refcount + e, 1);
        bits |= 1u << SMLA_ERR_REFCOUNT;
    }
}

// At most kFreeFew entries: one cluster, which joins its status bits and writes the word itself,
// so that the call is one launch. A thread's entries are on their way together.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
free_few_kernel(const CacheView c, int32_t* __restrict__ table, const int32_t* __restrict__ rows, int B, int total,
                int max_pages, unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int first = int(cl.block_rank()) * kPlanThreads + threadIdx.x;
    unsigned bits = 0;
    int32_t* at[kFreeEach];
    int e[kFreeEach];
#pragma unroll
    for (int k = 0; k < kFreeEach; ++k) {
        const int x = first + k * kPlanCtas * kPlanThreads, i = x / max_pages;
        e[k] = -1;
        if (x >= total) continue;
        const int b = rows ? __ldg(rows + i) : i;
        if (b < 0 || b >= B) { bits |= 1u << SMLA_ERR_INDEX; continue; }
        at[k] = table + int64_t(b) * max_pages + (x - i * max_pages);
        e[k] = __ldcg(at[k]);
    }
#pragma unroll
    for (int k = 0; k < kFreeEach; ++k)
        if (e[k] != -1) e[k] = atomicExch(at[k], -1);      // a row listed twice is given back once
#pragma unroll
    for (int k = 0; k < kFreeEach; ++k) give_back(c, e[k], bits);
    const bool index = __syncthreads_or(bits & (1u << SMLA_ERR_INDEX)) != 0;
    const bool count = __syncthreads_or(bits & (1u << SMLA_ERR_REFCOUNT)) != 0;
    if (threadIdx.x == 0) {
        sh.part = 0;
        sh.bits = (index ? 1u << SMLA_ERR_INDEX : 0u) | (count ? 1u << SMLA_ERR_REFCOUNT : 0u);
    }
    cl.sync();
    if (cl.block_rank() == 0 && threadIdx.x == 0) {
        int before, all;
        join(cl, sh, before, all, bits);
        *status = bits;
    }
    cl.sync();                                  // no CTA leaves while another reads its part
}

__global__ void __launch_bounds__(256)
free_kernel(const CacheView c, int32_t* __restrict__ table, const int32_t* __restrict__ rows, int B, int n,
            int max_pages, unsigned* status) {
    const int64_t threads = int64_t(gridDim.x) * blockDim.x;
    unsigned bits = 0;
    for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < int64_t(n) * max_pages; x += threads) {
        const int i = int(x / max_pages), j = int(x - int64_t(i) * max_pages);
        const int b = rows ? __ldg(rows + i) : i;
        if (b < 0 || b >= B) { bits |= 1u << SMLA_ERR_INDEX; continue; }
        int32_t* at = table + int64_t(b) * max_pages + j;
        if (__ldcg(at) == -1) continue;
        give_back(c, atomicExch(at, -1), bits);
    }
    if (bits) atomicOr(status, bits);
}

// Plan of a compaction, with `live` pages in use: the holes (free pages below live) in order in
// w.dst, the pages to move (live ones from `live` on) in reverse order in w.src, the
// place of each in that list in w.map; count[0] their number, count[1] = live. The
// reverse order needs no sum that only the CTA with page `live` in its share could give.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
compact_plan_kernel(const CacheView c, const PageScratch w, unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    grid_dep_launch();                          // the moving kernel's blocks wait for this one's end
    const int rank = int(cl.block_rank());
    int lo, hi, turn = 0;
    page_slice(c.num_pages, rank, lo, hi);
    const int mine = count_pages(c.refcount, lo, hi, sh, turn, [](int, int rc) { return rc > 0; });
    if (threadIdx.x == 0) { sh.part = mine; sh.bits = 0; }
    cl.sync();
    int before, live;
    unsigned bits;
    join(cl, sh, before, live, bits);
    // before this share: all pages are below `live` or this share has no hole
    const int holes_before = (lo < live ? lo : live) - before;
    if (lo < live)
        emit_pages(c.refcount, lo, hi, holes_before, live, sh, turn,
                   [&](int i, int rc) { return rc <= 0 && i < live && i < hi; },
                   [&](int r, int i) { w.dst[r] = i; });
    if (hi > live) {
        // ranks from the front within the share, counted down from the pages behind it
        const int behind = live - before - mine;
        const int below = lo < live ? count_pages(c.refcount, lo, live, sh, turn, [](int, int rc) { return rc > 0; }) : 0;
        const int here = mine - below;
        emit_pages(c.refcount, lo, hi, 0, here, sh, turn, [&](int i, int rc) { return rc > 0 && i >= live; },
                   [&](int r, int i) {
                       const int k = behind + here - 1 - r;
                       w.src[k] = i;
                       w.map[i] = k;
                   });
        if (lo <= live && threadIdx.x == 0) w.count[0] = behind + here;      // all that move
    }
    if (rank == 0 && threadIdx.x == 0) {
        w.count[1] = live;
        *status = 0;
        if (live == c.num_pages) w.count[0] = 0;
    }
    cl.sync();                                  // no CTA leaves while another reads its part
}

__global__ void __launch_bounds__(kCopyThreads)
compact_kernel(const CacheView c, const int32_t* __restrict__ table, int32_t* __restrict__ new_table,
               int32_t* __restrict__ new_refcount, int B, int max_pages, const PageScratch w,
               unsigned* status) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ CopyShared sh;
    grid_dep_wait();
    const int m = __ldcg(w.count), live = __ldcg(w.count + 1);
    // the k-th page that moves goes to the k-th hole; the list is in reverse order
    auto src = [&](int k) { return __ldcg(w.src + (m - 1 - k)); };
    auto dst = [&](int k) { return __ldcg(w.dst + k); };
    const int64_t threads = int64_t(gridDim.x) * kEntryThreads;
    const int64_t first = threadIdx.x < 32 ? INT64_MAX - threads      // (the copying warp has no entries)
                                           : int64_t(blockIdx.x) * kEntryThreads + threadIdx.x - 32;
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
                e = dst(m - 1 - __ldcg(w.map + e));
            }
        }
        new_table[x] = e;
    }
    for (int64_t i = first; i < c.num_pages; i += threads) {
        const int rc = __ldg(c.refcount + i);
        if (i >= live) new_refcount[i] = 0;
        else if (rc > 0) new_refcount[i] = rc;              // a hole's count comes with its page, below
    }
    for (int64_t k = first; k < m; k += threads) new_refcount[dst(int(k))] = __ldg(c.refcount + src(int(k)));
    copy_pairs(c, ring, sh, src, dst, m, status);
}

// count[0] = n if all dst differ from each other and from every src, else 0.
// map[] (zeroed) marks the dst pages.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
copy_check_kernel(const CacheView c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                  const PageScratch w, unsigned* status) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    grid_dep_launch();
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
    if (threadIdx.x == 0) { sh.part = twice; sh.bits = 0; }
    cl.sync();
    int before, all;
    unsigned bits;
    join(cl, sh, before, all, bits);
    if (cl.block_rank() == 0 && threadIdx.x == 0) {
        w.count[0] = all ? 0 : n;
        *status = all ? 1u << SMLA_ERR_OVERLAP : 0u;
    }
    cl.sync();
}

__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const CacheView c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            const PageScratch w, unsigned* status) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ CopyShared sh;
    grid_dep_wait();
    copy_pairs(c, ring, sh, [&](int k) { return __ldg(src + k); }, [&](int k) { return __ldg(dst + k); },
               __ldcg(w.count), status);
}

// Plan of a reordering: heir[p] the first child of row p (INT32_MAX: none; -2: none, and its last page
// goes to a copy), a.src / a.dst the pages to copy, need[i] the place of child i's copy in them (-1: none),
// count[0] their number (-1: too few pages; with kReorderFresh if some go to free pages), count[2] the first of those.
//
// What child i copies (-1: nothing), given its parent and whether it is the first.
__device__ __forceinline__ int tail_to_copy(const ReorderArgs& a, int p, bool first, unsigned& bits) {
    const CacheView& c = a.cache;
    const int len = clamp_len(__ldg(a.lens + p), int64_t(a.max_pages) << c.page_shift, bits);
    if (first || (len & ((1 << c.page_shift) - 1)) == 0) return -1;
    const int e = __ldg(a.table + int64_t(p) * a.max_pages + (len >> c.page_shift));
    if (e < 0 || e >= c.num_pages) { bits |= 1u << SMLA_ERR_INDEX; return -1; }
    if (__ldcg(c.refcount + e) <= 0) { bits |= 1u << SMLA_ERR_REFCOUNT; return -1; }
    return e;
}
// The last page of a row that ends, if it is partly filled and the row's alone (else -1).
__device__ __forceinline__ int tail_to_hand_on(const ReorderArgs& a, int p, unsigned& bits) {
    const CacheView& c = a.cache;
    const int len = clamp_len(__ldg(a.lens + p), int64_t(a.max_pages) << c.page_shift, bits);
    if ((len & ((1 << c.page_shift) - 1)) == 0) return -1;
    const int e = __ldg(a.table + int64_t(p) * a.max_pages + (len >> c.page_shift));
    return e >= 0 && e < c.num_pages && __ldcg(c.refcount + e) == 1 ? e : -1;
}
// Free pages for the copies from number `used` on; true if there are enough.
__device__ __forceinline__ bool pages_for_copies(const ReorderArgs& a, int used, int want, PlanShared& sh, int& turn,
                                                 cg::cluster_group& cl, unsigned& bits) {
    const CacheView& c = a.cache;
    int lo, hi;
    page_slice(c.num_pages, int(cl.block_rank()), lo, hi);
    const int mine = count_pages(c.refcount, lo, hi, sh, turn, is_free);
    if (threadIdx.x == 0) { sh.part = mine; sh.bits = bits; }
    cl.sync();
    int before, have;
    join(cl, sh, before, have, bits);
    const bool ok = want - used <= have;
    if (ok)
        emit_pages(c.refcount, lo, hi, used + before, want, sh, turn, is_free, [&](int r, int i) { a.dst[r] = i; });
    cl.sync();                                   // no CTA leaves while another reads its part
    return ok;
}

// Up to kReorderRows rows: every CTA finds children and last pages for itself, in shared memory, and only where the
// rows that end have too few last pages do they share out the search for free ones.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
reorder_plan_few_kernel(const ReorderArgs a) {
    __shared__ PlanShared sh;
    __shared__ int heir[kReorderRows], spare[kReorderRows];
    cg::cluster_group cl = cg::this_cluster();
    grid_dep_launch();                          // the moving kernel's blocks wait for this one's end
    const bool lead = cl.block_rank() == 0;
    unsigned bits = 0;
    int turn = 0;
    for (int p = threadIdx.x; p < a.B; p += kPlanThreads) heir[p] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const int p = __ldg(a.parents + i);
        if (p >= 0 && p < a.B) atomicMin(heir + p, i);
        else if (p != -1) bits |= 1u << SMLA_ERR_INDEX;
    }
    __syncthreads();
    int want = 0, spares = 0;
    for (int base = 0; base < a.n || base < a.B; base += kPlanThreads) {
        const int i = base + int(threadIdx.x);
        const int p = i < a.n ? __ldg(a.parents + i) : -1;
        int from = -1, to = -1;
        if (p >= 0 && p < a.B) from = tail_to_copy(a, p, heir[p] == i, bits);
        if (i < a.B && heir[i] == INT32_MAX) to = tail_to_hand_on(a, i, bits);
        int total;
        const int before = cta_scan(int(from >= 0) | int(to >= 0) << 16, sh, turn, &total);
        const int at = want + (before & 0xffff), place = spares + (before >> 16);
        if (i < a.B) spare[i] = to >= 0 ? place : -1;
        if (lead) {
            if (i < a.n) a.need[i] = from >= 0 ? at : -1;
            if (from >= 0) a.src[at] = from;
            if (to >= 0 && place < a.n) a.dst[place] = to;
        }
        want += total & 0xffff;
        spares += total >> 16;
    }
    bits = cta_bits(bits);
    const bool ok = want <= spares || pages_for_copies(a, spares, want, sh, turn, cl, bits);
    if (!lead) return;
    for (int p = threadIdx.x; p < a.B; p += kPlanThreads) a.heir[p] = spare[p] >= 0 && spare[p] < want ? -2 : heir[p];
    if (threadIdx.x == 0) {
        a.count[0] = !ok ? -1 : want | (want > spares ? kReorderFresh : 0);
        a.count[1] = 0;
        a.count[2] = spares;
        *a.status = bits | (ok ? 0u : 1u << SMLA_ERR_PAGES);
    }
}

// More rows: the cluster shares them out, through the workspace.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
reorder_plan_kernel(const ReorderArgs a) {
    __shared__ PlanShared sh;
    cg::cluster_group cl = cg::this_cluster();
    grid_dep_launch();
    const int rank = int(cl.block_rank()), first = rank * kPlanThreads + int(threadIdx.x);
    constexpr int kStep = kPlanCtas * kPlanThreads;
    unsigned bits = 0;
    int turn = 0;
    for (int p = first; p < a.B; p += kStep) __stcg(a.heir + p, INT32_MAX);
    cl.sync();
    for (int i = first; i < a.n; i += kStep) {
        const int p = __ldg(a.parents + i);
        if (p >= 0 && p < a.B) atomicMin(a.heir + p, i);
        else if (p != -1) bits |= 1u << SMLA_ERR_INDEX;
    }
    cl.sync();
    for (int i = first; i < a.n; i += kStep) {
        const int p = __ldg(a.parents + i);
        __stcg(a.tail + i, p >= 0 && p < a.B ? tail_to_copy(a, p, __ldcg(a.heir + p) == i, bits) : -1);
    }
    for (int p = first; p < a.B; p += kStep)
        __stcg(a.spare + p, __ldcg(a.heir + p) == INT32_MAX ? tail_to_hand_on(a, p, bits) : -1);
    bits = cta_bits(bits);
    cl.sync();
    const int want = scan_needs(a.n, INT32_MAX, sh, turn,
                                [&](int i) { return __ldcg(a.tail + i) >= 0 ? 1 : 0; },
                                [&](int i, int need, int at) {
                                    if (rank != 0) return;
                                    a.need[i] = need ? at : -1;
                                    if (need) a.src[at] = __ldcg(a.tail + i);
                                });
    const int spares = scan_needs(a.B, INT32_MAX, sh, turn,
                                  [&](int p) { return __ldcg(a.spare + p) >= 0 ? 1 : 0; },
                                  [&](int p, int need, int at) {
                                      if (rank != 0 || !need || at >= want) return;
                                      a.dst[at] = __ldcg(a.spare + p);
                                      a.heir[p] = -2;
                                  });
    // (the CTAs join their bits there)
    const bool ok = pages_for_copies(a, spares < want ? spares : want, want, sh, turn, cl, bits);
    if (rank == 0 && threadIdx.x == 0) {
        a.count[0] = !ok ? -1 : want | (want > spares ? kReorderFresh : 0);
        a.count[1] = 0;
        a.count[2] = spares;
        *a.status = bits | (ok ? 0u : 1u << SMLA_ERR_PAGES);
    }
}

// The new table, lengths and weights, the counts and the copies. Warp 0 copies pages; of the others seven see to tables
// and counts and the rest move weights (all see to tables if there are none), a row's 4 KB at a time.
__global__ void __launch_bounds__(kReorderThreads)
reorder_kernel(const ReorderArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ CopyShared sh;
    grid_dep_wait();
    const CacheView& c = a.cache;
    const int plan = __ldcg(a.count), m = plan < 0 ? -1 : plan & (kReorderFresh - 1), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t limit = int64_t(a.max_pages) << c.page_shift;
    auto len_of = [&](int p) {
        const int len = __ldg(a.lens + p);
        return len < 0 ? 0 : len > limit ? int(limit) : len;
    };
    const int table_warps = a.new_weights ? 7 : kReorderThreads / 32 - 1;
    if (warp > 0 && warp <= table_warps) {
        unsigned bits = 0;
        const int64_t step = int64_t(gridDim.x) * table_warps * 32;
        const int64_t first = (int64_t(blockIdx.x) * table_warps + warp - 1) * 32 + lane;
        for (int64_t x = first; x < int64_t(a.n) * a.max_pages; x += step) {
            const int i = int(x / a.max_pages), j = int(x - int64_t(i) * a.max_pages);
            const int p = __ldg(a.parents + i);
            int e = -1;
            if (m >= 0 && p >= 0 && p < a.B) {
                const int full = len_of(p) >> c.page_shift, heir = __ldcg(a.heir + p);
                const int old = __ldg(a.table + int64_t(p) * a.max_pages + j);
                if (heir == i) {
                    e = old;
                } else if (j < full) {
                    e = old;
                    if (e < 0 || e >= c.num_pages) {
                        bits |= 1u << SMLA_ERR_INDEX;
                        e = -1;
                    } else if (__ldcg(c.refcount + e) <= 0) {            // (no count rises from 0 before the last CTA)
                        bits |= 1u << SMLA_ERR_REFCOUNT;
                        e = -1;
                    } else {
                        atomicAdd(c.refcount + e, 1);
                    }
                } else if (j == full) {
                    const int k = __ldcg(a.need + i);
                    if (k >= 0) e = __ldcg(a.dst + k);
                }
            }
            a.new_table[x] = e;
            if (j == 0) a.new_lens[i] = m >= 0 && p >= 0 && p < a.B ? len_of(p) : 0;
        }
        if (m >= 0)
            for (int64_t x = first; x < int64_t(a.B) * a.max_pages; x += step) {
                const int p = int(x / a.max_pages), j = int(x - int64_t(p) * a.max_pages);
                const int heir = __ldcg(a.heir + p), e = __ldg(a.table + x);
                if (heir >= 0 && heir != INT32_MAX) continue;
                if (heir == -2 && j == len_of(p) >> c.page_shift) continue;
                give_back(c, e, bits);
            }
        if (bits) atomicOr(a.status, bits);
    } else if (warp > table_warps) {
        constexpr int kQuads = 256;              // of a piece: 8 a lane, on their way together
        const int64_t quads = limit / 4, pieces = (quads + kQuads - 1) / kQuads;
        const int warps = kReorderThreads / 32 - 1 - table_warps;
        for (int64_t u = int64_t(blockIdx.x) * warps + warp - 1 - table_warps; u < a.n * pieces; u += int64_t(gridDim.x) * warps) {
            const int i = int(u / pieces);
            const int64_t at = (u - i * pieces) * kQuads + lane;
            const int p = __ldg(a.parents + i);
            const int len = m >= 0 && p >= 0 && p < a.B ? len_of(p) : 0;
            const float4* src = reinterpret_cast<const float4*>(a.weights) + p * quads;
            float4* dst = reinterpret_cast<float4*>(a.new_weights) + i * quads;
            float4 v[kQuads / 32];
#pragma unroll
            for (int k = 0; k < kQuads / 32; ++k) {
                const int64_t q = at + 32 * k, left = len - 4 * q;
                v[k] = left > 0 ? __ldg(src + q) : make_float4(0.f, 0.f, 0.f, 0.f);
                if (left < 2) v[k].y = 0.f;
                if (left < 3) v[k].z = 0.f;
                if (left < 4) v[k].w = 0.f;
            }
#pragma unroll
            for (int k = 0; k < kQuads / 32; ++k)
                if (at + 32 * k < quads) dst[at + 32 * k] = v[k];
        }
    }
    if (m > 0)
        copy_pairs(c, ring, sh, [&](int k) { return __ldcg(a.src + k); }, [&](int k) { return __ldcg(a.dst + k); }, m,
                   a.status);
    // Free pages that copies took are counted by the last CTA, when no other looks at counts any more: the table may have
    // an entry of such a page, which is neither shared nor given back. (A page of a row that ended has its count. Doing
    // this without free pages too: 0.7 us more a call; one atomic in place of a look and one for each shared page, which
    // let one child take a page that the next had found free: 0.6 us less of 10.)
    if (plan < kReorderFresh) return;
    const int fresh = __ldcg(a.count + 2);
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.count + 1, 1) == int(gridDim.x) - 1;
    }
    __syncthreads();
    if (last)
#pragma unroll 4
        for (int k = fresh + int(threadIdx.x); k < m; k += kReorderThreads) {
            const int e = __ldcg(a.dst + k);
            if (e >= 0 && e < c.num_pages) c.refcount[e] = 1;
        }
}

namespace {

int sm_count() {
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// CTAs of a copying kernel: one an SM (its ring takes the shared memory), or fewer where the call
// cannot have more work.
int copy_grid(const CacheView& c, int64_t pages, int64_t entries) {
    const int64_t bytes = pages * (int64_t(kD) << c.page_shift);
    const int64_t a = (bytes + kCopyBytes - 1) / kCopyBytes, b = (entries + kEntryThreads - 1) / kEntryThreads;
    const int64_t most = a > b ? a : b, g = sm_count();
    return int(most < 1 ? 1 : most < g ? most : g);
}

int64_t blocks_for(int64_t n, int threads) { return (n + threads - 1) / threads; }

// Launches a kernel whose blocks may start before the one ahead of it on the stream is
// complete (they wait for that themselves).
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), bool (&attr_done)[64], int grid, int threads, cudaStream_t s,
                         Args... args) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopySmem);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = kCopySmem;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    note_launch();
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

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
    static bool attr_done[64] = {false};
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_early(fork_kernel, attr_done, copy_grid(c, n, int64_t(n) * max_pages), kCopyThreads, s, c, table, lens, parents,
                        child_table, B, n, max_pages, w, status);
}

cudaError_t launch_cache_reorder(const ReorderArgs& a, cudaStream_t s) {
    // Both sides, device time of a call and a copy before it: 1024 rows 16.8 us planned in shared memory, 21.8 through
    // the workspace; 32 rows 9.9 and 14.0.
    if (a.B <= kReorderRows && a.n <= 4 * kReorderRows) reorder_plan_few_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(a);
    else reorder_plan_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    static bool attr_done[64] = {false};
    int64_t entries = int64_t(a.n > a.B ? a.n : a.B) * a.max_pages;
    if (a.new_weights) entries = entries > 1 ? entries << (a.cache.page_shift - 2) : entries;
    return launch_early(reorder_kernel, attr_done, copy_grid(a.cache, a.n, entries), kReorderThreads, s, a);
}

cudaError_t launch_cache_free(const CacheView& c, int32_t* table, const int32_t* rows, int B, int n,
                              int max_pages, unsigned* status, cudaStream_t s) {
    const int64_t total = int64_t(n) * max_pages;
    // Up to 32768 entries one cluster and one launch (768 entries: 3.4 us, 16384: 5.6, 32768: 6.8, 65536:
    // 10.4); more take the whole GPU, after a launch that clears the word (6.3, 7.0, 6.9, 7.2 us).
    if (total <= kFreeFew) {
        free_few_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, table, rows, B, int(total), max_pages, status);
        note_launch();
        return cudaGetLastError();
    }
    const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return e;
    const int64_t most = 8 * int64_t(sm_count()), blocks = blocks_for(total, 256);
    const int grid = int(blocks < most ? blocks : most);
    free_kernel<<<grid, 256, 0, s>>>(c, table, rows, B, n, max_pages, status);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheView& c, const int32_t* table, int32_t* new_table,
                                 int32_t* new_refcount, int B, int max_pages, const PageScratch& w,
                                 unsigned* status, cudaStream_t s) {
    compact_plan_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, w, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    note_launch();
    static bool attr_done[64] = {false};
    const int64_t table_entries = int64_t(B) * max_pages;
    const int grid = copy_grid(c, c.num_pages / 2, table_entries > c.num_pages ? table_entries : c.num_pages);
    return launch_early(compact_kernel, attr_done, grid, kCopyThreads, s, c, table, new_table, new_refcount, B, max_pages, w, status);
}

cudaError_t launch_cache_copy(const CacheView& c, const int32_t* src, const int32_t* dst, int n,
                              const PageScratch& w, unsigned* status, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(w.map, 0, size_t(c.num_pages) * 4, s);
    if (e != cudaSuccess) return e;
    copy_check_kernel<<<kPlanCtas, kPlanThreads, 0, s>>>(c, src, dst, n, w, status);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    note_launch();
    static bool attr_done[64] = {false};
    return launch_early(copy_kernel, attr_done, copy_grid(c, n, n), kCopyThreads, s, c, src, dst, w, status);
}

}  // namespace smla
