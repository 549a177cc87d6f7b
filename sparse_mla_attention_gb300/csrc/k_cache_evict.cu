// k_cache_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence with more than `keep` positions the first `first`, the last `recent` and, of those between,
// the R = keep - first - recent of largest weight stay (ties: the lower position; NaN counts least), in
// the order of their positions, in fresh pages. The R-th largest weight is found by a radix descent over the
// weights' bits (a histogram of 2048 bins, and steps of seven bits among the weights of one bin as soon as they are
// few), so the choice is exact and the same in every run.
//
// Bound: latency, in the choice and in the copies (a warp follows positions, pages, scales and rows of a unit before it
// takes the next). 64 sequences of up to 8192 positions to 2048 each, pages and blocks of 64: 44 us with a free of the
// last call's pages, of which the copies take 31 (134 MB read and written: 4.3 TB/s), the choice 8 and the free 4; 3 of up
// to 81920 to 16384: 32 us, 15 and 12 and 4; one of 1500 to 1024: 16 us. The choice of a sequence in one CTA: weights
// into registers 1.1 us, histogram 0.9, its scan 0.4, collecting the bin 1,
// seven bits a step 0.7, the list 1.8; in eight, of 81920: 1.2 and 0.4 for the first barrier, 1.3, 0.5 joined, 0.8, 1.1,
// 0.9 joined, 1.2, 0.4, the counts 1.4, the list 1.2. Bisection of the few, a count and a barrier a step: 46 and 38 us (with
// lists gathered twice); bins read by every CTA from the first: 36 for the long ones. Three full histograms: 50 and 49
// us; rows looked up by the choice instead of the copies: 50.
//
// evict_plan_kernel: cluster 0 grants the free pages, the other CTAs choose, one sequence each.
// evict_copy_kernel: moves the rows. A block's scale is the largest of its rows'
// scales; the codes of rows of a smaller one are rounded to it.
#include <cuda_fp8.h>

#include "page_plan.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr int kEvictCopyThreads = 256;

// Two codes in the low half of v, times ratio, rounded again.
__device__ __forceinline__ uint32_t recode2(uint32_t v, float ratio) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return __nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t recode4(uint32_t v, float ratio) {
    return recode2(v, ratio) | recode2(v >> 16, ratio) << 16;
}
// The same where ratio is a power of two, in half precision: a code times 2^-14 or more is exact there, and what is
// less than 2^-10 (all codes times 2^-19) becomes 0 whatever its last bits.
__device__ __forceinline__ uint32_t shift4(uint32_t v, __half2 ratio) {
    const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v & 0xffffu), __NV_E4M3));
    const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v >> 16), __NV_E4M3));
    return uint32_t(__nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hmul2(lo, ratio)), __NV_SATFINITE, __NV_E4M3)) |
           uint32_t(__nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hmul2(hi, ratio)), __NV_SATFINITE, __NV_E4M3)) << 16;
}

// A weight's bits in an order of unsigned numbers; both zeros alike, NaN below all.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t x = __float_as_uint(w + 0.f);
    return w != w ? 0u : x & 0x80000000u ? ~x : x | 0x80000000u;
}

__device__ __forceinline__ int row_len(const EvictArgs& a, int b) {
    const int64_t limit = int64_t(a.max_pages) << a.cache.page_shift;
    const int len = __ldg(a.lens + b);
    return len < 0 ? 0 : len > limit ? int(limit) : len;
}

constexpr int kDigits = 2048;                    // bins of a pass: bits 31-21, 20-10 and 9-0 of a weight
constexpr int kRun = 16;                         // positions of a thread
constexpr int kTile = kPlanThreads * kRun;
constexpr int kFew = 4 * kPlanThreads;           // weights of one bin that its first CTA goes through seven bits at a time

struct ChooseShared {
    int hist[kDigits];                           // of this CTA
    int all[3][kDigits];                         // of the cluster, in its first CTA
    union {
        uint32_t few[kFew];                      // weights of the bin that the last one to stay is in; the first CTA's
        uint16_t stays[kTile];                   // positions of a tile that stay, in order
    };
    int digit, over, inside;                     // the bin of the rest-th largest, what lies above it and in it
    int n_few;                                   // of this CTA
    __align__(16) int fine[3][128];              // bins of the few
    int3 found;
    uint32_t prefix;
    int rest;
    int2 counts[kPlanCtas];                      // of each CTA's part: those above prefix, and equal
};

// The positions that sequence b keeps. kParts CTAs share the sequence (all of a cluster, or one), a run of positions
// each. A thread's keys stay in registers where the CTA's part is one tile (16384).
template <int kParts>
__device__ void choose(const EvictArgs& a, int b, int part, PlanShared& sh, ChooseShared& ch) {
    cg::cluster_group cl = cg::this_cluster();
    auto sync_all = [&]() { if (kParts > 1) cl.sync(); else __syncthreads(); };
    int turn = 0;
    const int64_t width = int64_t(a.max_pages) << a.cache.page_shift;
    const int len = row_len(a, b);
    const float* w = a.weights + b * width;
    int32_t* kept = a.kept + int64_t(b) * a.keep;
    const int64_t per = (int64_t(len) + kParts * kRun - 1) / (kParts * kRun) * kRun;
    const int64_t s0 = min(per * part, int64_t(len)), s1 = min(s0 + per, int64_t(len));
    const bool one_tile = s1 - s0 <= kTile;
    // all positions stay where there are no more than keep; else those between the first and the recent compete
    const int64_t mid0 = len <= a.keep ? len : a.first, mid1 = len <= a.keep ? len : len - a.recent;
    int rest = len <= a.keep ? 0 : a.keep - a.first - a.recent;          // of [mid0, mid1), which has more
    const bool by_weight = rest > 0;
    uint32_t key[kRun], runs, there;             // bits of the thread's positions that compete, and that exist
    auto load = [&](int64_t base) {
        const int64_t i0 = base + kRun * int64_t(threadIdx.x);
        auto below = [&](int64_t end) {          // bits of the positions before `end`
            return end <= i0 ? 0u : end >= i0 + kRun ? (1u << kRun) - 1 : (1u << int(end - i0)) - 1;
        };
        there = below(s1);
        runs = there & below(mid1) & ~below(mid0);
#pragma unroll
        for (int e = 0; e < kRun; e += 4) {      // (width is a multiple of 16: no quad passes a row's end)
            const float4 v = (there >> e) & 1 ? __ldg(reinterpret_cast<const float4*>(w + i0 + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
            key[e] = order_of(v.x); key[e + 1] = order_of(v.y); key[e + 2] = order_of(v.z); key[e + 3] = order_of(v.w);
        }
    };
    if (threadIdx.x == 0) ch.n_few = 0;
    if (threadIdx.x < 3 * 128) (&ch.fine[0][0])[threadIdx.x] = 0;
    if (kParts > 1 && part == 0)
        for (int i = threadIdx.x; i < 3 * kDigits; i += kPlanThreads) (&ch.all[0][0])[i] = 0;
    if (one_tile) load(s0);
    uint32_t prefix = 0;
    // Another CTA's shared memory exists once that CTA runs: every sequence waits for all of its CTAs, those whose
    // choice needs no weights too (they write their counts to the others below).
    if (kParts > 1) cl.sync();
    if (by_weight) {                             // (the same in every CTA of the sequence)
        ChooseShared* lead = kParts > 1 ? cl.map_shared_rank(&ch, 0) : &ch;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kDigits;
            const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
            ch.hist[threadIdx.x] = 0;
            ch.hist[threadIdx.x + 1024] = 0;
            __syncthreads();
            for (int64_t base = s0; base < s1; base += kTile) {
                if (!one_tile) load(base);
                if (runs == 0) continue;
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    if (((runs >> e) & 1) && (key[e] & mask) == prefix)
                        atomicAdd(ch.hist + ((key[e] >> shift) & uint32_t(bins - 1)), 1);
            }
            __syncthreads();
            const int* hist = ch.hist;
            if (kParts > 1) {                    // few bins hold anything: they are added to the first CTA's
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int d = int(threadIdx.x) + 1024 * k, h = ch.hist[d];
                    if (h) atomicAdd(lead->all[pass] + d, h);
                }
                cl.sync();
                hist = ch.all[pass];
            }
            if (part == 0) {                     // bins in falling order, two a thread: the sums before them
                const int d0 = bins - 1 - 2 * int(threadIdx.x), d1 = d0 - 1;
                const int h0 = d0 >= 0 ? hist[d0] : 0, h1 = d0 >= 0 ? hist[d1] : 0;
                int total;
                const int before = cta_scan(h0 + h1, sh, turn, &total);
                if (before < rest && rest <= before + h0 + h1) {
                    const bool second = rest > before + h0;
                    const int3 found = second ? make_int3(d1, before + h0, h1) : make_int3(d0, before, h0);
#pragma unroll
                    for (int r = 0; r < kParts; ++r) {
                        ChooseShared* to = kParts > 1 ? cl.map_shared_rank(&ch, r) : &ch;
                        to->digit = found.x;
                        to->over = found.y;
                        to->inside = found.z;
                    }
                }
            }
            sync_all();
            prefix |= uint32_t(ch.digit) << shift;
            rest -= ch.over;
            if (pass == 2 || ch.inside > kFew) continue;
            // the bin's weights in the first CTA, behind those of the CTAs before, and their rest-th largest there
            const uint32_t bin = ~0u << shift;
            const int lane = int(threadIdx.x & 31), n = ch.inside;
            int to0 = 0;
            if (kParts > 1) to0 = __reduce_add_sync(0xffffffffu, lane < part ? cl.map_shared_rank(&ch, lane)->hist[ch.digit] : 0);
            for (int64_t base = s0; base < s1; base += kTile) {
                if (!one_tile) load(base);
                uint32_t in = 0;
#pragma unroll
                for (int e = 0; e < kRun; ++e) in |= uint32_t((key[e] & bin) == prefix) << e;
                in &= runs;
                if (in == 0) continue;
                int to = to0 + atomicAdd(&ch.n_few, __popc(in));
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    if ((in >> e) & 1) lead->few[to++] = key[e];
            }
            sync_all();
            if (part == 0) {
                int mine[4];                     // what lies above prefix; -1: none
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = int(threadIdx.x) + kPlanThreads * k;
                    mine[k] = i < n ? int(ch.few[i] - prefix) : -1;
                }
                // seven bits of the rest-th largest at a time: a histogram of [lo, lo + 2^(s + 7)), `over` lie above
                int lo = 0, over = 0, s = shift == 21 ? 14 : 7;
                bool exact = false;
#pragma unroll 1
                for (int* fine = ch.fine[0]; s >= 0 && !exact; fine += 128, s -= 7) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = (mine[k] - lo) >> s;
                        if (mine[k] >= lo && d < 128) atomicAdd(fine + d, 1);
                    }
                    __syncthreads();
                    if (threadIdx.x < 32) {      // four bins a lane, the largest first
                        const int4 h = reinterpret_cast<const int4*>(fine)[31 - lane];
                        const int sum = h.x + h.y + h.z + h.w;
                        int before = sum;
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) {
                            const int x = __shfl_up_sync(0xffffffffu, before, d);
                            if (lane >= d) before += x;
                        }
                        before += over - sum;
                        if (before < rest && rest <= before + sum) {
                            int d = 127 - 4 * lane;
                            int in = h.w;
                            if (before + in < rest) { before += in; in = h.z; --d; }
                            if (before + in < rest) { before += in; in = h.y; --d; }
                            if (before + in < rest) { before += in; in = h.x; --d; }
                            // where all of the bin stay: those above the key before its first (there is one)
                            ch.found = make_int3(lo + (d << s), before, before + in == rest && (prefix | uint32_t(lo + (d << s))));
                        }
                    }
                    __syncthreads();
                    lo = ch.found.x;
                    over = ch.found.y;
                    exact = ch.found.z;
                }
                if (threadIdx.x < kParts) {
                    ChooseShared* to = kParts > 1 ? cl.map_shared_rank(&ch, threadIdx.x) : &ch;
                    to->prefix = prefix + uint32_t(lo) - (exact ? 1u : 0u);
                    to->rest = exact ? 0 : rest - over;
                }
            }
            sync_all();
            prefix = ch.prefix;
            rest = ch.rest;
            break;
        }
    }
    // keys above prefix stay, and the first `rest` equal ones
    uint32_t stay, tie;
    int total, before = 0;                       // those above prefix in the high half, equal ones in the low
    auto count = [&]() {
        stay = there & ~runs;
        tie = 0;
        if (by_weight && runs) {
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                stay |= uint32_t(key[e] > prefix) << e & runs;
                tie |= uint32_t(key[e] == prefix) << e & runs;
            }
        }
        before = cta_scan(__popc(stay) << 16 | __popc(tie), sh, turn, &total);
    };
    int64_t at = 0, tied = 0;                    // before the tile
    if (kParts > 1) {
        int2 mine = make_int2(0, 0);
        for (int64_t base = s0; base < s1; base += kTile) {
            if (!one_tile) load(base);
            count();
            mine.x += total >> 16;
            mine.y += total & 0xffff;
        }
        if (threadIdx.x < kParts) cl.map_shared_rank(&ch, threadIdx.x)->counts[part] = mine;
        cl.sync();                               // (the last look at another CTA's memory is behind every CTA here)
        for (int r = 0; r < part; ++r) {
            at += ch.counts[r].x;
            tied += ch.counts[r].y;
        }
    }
    at += min(tied, int64_t(rest));
    for (int64_t base = s0; base < s1; base += kTile) {
        if (!one_tile) load(base);
        if (kParts == 1 || !one_tile) count();
        const int64_t ties = tied + (before & 0xffff), done = min(tied, int64_t(rest));
        int to = (before >> 16) + int(min(ties, int64_t(rest)) - done);
        for (int64_t drop = ties + __popc(tie) - max(int64_t(rest), ties); drop > 0; --drop) tie ^= 1u << (31 - __clz(tie));
        stay |= tie;
        for (; stay; stay &= stay - 1) ch.stays[to++] = uint16_t(kRun * threadIdx.x + __ffs(stay) - 1);
        tied += total & 0xffff;
        const int n = (total >> 16) + int(min(tied, int64_t(rest)) - done);
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kPlanThreads) kept[at + i] = int(base) + ch.stays[i];
        at += n;
        __syncthreads();
    }
}

}  // namespace

template <int kParts>
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
evict_plan_kernel(const EvictArgs a) {
    __shared__ PlanShared sh;
    extern __shared__ __align__(16) uint8_t room[];
    grid_dep_launch();
    if (blockIdx.x >= kPlanCtas) {
        const int u = int(blockIdx.x) - kPlanCtas, b = u / kParts;
        if (b < a.B) choose<kParts>(a, b, u % kParts, sh, *reinterpret_cast<ChooseShared*>(room));
        return;
    }
    cg::cluster_group cl = cg::this_cluster();
    const CacheView& c = a.cache;
    const int64_t limit = int64_t(a.max_pages) << c.page_shift;
    unsigned bits = 0;
    int turn = 0;
    for (int b = int(blockIdx.x) * kPlanThreads + threadIdx.x; b < a.B; b += kPlanCtas * kPlanThreads) {
        const int len = clamp_len(__ldg(a.lens + b), limit, bits);
        a.need[b] = int((int64_t(len < a.keep ? len : a.keep) + (1 << c.page_shift) - 1) >> c.page_shift);
    }
    // A sequence's page that nobody owns may be among those that this call takes, which would be written as it is read:
    // nothing is granted then. (Counts change once all CTAs have looked.)
    constexpr int kStep = kPlanCtas * kPlanThreads;
#pragma unroll 4
    for (int64_t x = int64_t(blockIdx.x) * kPlanThreads + threadIdx.x; x < int64_t(a.B) * a.max_pages; x += kStep) {
        const int b = int(x / a.max_pages), j = int(x - int64_t(b) * a.max_pages);
        const int page = __ldg(a.table + x);
        if (int64_t(j) << c.page_shift < row_len(a, b) && page >= 0 && page < c.num_pages &&
            __ldcg(c.refcount + page) <= 0)
            bits |= 1u << SMLA_ERR_REFCOUNT;
    }
    const bool ok = grant_pages(c, a.B, a.need, a.start, a.fresh, bits, sh, turn, cl, a.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.granted[0] = ok;
}

// A warp moves up to 16 rows at a time, all of them in flight; it looks at the scales of the whole block.
__global__ void __launch_bounds__(kEvictCopyThreads, 2)
evict_copy_kernel(const EvictArgs a) {
    grid_dep_wait();
    const CacheView& c = a.cache;
    const int lane = threadIdx.x & 31;
    const int64_t threads = int64_t(gridDim.x) * kEvictCopyThreads, first = int64_t(blockIdx.x) * kEvictCopyThreads + threadIdx.x;
    const int64_t width = int64_t(a.max_pages) << c.page_shift;
    const bool ok = __ldcg(a.granted) != 0;
    const int block = 1 << c.block_shift, page_mask = (1 << c.page_shift) - 1;
    const int64_t per = (int64_t(a.keep) + 15) >> 4;
    bool bad = false;
    for (int64_t u = first >> 5; u < a.B * per; u += threads >> 5) {
        const int b = int(u / per);
        const int64_t r0 = (u - b * per) << 4;
        const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
        const int rows = int(min(n - r0, int64_t(16)));
        int32_t* kept = a.kept + int64_t(b) * a.keep;
        if (lane < 16 && lane >= rows && r0 + lane < a.keep) kept[r0 + lane] = -1;
        if (rows <= 0) continue;
        // the rows of the block, up to two a lane: where they lie (-1: no page) and their scales
        const int64_t block0 = r0 & ~int64_t(block - 1);
        const int32_t* table = a.table + int64_t(b) * a.max_pages;
        int p[2], from[2] = {-1, -1};
        float scale[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = lane + 32 * k;
            p[k] = r < block && block0 + r < n ? __ldcg(kept + block0 + r) : -1;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (p[k] >= 0) {
                const int page = __ldg(table + (p[k] >> c.page_shift));
                if (page >= 0 && page < c.num_pages) from[k] = (page << c.page_shift) + (p[k] & page_mask);
                else bad = true;
            }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (from[k] >= 0) scale[k] = __ldg(c.scales + (from[k] >> c.block_shift));
        // this warp's 16 of them
        const int half = int(r0 - block0) >> 5, lane0 = int(r0 - block0) & 31;
        const int mine = half ? from[1] : from[0];
        const float own = half ? scale[1] : scale[0];
        if (lane >= lane0 && lane < lane0 + rows)
            a.new_weights[b * width + r0 + lane - lane0] = __ldg(a.weights + b * width + (half ? p[1] : p[0]));
        if (!ok) continue;
        uint4 v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = __shfl_sync(0xffffffffu, mine, lane0 + r);
            v[r] = row >= 0 && r < rows ? __ldcg(reinterpret_cast<const uint4*>(c.pages + int64_t(row) * kD) + lane)
                                        : make_uint4(0, 0, 0, 0);
        }
        float size = fmaxf(scale[0], scale[1]);
#pragma unroll
        for (int d = 16; d; d >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
        const int page = __ldcg(a.fresh + __ldcg(a.start + b) + (r0 >> c.page_shift));
        const int64_t to = (int64_t(page) << c.page_shift) + (r0 & page_mask);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float was = __shfl_sync(0xffffffffu, own, lane0 + r);
            if (r >= rows) break;
            uint4 x = v[r];
            if (was != size) {
                const float ratio = was / size;
                if ((__float_as_uint(ratio) & 0x807fffffu) == 0) {
                    const __half2 h = __float2half2_rn(ratio);
                    x = make_uint4(shift4(x.x, h), shift4(x.y, h), shift4(x.z, h), shift4(x.w, h));
                } else {
                    x = make_uint4(recode4(x.x, ratio), recode4(x.y, ratio), recode4(x.z, ratio), recode4(x.w, ratio));
                }
            }
            *(reinterpret_cast<uint4*>(c.pages + (to + r) * kD) + lane) = x;
        }
        if (r0 == block0 && lane == 0) c.scales[to >> c.block_shift] = size;
    }
    if (bad) flag_status(a.status, SMLA_ERR_INDEX);
    // tables, lengths, and zeros behind the weights
    for (int64_t x = first; x < int64_t(a.B) * a.max_pages; x += threads) {
        const int b = int(x / a.max_pages), j = int(x - int64_t(b) * a.max_pages);
        const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
        a.new_table[x] = ok && j < __ldcg(a.need + b) ? __ldcg(a.fresh + __ldcg(a.start + b) + j) : -1;
        if (j == 0) a.new_lens[b] = ok ? n : 0;
    }
    const int64_t quads = width / 4;
    for (int64_t x = first; x < a.B * quads; x += threads) {
        const int b = int(x / quads);
        const int64_t i = 4 * (x - b * quads);
        const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
        float* out = a.new_weights + b * width + i;
        if (i >= n) *reinterpret_cast<float4*>(out) = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (i + 4 > n)
            for (int e = int(n - i); e < 4; ++e) out[e] = 0.f;
    }
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
    static bool attr_done[64] = {false};
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(evict_plan_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(sizeof(ChooseShared)));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(evict_plan_kernel<kPlanCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(sizeof(ChooseShared)));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // A sequence has one CTA, whose registers hold 16384 weights; wider tables give it a cluster. Both sides, device time:
    // 3 of 81920 61 us with one CTA each (it goes over its weights tile by tile), 32 with a cluster; 64 of 8192 44 and 83
    // (512 CTAs take turns), one of 1500 16 and 18.
    const int parts = (int64_t(a.max_pages) << a.cache.page_shift) > 16384 ? kPlanCtas : 1;
    const unsigned grid = unsigned(kPlanCtas + (int64_t(a.B) * parts + kPlanCtas - 1) / kPlanCtas * kPlanCtas);
    if (parts > 1) evict_plan_kernel<kPlanCtas><<<grid, kPlanThreads, sizeof(ChooseShared), s>>>(a);
    else evict_plan_kernel<1><<<grid, kPlanThreads, sizeof(ChooseShared), s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t units = int64_t(a.B) * ((int64_t(a.keep) + 15) / 16), blocks = (units + 7) / 8, most = int64_t(sms) * 2;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kEvictCopyThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    note_launch(2);
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, a);
}

}  // namespace smla
