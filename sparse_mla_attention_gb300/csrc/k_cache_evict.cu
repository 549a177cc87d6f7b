// k_cache_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence with more than `keep` positions the first `first`, the last `recent` and, of those between,
// the R = keep - first - recent of largest weight stay (ties: the lower position; NaN counts least), in
// the order of their positions, in fresh pages. The R-th largest weight is found by a radix descent over the
// weights' bits (three histograms of 2048 counts), so the choice is exact and the same in every run.
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
constexpr int kRun = 16;                         // positions of a thread: in one page and one scale block
constexpr int kTile = kPlanThreads * kRun;

struct ChooseShared {
    int hist[kDigits];                           // of this CTA
    int all[3][kDigits];                         // of the cluster, in its first CTA
    int digit, over;                             // the bin of the rest-th largest, and what lies above it
    int above, ties;                             // of this CTA's part, read by the others
};

// The positions that sequence b keeps, their weights and rows. kParts CTAs share the sequence (all of a cluster, or
// one), a run of positions each. A thread's keys stay in registers where the CTA's part is one tile (16384).
template <int kParts>
__device__ void choose(const EvictArgs& a, int b, int part, PlanShared& sh, ChooseShared& ch) {
    cg::cluster_group cl = cg::this_cluster();
    const CacheView& c = a.cache;
    int turn = 0;
    const int64_t width = int64_t(a.max_pages) << c.page_shift;
    const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
    const float* w = a.weights + b * width;
    int32_t* kept = a.kept + int64_t(b) * a.keep;
    float* out = a.new_weights + b * width;
    const int first = part * kPlanThreads + int(threadIdx.x);
    for (int64_t i = n + int64_t(first); i < width; i += kParts * kPlanThreads) out[i] = 0.f;
    for (int64_t i = n + int64_t(first); i < a.keep; i += kParts * kPlanThreads) kept[i] = -1;
    const int64_t per = (int64_t(len) + kParts * kRun - 1) / (kParts * kRun) * kRun;
    const int64_t s0 = min(per * part, int64_t(len)), s1 = min(s0 + per, int64_t(len));
    const bool one_tile = s1 - s0 <= kTile;
    // all positions stay where there are no more than keep; else those between the first and the recent compete
    const int64_t mid0 = len <= a.keep ? len : a.first, mid1 = len <= a.keep ? len : len - a.recent;
    int rest = len <= a.keep ? 0 : a.keep - a.first - a.recent;          // of [mid0, mid1), which has more
    const bool by_weight = rest > 0;
    uint32_t key[kRun];
    int64_t i0 = 0;                              // the thread's first position of the tile at hand
    auto load = [&](int64_t base) {
        i0 = base + kRun * int64_t(threadIdx.x);
#pragma unroll
        for (int e = 0; e < kRun; e += 4) {      // (width is a multiple of 16: no quad passes a row's end)
            const float4 v = i0 + e < s1 ? __ldg(reinterpret_cast<const float4*>(w + i0 + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
            key[e] = order_of(v.x); key[e + 1] = order_of(v.y); key[e + 2] = order_of(v.z); key[e + 3] = order_of(v.w);
        }
    };
    auto competes = [&](int e) { return i0 + e >= mid0 && i0 + e < mid1 && i0 + e < s1; };
    if (one_tile) load(s0);
    uint32_t prefix = 0;
    if (by_weight) {                             // (the same in every CTA of the sequence)
        if (kParts > 1) {
            if (part == 0)
                for (int i = threadIdx.x; i < 3 * kDigits; i += kPlanThreads) (&ch.all[0][0])[i] = 0;
            cl.sync();
        }
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kDigits;
            const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
            ch.hist[threadIdx.x] = 0;
            ch.hist[threadIdx.x + 1024] = 0;
            __syncthreads();
            for (int64_t base = s0; base < s1; base += kTile) {
                if (!one_tile) load(base);
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    if (competes(e) && (key[e] & mask) == prefix)
                        atomicAdd(ch.hist + ((key[e] >> shift) & uint32_t(bins - 1)), 1);
            }
            __syncthreads();
            const int* hist = ch.hist;
            if (kParts > 1) {                    // few bins hold anything: they are added to the first CTA's
                int* all = cl.map_shared_rank(ch.all[pass], 0);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int d = int(threadIdx.x) + 1024 * k, h = ch.hist[d];
                    if (h) atomicAdd(all + d, h);
                }
                cl.sync();
                hist = all;
            }
            // bins in falling order, two a thread: the sums before them
            const int d0 = bins - 1 - 2 * int(threadIdx.x), d1 = d0 - 1;
            const int h0 = d0 >= 0 ? hist[d0] : 0, h1 = d0 >= 0 ? hist[d1] : 0;
            int total;
            const int before = cta_scan(h0 + h1, sh, turn, &total);
            if (before < rest && rest <= before + h0 + h1) {
                const bool second = rest > before + h0;
                ch.digit = second ? d1 : d0;
                ch.over = second ? before + h0 : before;
            }
            __syncthreads();
            prefix |= uint32_t(ch.digit) << shift;
            rest -= ch.over;
        }
    }
    // keys above prefix stay (1), and the first `rest` equal ones (1 << 16)
    auto verdict = [&](int e) {
        if (i0 + e >= s1) return 0;
        if (!competes(e)) return 1;
        return !by_weight ? 0 : key[e] > prefix ? 1 : key[e] == prefix ? 1 << 16 : 0;
    };
    int64_t at = 0, tied_before = 0;
    if (kParts > 1) {
        int above = 0, ties = 0;
        for (int64_t base = s0; base < s1; base += kTile) {
            if (!one_tile) load(base);
            int count = 0, total;
#pragma unroll
            for (int e = 0; e < kRun; ++e) count += verdict(e);
            cta_scan(count & 0xffff, sh, turn, &total);
            above += total;
            cta_scan(count >> 16, sh, turn, &total);
            ties += total;
        }
        if (threadIdx.x == 0) { ch.above = above; ch.ties = ties; }
        cl.sync();
        for (int r = 0; r < part; ++r) {
            at += cl.map_shared_rank(&ch, r)->above;
            tied_before += cl.map_shared_rank(&ch, r)->ties;
        }
    }
    int t = int(tied_before);
    for (int64_t base = s0; base < s1; base += kTile) {
        if (!one_tile) load(base);
        int2 from = make_int2(-1, 0);            // the run's first row of the pool and its scale
        if (i0 < s1) {
            const int page = __ldg(a.table + int64_t(b) * a.max_pages + (i0 >> c.page_shift));
            if (page >= 0 && page < c.num_pages) {
                from.x = (page << c.page_shift) + int(i0 & ((1 << c.page_shift) - 1));
                from.y = __float_as_int(__ldg(c.scales + (from.x >> c.block_shift)));
            }
        }
        int count = 0, stay, tie;
#pragma unroll
        for (int e = 0; e < kRun; ++e) count += verdict(e);
        const int stays = cta_scan(count & 0xffff, sh, turn, &stay), tied0 = cta_scan(count >> 16, sh, turn, &tie);
        int64_t to = at + stays;
        int tied = t + tied0;
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            const int v = verdict(e);
            if (v == 1 || (v != 0 && tied < rest)) {
                const int64_t row = to + min(tied, rest);
                kept[row] = int(i0 + e);
                out[row] = __ldg(w + i0 + e);
                a.from[int64_t(b) * a.keep + row] = make_int2(from.x < 0 ? -1 : from.x + e, from.y);
            }
            to += v & 1;
            tied += v >> 16;
        }
        at += stay;
        t += tie;
    }
    if (kParts > 1) cl.sync();                   // no CTA leaves while another reads its counts
}

}  // namespace

template <int kParts>
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
evict_plan_kernel(const EvictArgs a) {
    __shared__ PlanShared sh;
    __shared__ ChooseShared ch;
    grid_dep_launch();
    if (blockIdx.x >= kPlanCtas) {
        const int u = int(blockIdx.x) - kPlanCtas, b = u / kParts;
        if (b < a.B) choose<kParts>(a, b, u % kParts, sh, ch);
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
    const bool ok = grant_pages(c, a.B, a.need, a.start, a.fresh, bits, sh, turn, cl, a.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.granted[0] = ok;
}

// A warp moves up to 16 rows at a time, all of them in flight; it looks at the scales of the whole block.
__global__ void __launch_bounds__(kEvictCopyThreads)
evict_copy_kernel(const EvictArgs a) {
    grid_dep_wait();
    const CacheView& c = a.cache;
    const int lane = threadIdx.x & 31;
    const int64_t threads = int64_t(gridDim.x) * kEvictCopyThreads, first = int64_t(blockIdx.x) * kEvictCopyThreads + threadIdx.x;
    const bool ok = __ldcg(a.granted) != 0;
    for (int64_t x = first; x < int64_t(a.B) * a.max_pages; x += threads) {
        const int b = int(x / a.max_pages), j = int(x - int64_t(b) * a.max_pages);
        a.new_table[x] = ok && j < __ldcg(a.need + b) ? __ldcg(a.fresh + __ldcg(a.start + b) + j) : -1;
        if (j == 0) {
            const int len = row_len(a, b);
            a.new_lens[b] = !ok ? 0 : len < a.keep ? len : a.keep;
        }
    }
    if (!ok) return;
    const int block = 1 << c.block_shift, page_mask = (1 << c.page_shift) - 1;
    const int64_t per = (int64_t(a.keep) + 15) >> 4;
    bool bad = false;
    for (int64_t u = first >> 5; u < a.B * per; u += threads >> 5) {
        const int b = int(u / per);
        const int64_t r0 = (u - b * per) << 4;
        const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
        const int rows = int(min(n - r0, int64_t(16)));
        if (rows <= 0) continue;
        const int64_t block0 = r0 & ~int64_t(block - 1);
        const int page = __ldcg(a.fresh + __ldcg(a.start + b) + (r0 >> c.page_shift));
        // the rows of the block, up to two a lane, and this warp's
        const int2* list = a.from + int64_t(b) * a.keep;
        float size = 0.f;
        for (int r = lane; r < block && block0 + r < n; r += 32) size = fmaxf(size, __int_as_float(__ldcg(list + block0 + r).y));
        const int2 own = lane < rows ? __ldcg(list + r0 + lane) : make_int2(-1, 0);
        bad |= lane < rows && own.x < 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
        const int64_t to = (int64_t(page) << c.page_shift) + (r0 & page_mask);
        uint4 v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = __shfl_sync(0xffffffffu, own.x, r);
            v[r] = row >= 0 ? __ldcg(reinterpret_cast<const uint4*>(c.pages + int64_t(row) * kD) + lane) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (r >= rows) break;
            const float scale = __int_as_float(__shfl_sync(0xffffffffu, own.y, r));
            uint4 x = v[r];
            if (scale != size) {
                const float ratio = scale / size;
                x = make_uint4(recode4(x.x, ratio), recode4(x.y, ratio), recode4(x.z, ratio), recode4(x.w, ratio));
            }
            *(reinterpret_cast<uint4*>(c.pages + (to + r) * kD) + lane) = x;
        }
        if (r0 == block0 && lane == 0) c.scales[to >> c.block_shift] = size;
    }
    if (bad) flag_status(a.status, SMLA_ERR_INDEX);
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // Long sequences have a cluster each.
    const int parts = (int64_t(a.max_pages) << a.cache.page_shift) > 16384 ? kPlanCtas : 1;
    const int64_t grid = kPlanCtas + (int64_t(a.B) * parts + kPlanCtas - 1) / kPlanCtas * kPlanCtas;
    if (parts > 1) evict_plan_kernel<kPlanCtas><<<unsigned(grid), kPlanThreads, 0, s>>>(a);
    else evict_plan_kernel<1><<<unsigned(grid), kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t units = int64_t(a.B) * ((int64_t(a.keep) + 15) / 16), blocks = (units + 7) / 8, most = int64_t(sms) * 4;
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
