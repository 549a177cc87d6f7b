// k_cache_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence with more than `keep` positions the first `first`, the last `recent` and, of those between,
// the R = keep - first - recent of largest weight stay (ties: the lower position; NaN counts least), in
// the order of their positions, in fresh pages. The R-th largest weight is found by a radix descent over the
// weights' bits (four histograms of 256 counts), so the choice is exact and the same in every run.
//
// evict_plan_kernel: cluster 0 grants the free pages, the other CTAs choose, one sequence each.
// evict_copy_kernel: moves the rows, a scale block at a time. A block's scale is the largest of its rows'
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

// The positions that sequence b keeps and their weights.
__device__ void choose(const EvictArgs& a, int b, PlanShared& sh, int* hist) {
    int turn = 0;
    const int64_t width = int64_t(a.max_pages) << a.cache.page_shift;
    const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
    const float* w = a.weights + b * width;
    int32_t* kept = a.kept + int64_t(b) * a.keep;
    float* out = a.new_weights + b * width;
    for (int64_t i = n + int64_t(threadIdx.x); i < width; i += kPlanThreads) out[i] = 0.f;
    for (int i = n + threadIdx.x; i < a.keep; i += kPlanThreads) kept[i] = -1;
    if (len <= a.keep) {
        for (int i = threadIdx.x; i < n; i += kPlanThreads) {
            kept[i] = i;
            out[i] = __ldg(w + i);
        }
        return;
    }
    const int lo = a.first, hi = len - a.recent;
    int rest = a.keep - a.first - a.recent;      // of [lo, hi), which has more
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int64_t i = lo + int(threadIdx.x); i < hi; i += kPlanThreads) {
            const uint32_t key = order_of(__ldg(w + i));
            if ((key & mask) == prefix) atomicAdd(hist + ((key >> shift) & 255u), 1);
        }
        __syncthreads();
        // the digit of the rest-th largest: thread d counts those of larger digits
        int above = 0, mine = 0;
        if (threadIdx.x < 256) {
            mine = hist[threadIdx.x];
            for (int d = threadIdx.x + 1; d < 256; ++d) above += hist[d];
            if (above < rest && rest <= above + mine) {
                hist[256] = int(threadIdx.x);
                hist[257] = above;
            }
            if (rest == 0 && threadIdx.x == 255) { hist[256] = 255; hist[257] = 0; }
        }
        __syncthreads();
        prefix |= uint32_t(hist[256]) << shift;
        rest -= hist[257];
        __syncthreads();
    }
    // keys above prefix stay, and the first `rest` equal ones
    int at = 0, ties = 0;
    for (int64_t base = 0; base < len; base += kPlanThreads) {
        const int64_t i = base + int(threadIdx.x);
        const float v = i < len ? __ldg(w + i) : 0.f;
        bool stays = false, tie = false;
        if (i < len) {
            if (i < lo || i >= hi) {
                stays = true;
            } else {
                const uint32_t key = order_of(v);
                stays = key > prefix && a.keep > a.first + a.recent;
                tie = key == prefix;
            }
        }
        int total;
        const int before = cta_scan(int(stays) | int(tie) << 16, sh, turn, &total);
        const int tied = ties + (before >> 16);
        if (tie) stays = tied < rest;
        if (stays) {
            const int to = at + (before & 0xffff) + (tied < rest ? tied : rest);
            kept[to] = int(i);
            out[to] = v;
        }
        at += total & 0xffff;
        ties += total >> 16;
    }
}

}  // namespace

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
evict_plan_kernel(const EvictArgs a) {
    __shared__ PlanShared sh;
    __shared__ int hist[258];
    grid_dep_launch();
    if (blockIdx.x >= kPlanCtas) {
        const int b = int(blockIdx.x) - kPlanCtas;
        if (b < a.B) choose(a, b, sh, hist);
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

__global__ void __launch_bounds__(kEvictCopyThreads)
evict_copy_kernel(const EvictArgs a) {
    __shared__ int src[64];
    __shared__ float scale[64];
    grid_dep_wait();
    const CacheView& c = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t threads = int64_t(gridDim.x) * kEvictCopyThreads;
    const bool ok = __ldcg(a.granted) != 0;
    for (int64_t x = int64_t(blockIdx.x) * kEvictCopyThreads + threadIdx.x; x < int64_t(a.B) * a.max_pages; x += threads) {
        const int b = int(x / a.max_pages), j = int(x - int64_t(b) * a.max_pages);
        a.new_table[x] = ok && j < __ldcg(a.need + b) ? __ldcg(a.fresh + __ldcg(a.start + b) + j) : -1;
        if (j == 0) {
            const int len = row_len(a, b);
            a.new_lens[b] = !ok ? 0 : len < a.keep ? len : a.keep;
        }
    }
    if (!ok) return;
    const int block = 1 << c.block_shift, page_mask = (1 << c.page_shift) - 1;
    const int per = (a.keep + block - 1) >> c.block_shift;
    for (int64_t u = blockIdx.x; u < int64_t(a.B) * per; u += gridDim.x) {
        const int b = int(u / per), r0 = int(u - int64_t(b) * per) << c.block_shift;
        const int len = row_len(a, b), n = len < a.keep ? len : a.keep;
        const int rows = n - r0 < block ? n - r0 : block;
        if (rows <= 0) continue;
        __syncthreads();
        if (threadIdx.x < rows) {
            const int p = __ldcg(a.kept + int64_t(b) * a.keep + r0 + threadIdx.x);
            const int page = __ldg(a.table + int64_t(b) * a.max_pages + (p >> c.page_shift));
            const bool there = page >= 0 && page < c.num_pages;
            const int row = there ? (page << c.page_shift) + (p & page_mask) : -1;
            if (!there) flag_status(a.status, SMLA_ERR_INDEX);
            src[threadIdx.x] = row;
            scale[threadIdx.x] = there ? c.scales[row >> c.block_shift] : 0.f;
        }
        __syncthreads();
        float size = 0.f;
        for (int r = lane; r < rows; r += 32) size = fmaxf(size, scale[r]);
#pragma unroll
        for (int d = 16; d; d >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, d));
        const int64_t to = (int64_t(__ldcg(a.fresh + __ldcg(a.start + b) + (r0 >> c.page_shift))) << c.page_shift) +
                           (r0 & page_mask);
        for (int r = warp; r < rows; r += kEvictCopyThreads / 32) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (src[r] >= 0) v = *(reinterpret_cast<const uint4*>(c.pages + int64_t(src[r]) * kD) + lane);
            if (scale[r] != size) {
                const float ratio = scale[r] / size;
                v = make_uint4(recode4(v.x, ratio), recode4(v.y, ratio), recode4(v.z, ratio), recode4(v.w, ratio));
            }
            *(reinterpret_cast<uint4*>(c.pages + (to + r) * kD) + lane) = v;
        }
        if (threadIdx.x == 0) c.scales[to >> c.block_shift] = size;
    }
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
    const int rows = (a.B + kPlanCtas - 1) / kPlanCtas * kPlanCtas;
    evict_plan_kernel<<<kPlanCtas + rows, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t units = int64_t(a.B) * ((a.keep + (1 << a.cache.block_shift) - 1) >> a.cache.block_shift);
    const int64_t most = int64_t(sms) * 8;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(units < most ? units : most));
    cfg.blockDim = dim3(kEvictCopyThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    note_launch(2);
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, a);
}

}  // namespace smla
