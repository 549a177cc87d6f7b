// k_cache_weights.cu -- the attention weight that each cached position gets.
//
// For sequence b with the tokens t in [cu[b], cu[b+1]) and position p < lens[t] of any of them:
//   weights[b,p] = decay * earlier[b,p] + sum_t sum_h exp(scale * <q[t,h,:], x_p> - lse[t,h]) [p < lens[t]],
//   x_p = e4m3 code * block scale.
//
// One CTA takes 16 positions, widened in shared memory; its warps take the tokens' heads in turn, and the
// warps' sums are added in their order.
#include <cuda_fp8.h>

#include "smla_internal.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr int kCwTile = 16, kCwThreads = 256, kCwWarps = kCwThreads / 32;
constexpr float kCwLog2e = 1.4426950408889634f;

}  // namespace

__global__ void __launch_bounds__(kCwThreads)
cache_weights_kernel(const WeightsArgs a) {
    __shared__ float x[kCwTile][kD];
    __shared__ float part[kCwWarps][kCwTile];
    __shared__ int row_of[kCwTile];
    const CacheView& c = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t width = int64_t(a.max_pages) << c.page_shift, tiles = width / kCwTile;
    if (a.B == 0) return;
    for (int64_t u = blockIdx.x; u < a.B * tiles; u += gridDim.x) {
        const int b = int(u / tiles);
        const int64_t p0 = (u - b * tiles) * kCwTile;
        int c0 = b, c1 = b < a.T ? b + 1 : b;
        if (a.cu) { c0 = __ldg(a.cu + b); c1 = __ldg(a.cu + b + 1); }
        if (c0 < 0 || c1 < c0 || c1 > a.T) {
            if (p0 == 0 && threadIdx.x == 0) flag_status(a.status, SMLA_ERR_INDEX);
            continue;
        }
        int64_t seen = 0;
        for (int t = c0; t < c1; ++t) {
            const int len = __ldg(a.lens + t);
            if ((len < 0 || len > width) && p0 == 0 && threadIdx.x == 0) flag_status(a.status, SMLA_ERR_INDEX);
            seen = max(seen, min(int64_t(len), width));
        }
        if (p0 >= seen) continue;
        __syncthreads();
        if (threadIdx.x < kCwTile) {
            const int64_t p = p0 + threadIdx.x;
            const int page = p < seen ? __ldg(a.table + b * int64_t(a.max_pages) + (p >> c.page_shift)) : -1;
            const bool there = page >= 0 && page < c.num_pages;
            if (p < seen && !there) flag_status(a.status, SMLA_ERR_INDEX);
            row_of[threadIdx.x] = there ? (page << c.page_shift) + int(p & ((1 << c.page_shift) - 1)) : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kCwTile * kD; i += kCwThreads) {
            const int r = i / kD, row = row_of[r];
            __nv_fp8_e4m3 code;
            code.__x = row < 0 ? 0 : c.pages[int64_t(row) * kD + i % kD];
            x[r][i % kD] = row < 0 ? 0.f : float(code) * c.scales[row >> c.block_shift];
        }
        __syncthreads();
        float sum = 0.f;                         // of position p0 + lane
        for (int64_t k = int64_t(c0) * a.H + warp; k < int64_t(c1) * a.H; k += kCwWarps) {
            const int len = __ldg(a.lens + k / a.H);
            if (p0 >= len) continue;
            const float lse = __ldg(a.lse + k);
            float q[16];
            bool odd = false;                    // an infinity or a NaN makes the head's weights NaN
            for (int e = 0; e < 16; ++e) {
                const uint32_t bits = a.q[k * kD + lane + 32 * e];
                q[e] = __uint_as_float(bits << 16);
                odd |= (bits & 0x7f80u) == 0x7f80u;
            }
            odd = __any_sync(0xffffffffu, odd) != 0;
            for (int r = 0; r < kCwTile; ++r) {
                float s = odd ? __int_as_float(0x7fffffff) : 0.f;
                for (int e = 0; e < 16; ++e) s = fmaf(q[e], x[r][lane + 32 * e], s);
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (lane == r && p0 + r < len && lse != -INFINITY && row_of[r] >= 0)
                    sum += exp2f((s * a.scale - lse) * kCwLog2e);
            }
        }
        if (lane < kCwTile) part[warp][lane] = sum;
        __syncthreads();
        if (threadIdx.x < kCwTile && p0 + threadIdx.x < seen) {
            const int64_t at = b * width + p0 + threadIdx.x;
            float total = a.decay != 0.f ? a.decay * a.earlier[at] : 0.f;
            for (int w = 0; w < kCwWarps; ++w) total += part[w][threadIdx.x];
            a.weights[at] = total;
        }
    }
}

size_t weights_scratch_bytes(int, int) { return 0; }

cudaError_t launch_cache_weights(const WeightsArgs& a, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return e;
    cache_weights_kernel<<<152 * 6, kCwThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

}  // namespace smla
