// k_fwd_paged.cu -- attention over the paged 8-bit cache.
//
// For token t (sequence seq[t]) and head h, over the valid ranks r (positions
// below lens[t], all of them or the picks topk[t, :]):
//   s_r = scale * <q[t,h,:], x_r>, lse = log(exp(sink_h) + sum exp(s_r)),
//   o = sum_r exp(s_r - lse) * x_r,   x_r = e4m3 code * block scale.
//
// One CTA per token and group of 16 heads, one warp per head (lane l holds
// columns 16l .. 16l+15 of q and of o), rows of 32 ranks staged in shared
// memory as bytes; one pass with a running maximum and sum, all in fp32.
#include <cuda_fp8.h>

#include "smla_internal.cuh"

namespace smla {

namespace {

constexpr int kPgHeads = 16;
constexpr int kPgTile = 32;

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}

__device__ __forceinline__ void unpack16(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3x2_to_float2(w[i]), b = e4m3x2_to_float2(w[i] >> 16);
        x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
    }
}

}  // namespace

__global__ void __launch_bounds__(kPgHeads * 32) fwd_paged_kernel(const PagedArgs p) {
    __shared__ uint4 tile[kPgTile][kD / 16];
    __shared__ int64_t row_of[kPgTile];
    __shared__ float scale_of[kPgTile];
    const int t = blockIdx.x, h = blockIdx.y * kPgHeads + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const CacheView& c = p.cache;
    const int64_t limit = int64_t(p.max_pages) << c.page_shift;
    int len = __ldg(p.lens + t);
    if (len < 0 || len > limit) {
        if (threadIdx.x == 0) flag_status(p.status, SMLA_ERR_INDEX);
        len = len < 0 ? 0 : int(limit);
    }
    const int b = p.seq ? __ldg(p.seq + t) : t;
    if (b < 0 || b >= p.B) {
        if (threadIdx.x == 0) flag_status(p.status, SMLA_ERR_INDEX);
        len = 0;
    }
    const int ranks = p.topk ? (len > 0 ? p.K : 0) : len;
    float qf[16], acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    const uint4* qrow = reinterpret_cast<const uint4*>(p.q) + (int64_t(t) * p.H + h) * (kD / 8) + 2 * lane;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 v = __ldg(qrow + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) { qf[8 * k + 2 * e] = bf16_lo(w[e]); qf[8 * k + 2 * e + 1] = bf16_hi(w[e]); }
    }
    const float sink = p.sink ? __ldg(p.sink + h) : -INFINITY;
    float m = sink, l = p.sink ? 1.f : 0.f;
    for (int r0 = 0; r0 < ranks; r0 += kPgTile) {
        __syncthreads();
        if (threadIdx.x < kPgTile) {
            const int r = r0 + int(threadIdx.x);
            int pos = -1;
            if (r < ranks) {
                pos = p.topk ? __ldg(p.topk + int64_t(t) * p.K + r) : r;
                if (pos < -1 || pos >= len) { flag_status(p.status, SMLA_ERR_INDEX); pos = -1; }
            }
            int64_t row = -1;
            float sc = 0.f;
            if (pos >= 0) {
                const int page = __ldg(p.table + int64_t(b) * p.max_pages + (pos >> c.page_shift));
                if (page < 0 || page >= c.num_pages) {
                    flag_status(p.status, SMLA_ERR_INDEX);
                } else {
                    row = (int64_t(page) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
                    sc = __ldg(c.scales + (row >> c.block_shift));
                }
            }
            row_of[threadIdx.x] = row;
            scale_of[threadIdx.x] = sc;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kPgTile * (kD / 16); i += blockDim.x) {
            const int rr = i / (kD / 16), col = i % (kD / 16);
            const int64_t row = row_of[rr];
            tile[rr][col] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(c.pages + row * kD) + col)
                                     : make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        float my_s = -INFINITY;
        for (int rr = 0; rr < kPgTile; ++rr) {
            float x[16], part = 0.f;
            unpack16(tile[rr][lane], x);
#pragma unroll
            for (int k = 0; k < 16; ++k) part = fmaf(qf[k], x[k], part);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            if (lane == rr) my_s = part * scale_of[rr] * p.scale;
        }
        const bool valid = row_of[lane] >= 0;
        if (!valid) my_s = -INFINITY;
        float tmax = my_s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, off));
        const float m_new = fmaxf(m, tmax);
        if (!__any_sync(0xffffffffu, valid)) continue;
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float e = valid ? expf(my_s - base) : 0.f;
        const float corr = m == -INFINITY ? 0.f : expf(m - base);
        float sum = e;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * corr + sum;
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] *= corr;
        for (int rr = 0; rr < kPgTile; ++rr) {
            if (row_of[rr] < 0) continue;
            const float w = __shfl_sync(0xffffffffu, e, rr) * scale_of[rr];
            float x[16];
            unpack16(tile[rr][lane], x);
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[k] = fmaf(w, x[k], acc[k]);
        }
        m = m_new;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint4* orow = reinterpret_cast<uint4*>(p.o) + (int64_t(t) * p.H + h) * (kD / 8) + 2 * lane;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        orow[k] = make_uint4(pack_bf16x2(acc[8 * k] * inv, acc[8 * k + 1] * inv),
                             pack_bf16x2(acc[8 * k + 2] * inv, acc[8 * k + 3] * inv),
                             pack_bf16x2(acc[8 * k + 4] * inv, acc[8 * k + 5] * inv),
                             pack_bf16x2(acc[8 * k + 6] * inv, acc[8 * k + 7] * inv));
    if (lane == 0) p.lse[int64_t(t) * p.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t paged_scratch_bytes(int, int) { return 0; }

cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t s) {
    fwd_paged_kernel<<<dim3(a.T, a.H / kPgHeads), kPgHeads * 32, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}

}  // namespace smla
