// k_cache_write.cu -- rows into the paged 8-bit cache.
//
// For each scale block that the new rows touch: amax over the block's new
// finite values, e = the least integer >= -100 with amax <= 448 * 2^e, scale =
// 2^e (or the block's present scale where earlier rows of the sequence are in
// it and it is larger), codes = rne_e4m3(x / scale). A power of two makes x /
// scale exact, so each code is the e4m3 value nearest to the bf16 input, and a
// growing scale moves earlier codes by whole exponents (exact but for e4m3
// subnormals).
//
// Bound: HBM. A row is read once (1 KB) and its codes written once (512 B); a
// CTA holds its whole block (at most 64 rows) in registers between the
// maximum and the conversion.
#include <cuda_fp8.h>

#include "smla_internal.cuh"

namespace smla {

namespace {

// bf16 pair -> two e4m3 codes of x * inv (inv a power of two) or x / scale.
__device__ __forceinline__ uint32_t encode2(uint32_t v, float inv, float scale, bool exact) {
    float a = bf16_lo(v), b = bf16_hi(v);
    a = exact ? a * inv : a / scale;
    b = exact ? b * inv : b / scale;
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Two codes in the low half of v, times ratio, rounded again.
__device__ __forceinline__ uint32_t recode2(uint32_t v, float ratio) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return __nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace

// One CTA per slot; slots are handed out so that no sum over sequences is
// needed: sequence b owns the slots from floor(cu[b] / kBlock) + 2b on, at least
// as many as the blocks its rows can touch (floor(n / kBlock) + 2).
template <int kBlock>
__global__ void __launch_bounds__(kBlock * 8)
cache_write_kernel(const CacheView c, const int32_t* __restrict__ table,
                   const int32_t* __restrict__ start, const int32_t* __restrict__ cu,
                   const uint4* __restrict__ rows, int B, int max_pages, int n_rows,
                   unsigned* status) {
    constexpr int kWarps = kBlock / 4;
    __shared__ uint32_t warp_max[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t slot = blockIdx.x;
    // the last b with cu[b] / kBlock + 2b <= slot, 32 probes at a time: a halving search is a
    // chain of loads, and a call for one token a sequence is little else
    int b = 0, above = B;
    while (above - b > 1) {
        const int step = (above - b + 31) / 32, mid = b + lane * step;
        const bool yes = mid < above &&
                         (lane == 0 || int64_t(__ldg(cu + mid) / kBlock) + 2 * int64_t(mid) <= slot);
        b += (__popc(__ballot_sync(0xffffffffu, yes)) - 1) * step;
        above = min(above, b + step);
    }
    const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1), st = __ldg(start + b);
    const int64_t j = slot - (int64_t(c0 / kBlock) + 2 * int64_t(b));
    if (c0 < 0 || c1 < c0 || c1 > n_rows || (c1 > c0 && st < 0) || j < 0) {
        if (threadIdx.x == 0) flag_status(status, SMLA_ERR_INDEX);
        return;
    }
    const int64_t p0 = (int64_t(st) / kBlock + j) * kBlock;          // first position of the block
    const int64_t end = int64_t(st) + (c1 - c0);
    const int lo = int(p0 < st ? st - p0 : 0);
    const int hi = int(end - p0 < kBlock ? end - p0 : kBlock);       // new rows: [lo, hi) of the block
    if (hi <= lo) return;
    const int64_t pslot = p0 >> c.page_shift;
    const int page = pslot < max_pages ? __ldg(table + int64_t(b) * max_pages + pslot) : -1;
    const uint4* src = rows + (int64_t(c0) + (p0 - st)) * (kD / 8);  // row 0 of the block

    uint4 v[4][2];                               // (on their way while the page is looked up)
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp + i * kWarps;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[i][k] = r >= lo && r < hi ? __ldcs(src + int64_t(r) * (kD / 8) + 32 * k + lane)
                                        : make_uint4(0, 0, 0, 0);
    }
    if (page < 0 || page >= c.num_pages) {
        if (threadIdx.x == 0) flag_status(status, SMLA_ERR_INDEX);
        return;
    }
    const int64_t row0 = (int64_t(page) << c.page_shift) + (p0 & ((1 << c.page_shift) - 1));
    float* scale_at = c.scales + (row0 >> c.block_shift);
    const float old = lo > 0 ? *scale_at : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[e] & 0x7fff7fffu;
                top = __vmaxu2(top, a & __vcmpltu2(a, 0x7f807f80u));     // finite values only
            }
        }
    top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, warp_max[w]);
    // top holds the bf16 bits of amax: 448 = 1.75 * 2^8
    int e = int(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    if (e < -100) e = -100;
    float scale = __int_as_float((e + 127) << 23), inv = __int_as_float((127 - e) << 23);
    bool exact = true;
    if (lo > 0) {
        const bool keep = old >= scale;
        if (keep) {
            scale = old;
            const uint32_t bits = __float_as_uint(old);
            exact = (bits & 0x7fffffu) == 0 && bits < (252u << 23);
            inv = exact ? __uint_as_float((254u << 23) - bits) : 0.f;
        } else {
            const float ratio = old / scale;
            for (int r = warp; r < lo; r += kWarps) {
                uint4* at = reinterpret_cast<uint4*>(c.pages + (row0 + r) * kD) + lane;
                uint4 x = *at;
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = recode2(w[q], ratio) | recode2(w[q] >> 16, ratio) << 16;
                *at = x;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp + i * kWarps;
        if (r < lo || r >= hi) continue;
        uint2* dst = reinterpret_cast<uint2*>(c.pages + (row0 + r) * kD) + lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint2 w;
            w.x = encode2(v[i][k].x, inv, scale, exact) | encode2(v[i][k].y, inv, scale, exact) << 16;
            w.y = encode2(v[i][k].z, inv, scale, exact) | encode2(v[i][k].w, inv, scale, exact) << 16;
            dst[32 * k] = w;
        }
    }
    if (threadIdx.x == 0) *scale_at = scale;
}

cudaError_t launch_cache_write(const CacheView& c, const int32_t* table, const int32_t* start,
                               const int32_t* cu, const uint16_t* rows, int B, int max_pages,
                               int n_rows, unsigned* status, cudaStream_t s) {
    const int block = 1 << c.block_shift;
    const unsigned grid = unsigned(n_rows / block) + 2u * unsigned(B);
    const uint4* r = reinterpret_cast<const uint4*>(rows);
    if (block == 16)
        cache_write_kernel<16><<<grid, 128, 0, s>>>(c, table, start, cu, r, B, max_pages, n_rows, status);
    else if (block == 32)
        cache_write_kernel<32><<<grid, 256, 0, s>>>(c, table, start, cu, r, B, max_pages, n_rows, status);
    else
        cache_write_kernel<64><<<grid, 512, 0, s>>>(c, table, start, cu, r, B, max_pages, n_rows, status);
    note_launch();
    return cudaGetLastError();
}

}  // namespace smla
