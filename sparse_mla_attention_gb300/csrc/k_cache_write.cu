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
// Bound: HBM. A row is read once (1 KB) and its codes written once (512 B). The
// CTAs stay on the SMs and take block after block: a bulk copy brings the next
// one to shared memory while the one at hand, in registers since its maximum was
// taken, is converted and stored. 78,000 rows of 24 prompts (64-row blocks): 25.4 us, 4.7
// TB/s of reads and writes (one block a CTA, loaded to registers, and the status word
// cleared by a launch of its own: 29 us). One row for each of 128 sequences: 5.3 us (8.3),
// the latency of a launch and of five loads in a row. CTA 0's look at every slot is hidden only
// while the slots are few: 619,000 rows take 172 us in blocks of 64, 169 in blocks of 32 and 330 in
// blocks of 16, where it is the bound.
#include <cuda_fp8.h>

#include "smla_internal.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr uint64_t kWriteWaitNs = 2000000000u;

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

// The new rows [lo, hi) of a scale block: its first position, the row of `rows` that would be the
// block's first, the sequence. hi 0: none.
struct Piece {
    int lo, hi, b;
    int64_t p0, row0;
};

// Sequences own slots, so that none has to sum over the others: sequence b those from
// floor(cu[b] / kBlock) + 2b on, at least as many as the blocks its rows can touch
// (floor(n / kBlock) + 2).
template <int kBlock>
__device__ __forceinline__ int64_t first_slot(const int32_t* cu, int b) {
    return int64_t(__ldg(cu + b) / kBlock) + 2 * int64_t(b);
}

// What slot `slot` of sequence b is; *bad if the sequence's numbers are.
template <int kBlock>
__device__ __forceinline__ Piece piece_of(const int32_t* start, const int32_t* cu, int b, int64_t slot, int n_rows,
                                          bool* bad) {
    const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1), st = __ldg(start + b);
    const int64_t j = slot - (int64_t(c0 / kBlock) + 2 * int64_t(b));
    *bad = c0 < 0 || c1 < c0 || c1 > n_rows || (c1 > c0 && st < 0);
    Piece x{0, 0, b, 0, 0};
    if (*bad || j < 0) return x;
    x.p0 = (int64_t(st) / kBlock + j) * kBlock;
    const int64_t end = int64_t(st) + (c1 - c0);
    x.lo = int(x.p0 < st ? st - x.p0 : 0);
    x.hi = int(end - x.p0 < kBlock ? end - x.p0 : kBlock);
    x.row0 = int64_t(c0) + (x.p0 - st);
    if (x.hi <= x.lo) x.hi = 0;
    return x;
}

// The page of a piece, -1 if there is none.
__device__ __forceinline__ int page_of(const CacheView& c, const int32_t* table, int max_pages, const Piece& x) {
    const int64_t at = x.p0 >> c.page_shift;
    const int page = at < max_pages ? __ldg(table + int64_t(x.b) * max_pages + at) : -1;
    return page >= 0 && page < c.num_pages ? page : -1;
}

}  // namespace

// CTA 0 looks at every sequence and slot and writes the call's status word, so that the
// call is one launch; the others take the slots in turn and leave out the bad ones.
template <int kBlock>
__global__ void __launch_bounds__(kBlock * 8, 128 / kBlock)
cache_write_kernel(const CacheView c, const int32_t* __restrict__ table,
                   const int32_t* __restrict__ start, const int32_t* __restrict__ cu,
                   const uint8_t* __restrict__ rows, int B, int max_pages, int n_rows, int64_t slots,
                   unsigned* status) {
    constexpr int kWarps = kBlock / 4, kThreads = kBlock * 8;
    extern __shared__ __align__(128) uint8_t stage[];        // kBlock rows
    __shared__ uint32_t warp_max[2][kWarps];
    __shared__ uint64_t full;
    __shared__ int late;                                     // a wait ran out
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad = false;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < B; b += kThreads) {
            bool x;
            piece_of<kBlock>(start, cu, b, 0, n_rows, &x);
            bad |= x;
        }
        for (int64_t slot = threadIdx.x; slot < slots; slot += kThreads) {
            int b = 0, above = B;
            while (above - b > 1) {
                const int mid = b + (above - b) / 2;
                if (first_slot<kBlock>(cu, mid) <= slot) b = mid; else above = mid;
            }
            bool x;
            const Piece at = piece_of<kBlock>(start, cu, b, slot, n_rows, &x);
            bad |= at.hi > 0 && page_of(c, table, max_pages, at) < 0;
        }
        const bool any = __syncthreads_or(bad) != 0;
        if (threadIdx.x == 0) *status = any ? 1u << SMLA_ERR_INDEX : 0u;
        return;
    }
    int64_t slot = int64_t(blockIdx.x) - 1;
    // this CTA's next slot that has rows
    auto next = [&]() {
        Piece x{0, 0, 0, 0, 0};
        for (; slot < slots && x.hi == 0; slot += gridDim.x - 1) {
            // the last b with first_slot(b) <= slot, 32 probes at a time: a halving search is a
            // chain of loads, and a call for one token a sequence is little else
            int b = 0, above = B;
            while (above - b > 1) {
                const int step = (above - b + 31) / 32, mid = b + lane * step;
                const bool yes = mid < above && (lane == 0 || first_slot<kBlock>(cu, mid) <= slot);
                b += (__popc(__ballot_sync(0xffffffffu, yes)) - 1) * step;
                above = min(above, b + step);
            }
            x = piece_of<kBlock>(start, cu, b, slot, n_rows, &bad);
        }
        return x;
    };
    auto load = [&](const Piece& x) {
        if (threadIdx.x != 0 || x.hi == 0) return;
        const uint32_t bytes = uint32_t(x.hi - x.lo) * (kD * 2);
        mbar_arrive_expect_tx(&full, bytes);
        bulk_load(stage + x.lo * (kD * 2), rows + (x.row0 + x.lo) * (kD * 2), bytes, &full);
    };
    if (threadIdx.x == 0) {
        late = 0;
        mbar_init(&full, 1);
        fence_mbar_init();
    }
    Piece cur = next();
    load(cur);
    __syncthreads();                             // (the barrier is made)
    for (uint32_t n = 0; cur.hi > 0; ++n) {
        const int lo = cur.lo, hi = cur.hi;
        const int page = page_of(c, table, max_pages, cur);
        const int64_t row0 = page < 0 ? 0 : (int64_t(page) << c.page_shift) + (cur.p0 & ((1 << c.page_shift) - 1));
        float* scale_at = c.scales + (row0 >> c.block_shift);
        const float old = lo > 0 ? *scale_at : 0.f;
        const Piece then = next();
        if (!mbar_wait(&full, n & 1u, kWriteWaitNs)) {
            flag_status(status, SMLA_ERR_TIMEOUT);           // (long after CTA 0 wrote the word)
            late = 1;
        }
        uint4 v[4][2];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = warp + i * kWarps;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                v[i][k] = r >= lo && r < hi
                              ? *reinterpret_cast<const uint4*>(stage + r * (kD * 2) + 512 * k + 16 * lane)
                              : make_uint4(0, 0, 0, 0);
        }
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
        if (lane == 0) warp_max[n & 1][warp] = top;
        __syncthreads();
        if (late) {                              // the copy in flight lands before the CTA's memory is another's
            if (threadIdx.x == 0) mbar_wait(&full, n & 1u, kWriteWaitNs / 8);
            return;
        }
        load(then);                              // all have their rows: the next block's may come
        cur = then;
        if (page < 0) continue;
        top = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = max(top, warp_max[n & 1][w]);
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
}

namespace {

template <int kBlock>
cudaError_t launch_write(const CacheView& c, const int32_t* table, const int32_t* start, const int32_t* cu,
                         const uint8_t* rows, int B, int max_pages, int n_rows, unsigned* status, cudaStream_t s) {
    constexpr int kBytes = kBlock * kD * 2, kPerSm = 128 / kBlock;
    static bool attr_done[64] = {false};
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    if (kBytes > 48 * 1024 && dev >= 0 && dev < 64 && !attr_done[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(cache_write_kernel<kBlock>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t slots = n_rows / kBlock + 2 * int64_t(B), most = int64_t(sms) * kPerSm;
    const unsigned grid = unsigned(slots + 1 < most ? slots + 1 : most);
    cache_write_kernel<kBlock><<<grid, kBlock * 8, kBytes, s>>>(c, table, start, cu, rows, B, max_pages, n_rows, slots,
                                                                status);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const int32_t* table, const int32_t* start,
                               const int32_t* cu, const uint16_t* rows, int B, int max_pages,
                               int n_rows, unsigned* status, cudaStream_t s) {
    const uint8_t* r = reinterpret_cast<const uint8_t*>(rows);
    switch (c.block_shift) {
        case 4: return launch_write<16>(c, table, start, cu, r, B, max_pages, n_rows, status, s);
        case 5: return launch_write<32>(c, table, start, cu, r, B, max_pages, n_rows, status, s);
        default: return launch_write<64>(c, table, start, cu, r, B, max_pages, n_rows, status, s);
    }
}

}  // namespace smla
