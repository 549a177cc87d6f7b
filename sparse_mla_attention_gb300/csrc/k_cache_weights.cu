// k_cache_weights.cu -- the attention weight that each cached position gets, on the tensor cores.
//
// For sequence b with the tokens t in [cu[b], cu[b+1]) and position p < lens[t] of any of them:
//   weights[b,p] = decay * earlier[b,p] + sum_t sum_h exp(scale * <q[t,h,:], x_p> - lse[t,h]) [p < lens[t]],
//   x_p = e4m3 code * block scale.
// It needs the final lse, so it cannot ride on the attention's own pass; the scores kept for it would take 2 H
// bytes a position, where reading the row again takes 512.
//
// S^T = X Q^T: M = 128 positions (a tile of the cache as it lies, kind::f8f6f4), N = rows of q, K = 512. A position is
// a lane of TMEM then, and the sum over tokens and heads a thread's own: no shuffles, no atomics, one order. A row of
// garbage (behind the end, without a page) stays in its lane, so whole pages are loaded and nothing is masked before
// the sum.
// q is split as in the attention: a row's power of two 2^e, hi = e4m3(q / 2^e), lo = e4m3(16 (q / 2^e - hi)), hi and
// lo as columns of one product. weights_q_kernel does that once a call and writes each chunk of up to 128 rows
// (token, head) as the very bytes that shared memory wants, with the factors of its columns.
//
// weights_kernel: persistent, one CTA an SM. The units (tile, chunk of a sequence's q) are dealt out in tiles; a
// CTA goes through its tiles once for each chunk, q staying, the cache streaming. Warps: 0-3 and 4-7 sums, on
// alternate tiles, 8 and 10 loads of the cache and of q, 9 products. Shared memory: q 128 KB (one chunk of 128 rows, or two of up to 64 rows in
// turn; reloaded in quarters of K as the last tile gets done with them), ring of 6 blocks of 128 rows x 128 bytes.
// TMEM: two buffers of 256 columns.
//
// Every mbarrier wait is bounded; a timeout sets SMLA_ERR_TIMEOUT, stops the CTA's loops, waits (bounded) for its own
// copies and MMAs and frees TMEM.
#include <cfloat>

#include <cuda_fp8.h>

#include "smla_internal.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace smla {
using namespace sm100;

namespace {

constexpr uint32_t kCwWaitNs = 2000000000u;
constexpr float kCwLog2e = 1.4426950408889634f;
constexpr int kCwTile = 128;                     // positions
constexpr int kCwRows = 128;                     // rows of q of a chunk at most
constexpr int kCwSlots = 6, kCwSlotBytes = kCwTile * 128;
constexpr int kCwQSlots = 8, kCwQSlotBytes = 16384;
constexpr int kCwLoadWarp = 8, kCwMmaWarp = 9, kCwQWarp = 10, kCwThreads = 352;
constexpr int kCwSplitThreads = 256;
constexpr int kCwMaxBlocks = 1024;               // of the splitting kernel

// Two floats at a time.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

struct CwShared {
    uint64_t full[kCwSlots], empty[kCwSlots];
    uint64_t q_full[kCwQSlots], q_empty[kCwQSlots];
    uint64_t f_full[2], f_empty[2];              // the factors of a chunk's columns
    uint64_t t_full[2], t_empty[2], drain;
    uint32_t tbase;
    volatile int abort_flag;
    int b0;                                      // first sequence with work of this CTA
    int64_t at0, lo, hi;                         // its first unit; the CTA's units
    int64_t sum[kCwThreads / 32];
};

constexpr int kCwQAt = kCwSlots * kCwSlotBytes;
constexpr int kCwFactorAt = kCwQAt + kCwQSlots * kCwQSlotBytes;
constexpr int kCwSharedAt = kCwFactorAt + 2 * kCwRows * int(sizeof(float2));
constexpr int kCwSmem = kCwSharedAt + int(sizeof(CwShared));
static_assert(kCwSmem <= 232448, "shared memory of one CTA is at most 227 KB");

struct CwParams {
    WeightsArgs a;
    uint8_t* image;                              // [T * H] rows of q as shared memory has them, 1 KB each
    float* factor;                               // [2][T * H] score factor, -lse in log2 units
    unsigned* bits;                              // status bits of each block of the splitting kernel
    int blocks;
};

__device__ __forceinline__ bool cw_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint32_t t0 = globaltimer_lo_ns();
        do {
#pragma unroll 1
            for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
            if (!ok && globaltimer_lo_ns() - t0 > kCwWaitNs) {
                *abort_flag = 1;
                flag_status(status, SMLA_ERR_TIMEOUT);
            }
        } while (!ok && !*abort_flag);
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ int cw_len(const WeightsArgs& a, int t) {
    const int64_t limit = int64_t(a.max_pages) << a.cache.page_shift;
    const int len = __ldg(a.lens + t);
    return len < 0 ? 0 : len > limit ? int(limit) : len;
}

// Sequence b's tokens; false if its entries of cu are out of order or range.
__device__ __forceinline__ bool cw_tokens(const WeightsArgs& a, int b, int& c0, int& c1) {
    c0 = b < a.T ? b : a.T;
    c1 = b < a.T ? b + 1 : a.T;
    if (!a.cu) return true;
    c0 = __ldg(a.cu + b);
    c1 = __ldg(a.cu + b + 1);
    return c0 >= 0 && c1 >= c0 && c1 <= a.T;
}

// Rows of a sequence's chunks (but for the last): up to 64 rows are one chunk and need half of the room.
__device__ __forceinline__ int cw_chunk_rows(int rows) { return rows <= kCwRows / 2 ? rows : kCwRows; }

__device__ __forceinline__ uint32_t cw_e4m3x2(__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 cw_e4m3x2_half(uint32_t v) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v), __NV_E4M3));
}

// Positions that some token of a sequence sees (0: nothing to do). The whole warp asks for one sequence.
__device__ __forceinline__ int cw_seen(const WeightsArgs& a, int c0, int c1) {
    int most = 0;
#pragma unroll 4
    for (int t = c0 + int(threadIdx.x & 31); t < c1; t += 32) most = max(most, cw_len(a, t));
    return __reduce_max_sync(0xffffffffu, most);
}

struct CwSize {
    int tiles, chunk_rows, chunks;
    __device__ __forceinline__ CwSize(int seen, int rows)
        : tiles((seen + kCwTile - 1) / kCwTile), chunk_rows(cw_chunk_rows(rows)),
          chunks(rows > 0 ? (rows + chunk_rows - 1) / chunk_rows : 0) {}
    __device__ __forceinline__ int64_t units() const { return int64_t(tiles) * chunks; }
};

// Where a CTA's work lies: items (sequence b, its tiles [k0, k1)), all chunks of each. A warp walks together.
struct CwWalk {
    int b, c0, c1, seen, k0, k1;
    int rows, chunk_rows, chunks;
    int64_t at, units, lo, hi;
    __device__ __forceinline__ CwWalk(const CwShared& sh) : b(sh.b0 - 1), at(sh.at0), units(0), lo(sh.lo), hi(sh.hi) {}
    __device__ __forceinline__ bool next(const CwParams& p) {
        do {
            at += units;
            units = 0;
            k0 = k1 = 0;
            ++b;
            if (at >= hi || b >= p.a.B) return false;
            if (!cw_tokens(p.a, b, c0, c1) || c0 == c1) continue;
            seen = cw_seen(p.a, c0, c1);
            rows = (c1 - c0) * p.a.H;
            const CwSize n(seen, rows);
            chunk_rows = n.chunk_rows;
            chunks = n.chunks;
            units = n.units();
            // tile k is whose the unit at + k * chunks is
            k0 = at >= lo ? 0 : int(min(int64_t(n.tiles), (lo - at + chunks - 1) / chunks));
            k1 = int(min(int64_t(n.tiles), (hi - at + chunks - 1) / chunks));
        } while (k0 >= k1);
        return true;
    }
    __device__ __forceinline__ int chunk_size(int j) const {
        const int left = rows - j * chunk_rows;
        return left < chunk_rows ? left : chunk_rows;
    }
};

// Units of sequence b; the whole warp asks.
__device__ __forceinline__ int64_t cw_units(const CwParams& p, int b) {
    int c0, c1;
    if (!cw_tokens(p.a, b, c0, c1) || c0 == c1) return 0;
    return CwSize(cw_seen(p.a, c0, c1), (c1 - c0) * p.a.H).units();
}

// The CTA's share of the units and the sequence that it begins in.
__device__ void cw_locate(const CwParams& p, CwShared& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (p.a.B + kCwThreads - 1) / kCwThreads;
    const int b0 = int(min(int64_t(threadIdx.x) * run, int64_t(p.a.B))), b1 = min(b0 + run, p.a.B);
    int64_t mine = 0;
    for (int i = 0; i < run; ++i) {
        // a lane its own sequence if that has one token, the warp together one after the other that have more
        const int b = b0 + i;
        int c0 = 0, c1 = 0;
        const bool live = b < b1 && cw_tokens(p.a, b, c0, c1) && c1 > c0;
        int seen = live && c1 == c0 + 1 ? cw_len(p.a, c0) : 0;
        for (unsigned more = __ballot_sync(0xffffffffu, live && c1 > c0 + 1); more; more &= more - 1) {
            const int l = __ffs(more) - 1;
            const int most = cw_seen(p.a, __shfl_sync(0xffffffffu, c0, l), __shfl_sync(0xffffffffu, c1, l));
            if (lane == l) seen = most;
        }
        if (live) mine += CwSize(seen, (c1 - c0) * p.a.H).units();
    }
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh.sum[warp] = x;
    if (threadIdx.x == 0) sh.b0 = p.a.B;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kCwThreads / 32; ++w) {
        if (w < warp) before += sh.sum[w];
        total += sh.sum[w];
    }
    int64_t at = before + x - mine;
    const int64_t per = total / gridDim.x, rem = total - per * gridDim.x, c = blockIdx.x;
    const int64_t lo = per * c + min(c, rem), hi = lo + per + (c < rem ? 1 : 0);
    if (threadIdx.x == 0) { sh.lo = lo; sh.hi = hi; }
    const unsigned finder = __ballot_sync(0xffffffffu, lo < hi && at <= lo && lo < at + mine);
    if (finder) {
        int b = __shfl_sync(0xffffffffu, b0, __ffs(finder) - 1);
        at = __shfl_sync(0xffffffffu, at, __ffs(finder) - 1);
        for (int64_t n = cw_units(p, b); lo >= at + n; n = cw_units(p, b)) {
            at += n;
            ++b;
        }
        if (lane == 0) { sh.b0 = b; sh.at0 = at; }
    }
}

}  // namespace

// q into parts. The other kernel's blocks start when what ran before this one is complete and wait for its end before
// they look at its results; what the caller gave them (cache, table, lengths) they may read at once.
__global__ void __launch_bounds__(kCwSplitThreads)
weights_q_kernel(const CwParams p) {
    const WeightsArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t warps = int64_t(gridDim.x) * (kCwSplitThreads / 32);
    const int64_t first = int64_t(blockIdx.x) * (kCwSplitThreads / 32) + (threadIdx.x >> 5);
    const int64_t limit = int64_t(a.max_pages) << a.cache.page_shift;
    bool bad = false;
    for (int64_t g = first; g < int64_t(a.T) * a.H; g += warps) {
        const int t = int(g / a.H);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + g * kD) + 2 * lane;
        const uint4 x0 = __ldg(src), x1 = __ldg(src + 1);
        const float lse = __ldg(a.lse + g);
        int b = t;
        if (a.cu) {
            // the last b with cu[b] <= t, 32 probes at a time
            b = 0;
            for (int above = a.B; above - b > 1;) {
                const int step = (above - b + 31) / 32, mid = b + lane * step;
                const bool yes = mid < above && (lane == 0 || __ldg(a.cu + mid) <= t);
                b += (__popc(__ballot_sync(0xffffffffu, yes)) - 1) * step;
                above = min(above, b + step);
            }
        }
        int c0, c1;
        if (!cw_tokens(a, b, c0, c1) || t < c0 || t >= c1) continue;
        uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
        // the least 2^e with top <= 448 * 2^e (448 = 1.75 * 2^8)
        int e = int(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
        const bool odd = top >= 0x7f80u, blind = lse == -INFINITY;
        e = odd || top == 0 ? 0 : e < -100 ? -100 : e;           // (120 at most)
        const float inv = __int_as_float((127 - e) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (odd || blind) w[i] = 0;
            // half precision holds a scaled value and what e4m3 leaves of it exactly
            const __half2 v = __floats2half2_rn(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
            const uint32_t h = cw_e4m3x2(v);
            const uint32_t l = cw_e4m3x2(__hmul2(__hsub2(v, cw_e4m3x2_half(h)), __float2half2_rn(16.f)));
            if (i & 1) { hi[i >> 1] |= h << 16; lo[i >> 1] |= l << 16; } else { hi[i >> 1] = h; lo[i >> 1] = l; }
        }
        const int rows = (c1 - c0) * a.H, per = cw_chunk_rows(rows);
        const int64_t g0 = int64_t(c0) * a.H;
        const int l = int((g - g0) % per), left = rows - (int(g - g0) - l), r = left < per ? left : per;
        // K block (8 lanes each), rows hi then rows lo, 16-byte pieces swizzled
        uint8_t* at = p.image + (g - l) * 1024 + (lane >> 3) * (r * 256);
        *reinterpret_cast<uint4*>(at + l * 128 + (((lane & 7) ^ (l & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + (r + l) * 128 + (((lane & 7) ^ (l & 7)) << 4)) =
            make_uint4(lo[0], lo[1], lo[2], lo[3]);                // (r is a multiple of 16)
        if (lane == 0) {
            p.factor[g] = odd && !blind ? __int_as_float(0x7fffffff)
                                        : fminf(__int_as_float((127 + e) << 23) * a.scale * kCwLog2e, FLT_MAX);
            p.factor[int64_t(a.T) * a.H + g] = blind ? -INFINITY : -lse * kCwLog2e;
        }
    }
    for (int64_t b = first; b < a.B; b += warps) {
        int c0, c1;
        const bool ok = cw_tokens(a, int(b), c0, c1);
        bad |= !ok;
        for (int t = c0 + lane; ok && t < c1; t += 32) {
            const int len = __ldg(a.lens + t);
            bad |= len < 0 || len > limit;
        }
    }
    bad = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0) {
        p.bits[blockIdx.x] = bad ? 1u << SMLA_ERR_INDEX : 0u;
        if (blockIdx.x == 0) *a.status = 0;      // the other kernel adds to it
    }
}

__global__ void __launch_bounds__(kCwThreads, 1)
weights_kernel(const __grid_constant__ CUtensorMap map_box, const CwParams p) {
    extern __shared__ __align__(1024) uint8_t ring[];
    CwShared& sh = *reinterpret_cast<CwShared*>(ring + kCwSharedAt);
    uint8_t* qbuf = ring + kCwQAt;
    float* factors = reinterpret_cast<float*>(ring + kCwFactorAt);
    const WeightsArgs& a = p.a;
    const CacheView& c = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* ab = &sh.abort_flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kCwSlots; ++i) { mbar_init(&sh.full[i], 1); mbar_init(&sh.empty[i], 1); }
        for (int i = 0; i < kCwQSlots; ++i) { mbar_init(&sh.q_full[i], 1); mbar_init(&sh.q_empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.f_full[i], 1);
            mbar_init(&sh.f_empty[i], 8);
            mbar_init(&sh.t_full[i], 1);
            mbar_init(&sh.t_empty[i], 8);        // both teams see every phase
        }
        mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCwMmaWarp) { tmem_alloc(&sh.tbase, 512); tmem_relinquish(); }
    cw_locate(p, sh);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tbase;
    const int page_mask = (1 << c.page_shift) - 1;
    const int box_rows = page_mask + 1 < kCwTile ? page_mask + 1 : kCwTile;
    CwWalk w(sh);

    if (warp == kCwLoadWarp) {
        // ------------------------------------------------------- loads of the cache
        uint32_t use = 0;
        bool ok = true;
        const int boxes = kCwTile / box_rows;
        while (ok && w.next(p)) {
            // lane's page of a tile: of the rows [lane * box_rows, ...)
            auto row_of = [&](int k) {
                const int64_t pos = int64_t(k) * kCwTile + lane * box_rows;
                if (lane >= boxes || pos >= w.seen) return -1;
                const int page = __ldg(a.table + int64_t(w.b) * a.max_pages + (pos >> c.page_shift));
                return page >= 0 && page < c.num_pages ? (page << c.page_shift) + int(pos & page_mask) : -1;
            };
            int row = row_of(w.k0);
            for (int j = 0; j < w.chunks && ok; ++j)
                for (int k = w.k0; k < w.k1 && ok; ++k) {
                    const int next_row = row_of(k + 1 < w.k1 ? k + 1 : w.k0);
                    const int live = __popc(__ballot_sync(0xffffffffu, row >= 0));
#pragma unroll 1
                    for (int kb = 0; kb < 4; ++kb) {
                        const int slot = int(use % kCwSlots);
                        ok = cw_wait(&sh.empty[slot], ((use / kCwSlots) & 1u) ^ 1u, ab, a.status);
                        if (!ok) break;
                        ++use;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], uint32_t(live * box_rows) * 128);
                        __syncwarp();
                        if (row >= 0)
                            tma_load_2d(ring + slot * kCwSlotBytes + lane * box_rows * 128, &map_box, kb * 128, row,
                                        &sh.full[slot]);
                        __syncwarp();
                    }
                    row = next_row;
                }
        }
        __syncwarp();
        if (sh.abort_flag)                       // the loads already issued land before the CTA exits
            for (uint32_t n = use > kCwSlots ? use - kCwSlots : 0; n < use; ++n)
                mbar_wait(&sh.full[n % kCwSlots], (n / kCwSlots) & 1u, kCwWaitNs / 8);
        __syncwarp();
    } else if (warp == kCwQWarp) {
        // ------------------------------------------------------- loads of q and its factors
        uint32_t q_uses = 0, f_uses = 0;         // q_uses: a parity bit a slot
        int half = 0;
        bool ok = true;
        grid_dep_wait();                         // the splitting kernel is complete
        if (blockIdx.x == 0) {
            unsigned bits = 0;
            for (int i = lane; i < p.blocks; i += 32) bits |= __ldcg(p.bits + i);
            if (bits) atomicOr(a.status, bits);
            __syncwarp();
        }
        while (ok && w.next(p)) {
            for (int j = 0; j < w.chunks && ok; ++j) {
                const int r = w.chunk_size(j), f = f_uses & 1;
                const int64_t g = (int64_t(w.c0) * a.H) + int64_t(j) * w.chunk_rows;
                const bool big = r > kCwRows / 2;
                ok = cw_wait(&sh.f_empty[f], ((f_uses >> 1) & 1u) ^ 1u, ab, a.status);
                if (!ok) break;
                ++f_uses;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.f_full[f], uint32_t(r) * 8);
                    bulk_load(factors + 2 * f * kCwRows, p.factor + g, uint32_t(r) * 4, &sh.f_full[f]);
                    bulk_load(factors + (2 * f + 1) * kCwRows, p.factor + int64_t(a.T) * a.H + g, uint32_t(r) * 4,
                              &sh.f_full[f]);
                }
#pragma unroll 1
                for (int kb = 0; kb < 4; ++kb) {
                    // a quarter of K: slots 2 kb and the next, or slot kb of a half
                    const int s = big ? 2 * kb : 4 * half + kb;
                    ok = cw_wait(&sh.q_empty[s], ((q_uses >> s) & 1u) ^ 1u, ab, a.status);
                    if (ok && big) ok = cw_wait(&sh.q_empty[s + 1], ((q_uses >> (s + 1)) & 1u) ^ 1u, ab, a.status);
                    if (!ok) break;
                    q_uses ^= (big ? 3u : 1u) << s;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sh.q_full[s], uint32_t(r) * 256);
                        bulk_load(qbuf + s * kCwQSlotBytes, p.image + g * 1024 + kb * (r * 256), uint32_t(r) * 256,
                                  &sh.q_full[s]);
                        if (big) mbar_arrive(&sh.q_full[s + 1]);
                    }
                    __syncwarp();
                }
                if (!big) half ^= 1;
            }
        }
        __syncwarp();
        if (sh.abort_flag) {                     // the loads already issued land before the CTA exits
            for (int i = 0; i < kCwQSlots; ++i) mbar_wait(&sh.q_full[i], ((q_uses >> i) & 1u) ^ 1u, kCwWaitNs / 8);
            for (uint32_t n = f_uses > 2 ? f_uses - 2 : 0; n < f_uses; ++n)
                mbar_wait(&sh.f_full[n & 1], (n >> 1) & 1u, kCwWaitNs / 8);
        }
        __syncwarp();
    } else if (warp == kCwMmaWarp) {
        // ------------------------------------------------------------ products
        const uint64_t ring_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t q_desc = sdesc_sw128(smem_u32(qbuf), 16, 1024);
        const bool leader = elect_one();
        uint32_t use = 0, q_uses = 0, tile = 0;
        int half = 0;
        bool ok = true;
        while (ok && w.next(p)) {
            for (int j = 0; j < w.chunks && ok; ++j) {
                const int r = w.chunk_size(j);
                const bool big = r > kCwRows / 2;
                const uint32_t idesc = idesc_f8(128, 2 * r, false, false);
                const uint32_t q_next = q_uses ^ (big ? 0xffu : 0xfu << (4 * half));
                for (int k = w.k0; k < w.k1 && ok; ++k) {
                    const int buf = tile & 1;
                    ok = cw_wait(&sh.t_empty[buf], ((tile >> 1) & 1u) ^ 1u, ab, a.status);
                    ++tile;
#pragma unroll 1
                    for (int kb = 0; kb < 4 && ok; ++kb) {
                        const int s = big ? 2 * kb : 4 * half + kb;
                        if (k == w.k0) {
                            ok = cw_wait(&sh.q_full[s], (q_uses >> s) & 1u, ab, a.status);
                            if (ok && big) ok = cw_wait(&sh.q_full[s + 1], (q_uses >> (s + 1)) & 1u, ab, a.status);
                            if (!ok) break;
                        }
                        const int slot = int(use % kCwSlots);
                        ok = cw_wait(&sh.full[slot], (use / kCwSlots) & 1u, ab, a.status);
                        if (!ok) break;
                        ++use;
                        tc_fence_after();
                        const uint64_t xa = ring_desc + uint32_t(slot) * (kCwSlotBytes >> 4);
                        const uint64_t qa = q_desc + uint32_t(s) * (kCwQSlotBytes >> 4);
                        if (leader) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_f8_ss(tbase + 256 * buf, xa + 2 * i, qa + 2 * i, idesc, (kb | i) != 0);
                            mma_commit(&sh.empty[slot]);
                            if (k == w.k1 - 1) {
                                mma_commit(&sh.q_empty[s]);
                                if (big) mma_commit(&sh.q_empty[s + 1]);
                            }
                            if (kb == 3) mma_commit(&sh.t_full[buf]);
                        }
                        __syncwarp();
                    }
                }
                q_uses = q_next;
                if (!big) half ^= 1;
            }
        }
        if (leader) {
            mma_commit(&sh.drain);
            mbar_wait(&sh.drain, 0, kCwWaitNs);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- sums
        const int team = warp >> 2, quarter = warp & 3;
        const int64_t width = int64_t(a.max_pages) << c.page_shift;
        uint32_t f_uses = 0, tile = 0;
        bool ok = true, bad = false;
        while (ok && w.next(p)) {
            const int64_t line = w.b * width;
            // This thread's position of a tile: its page, two of the team's tiles ahead, its block scale (-1: none), one
            // ahead, so that no load is waited for.
            auto page_of = [&](int k) {
                const int64_t pos = int64_t(k) * kCwTile + 32 * quarter + lane;
                return k < w.k1 && pos < w.seen ? __ldg(a.table + int64_t(w.b) * a.max_pages + (pos >> c.page_shift)) : INT32_MAX;
            };
            auto scale_of = [&](int k, int page) {
                if (page < 0 || page >= c.num_pages) {
                    bad |= page != INT32_MAX;
                    return -1.f;
                }
                const int64_t pos = int64_t(k) * kCwTile + 32 * quarter + lane;
                return __ldg(c.scales + (((page << c.page_shift) + int(pos & page_mask)) >> c.block_shift));
            };
            const int k_first = w.k0 + team;
            auto after = [&](int k) { return k + 2 < w.k1 ? k + 2 : k_first; };
            float next_scale = scale_of(k_first, page_of(k_first));
            int next_page = page_of(after(k_first));
            for (int j = 0; j < w.chunks && ok; ++j) {
                const int r = w.chunk_size(j), f = f_uses & 1;
                // positions that every token of the chunk sees
                const int t0 = w.c0 + j * w.chunk_rows / a.H, t1 = w.c0 + (j * w.chunk_rows + r - 1) / a.H;
                int least = INT32_MAX;
                for (int t = t0 + lane; t <= t1; t += 32) least = min(least, cw_len(a, t));
                least = __reduce_min_sync(0xffffffffu, least);
                ok = cw_wait(&sh.f_full[f], (f_uses >> 1) & 1u, ab, a.status);
                if (!ok) break;
                ++f_uses;
                const float* fac = factors + 2 * f * kCwRows;
                // what the sum is added to: the chunks before, or the caller's
                const float* base = j > 0 ? a.weights : a.earlier;
                const float keep = j > 0 ? 1.f : a.decay;
                for (int k = w.k0; k < w.k1; ++k, ++tile) {
                    const int buf = tile & 1;
                    const bool own = ((k - w.k0) & 1) == team;
                    const int64_t pos = int64_t(k) * kCwTile + 32 * quarter + lane;
                    const float scale = next_scale;
                    float before = 0.f;
                    if (own) {
                        if (pos < w.seen && keep != 0.f) before = base[line + pos];
                        const int k_next = after(k);
                        next_scale = scale_of(k_next, next_page);
                        next_page = page_of(after(k_next));
                    }
                    ok = cw_wait(&sh.t_full[buf], (tile >> 1) & 1u, ab, a.status);
                    if (!ok) break;
                    if (!own) {
                        if (lane == 0) mbar_arrive(&sh.t_empty[buf]);
                        continue;
                    }
                    tc_fence_after();
                    const uint32_t trow = tbase + 256 * buf + (uint32_t(quarter * 32) << 16);
                    const bool all = (k + 1) * int64_t(kCwTile) <= least;
                    const uint64_t scale2 = pair_of(scale, scale), sixteenth = pair_of(0.0625f, 0.0625f);
                    float sum = 0.f;
                    uint32_t hi[2][16], lo[2][16];
                    auto read = [&](int n, int b) {
                        tmem_ld16(trow + n, hi[b]);
                        tmem_ld16(trow + r + n, lo[b]);
                    };
                    auto add = [&](int n, int b) {           // two columns at a time
                        uint64_t part[2] = {0, 0};
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const ulonglong2 fx = *reinterpret_cast<const ulonglong2*>(fac + n + e);
                            const ulonglong2 fy = *reinterpret_cast<const ulonglong2*>(fac + kCwRows + n + e);
#pragma unroll
                            for (int d = 0; d < 4; d += 2) {
                                const uint64_t s = fma2(pair_of(lo[b][e + d], lo[b][e + d + 1]), sixteenth,
                                                        pair_of(hi[b][e + d], hi[b][e + d + 1]));
                                const float2 x = floats_of(fma2(mul2(s, scale2), d ? fx.y : fx.x, d ? fy.y : fy.x));
                                part[d >> 1] = add2(part[d >> 1], pair_of(ex2_approx(x.x), ex2_approx(x.y)));
                            }
                        }
                        const float2 both = floats_of(add2(part[0], part[1]));
                        // (tokens have multiples of 16 rows)
                        if (all || pos < cw_len(a, w.c0 + (j * w.chunk_rows + n) / a.H)) sum += both.x + both.y;
                    };
                    read(0, 0);
#pragma unroll 1
                    for (int n = 0; n < r; n += 32) {
                        tmem_wait_ld();
                        if (n + 16 < r) read(n + 16, 1);
                        add(n, 0);
                        if (n + 16 >= r) break;
                        tmem_wait_ld();
                        if (n + 32 < r) read(n + 32, 0);
                        add(n + 16, 1);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.t_empty[buf]);
                    if (pos < w.seen) a.weights[line + pos] = fmaf(before, keep, scale >= 0.f ? sum : 0.f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.f_empty[f]);
            }
        }
        if (bad) flag_status(a.status, SMLA_ERR_INDEX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kCwMmaWarp) tmem_dealloc(tbase, 512);
}

namespace {

struct CwPlan { size_t image, factor, bits, bytes; };

CwPlan plan_weights(int64_t T, int64_t H) {
    CwPlan x{};
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes > 0 ? bytes : 1, 256); return o; };
    x.image = take(size_t(T) * H * 1024);
    x.factor = take(size_t(T) * H * sizeof(float2));
    x.bits = take(size_t(kCwMaxBlocks) * 4);
    x.bytes = off;
    return x;
}

}  // namespace

size_t weights_scratch_bytes(int T, int H) { return plan_weights(T, H).bytes; }

cudaError_t launch_cache_weights(const WeightsArgs& a, cudaStream_t s) {
    static bool attr_done[64] = {false};
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCwSmem);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const CwPlan plan = plan_weights(a.T, a.H);
    const CacheView& c = a.cache;
    CUtensorMap mb;
    const uint32_t box = (1 << c.page_shift) < kCwTile ? uint32_t(1) << c.page_shift : uint32_t(kCwTile);
    if (!make_tmap_u8_rows(&mb, c.pages, uint64_t(c.num_pages) << c.page_shift, box)) return cudaErrorInvalidValue;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    CwParams p{};
    p.a = a;
    p.image = reinterpret_cast<uint8_t*>(a.scratch + plan.image);
    p.factor = reinterpret_cast<float*>(a.scratch + plan.factor);
    p.bits = reinterpret_cast<unsigned*>(a.scratch + plan.bits);
    const int64_t rows = int64_t(a.T) * a.H, most = rows > a.B ? rows : a.B;
    const int64_t blocks = (most + kCwSplitThreads / 32 - 1) / (kCwSplitThreads / 32);
    p.blocks = int(blocks < kCwMaxBlocks ? blocks : kCwMaxBlocks);
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.blocks);
    cfg.blockDim = dim3(kCwSplitThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, weights_q_kernel, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(kCwThreads);
    cfg.dynamicSmemBytes = kCwSmem;
    note_launch(2);
    return cudaLaunchKernelEx(&cfg, weights_kernel, mb, p);
}

}  // namespace smla
