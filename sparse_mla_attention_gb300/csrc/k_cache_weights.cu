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
// alternate tiles, 8 and 10 loads of the cache and of q, 9 products. Shared memory: q 128 KB (one chunk of 128 rows, or
// two of up to 64 rows in turn; reloaded in quarters of K as the last tile gets done with them), ring of 6 blocks of 128
// rows x 128 bytes. TMEM: two buffers of 256 columns.
// Many rows of q (kCwManyRows): streaming the cache once a chunk is bound by L2 (207 us where the other takes 132), so
// weights_resident_kernel keeps three tiles in TMEM and streams q; see there.
//
// Bound: HBM for few rows: 128 sequences of up to 5120 positions, 64 heads 53 us, 96 of up to 6001, 16 heads 44 us,
// 5.0 and 5.1 TB/s over all; from the first tile to the last (40 of the 53 us) 6.6 TB/s. The rest is the splitting
// kernel's start (2 us), the deal (2), look-ups and first loads (3 to 4) and the last tile's way out. More or fewer ring
// slots: 4 / 5 / 6 / 9 56.7 / 54.4 / 53.7 / - and 45.9 / 44.4 / 44.0 / 43.9 us; the same pages asked of L2 three tiles ahead: 58.8
// and 48.8. One token of 777 positions: 8 us. Many rows: the tensor core (78% busy): 4 prompts of up to 20000
// positions, 32 tokens, 128 heads 132 us, 1.62 PFLOP/s, of which the 8-bit products are twice as many.
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
constexpr int kCwMmaWarp2 = 11, kCwLThreads = 384;
// With the cache resident: rows of a chunk, chunks in flight, tiles of a pass.
constexpr int kCwLRows = 32, kCwLSlots = 4, kCwLQSlots = 4, kCwLTiles = 3;
constexpr int kCwLQBytes = kCwLRows * 1024;
constexpr uint32_t kCwLColS = 128 * kCwLTiles;   // TMEM: a tile 128 columns each, then two buffers
constexpr uint32_t kCwLCols = (512 - kCwLColS) / 2;
static_assert(2 * kCwLRows <= int(kCwLCols), "a product has a column for each row of q and part");
constexpr int kCwMaxCtas = 160;
constexpr int kCwSplitThreads = 256;
// Rows of q a sequence, on average, above which the cache is resident. Device time in us, streaming / resident (sequences
// x positions, heads, rows): 64 x 3000, 128, 192: 42.5 / 63.3, 386: 77.0 / 87.0, 768: 137 / 125; 16 x 4000, 64, 288: 30.9 /
// 30.3, 392: 37.2 / 34.6, 760: 59.8 / 49.6; 2 x 30000, 128, 448: 35.5 / 31.4, 1216: 79.0 / 50.6; 1 x 2000, 128, 4096: 125 /
// 24.6 (streaming, a tile's chunks are one CTA's).
// The rule sees the average alone, as cu is on the device. In a batch of single tokens and one sequence of many, that
// sequence's tiles, all chunks of each, stay on a few CTAs where the cache streams: 255 x 1 token and one of 512, 2000
// positions, 128 heads, 383 rows: 2166 / 337; 127 x 1 and one of 64, 3000, 128, 191: 300 / 133; 31 x 1 and one of 32, 20000,
// 128, 252: 184 / 236. Two calls, one for the single tokens and one for the many, are the way around it.
constexpr int kCwManyRows = 400;
constexpr int kCwMaxBlocks = 608;                // of the splitting kernel: four an SM leave room for the other's, which start meanwhile

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

// Where a CTA's work begins and ends.
struct CwPlace {
    int b0;                                      // first sequence with work of this CTA,
    int c0, c1, seen;                            // its tokens and what they see
    int64_t at0, lo, hi;                         // its first unit; the CTA's units
    int64_t per, rem;                            // of a CTA; the first rem have one more
    int64_t sum[kCwLThreads / 32];
};

struct CwShared {
    uint64_t full[kCwSlots], empty[kCwSlots];
    uint64_t q_full[kCwQSlots], q_empty[kCwQSlots];
    uint64_t f_full[2], f_empty[2];              // the factors of a chunk's columns
    uint64_t t_full[2], t_empty[2], drain;
    CwPlace at;
    uint32_t tbase;
    volatile int abort_flag;
};

constexpr int kCwQAt = kCwSlots * kCwSlotBytes;
constexpr int kCwFactorAt = kCwQAt + kCwQSlots * kCwQSlotBytes;
constexpr int kCwSharedAt = kCwFactorAt + 2 * kCwRows * int(sizeof(float2));
constexpr int kCwSmem = kCwSharedAt + int(sizeof(CwShared));
static_assert(kCwSmem <= 232448, "shared memory of one CTA is at most 227 KB");

struct CwParams {
    WeightsArgs a;
    uint8_t* image;                              // [T * H] rows of q as shared memory has them, 1 KB each
    float* factor;                               // [3][T * H] of a row: score factor, -lse in log2 units, lens (int bits)
    unsigned* bits;                              // status bits of each block of the splitting kernel
    int blocks;
    int resident;                                // which of the two kernels follows the splitting one
    // of the resident kernel's CTAs: sums of a pass whose chunks they have from one after the first on (0) or up to one
    // before the last (1); and, for the CTA with the last one, the pass: {sequence (-1: none), pass, CTA with the first}
    float* parts;                                // [CTAs][2][3][128]
    int4* meta;                                  // [CTAs]
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

// Rows of a sequence's chunks (but for the last). Where the cache streams, up to 64 rows are one chunk and need half of
// the room.
__device__ __forceinline__ int cw_chunk_rows(int rows, int resident) {
    return resident ? kCwLRows : rows <= kCwRows / 2 ? rows : kCwRows;
}

__device__ __forceinline__ uint32_t cw_e4m3x2(__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 cw_e4m3x2_half(uint32_t v) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v), __NV_E4M3));
}

// (The shuffles tell the compiler that a warp's lanes agree: descriptors stay in uniform registers.)
__device__ __forceinline__ int cw_same(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Positions that some token of a sequence sees (0: nothing to do). The whole warp asks for one sequence.
__device__ __forceinline__ int cw_seen(const WeightsArgs& a, int c0, int c1) {
    int most = 0;
#pragma unroll 4
    for (int t = c0 + int(threadIdx.x & 31); t < c1; t += 32) most = max(most, cw_len(a, t));
    return __reduce_max_sync(0xffffffffu, most);
}

// Sequence b's tokens and what they see, for a whole warp; the first one's are at hand. False: it has none.
__device__ __forceinline__ bool cw_look(const WeightsArgs& a, const CwPlace& place, int b, int& c0, int& c1, int& seen) {
    if (b == place.b0) {
        c0 = cw_same(place.c0);
        c1 = cw_same(place.c1);
        seen = cw_same(place.seen);
        return true;
    }
    if (!cw_tokens(a, b, c0, c1) || c0 == c1) return false;
    c0 = cw_same(c0);
    c1 = cw_same(c1);
    seen = cw_seen(a, c0, c1);
    return true;
}

struct CwSize {
    int tiles, chunk_rows, chunks;
    __device__ __forceinline__ CwSize(int seen, int rows, int resident)
        : tiles((seen + kCwTile - 1) / kCwTile), chunk_rows(cw_chunk_rows(rows, resident)),
          chunks(rows > 0 ? (rows + chunk_rows - 1) / chunk_rows : 0) {}
    // what is dealt out: (tile, chunk), or (three tiles, chunk) where the cache is resident
    __device__ __forceinline__ int64_t units(int resident) const {
        return int64_t(resident ? (tiles + kCwLTiles - 1) / kCwLTiles : tiles) * chunks;
    }
};

// The weights of 16 columns of a position, two at a time.
__device__ __forceinline__ float cw_sum16(const uint32_t (&hi)[16], const uint32_t (&lo)[16], uint64_t scale2,
                                          const float* fx, const float* fy) {
    const uint64_t sixteenth = pair_of(0.0625f, 0.0625f);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(fx + e), y = *reinterpret_cast<const ulonglong2*>(fy + e);
#pragma unroll
        for (int d = 0; d < 4; d += 2) {
            const uint64_t s = fma2(pair_of(lo[e + d], lo[e + d + 1]), sixteenth, pair_of(hi[e + d], hi[e + d + 1]));
            const float2 w = floats_of(fma2(mul2(s, scale2), d ? x.y : x.x, d ? y.y : y.x));
            part[d >> 1] = add2(part[d >> 1], pair_of(ex2_approx(w.x), ex2_approx(w.y)));
        }
    }
    const float2 both = floats_of(add2(part[0], part[1]));
    return both.x + both.y;
}

// Where a CTA's work lies: items (sequence b, its tiles [k0, k1)), all chunks of each. A warp walks together.
struct CwWalk {
    int b, c0, c1, seen, k0, k1;
    int rows, chunk_rows, chunks;
    int64_t at, units, lo, hi;
    const CwPlace* place;
    __device__ __forceinline__ CwWalk(const CwPlace& sh)
        : b(sh.b0 - 1), at(sh.at0), units(0), lo(sh.lo), hi(sh.hi), place(&sh) {}
    __device__ __forceinline__ bool next(const CwParams& p) {
        do {
            at += units;
            units = 0;
            k0 = k1 = 0;
            ++b;
            if (at >= hi || b >= p.a.B) return false;
            if (!cw_look(p.a, *place, b, c0, c1, seen)) continue;
            rows = (c1 - c0) * p.a.H;
            const CwSize n(seen, rows, p.resident);
            chunk_rows = n.chunk_rows;
            chunks = n.chunks;
            units = n.units(p.resident);
            // tile k is whose the unit at + k * chunks is
            k0 = cw_same(at >= lo ? 0 : int(min(int64_t(n.tiles), (lo - at + chunks - 1) / chunks)));
            k1 = cw_same(int(min(int64_t(n.tiles), (hi - at + chunks - 1) / chunks)));
        } while (k0 >= k1);
        return true;
    }
    __device__ __forceinline__ int chunk_size(int j) const {
        const int left = rows - j * chunk_rows;
        return left < chunk_rows ? left : chunk_rows;
    }
};

// The resident kernel's work: items (sequence b, its units [u0, u1): three tiles from 3 (u / chunks) on, chunk u % chunks).
struct CwUnits {
    int b, c0, c1, seen, rows, tiles, chunks;
    int64_t at, units, lo, hi, u0, u1;
    const CwPlace* place;
    CwUnits() = default;
    __device__ __forceinline__ CwUnits(const CwPlace& sh)
        : b(sh.b0 - 1), at(sh.at0), units(0), lo(sh.lo), hi(sh.hi), place(&sh) {}
    __device__ __forceinline__ bool next(const CwParams& p) {
        do {
            at += units;
            units = u0 = u1 = 0;
            ++b;
            if (at >= hi || b >= p.a.B) return false;
            if (!cw_look(p.a, *place, b, c0, c1, seen)) continue;
            rows = (c1 - c0) * p.a.H;
            const CwSize n(seen, rows, 1);
            tiles = n.tiles;
            chunks = n.chunks;
            units = n.units(1);
            u0 = max(lo - at, int64_t(0));
            u1 = min(hi - at, units);
        } while (u0 >= u1);
        return true;
    }
    // the item's passes [first(), last()], a pass's tiles, and its chunks [from(k), to(k))
    __device__ __forceinline__ int first() const { return cw_same(int(u0 / chunks)); }
    __device__ __forceinline__ int last() const { return cw_same(int((u1 - 1) / chunks)); }
    __device__ __forceinline__ int width(int k) const { return cw_same(min(tiles - k * kCwLTiles, kCwLTiles)); }
    __device__ __forceinline__ int from(int k) const { return cw_same(int(max(u0 - int64_t(k) * chunks, int64_t(0)))); }
    __device__ __forceinline__ int to(int k) const { return cw_same(int(min(u1 - int64_t(k) * chunks, int64_t(chunks)))); }
    __device__ __forceinline__ int chunk_size(int j) const {
        const int left = rows - j * kCwLRows;
        return left < kCwLRows ? left : kCwLRows;
    }
};

struct CwLShared {
    uint64_t full[kCwLSlots], empty[kCwLSlots];
    uint64_t q_full[kCwLQSlots], q_empty[kCwLQSlots];
    uint64_t x_full;                             // the tiles of a pass are in TMEM
    uint64_t t_full[2], t_empty[2], drain[2];
    CwPlace at;
    uint32_t tbase;
    volatile int abort_flag;
    float sums[kCwLTiles][kCwTile];              // of the second team
    CwUnits item;                                // of the sums' warps
    int more;
};
constexpr int kCwLQAt = kCwLSlots * kCwSlotBytes;
constexpr int kCwLFactorAt = kCwLQAt + kCwLQSlots * kCwLQBytes;
constexpr int kCwLSharedAt = kCwLFactorAt + kCwLQSlots * 3 * kCwLRows * 4;
constexpr int kCwLSmem = kCwLSharedAt + int(sizeof(CwLShared));
static_assert(kCwLSmem <= 232448, "shared memory of one CTA is at most 227 KB");

// Units of sequence b; the whole warp asks.
__device__ __forceinline__ int64_t cw_units(const CwParams& p, int b) {
    int c0, c1;
    if (!cw_tokens(p.a, b, c0, c1) || c0 == c1) return 0;
    return CwSize(cw_seen(p.a, c0, c1), (c1 - c0) * p.a.H, p.resident).units(p.resident);
}

// The CTA that has a unit.
__device__ __forceinline__ int cw_owner(const CwPlace& sh, int64_t unit) {
    const int64_t longer = sh.rem * (sh.per + 1);
    return int(unit < longer ? unit / (sh.per + 1) : sh.rem + (unit - longer) / sh.per);
}

// The CTA's share of the units and the sequence that it begins in.
__device__ void cw_locate(const CwParams& p, CwPlace& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (p.a.B + int(blockDim.x) - 1) / int(blockDim.x);
    const int b0 = int(min(int64_t(threadIdx.x) * run, int64_t(p.a.B))), b1 = min(b0 + run, p.a.B);
    int64_t mine = 0;
    int c0 = 0, c1 = 0, seen = 0;                // of the last sequence looked at
    for (int i = 0; i < run; ++i) {
        // a lane its own sequence if that has one token, the warp together one after the other that have more
        const int b = b0 + i;
        const bool live = b < b1 && cw_tokens(p.a, b, c0, c1) && c1 > c0;
        seen = live && c1 == c0 + 1 ? cw_len(p.a, c0) : 0;
        for (unsigned more = __ballot_sync(0xffffffffu, live && c1 > c0 + 1); more; more &= more - 1) {
            const int l = __ffs(more) - 1;
            const int most = cw_seen(p.a, __shfl_sync(0xffffffffu, c0, l), __shfl_sync(0xffffffffu, c1, l));
            if (lane == l) seen = most;
        }
        if (live) mine += CwSize(seen, (c1 - c0) * p.a.H, p.resident).units(p.resident);
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
    for (int w = 0; w < int(blockDim.x) / 32; ++w) {
        if (w < warp) before += sh.sum[w];
        total += sh.sum[w];
    }
    int64_t at = before + x - mine;
    const int64_t per = total / gridDim.x, rem = total - per * gridDim.x, c = blockIdx.x;
    const int64_t lo = per * c + min(c, rem), hi = lo + per + (c < rem ? 1 : 0);
    if (threadIdx.x == 0) { sh.lo = lo; sh.hi = hi; sh.per = per; sh.rem = rem; }
    const unsigned finder = __ballot_sync(0xffffffffu, lo < hi && at <= lo && lo < at + mine);
    if (finder) {
        int b = __shfl_sync(0xffffffffu, b0, __ffs(finder) - 1);
        at = __shfl_sync(0xffffffffu, at, __ffs(finder) - 1);
        if (run > 1) {
            for (int64_t n = cw_units(p, b); lo >= at + n; n = cw_units(p, b)) {
                at += n;
                ++b;
            }
            cw_tokens(p.a, b, c0, c1);
            seen = cw_seen(p.a, c0, c1);
        }
        if (lane == __ffs(finder) - 1) { sh.b0 = b; sh.at0 = at; sh.c0 = c0; sh.c1 = c1; sh.seen = seen; }
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
        const int rows = (c1 - c0) * a.H, per = cw_chunk_rows(rows, p.resident);
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
            p.factor[2 * int64_t(a.T) * a.H + g] = __int_as_float(cw_len(a, t));
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
    cw_locate(p, sh.at);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = uint32_t(cw_same(int(sh.tbase)));
    const int page_mask = (1 << c.page_shift) - 1;
    const int box_rows = page_mask + 1 < kCwTile ? page_mask + 1 : kCwTile;
    CwWalk w(sh.at);
    uint32_t use = 0, q_uses = 0, f_uses = 0;    // of the ring, of q's slots (a parity bit each), of the factors

    if (warp == kCwLoadWarp) {
        // ------------------------------------------------------- loads of the cache
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
    } else if (warp == kCwQWarp) {
        // ------------------------------------------------------- loads of q and its factors
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
    } else if (warp == kCwMmaWarp) {
        // ------------------------------------------------------------ products
        const uint64_t ring_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t q_desc = sdesc_sw128(smem_u32(qbuf), 16, 1024);
        const bool leader = elect_one();
        uint32_t tile = 0;
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
        uint32_t tile = 0;
        bool ok = true, bad = false;
        while (ok && w.next(p)) {
            const int64_t line = w.b * width;
            // This thread's position of a tile: its page, two of the team's tiles ahead, its block scale and whether it
            // has a row, one ahead, so that no load is waited for.
            auto seen_in = [&](int k) { return k < w.k1 && int64_t(k) * kCwTile + 32 * quarter + lane < w.seen; };
            auto page_of = [&](int k) {
                const int64_t pos = int64_t(k) * kCwTile + 32 * quarter + lane;
                return seen_in(k) ? __ldg(a.table + int64_t(w.b) * a.max_pages + (pos >> c.page_shift)) : -1;
            };
            bool next_there = false;
            auto scale_of = [&](int k, int page) {
                next_there = page >= 0 && page < c.num_pages;            // (a page was looked up for positions that are seen)
                bad |= !next_there && seen_in(k);
                if (!next_there) return 0.f;
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
                const float* seen = p.factor + (2 * int64_t(a.T) + w.c0) * a.H + int64_t(j) * w.chunk_rows;
                // what the sum is added to: the chunks before, or the caller's
                const float* base = j > 0 ? a.weights : a.earlier;
                const float keep = j > 0 ? 1.f : a.decay;
                for (int k = w.k0; k < w.k1; ++k, ++tile) {
                    const int buf = tile & 1;
                    const bool own = ((k - w.k0) & 1) == team;
                    const int64_t pos = int64_t(k) * kCwTile + 32 * quarter + lane;
                    const float scale = next_scale;
                    const bool there = next_there;
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
                    const uint64_t scale2 = pair_of(scale, scale);
                    float sum = 0.f;
                    uint32_t hi[2][16], lo[2][16];
                    auto read = [&](int n, int b) {
                        tmem_ld16(trow + n, hi[b]);
                        tmem_ld16(trow + r + n, lo[b]);
                    };
                    auto add = [&](int n, int b) {
                        const float part = cw_sum16(hi[b], lo[b], scale2, fac + n, fac + kCwRows + n);
                        // (tokens have multiples of 16 rows)
                        if (all || pos < __float_as_int(__ldcg(seen + n))) sum += part;
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
                    if (pos < w.seen) a.weights[line + pos] = fmaf(before, keep, there ? sum : 0.f);
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
    // Whichever warp gave up a wait, all are out of their loops here: the loads already issued land before the CTA exits.
    if (sh.abort_flag && warp == kCwLoadWarp) {
        for (uint32_t n = use > kCwSlots ? use - kCwSlots : 0; n < use; ++n)
            mbar_wait(&sh.full[n % kCwSlots], (n / kCwSlots) & 1u, kCwWaitNs / 8);
    } else if (sh.abort_flag && warp == kCwQWarp) {
        for (int i = 0; i < kCwQSlots; ++i) mbar_wait(&sh.q_full[i], ((q_uses >> i) & 1u) ^ 1u, kCwWaitNs / 8);
        for (uint32_t n = f_uses > 2 ? f_uses - 2 : 0; n < f_uses; ++n)
            mbar_wait(&sh.f_full[n & 1], (n >> 1) & 1u, kCwWaitNs / 8);
    }
}

// The same with the cache resident, for sequences of many rows of q: passes of three tiles, which go from shared
// memory to TMEM (as A operands, 128 columns each) and stay there while the sequence's q streams past in chunks of
// 32 rows, one bulk copy each, four in flight. The units (three tiles, chunk) are dealt out one by one; a pass whose
// chunks several CTAs have is joined by weights_join_kernel. Warps as above, and 11 for products too; the teams take the
// products in turn (tiles within chunks), keep their sums of a pass in registers and join them at its end.
// Why so: with the cache as the streamed operand each product of 128 x 128 x 512 takes 64 KB from L2, 9 TB/s at the
// tensor core's rate over all SMs; with three tiles resident it takes 43. Three tiles and 64 columns twice fill TMEM. A
// as a TMEM operand leaves shared memory's rate to q (as a shared one with 64 columns it would need 1.5 times that rate).
// Products of 16 x (128 x 64 x 32) take 512 to 535 cycles, back to back within a chunk; one issuing warp left 250 to 400
// between them (224 us). Passes by tile, not by three: the CTAs with a fourth tile took 1.5 times as long (169 us).
__global__ void __launch_bounds__(kCwLThreads, 1)
weights_resident_kernel(const __grid_constant__ CUtensorMap map_box, const CwParams p) {
    extern __shared__ __align__(1024) uint8_t ring[];
    CwLShared& sh = *reinterpret_cast<CwLShared*>(ring + kCwLSharedAt);
    uint8_t* qbuf = ring + kCwLQAt;
    float* factors = reinterpret_cast<float*>(ring + kCwLFactorAt);
    const WeightsArgs& a = p.a;
    const CacheView& c = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* ab = &sh.abort_flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kCwLSlots; ++i) { mbar_init(&sh.full[i], 1); mbar_init(&sh.empty[i], 4); }
        // a chunk's slot is free when its products are done and both teams are done with its factors
        for (int i = 0; i < kCwLQSlots; ++i) { mbar_init(&sh.q_full[i], 1); mbar_init(&sh.q_empty[i], 10); }
        mbar_init(&sh.x_full, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.t_full[i], 1);
            mbar_init(&sh.t_empty[i], 4);
            mbar_init(&sh.drain[i], 1);
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCwMmaWarp) { tmem_alloc(&sh.tbase, 512); tmem_relinquish(); }
    cw_locate(p, sh.at);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = uint32_t(cw_same(int(sh.tbase)));
    const int page_mask = (1 << c.page_shift) - 1;
    const int box_rows = page_mask + 1 < kCwTile ? page_mask + 1 : kCwTile;
    CwUnits w(sh.at);
    uint32_t use = 0;                            // of the ring, or of q's slots

    if (warp == kCwLoadWarp) {
        // ------------------------------------------------------- loads of the cache
        bool ok = true;
        const int boxes = kCwTile / box_rows;
        while (ok && w.next(p)) {
            const int end = min((w.last() + 1) * kCwLTiles, w.tiles);
            for (int k = w.first() * kCwLTiles; k < end && ok; ++k) {
                const int64_t pos = int64_t(k) * kCwTile + lane * box_rows;
                int row = -1;
                if (lane < boxes && pos < w.seen) {
                    const int page = __ldg(a.table + int64_t(w.b) * a.max_pages + (pos >> c.page_shift));
                    if (page >= 0 && page < c.num_pages) row = (page << c.page_shift) + int(pos & page_mask);
                }
                const int live = __popc(__ballot_sync(0xffffffffu, row >= 0));
#pragma unroll 1
                for (int kb = 0; kb < 4; ++kb) {
                    const int slot = int(use % kCwLSlots);
                    ok = cw_wait(&sh.empty[slot], ((use / kCwLSlots) & 1u) ^ 1u, ab, a.status);
                    if (!ok) break;
                    ++use;
                    if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], uint32_t(live * box_rows) * 128);
                    __syncwarp();
                    if (row >= 0)
                        tma_load_2d(ring + slot * kCwSlotBytes + lane * box_rows * 128, &map_box, kb * 128, row,
                                    &sh.full[slot]);
                    __syncwarp();
                }
            }
        }
        __syncwarp();
    } else if (warp == kCwQWarp) {
        // ------------------------------------------------------- loads of q and its factors
        bool ok = true;
        grid_dep_wait();                         // the splitting kernel is complete
        if (blockIdx.x == 0) {
            unsigned bits = 0;
            for (int i = lane; i < p.blocks; i += 32) bits |= __ldcg(p.bits + i);
            if (bits) atomicOr(a.status, bits);
            __syncwarp();
        }
        while (ok && w.next(p)) {
            const int last = w.last();
            for (int k = w.first(); k <= last && ok; ++k) {
                const int j1 = w.to(k);
                for (int j = w.from(k); j < j1 && ok; ++j) {
                    const int r = w.chunk_size(j), slot = int(use % kCwLQSlots);
                    const int64_t g = (int64_t(w.c0) * a.H) + int64_t(j) * kCwLRows;
                    ok = cw_wait(&sh.q_empty[slot], ((use / kCwLQSlots) & 1u) ^ 1u, ab, a.status);
                    if (!ok) break;
                    ++use;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sh.q_full[slot], uint32_t(r) * 1036);
                        for (int i = 0; i < 3; ++i)
                            bulk_load(factors + (3 * slot + i) * kCwLRows, p.factor + i * int64_t(a.T) * a.H + g,
                                      uint32_t(r) * 4, &sh.q_full[slot]);
                        bulk_load(qbuf + slot * kCwLQBytes, p.image + g * 1024, uint32_t(r) * 1024, &sh.q_full[slot]);
                    }
                    __syncwarp();
                }
            }
        }
        __syncwarp();
    } else if (warp == kCwMmaWarp || warp == kCwMmaWarp2) {
        // ------------------------------------------------------------ products
        // Two warps take them in turn, a buffer each: one's waits and its way to the next product (some 250 cycles,
        // with the tensor core idle when there was one warp) pass while the other's are issued.
        const uint64_t q_desc = sdesc_sw128(smem_u32(qbuf), 16, 1024);
        const int buf = warp == kCwMmaWarp ? 0 : 1;
        const bool leader = elect_one();
        uint32_t tile = 0, pass = 0;
        bool ok = true;
        while (ok && w.next(p)) {
            const int last = w.last();
            for (int k = w.first(); k <= last && ok; ++k, ++pass) {
                const int n = w.width(k), j1 = w.to(k);
                ok = cw_wait(&sh.x_full, pass & 1u, ab, a.status);
                for (int j = w.from(k); j < j1 && ok; ++j) {
                    const int r = w.chunk_size(j), slot = int(use % kCwLQSlots);
                    const uint32_t idesc = idesc_f8(128, 2 * r, false, false);
                    ok = cw_wait(&sh.q_full[slot], (use / kCwLQSlots) & 1u, ab, a.status);
                    ++use;
#pragma unroll 1
                    for (int i = (int(tile) & 1) == buf ? 0 : 1; i < n && ok; i += 2) {
                        const uint32_t at = tile + i;
                        ok = cw_wait(&sh.t_empty[buf], ((at >> 1) & 1u) ^ 1u, ab, a.status);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            uint64_t qa = q_desc + uint32_t(slot) * (kCwLQBytes >> 4);
                            uint32_t xa = tbase + 128 * i;
#pragma unroll 1
                            for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    mma_f8_ts(tbase + kCwLColS + kCwLCols * buf, xa + 8 * d, qa + 2 * d, idesc, (kb | d) != 0);
                                qa += uint32_t(r * 256) >> 4;
                                xa += 32;
                            }
                            mma_commit(&sh.t_full[buf]);
                            if (i + 2 >= n) mma_commit(&sh.q_empty[slot]);       // this warp's last of the chunk
                        }
                        __syncwarp();
                    }
                    // (a chunk of one product is the other warp's alone)
                    if (leader && n == 1 && int(tile & 1) != buf) mbar_arrive(&sh.q_empty[slot]);
                    tile += n;
                    __syncwarp();
                }
            }
        }
        if (leader) {
            mma_commit(&sh.drain[buf]);
            mbar_wait(&sh.drain[buf], 0, kCwWaitNs);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------- the tiles into TMEM, and sums
        const int team = warp >> 2, quarter = warp & 3;
        const uint32_t trow = tbase + (uint32_t(quarter * 32) << 16);
        const int row_in = 32 * quarter + lane;  // this thread's position in a tile
        const int64_t width = int64_t(a.max_pages) << c.page_shift;
        uint32_t x_use = 0, tile = 0;
        int4 joins = make_int4(-1, 0, 0, 0);
        bool ok = true, bad = false;
        for (;;) {
            // One warp looks for the next item and the others take its word: they meet at barriers in each pass, and
            // would not leave them if they saw different numbers.
            if (warp == 0) {
                const bool more = ok && w.next(p);
                if (lane == 0) { sh.item = w; sh.more = more; }
            }
            asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory");
            if (!sh.more) break;
            w = sh.item;
            const int64_t line = w.b * width;
            const int last = w.last();
            for (int k = w.first(); k <= last && ok; ++k) {
                const int tiles = w.width(k), j0 = w.from(k), j1 = w.to(k);
                const int64_t pos0 = int64_t(k) * (kCwLTiles * kCwTile) + row_in;
                float scale[kCwLTiles], sum[kCwLTiles];
                uint32_t there = 0;              // a bit a tile: the position has a row
#pragma unroll
                for (int i = 0; i < kCwLTiles; ++i) {
                    const int64_t pos = pos0 + i * kCwTile;
                    scale[i] = 0.f;
                    sum[i] = 0.f;
                    if (i >= tiles || pos >= w.seen) continue;
                    const int page = __ldg(a.table + int64_t(w.b) * a.max_pages + (pos >> c.page_shift));
                    if (page < 0 || page >= c.num_pages) {
                        bad = true;
                        continue;
                    }
                    there |= 1u << i;
                    scale[i] = __ldg(c.scales + (((page << c.page_shift) + int(pos & page_mask)) >> c.block_shift));
                }
                // the blocks of 128 columns in turn, a team every other one
                for (int i = 0; i < 4 * tiles && ok; ++i, ++x_use) {
                    if (int(x_use & 1) != team) continue;
                    const int slot = int(x_use % kCwLSlots);
                    ok = cw_wait(&sh.full[slot], (x_use / kCwLSlots) & 1u, ab, a.status);
                    if (!ok) break;
                    const uint8_t* from = ring + slot * kCwSlotBytes + row_in * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[16];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint4 y = *reinterpret_cast<const uint4*>(from + (((4 * h + d) ^ (lane & 7)) << 4));
                            v[4 * d] = y.x; v[4 * d + 1] = y.y; v[4 * d + 2] = y.z; v[4 * d + 3] = y.w;
                        }
                        tmem_st16(trow + 128 * (i >> 2) + 32 * (i & 3) + 16 * h, v);
                    }
                    fence_proxy_async_smem();    // the slot's next load comes after these reads
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.empty[slot]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.x_full);
                for (int j = j0; j < j1 && ok; ++j) {
                    const int r = w.chunk_size(j), slot = int(use % kCwLQSlots);
                    ++use;
                    const float* fac = factors + slot * 3 * kCwLRows;
                    ok = cw_wait(&sh.q_full[slot], ((use - 1) / kCwLQSlots) & 1u, ab, a.status);
#pragma unroll
                    for (int i = 0; i < kCwLTiles; ++i) {
                        if (!ok || i >= tiles) continue;
                        const int buf = tile & 1;
                        const uint32_t turn = (tile++ >> 1) & 1u;
                        if (buf != team) continue;
                        ok = cw_wait(&sh.t_full[buf], turn, ab, a.status);
                        if (!ok) continue;
                        tc_fence_after();
                        const uint32_t at = trow + kCwLColS + kCwLCols * buf;
                        constexpr int kBlocks = kCwLRows / 16;
                        uint32_t hi[kBlocks][16], lo[kBlocks][16];
#pragma unroll
                        for (int n = 0; n < kBlocks; ++n)
                            if (16 * n < r) {
                                tmem_ld16(at + 16 * n, hi[n]);
                                tmem_ld16(at + r + 16 * n, lo[n]);
                            }
                        tmem_wait_ld();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.t_empty[buf]);
                        const uint64_t scale2 = pair_of(scale[i], scale[i]);
#pragma unroll
                        for (int n = 0; n < kBlocks; ++n) {
                            if (16 * n >= r) break;
                            const float part = cw_sum16(hi[n], lo[n], scale2, fac + 16 * n, fac + kCwLRows + 16 * n);
                            // (tokens have multiples of 16 rows)
                            if (pos0 + i * kCwTile < __float_as_int(fac[2 * kCwLRows + 16 * n])) sum[i] += part;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.q_empty[slot]);
                }
                // The teams' sums together; behind the second barrier all of the pass's products are done and the
                // tiles may go.
                if (team == 1)
#pragma unroll
                    for (int i = 0; i < kCwLTiles; ++i) sh.sums[i][row_in] = sum[i];
                // (if a wait ran out in one of these warps, all of them stop here)
                uint32_t stop;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\t"
                    "setp.ne.u32 p, %1, 0;\n\t"
                    "barrier.cta.red.or.pred.aligned q, 1, 256, p;\n\t"
                    "selp.u32 %0, 1, 0, q;\n\t}"
                    : "=r"(stop)
                    : "r"(uint32_t(!ok))
                    : "memory");
                ok = stop == 0;
                if (team == 0)
#pragma unroll
                    for (int i = 0; i < kCwLTiles; ++i) {
                        if (i >= tiles || !ok) continue;
                        const int64_t pos = pos0 + i * kCwTile;
                        const float both = (there >> i) & 1 ? sum[i] + sh.sums[i][row_in] : 0.f;
                        if (j0 > 0 || j1 < w.chunks) {
                            p.parts[((2 * blockIdx.x + (j0 > 0 ? 0 : 1)) * kCwLTiles + i) * kCwTile + row_in] = both;
                        } else if (pos < w.seen) {
                            a.weights[line + pos] = a.decay != 0.f ? fmaf(a.decay, a.earlier[line + pos], both) : both;
                        }
                    }
                if (j0 > 0 && j1 == w.chunks) joins = make_int4(w.b, k, cw_owner(sh.at, w.at + int64_t(k) * w.chunks), 0);
                asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory");
                tc_fence_after();
            }
        }
        if (threadIdx.x == 0) p.meta[blockIdx.x] = joins;
        if (bad) flag_status(a.status, SMLA_ERR_INDEX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kCwMmaWarp) tmem_dealloc(tbase, 512);
    // Whichever warp gave up a wait, all are out of their loops here: the loads already issued land before the CTA exits.
    if (sh.abort_flag && warp == kCwLoadWarp)
        for (uint32_t n = use > kCwLSlots ? use - kCwLSlots : 0; n < use; ++n)
            mbar_wait(&sh.full[n % kCwLSlots], (n / kCwLSlots) & 1u, kCwWaitNs / 8);
    else if (sh.abort_flag && warp == kCwQWarp)
        for (uint32_t n = use > kCwLQSlots ? use - kCwLQSlots : 0; n < use; ++n)
            mbar_wait(&sh.q_full[n % kCwLQSlots], (n / kCwLQSlots) & 1u, kCwWaitNs / 8);
}

// The passes that several CTAs of the resident kernel have a part in, their parts in order: a block for each CTA and tile.
__global__ void __launch_bounds__(kCwTile)
weights_join_kernel(const CwParams p) {
    grid_dep_wait();
    const WeightsArgs& a = p.a;
    const int4 pass = __ldcg(p.meta + blockIdx.x);
    if (pass.x < 0) return;
    const int row = blockIdx.y * kCwTile + threadIdx.x;
    float sum = __ldcg(p.parts + (2 * pass.z + 1) * (kCwLTiles * kCwTile) + row);
#pragma unroll 8
    for (int i = pass.z + 1; i <= int(blockIdx.x); ++i) sum += __ldcg(p.parts + 2 * i * (kCwLTiles * kCwTile) + row);
    int c0, c1;
    cw_tokens(a, pass.x, c0, c1);
    const int seen = cw_seen(a, c0, c1);
    const int64_t pos = int64_t(pass.y) * (kCwLTiles * kCwTile) + row;
    const int64_t at = pass.x * (int64_t(a.max_pages) << a.cache.page_shift) + pos;
    if (pos < seen) a.weights[at] = a.decay != 0.f ? fmaf(a.decay, a.earlier[at], sum) : sum;
}

namespace {

struct CwPlan { size_t image, factor, bits, parts, meta, bytes; };

CwPlan plan_weights(int64_t T, int64_t H) {
    CwPlan x{};
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes > 0 ? bytes : 1, 256); return o; };
    x.image = take(size_t(T) * H * 1024);
    x.factor = take(size_t(T) * H * 3 * sizeof(float));
    x.bits = take(size_t(kCwMaxBlocks) * 4);
    x.parts = take(size_t(kCwMaxCtas) * 2 * kCwLTiles * kCwTile * 4);
    x.meta = take(size_t(kCwMaxCtas) * sizeof(int4));
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
        cudaError_t e = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCwSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(weights_resident_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCwLSmem);
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
    p.parts = reinterpret_cast<float*>(a.scratch + plan.parts);
    p.meta = reinterpret_cast<int4*>(a.scratch + plan.meta);
    p.resident = int64_t(a.T) * a.H > kCwManyRows * int64_t(a.B);
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
    cfg.gridDim = dim3(sms < kCwMaxCtas ? sms : kCwMaxCtas);
    cfg.blockDim = dim3(p.resident ? kCwLThreads : kCwThreads);
    cfg.dynamicSmemBytes = p.resident ? kCwLSmem : kCwSmem;
    note_launch(2);
    if (!p.resident) return cudaLaunchKernelEx(&cfg, weights_kernel, mb, p);
    e = cudaLaunchKernelEx(&cfg, weights_resident_kernel, mb, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim.y = kCwLTiles;
    cfg.blockDim = dim3(kCwTile);
    cfg.dynamicSmemBytes = 0;
    note_launch();
    return cudaLaunchKernelEx(&cfg, weights_join_kernel, p);
}

}  // namespace smla
