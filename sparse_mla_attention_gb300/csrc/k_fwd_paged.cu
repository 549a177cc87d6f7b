// k_fwd_paged.cu -- attention over the paged 8-bit cache on the tensor cores.
//
// For token t (sequence seq[t]) and head h, over the valid ranks r (positions
// below lens[t], all of them or the picks topk[t, :]):
//   s_r = scale * <q[t,h,:], x_r>, lse = log(exp(sink_h) + sum exp(s_r)),
//   o = sum_r exp(s_r - lse) * x_r,   x_r = e4m3 code * block scale.
//
// The codes go from the cache to the tensor cores as they are (kind::f8f6f4);
// what meets them is split so that nothing but the codes is 8 bits wide:
//  * q: a row's power-of-two scale 2^e, then hi = e4m3(q / 2^e) and lo =
//    e4m3(16 (q / 2^e - hi)): e4m3 has 4 significant bits and bf16 8, so hi +
//    lo / 16 is q itself (to 2^-23 of the row's largest value for small ones).
//  * the weights w = exp(s - m) * block scale: e4m3(w) and, of what is left,
//    e5m2(w - e4m3(w)), whose range reaches further down: off by at most 2^-7 w
//    (bf16: 2^-8), and 2^-20 of the largest weight for small ones. Both parts
//    accumulate into one fp32 accumulator; the denominator sums unrounded weights.
// Block scales: s_r is multiplied by its row's scale in fp32, and w carries it (2^-100 at least).
//
// S = Q K^T: M = 128 (up to 64 heads; lanes 16i .. 16i+15 of each lane quarter's first half
// hold hi, its second half lo), N = 64 ranks, K = 512, A = Q from TMEM.
// O^T = V^T W^T: M = 128 columns of D (four blocks), N = heads, K = 64 ranks hi
// then 64 ranks lo; A = the very tile that S read, as its MN-major transpose.
// TMEM: S two buffers of 64 columns, Q 128 columns, O^T 4 x 64 columns.
//
// fwd_paged_kernel: persistent, one CTA per SM. The tiles (64 ranks) of all
// tokens, in order, are dealt out evenly: CTA c of a head group takes the
// tiles [c X / G, (c+1) X / G), finds its first token by a scan over lens, and
// works through its items (a token's part of the range). An item that holds a
// whole token writes o and lse; a part of a token goes to the workspace as fp32
// (unnormalised O, maximum, sum), and combine_paged_kernel joins the parts in order.
// Warps: 0-3 and 4-7 softmax, on alternate tiles (a thread has one head and half of
// the tile's ranks: the two lanes of a head swap their halves of S, which adds hi and
// lo), 8-11 q conversion and output, 12 S products, 13 O products, 14-17 loads (TMA
// boxes where a tile's rows lie in whole pages, copies row by row otherwise). A masked
// rank's row is zeros with weight 0: no byte of a row that nothing names is ever read.
//
// Why so: the cache is read once a head group, in 8 bits, and never widened: bf16 copies of
// a tile would take twice the shared memory and more conversions than the tile has
// products to hide them. With up to 64 heads, hi and lo of q fill the 128 rows of one MMA
// for S; O is taken transposed because its 64 heads are then N, and V needs no copy.
// 64 ranks a tile: S takes two buffers of 64 TMEM columns beside Q and O, which fill the
// other 384. Two teams, because a tile's softmax is a chain of waits.
// Bound: 152 CTAs with one item of 8 to 64 tiles each take 17.9 us + 0.95 a tile at 64 heads (1970
// cycles a tile: its products take ~1600, 16 of 62 for O and 16 of 38 for S, reading it at shared
// memory's rate; reading 32 KB at the SM's share of HBM takes ~1500; a team has two tiles' time for
// a chain of loads, swaps, exponentials and conversions), 12.8 us + 0.82 at 16 heads, which are
// bound by the loads. No unit is full (profiled at 64 heads: DRAM 47% of its rate, issue slots
// 44% and tensor pipe 41% of the time). The fixed part is the start, the look-ups, the first q's
// split, the output and the second launch; second items and split tokens come on top.
// Measured (one GB300, device time of a call with its join, in a graph, scores of N(0,1); in brackets
// four times as far apart, where O is rescaled every few tiles):
//   128 sequences of up to 5120 positions, 64 heads: 78 us (91), 3.3 TB/s of cache, 0.83 PFLOP/s
//   96 of up to 6001, 16 heads: 55 us (59), 4.0 TB/s;  3 of 81920, 128 heads: 64.5 us (77), 0.90 PFLOP/s
//   256 tokens x 512 picks, 128 heads: 76 us (83);  one token of 777 positions: 14.5 us: the two
//   launches, the look-ups' latency, q, one tile, the output and the join.
//
// Every mbarrier wait is bounded; a timeout sets SMLA_ERR_TIMEOUT, stops the
// CTA's loops, waits (bounded) for its own copies and MMAs and frees TMEM.
#include <cfloat>

#include <cuda_fp8.h>

#include "smla_internal.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace smla {
using namespace sm100;

namespace {

constexpr uint32_t kPgWaitNs = 2000000000u;
constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;
constexpr int kPgTile = 64;                      // ranks per tile
constexpr int kPgSlots = 6;
constexpr int kPgLead = 4;
constexpr int kPgSlotBytes = kPgTile * kD;       // 32 KB: four blocks of 64 rows x 128 bytes
constexpr int kPgBlockBytes = kPgTile * 128;
constexpr int kPgHeads = 64;                     // heads of a group at most
constexpr int kPgPBytes = kPgHeads * 128;        // weights of a tile: 64 bytes hi, 64 bytes lo a head
constexpr int kPgOutWarp = 8, kPgMmaWarp = 12, kPgLoadWarp = 14, kPgLoadWarps = 4;
constexpr int kPgThreads = (kPgLoadWarp + kPgLoadWarps) * 32;
constexpr int kPgMaxCtas = 160;
// TMEM columns
constexpr uint32_t kPgColS = 0, kPgColQ = 128, kPgColO = 256;
// Weights are scaled so that the running reference's is 2^kPgBias; the
// reference follows the maximum when it is passed by more than 2^kPgSlack
// (e4m3 ends at 448 > 2^(kPgBias + kPgSlack)). A weight below 2^-7 is off by up to 2^-14, so
// each bit of bias is a bit of precision for small weights, and each bit of slack saves rescalings
// of O. 128 sequences of up to 5120 positions, 64 heads, device time in us with bias 4 / 5 / 6 / 7 and
// slack 8.75 - bias: scores of N(0,1) 77.8 / 78.0 / 78.8 / 83.6, four times as far apart 87.5 / 89.5 /
// 91.1 / 93.0. A head with half of its weight on one row and half on 32,767 nearly equal ones: o off by
// 5.8e-3 of its norm with bias 4, by less than a tenth of its rounding to bf16 with 6.
constexpr float kPgBias = 6.f, kPgSlack = 2.75f;

struct PgShared {
    uint64_t full[kPgSlots], empty[kPgSlots], q_load[4];
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t q_full, q_empty, o_full, o_empty, dec[4], fixed[2], drain[2];
    uint32_t tbase;
    unsigned status;                             // this CTA's status bits
    volatile int abort_flag;
    volatile int far;                            // the CTA has met a scale outside [2^-45, 2^45]
    int t0, k0, count;                           // the CTA's first token, tile in it, tiles in all
    int sum[kPgThreads / 32];
    __align__(16) uint32_t need[2][2][4];        // team, parity of its count, lane quarter: rescale O first
    // of each rank: block scale and its log2, or 0 and -inf (masked); 1 / scale. A scale counts as 2^-100 at least in
    // the logarithm and the reciprocal.
    __align__(16) float2 scale[kPgSlots][kPgTile];
    __align__(16) float inv[kPgSlots][kPgTile];
    __align__(16) float fac[2][2][kPgHeads];     // rescaling factors (team, parity of its count)
    // per item & 1 (an item's q is split only when the output of the item two before is done)
    float qfac[2][kPgHeads];                     // score factor of a head's q: 2^e * scale * log2(e)
    // item & 3 (an output warp may split the q of the item after next while another still reads the done item's)
    float qodd[4][kPgHeads];                     // NaN where a head's q holds an infinity or a NaN, else 0
    float st_ref[kPgHeads];                      // running reference of a head
    float ref[2][2][kPgHeads], l[2][2][kPgHeads];         // and team: reference and sum of a head
    __align__(16) float fin[4][kPgHeads];        // per output warp: 1 / denominator
};

constexpr int kPgStageBytes = 2048;              // an output warp's staging: two halves
// The ring comes first: swizzled tiles want a base that is a multiple of 1024, as the array's is declared to be.
constexpr int kPgSharedAt = kPgSlots * kPgSlotBytes + 2 * kPgPBytes + 4 * kPgStageBytes;
constexpr int kPgSmem = kPgSharedAt + int(sizeof(PgShared));
static_assert(kPgSmem <= 232448, "shared memory of one CTA is at most 227 KB");

struct PgParams {
    const int32_t* table; const int32_t* seq; const int32_t* lens; const int32_t* topk;
    const uint8_t* pages; const float* scales; const float* sink;
    uint16_t* o; float* lse;
    int T, H, K, B, max_pages, num_pages, page_shift, block_shift;
    int groups, group_heads;                     // head groups, heads of a full one
    int ctas;                                    // CTAs of a group
    float scale;
    unsigned* status;                            // the call's status word
    unsigned* cta_status;                        // [CTAs]
    int4* meta;                                  // [CTAs] end of a split token: {t, first CTA, its part, 0} (t -1: none)
    float2* part_ml;                             // [CTAs][2][group_heads] maximum (log2) and sum
    float* part_o;                               // [CTAs][2][group_heads / 4][512][4] (head h: block h / 4, h % 4)
};

// Every lane waits, for at most about two seconds; the warp goes on only if all of them
// saw the phase. Short on purpose (the kernel has many waits, its warps run different
// code, and instruction fetches count), and quiet: a waiting warp sleeps in
// try_wait and looks at the timer only now and then.
__device__ __forceinline__ bool pg_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned* status) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint32_t t0 = globaltimer_lo_ns();
        do {
#pragma unroll 1
            for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
            if (!ok && globaltimer_lo_ns() - t0 > kPgWaitNs) {
                *abort_flag = 1;
                flag_status(status, SMLA_ERR_TIMEOUT);
            }
        } while (!ok && !*abort_flag);
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ int pg_len(const PgParams& p, int t) {
    const int64_t limit = int64_t(p.max_pages) << p.page_shift;
    const int len = __ldg(p.lens + t);
    return len < 0 ? 0 : len > limit ? int(limit) : len;
}

// Tiles of token t; at least one, so that every token is somebody's item.
__device__ __forceinline__ int pg_tiles(const PgParams& p, int t) {
    const int n = p.topk ? p.K : pg_len(p, t);
    return n < 1 ? 1 : (n + kPgTile - 1) / kPgTile;
}

// The ring's uses are the items' q (two each) and tiles; use g is in slot g % kPgSlots. The
// first item's q comes first, every other item's kPgLead tiles before the end of the item
// ahead of it (PgWalk::early), so that it is loaded and split before it is needed.
// A parity wait tells a phase only from the one before, so whoever waits for a barrier
// sees each of its phases in turn: `empty` counts every use (each loading warp has a
// part in each), `full` the tiles alone (the S warp keeps a parity bit a slot), and q
// has barriers of its own, q_load[item & 3] (the uses between the q of an item and of
// the fourth after it go round the ring).
static_assert(kPgSlots % 2 == 0 && kPgSlots >= 6, "a slot belongs to one of the two softmax teams");
__device__ __forceinline__ int pg_slot(int g) { return g % kPgSlots; }
__device__ __forceinline__ uint32_t pg_parity(uint32_t bits, int slot) { return (bits >> slot) & 1u; }

// The tiles (fewer than 2^31) are dealt out in runs of per or (the first rem CTAs) per + 1.
struct PgDeal {
    unsigned per, rem;
    __device__ __forceinline__ PgDeal(unsigned total, unsigned ctas) : per(total / ctas), rem(total - per * ctas) {}
    __device__ __forceinline__ unsigned first(unsigned c) const { return per * c + (c < rem ? c : rem); }
    __device__ __forceinline__ unsigned owner(unsigned tile) const {
        const unsigned longer = rem * (per + 1);
        return tile < longer ? tile / (per + 1) : rem + (tile - longer) / per;
    }
};

__device__ __forceinline__ uint32_t e4m3x2(__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_half(uint32_t v) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v), __NV_E4M3));
}
__device__ __forceinline__ uint32_t e5m2x2(__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E5M2);
}
// 1 / x by the PTX rcp.approx.f32 instruction (relative error at most 2^-23, subnormal results kept).
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x 2^d for d down to -250 (in two steps: the factor alone may be less than a float holds).
__device__ __forceinline__ float mul_ex2(float x, float d) {
    const float h = ex2_approx(0.5f * d);
    return x * h * h;
}
// The CTA's share of the tiles. Picks: every token has as many tiles. All
// positions: sums the tiles of the tokens (thread i those of a run of tokens), then
// the thread whose run holds the CTA's first tile finds its token.
__device__ void pg_locate(const PgParams& p, PgShared& sh, unsigned c, unsigned ctas) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned total, at;
    int t0 = 0, mine = 0;
    if (p.topk) {
        const int n = pg_tiles(p, 0);
        total = unsigned(p.T) * n;
        at = 0;
    } else {
        const int run = (p.T + kPgThreads - 1) / kPgThreads;
        t0 = min(int(threadIdx.x) * run, p.T);
        const int t1 = min(t0 + run, p.T);
#pragma unroll 4
        for (int t = t0; t < t1; ++t) mine += pg_tiles(p, t);
        int x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) sh.sum[warp] = x;
        __syncthreads();
        static_assert(kPgThreads <= 1024, "a lane for each warp's sum");
        int y = lane < kPgThreads / 32 ? sh.sum[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        total = unsigned(__shfl_sync(0xffffffffu, y, 31));
        const int before = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
        at = unsigned((warp ? before : 0) + x - mine);
    }
    const PgDeal deal(total, ctas);
    const unsigned a = deal.first(c), b = deal.first(c + 1);
    if (threadIdx.x == 0) sh.count = int(b - a);
    const bool mine_to_find = p.topk ? threadIdx.x == 0 : at <= a && a < at + unsigned(mine);
    if (a < b && mine_to_find) {
        int t = t0, n = pg_tiles(p, t);
        if (p.topk) {
            t = int(a / unsigned(n));
            at = unsigned(t) * n;
        } else {
#pragma unroll 1
            while (a >= at + unsigned(n)) {
                at += unsigned(n);
                n = pg_tiles(p, ++t);
            }
        }
        sh.t0 = t;
        sh.k0 = int(a - at);
        // this CTA ends a token that began in an earlier one: it names the parts to join
        int4 end = make_int4(-1, 0, 0, 0);
        if (a > at && b - at >= unsigned(n)) {
            const unsigned first = deal.owner(at);
            end = make_int4(t, int(first), deal.first(first) == at ? 0 : 1, 0);
        }
        p.meta[blockIdx.x] = end;
    } else if (a >= b && threadIdx.x == 0) {
        p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
}

// The CTA's items: parts [k0, k0 + n) of the tiles of token t.
struct PgWalk {
    int t, k0, left;
    // (the shuffles tell the compiler that a warp's lanes agree)
    __device__ __forceinline__ PgWalk(const PgShared& sh)
        : t(__shfl_sync(0xffffffffu, sh.t0, 0)), k0(__shfl_sync(0xffffffffu, sh.k0, 0)),
          left(__shfl_sync(0xffffffffu, sh.count, 0)) {}
    __device__ __forceinline__ int tiles(const PgParams& p) const {
        const int n = __shfl_sync(0xffffffffu, pg_tiles(p, t), 0) - k0;
        return n < left ? n : left;
    }
    // the tile of an item of n that the next item's q is loaded ahead of (-1: no next item)
    __device__ __forceinline__ int early(int n) const { return left <= n ? -1 : n > kPgLead ? n - kPgLead : 0; }
    __device__ __forceinline__ void next(int n) { left -= n; ++t; k0 = 0; }
};

}  // namespace

__global__ void __launch_bounds__(kPgThreads, 1)
fwd_paged_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_box,
                 const PgParams p) {
    extern __shared__ __align__(1024) uint8_t ring[];
    PgShared& sh = *reinterpret_cast<PgShared*>(ring + kPgSharedAt);
    uint8_t* pbuf = ring + kPgSlots * kPgSlotBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = int(blockIdx.x) % p.groups, cta = int(blockIdx.x) / p.groups;
    const int ctas = int(gridDim.x) / p.groups;
    const int head0 = group * p.group_heads;
    const int heads = p.H - head0 < p.group_heads ? p.H - head0 : p.group_heads;
    volatile int* ab = &sh.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPgSlots; ++s) {
            mbar_init(&sh.full[s], kPgLoadWarps);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.s_full[b], 2);         // MMA completion and the issuing thread
            mbar_init(&sh.s_empty[b], 4);
            mbar_init(&sh.p_full[b], 4);
            mbar_init(&sh.p_empty[b], 1);
        }
        for (int b = 0; b < 4; ++b) mbar_init(&sh.q_load[b], 2 * kPgLoadWarps);
        mbar_init(&sh.q_full, 4);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.o_full, 2);                // MMA completion and the issuing thread
        mbar_init(&sh.o_empty, 4);
        mbar_init(&sh.fixed[0], 4);
        mbar_init(&sh.fixed[1], 4);
        for (int q = 0; q < 4; ++q) mbar_init(&sh.dec[q], 1);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        sh.abort_flag = 0;
        sh.far = 0;
        sh.status = 0;
        fence_mbar_init();
    }
    if (warp == kPgMmaWarp) { tmem_alloc(&sh.tbase, 512); tmem_relinquish(); }
    grid_dep_wait();                             // what ran before is complete: nothing global was touched yet
    pg_locate(p, sh, unsigned(cta), unsigned(ctas));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tbase;

    if (warp >= kPgLoadWarp) {
        // --------------------------------------------------------------- loads
        // Every warp has a part in each ring use: of an item's q (two uses of four 64-column
        // boxes) one box; of a tile whose rows lie in whole runs of 16 (all positions,
        // none masked) one column block of all 64 ranks, as TMA boxes; of other tiles 16 ranks,
        // copied 16 bytes a lane (a warp issues a four-row TMA gather per 100 cycles, 16 a tile;
        // the same bytes as copies take 16 instructions).
        // Picks: positions are loaded two tiles ahead, pages and scales one tile ahead.
        const int lw = warp - kPgLoadWarp;
        const int64_t limit = int64_t(p.max_pages) << p.page_shift;
        const int page_mask = (1 << p.page_shift) - 1;
        const int box_rows = page_mask + 1 < kPgTile ? page_mask + 1 : kPgTile;
        bool bad = false;
        int g = 0, item = 0;
        uint32_t loads = 0;                      // parity of each slot's last tile load
        int q_last = -1;
        bool ok = true;
        // Gathered tiles whose copies are in flight, oldest first: the copies are this warp's own
        // (cp.async), so it is the one to see them land, make them visible to the tensor
        // core and arrive. It never sleeps on a slot before that.
        int flying = 0, fly0 = 0, fly1 = 0;
        auto land_all = [&]() {
            if (flying == 0) return;
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.full[fly0]);
                if (flying > 1) mbar_arrive(&sh.full[fly1]);
            }
            flying = 0;
        };
        auto wait_slot = [&](int slot, uint32_t parity) {
            if (flying && !__all_sync(0xffffffffu, mbar_try_test(&sh.empty[slot], parity))) land_all();
            return pg_wait_warp(&sh.empty[slot], parity, ab, &sh.status);
        };
        auto load_q = [&](int of, int t) {
            for (int k = 0; k < 2 && ok; ++k, ++g) {
                const int slot = pg_slot(g);
                ok = wait_slot(slot, (uint32_t(g / kPgSlots) & 1u) ^ 1u);
                if (!ok) break;
                q_last = of;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_load[of & 3], uint32_t(p.group_heads) * 128u);
                    tma_load_2d(ring + slot * kPgSlotBytes + lw * kPgBlockBytes, &map_q, (4 * k + lw) * 64,
                                t * p.H + head0, &sh.q_load[of & 3]);
                }
            }
        };
        // the first q's uses: its slots are free at the start
        if (sh.count > 0) load_q(0, sh.t0);
        // Look-ups ahead of the loads: tile after tile over all items.
        PgWalk wa(sh);
        int na = 0, ia = 0, ba = 0, lena = 0;
        auto open_item = [&]() {
            ia = 0;
            na = 0;
            if (wa.left <= 0) return;
            na = wa.tiles(p);
            lena = __ldg(p.lens + wa.t);
            if (lena < 0 || lena > limit) { bad = true; lena = lena < 0 ? 0 : int(limit); }
            ba = p.seq ? __ldg(p.seq + wa.t) : wa.t;
            if (lena > 0 && (ba < 0 || ba >= p.B)) { bad = true; lena = 0; }
        };
        // Lane's position in the next tile, as it stands in topk; for all positions that of the
        // first rank of run (lane & 3) of 16
        struct Ahead { int pos, len, b; };
        auto look = [&]() {
            Ahead x{-1, 0, 0};
            if (na > 0) {
                const int r0 = kPgTile * (wa.k0 + ia);
                x.len = lena;
                x.b = ba;
                if (p.topk) {
                    const int r = r0 + 16 * lw + (lane & 15);
                    x.pos = r < p.K ? __ldg(p.topk + int64_t(wa.t) * p.K + r) : -1;
                } else {
                    x.pos = r0 + 16 * (lane & 3);
                }
                if (++ia == na) {
                    wa.next(na);
                    open_item();
                }
            }
            return x;
        };
        auto page_of = [&](const Ahead& x) {     // -1: masked
            if (p.topk) bad |= x.len > 0 && (x.pos < -1 || x.pos >= x.len);
            if (x.pos < 0 || x.pos >= x.len) return -1;
            return __ldg(p.table + int64_t(x.b) * p.max_pages + (x.pos >> p.page_shift));
        };
        auto row_of = [&](const Ahead& x, int page) {
            const bool v = x.pos >= 0 && x.pos < x.len;
            bad |= v && (page < 0 || page >= p.num_pages);
            return v && page >= 0 && page < p.num_pages ? (page << p.page_shift) + (x.pos & page_mask) : -1;
        };
        open_item();
        Ahead x0 = look(), x1 = look();          // the tile at hand and the next one
        int row = row_of(x0, page_of(x0));
        float sc = row >= 0 ? __ldg(p.scales + (row >> p.block_shift)) : -1.f;

        for (PgWalk w(sh); w.left > 0 && ok; ++item) {
            const int n = w.tiles(p), early = w.early(n);
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++g) {
                if (i == early) load_q(item + 1, w.t + 1);
                const int slot = pg_slot(g);
                uint8_t* dst = ring + slot * kPgSlotBytes;
                const int page1 = page_of(x1);
                const Ahead x2 = look();
                if (ok) ok = wait_slot(slot, (uint32_t(g / kPgSlots) & 1u) ^ 1u);
                if (!ok) break;
                loads ^= 1u << slot;             // full's phase of this load has the parity before
                const int left = x0.len - (x0.pos - 16 * (lane & 3));    // all positions: from the tile's first on
                const bool boxes = !p.topk && __all_sync(0xffffffffu, row >= 0 && left >= kPgTile) != 0;
                float sc16 = sc;                 // scale of the warp's rank (lane & 15)
                if (boxes) {
                    if (lane == 0) mbar_expect_tx(&sh.full[slot], kPgBlockBytes);
#pragma unroll 1
                    for (int r = 0; r < kPgTile; r += box_rows) {
                        const int y = __shfl_sync(0xffffffffu, row, r >> 4);
                        if (lane == 0)
                            tma_load_2d(dst + lw * kPgBlockBytes + r * 128, &map_box, lw * 128, y, &sh.full[slot]);
                    }
                    sc16 = __shfl_sync(0xffffffffu, sc, lw);
                } else {
                    int mine = row;
                    if (!p.topk) {               // ranks 16 lw + (lane & 15), as far as the sequence goes
                        mine = __shfl_sync(0xffffffffu, row, lw);
                        sc16 = __shfl_sync(0xffffffffu, sc, lw);
                        const bool v = mine >= 0 && 16 * lw + (lane & 15) < left;
                        mine = v ? mine + (lane & 15) : -1;
                        sc16 = v ? sc16 : -1.f;
                    }
                    // four rows of 128 bytes an instruction; a masked rank's row is zeros, unread
                    uint8_t* at = dst + (16 * lw + (lane >> 3)) * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = __shfl_sync(0xffffffffu, mine, 4 * q + (lane >> 3));
                        const uint8_t* src = p.pages + int64_t(r < 0 ? 0 : r) * kD + (lane & 7) * 16;
                        uint8_t* to = at + q * 512 + (((lane & 7) ^ ((4 * q + (lane >> 3)) & 7)) << 4);
#pragma unroll
                        for (int cb = 0; cb < 4; ++cb)
                            cp_async16_zfill(to + cb * kPgBlockBytes, src + cb * 128, r < 0 ? 0u : 16u);
                    }
                    cp_async_commit();
                }
                if (lane < 16) {
                    const float least = fmaxf(sc16, 0x1p-100f);
                    sh.scale[slot][16 * lw + lane] = make_float2(fmaxf(sc16, 0.f), sc16 >= 0.f ? __log2f(least) : -INFINITY);
                    sh.inv[slot][16 * lw + lane] = rcp_approx(least);
                }
                if (sc16 > 0x1p45f || (sc16 >= 0.f && sc16 < 0x1p-45f)) sh.far = 1;
                __syncwarp();
                if (boxes) {
                    if (lane == 0) mbar_arrive(&sh.full[slot]);
                } else {
                    if (flying == 2) {           // the oldest lands first
                        cp_async_wait<2>();
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.full[fly0]);
                        fly0 = fly1;
                        flying = 1;
                    }
                    if (flying == 0) fly0 = slot; else fly1 = slot;
                    ++flying;
                }
                // the next tile's rows and scales
                row = row_of(x1, page1);
                sc = row >= 0 ? __ldg(p.scales + (row >> p.block_shift)) : -1.f;
                x0 = x1;
                x1 = x2;
            }
            w.next(n);
        }
        land_all();
        if (bad) flag_status(&sh.status, SMLA_ERR_INDEX);
        if (sh.abort_flag) {     // the loads already issued land before the CTA exits
            for (int slot = 0; slot < kPgSlots; ++slot)
                mbar_wait(&sh.full[slot], pg_parity(loads, slot) ^ 1u, kPgWaitNs / 8);
            for (int q = q_last > 2 ? q_last - 2 : 0; q <= q_last; ++q)
                mbar_wait(&sh.q_load[q & 3], uint32_t(q >> 2) & 1u, kPgWaitNs / 8);
        }
        __syncwarp();
    } else if (warp >= kPgMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        // One warp issues the S products, one the O products: small MMAs keep the tensor core
        // busy only if the waits for one kind pass while the other is issued. The whole warp
        // walks the tiles, so that descriptors stay in uniform registers; one elected lane issues.
        const uint64_t ring_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
        const bool leader = elect_one();
        int g = 2, tile = 0, item = 0;
        bool ok = true;
        if (warp == kPgMmaWarp) {
            const uint32_t id_s = idesc_f8(128, kPgTile, false, false);
            uint32_t seen = 0;
            int q_at = 0, q_next = 0;            // the item's q uses, and the next one's
            for (PgWalk w(sh); w.left > 0 && ok; ++item) {
                const int n = w.tiles(p), early = w.early(n);
                q_at = q_next;
#pragma unroll 1
                for (int i = 0; i < n; ++i, ++g, ++tile) {
                    if (i == early) { q_next = g; g += 2; }
                    const int slot = pg_slot(g), b = tile & 1;
                    if (i == 0) {
                        ok = pg_wait_warp(&sh.q_full, uint32_t(item) & 1u, ab, &sh.status);
                        if (ok && leader) {      // q is in TMEM: its slots are free
                            mbar_arrive(&sh.empty[pg_slot(q_at)]);
                            mbar_arrive(&sh.empty[pg_slot(q_at + 1)]);
                        }
                    }
                    if (ok) ok = pg_wait_warp(&sh.s_empty[b], (uint32_t(tile >> 1) & 1u) ^ 1u, ab, &sh.status);
                    if (ok) ok = pg_wait_warp(&sh.full[slot], pg_parity(seen, slot), ab, &sh.status);
                    if (!ok) break;
                    seen ^= 1u << slot;
                    tc_fence_after();
                    uint64_t ka = ring_desc + uint32_t(slot) * (kPgSlotBytes >> 4);
                    if (leader) {
                        uint32_t qa = tbase + kPgColQ;
#pragma unroll 1
                        for (int cb = 0; cb < 4; ++cb) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f8_ts(tbase + kPgColS + kPgTile * b, qa + 8 * k, ka + 2 * k, id_s, (cb | k) != 0);
                            ka += kPgBlockBytes >> 4;
                            qa += 32;
                        }
                        mbar_arrive(&sh.s_full[b]);
                        mma_commit(&sh.s_full[b]);
                        if (i == n - 1) mma_commit(&sh.q_empty);
                    }
                    __syncwarp();
                }
                w.next(n);
            }
        } else {
            int fixes0 = 0, fixes1 = 0;          // times that each team rescaled O
            const uint64_t p_desc = sdesc_sw128(smem_u32(pbuf), 16, 1024);
            const uint32_t id_hi = idesc_f8(128, heads, true, false), id_lo = idesc_f8(128, heads, true, true);
            for (PgWalk w(sh); w.left > 0 && ok; ++item) {
                const int n = w.tiles(p), early = w.early(n);
#pragma unroll 1
                for (int i = 0; i < n; ++i, ++g, ++tile) {
                    if (i == early) g += 2;
                    const int slot = pg_slot(g), b = tile & 1;
                    if (i == 0 && item > 0) ok = pg_wait_warp(&sh.o_empty, uint32_t(item - 1) & 1u, ab, &sh.status);
                    if (ok) ok = pg_wait_warp(&sh.p_full[b], uint32_t(tile >> 1) & 1u, ab, &sh.status);
                    if (!ok) break;
                    const uint4 need = *reinterpret_cast<const uint4*>(sh.need[b][(tile >> 1) & 1]);
                    if (need.x | need.y | need.z | need.w) {
                        ok = pg_wait_warp(&sh.fixed[b], uint32_t(b ? fixes1 : fixes0) & 1u, ab, &sh.status);
                        if (!ok) break;
                        if (b) ++fixes1; else ++fixes0;
                    }
                    tc_fence_after();
                    uint64_t va = ring_desc + uint32_t(slot) * (kPgSlotBytes >> 4);
                    const uint64_t wa = p_desc + uint32_t(b) * (kPgPBytes >> 4);
                    if (leader) {
                        uint32_t acc = tbase + kPgColO;
#pragma unroll 1
                        for (int db = 0; db < 4; ++db) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)      // hi ranks 0-31, 32-63, then lo
                                mma_f8_ss(acc, va + (((k & 1) * 4096) >> 4), wa + 2 * k, k < 2 ? id_hi : id_lo,
                                          (i | k) != 0);
                            va += kPgBlockBytes >> 4;
                            acc += 64;
                        }
                        mma_commit(&sh.empty[slot]);
                        mma_commit(&sh.p_empty[b]);
                        if (i == n - 1) {
                            mbar_arrive(&sh.o_full);
                            mma_commit(&sh.o_full);
                        }
                    }
                    __syncwarp();
                }
                w.next(n);
            }
        }
        if (leader) {
            uint64_t* bar = &sh.drain[warp - kPgMmaWarp];
            mma_commit(bar);
            mbar_wait(bar, 0, kPgWaitNs);
        }
        __syncwarp();
    } else if (warp < kPgOutWarp) {
        // -------------------------------------------------------------- softmax
        // Two teams of four warps take the tiles in turn (a tile's team is its slot's
        // parity). A head's reference r is kept so that weights 2^(s + log2(block scale) - r + bias)
        // stay below e4m3's largest value: it starts as the first tile's largest sum of score and
        // log2 of scale and follows when a tile passes it by more than the slack. (The sum is a
        // rank's own: the largest score plus log2 of the largest scale may be two ranks', and
        // then costs every weight range.) It passes from team to team along dec[quarter]; O is
        // rescaled for a tile by its team, before its O product but after its weights are
        // written, so that no warp waits for the others' verdicts on the way.
        const int team = warp >> 2, quarter = warp & 3;
        const int part = lane >> 4, head = 16 * quarter + (lane & 15);
        const bool active = 16 * quarter < heads;
        const uint32_t trow = tbase + (uint32_t(quarter * 32) << 16);
        const float lo_factor = part ? 0.0625f : 1.f;
        uint8_t* prow = pbuf + team * kPgPBytes + head * 128;
        int g = 2, tile = 0, item = 0, mine = -1;        // mine: the team's last tile
        bool ok = true;
        // rescales O for the team's last tile, if one of its warps asked for it
        auto fix = [&]() {
            if (mine < 0) return;
            const int c = (mine >> 1) & 1;
            ok = pg_wait_warp(&sh.p_full[team], uint32_t(c), ab, &sh.status);
            if (!ok) return;
            const uint4 need = *reinterpret_cast<const uint4*>(sh.need[team][c]);
            if ((need.x | need.y | need.z | need.w) == 0) return;
            // the O products before that tile's are complete (the one before last is, since the
            // weights could be written: so the parity means the last one's phase)
            ok = pg_wait_warp(&sh.p_empty[team ^ 1], uint32_t((mine - 1) >> 1) & 1u, ab, &sh.status);
            if (!ok) return;
            tc_fence_after();
            // a warp's TMEM lanes are columns of D, not heads: every warp rescales the sixteen heads
            // that a warp asked for, the next columns on their way while these are multiplied
#pragma unroll 1
            for (int h = 0; h < heads; h += 16) {
                if (sh.need[team][c][h >> 4] == 0) continue;
                const uint32_t at = trow + kPgColO + h;
                const float* fac = sh.fac[team][c] + h;
                uint32_t v[2][16];
                tmem_ld16(at, v[0]);
#pragma unroll
                for (int db = 0; db < 4; ++db) {
                    tmem_wait_ld();
                    if (db < 3) tmem_ld16(at + 64 * (db + 1), v[(db + 1) & 1]);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[db & 1][e] = __float_as_uint(__uint_as_float(v[db & 1][e]) * fac[e]);
                    tmem_st16(at + 64 * db, v[db & 1]);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.fixed[team]);
        };
        for (PgWalk w(sh); w.left > 0 && ok; ++item) {
            const int n = w.tiles(p), early = w.early(n);
            float own_ref = -INFINITY, l = 0.f, f = 0.f;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i, ++g, ++tile) {
                if (i == early) g += 2;
                const int slot = pg_slot(g);
                if ((slot & 1) != team) continue;
                fix();
                if (!ok) break;
                mine = tile;
                const uint32_t use = uint32_t(tile >> 1) & 1u;      // parity of the team's count of tiles
                ok = pg_wait_warp(&sh.s_full[team], use, ab, &sh.status);
                if (!ok) break;
                tc_fence_after();
                if (i < 2) f = sh.qfac[item & 1][head] * lo_factor;
                const float4* scp = reinterpret_cast<const float4*>(&sh.scale[slot][32 * part]);
                const float4* invp = reinterpret_cast<const float4*>(&sh.inv[slot][32 * part]);
                float s[32];                     // score plus log2 of the block scale: log2 of the weight
                float mx = -INFINITY;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // the head's other lane has the other part of q: swap halves and add
                    uint32_t v0[16], v1[16];
                    tmem_ld16(trow + kPgColS + kPgTile * team + 16 * q, v0);
                    tmem_ld16(trow + kPgColS + kPgTile * team + 32 + 16 * q, v1);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 c2 = scp[8 * q + e / 2];       // two ranks: scale and its log2
                        const float g0 = __uint_as_float(part ? v0[e] : v1[e]) * f;
                        const float g1 = __uint_as_float(part ? v0[e + 1] : v1[e + 1]) * f;
                        const float x0 = fmaf(__uint_as_float(part ? v1[e] : v0[e]), f,
                                              __shfl_xor_sync(0xffffffffu, g0, 16));
                        const float x1 = fmaf(__uint_as_float(part ? v1[e + 1] : v0[e + 1]), f,
                                              __shfl_xor_sync(0xffffffffu, g1, 16));
                        s[16 * q + e] = fmaf(x0, c2.x, c2.y);
                        s[16 * q + e + 1] = fmaf(x1, c2.z, c2.w);
                        mx = fmaxf(mx, fmaxf(s[16 * q + e], s[16 * q + e + 1]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty[team]);
                const float top = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                // the reference after the tile before this one
                if (tile > 0) ok = pg_wait_warp(&sh.dec[quarter], uint32_t(tile - 1) & 1u, ab, &sh.status);
                if (!ok) break;
                const float old = i == 0 ? top : sh.st_ref[head];
                const bool grow = active && top > old + kPgSlack;
                const float ref = grow ? top : old;
                const bool need = __any_sync(0xffffffffu, grow) != 0;
                if (part == 0) {
                    sh.st_ref[head] = ref;
                    sh.fac[team][use][head] = grow && old != -INFINITY ? ex2_approx(old - ref) : 1.f;
                }
                if (lane == 0) sh.need[team][use][quarter] = need;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.dec[quarter]);
                l = own_ref != ref && own_ref != -INFINITY ? mul_ex2(l, own_ref - ref) : l;
                own_ref = ref;
                // the team's weights before these are used up
                ok = pg_wait_warp(&sh.p_empty[team], use ^ 1u, ab, &sh.status);
                if (!ok) break;
                if (active) {
                    const float off = kPgBias - (ref == -INFINITY ? 0.f : ref);
                    // The denominator takes w / scale. Beside a scale 2^90 times as large a weight may be less than a
                    // float holds, its rank's term of the denominator not: then the term is taken for itself.
                    const bool wide = sh.far != 0;
                    if (__builtin_expect(wide, 0)) {
                        float copy[32];                      // (in local memory: short code that hardly ever runs)
#pragma unroll
                        for (int e = 0; e < 32; ++e) copy[e] = s[e];
#pragma unroll 1
                        for (int e = 0; e < 32; ++e) {
                            const float x = copy[e];
                            l += x == -INFINITY ? 0.f : ex2_approx(x - sh.scale[slot][32 * part + e].y + off);
                        }
                    }
                    float l0 = 0.f, l1 = 0.f;        // (two sums: a chain each)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {            // 16 ranks: 16 bytes hi and 16 bytes lo
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e4 = 0; e4 < 4; ++e4) {
                            uint32_t hl[2], ll[2];
                            const float4 i4 = invp[4 * q + e4];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int e = 16 * q + 4 * e4 + 2 * k;
                                const float w0 = ex2_approx(s[e] + off), w1 = ex2_approx(s[e + 1] + off);
                                l0 = fmaf(w0, k ? i4.z : i4.x, l0);
                                l1 = fmaf(w1, k ? i4.w : i4.y, l1);
                                // half precision holds a weight to 2^-12, and its e4m3 part exactly
                                const __half2 x = __floats2half2_rn(w0, w1);
                                hl[k] = e4m3x2(x);
                                ll[k] = e5m2x2(__hsub2(x, e4m3x2_half(hl[k])));
                            }
                            hi[e4] = hl[0] | hl[1] << 16;
                            lo[e4] = ll[0] | ll[1] << 16;
                        }
                        const int ch = 2 * part + q;
                        *reinterpret_cast<uint4*>(prow + ((ch ^ (head & 7)) << 4)) =
                            make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(prow + (((4 + ch) ^ (head & 7)) << 4)) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (!wide) l += l0 + l1;
                    const float both = l + __shfl_xor_sync(0xffffffffu, l, 16);
                    if (part == 0) {
                        sh.ref[item & 1][team][head] = ref;
                        sh.l[item & 1][team][head] = both;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[team]);
            }
            w.next(n);
        }
        if (ok) fix();
    } else {
        // ------------------------------------- q into TMEM, output out of TMEM
        const int quarter = warp & 3, part = lane >> 4, head = 16 * quarter + (lane & 15);
        const bool active = 16 * quarter < heads;
        const uint32_t trow = tbase + (uint32_t(quarter * 32) << 16);
        uint8_t* stage = pbuf + 2 * kPgPBytes + quarter * kPgStageBytes;
        int g = 2, item = 0, q_next = 0;
        bool ok = true;
        int t_prev = 0;
        bool whole_prev = false;
        int teams_prev = 0, teams_next = 0;
        float sinks[2];                          // of heads lane and lane + 32, in log2 units
#pragma unroll
        for (int k = 0; k < 2; ++k)
            sinks[k] = p.sink && lane + 32 * k < heads ? __ldg(p.sink + head0 + lane + 32 * k) * kPgLog2e : -INFINITY;

        for (PgWalk w(sh);; ++item) {
            const bool more = w.left > 0;
            const int n = more ? w.tiles(p) : 0;
            if (more) {
                const int s0 = pg_slot(q_next), s1 = pg_slot(q_next + 1), early = w.early(n);
                teams_next = n > 1 ? 3 : 1 << (g & 1);   // the softmax teams that have tiles of the item
                q_next = g + early;
                g += early < 0 ? n : n + 2;
                ok = pg_wait_warp(&sh.q_load[item & 3], uint32_t(item >> 2) & 1u, ab, &sh.status);
                if (!ok) break;
                uint8_t* qhalf = ring + (part ? s1 : s0) * kPgSlotBytes + head * 128;
                int at8[8];                      // the 16-byte pieces of a 128-byte row, swizzled
#pragma unroll
                for (int k = 0; k < 8; ++k) at8[k] = (k ^ (head & 7)) << 4;
                if (active) {
                    // largest |q| of the row; each of the head's lanes has one half
                    uint32_t top = 0;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint4 x = *reinterpret_cast<const uint4*>(qhalf + c * kPgBlockBytes + at8[k]);
                            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                         __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                        }
                    top = max(top >> 16, top & 0xffffu);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    int e2 = int(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
                    // An infinity or a NaN makes the head's output NaN, where the token has a valid rank. The
                    // scores would carry it to masked ranks too, so the row goes on as zeros and the sum is made
                    // NaN at the end, if there is one.
                    const bool odd = top >= 0x7f80u;
                    if (odd)
#pragma unroll 1
                        for (int c = 0; c < 32; ++c)
                            *reinterpret_cast<uint4*>(qhalf + (c >> 3) * kPgBlockBytes + ((c & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    e2 = odd || top == 0 ? 0 : e2 < -100 ? -100 : e2;        // (120 at most)
                    const float inv = __int_as_float((127 - e2) << 23);
                    if (part == 0) {
                        // (finite, so that a masked rank's zero stays one)
                        sh.qfac[item & 1][head] = fminf(__int_as_float((127 + e2) << 23) * p.scale * kPgLog2e, FLT_MAX);
                        sh.qodd[item & 3][head] = odd ? __int_as_float(0x7fffffff) : 0.f;
                    }
                    // in place: eight values become eight bytes hi and eight bytes lo
#pragma unroll 1
                    for (int c = 0; c < 32; c += 2) {
                        uint8_t* at = qhalf + (c >> 3) * kPgBlockBytes;
                        uint4* at0 = reinterpret_cast<uint4*>(at + (((c & 7) ^ (head & 7)) << 4));
                        uint4* at1 = reinterpret_cast<uint4*>(at + ((((c & 7) + 1) ^ (head & 7)) << 4));
                        uint4 x[2] = {*at0, *at1};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // half precision holds a scaled value and what e4m3 leaves of it exactly
                                const __half2 v = __floats2half2_rn(bf16_lo(xs[e]) * inv, bf16_hi(xs[e]) * inv);
                                hi[e] = e4m3x2(v);
                                lo[e] = e4m3x2(__hmul2(__hsub2(v, e4m3x2_half(hi[e])), __float2half2_rn(16.f)));
                            }
                            x[k] = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, lo[0] | lo[1] << 16,
                                              lo[2] | lo[3] << 16);
                        }
                        *at0 = x[0];
                        *at1 = x[1];
                    }
                }
                __syncwarp();
                if (item > 0) ok = pg_wait_warp(&sh.q_empty, uint32_t(item - 1) & 1u, ab, &sh.status);
                if (!ok) break;
                if (active) {
                    tc_fence_after();
                    const uint8_t* q0 = ring + s0 * kPgSlotBytes + head * 128 + 8 * part;
                    const uint8_t* q1 = ring + s1 * kPgSlotBytes + head * 128 + 8 * part;
#pragma unroll 2
                    for (int c = 0; c < 8; ++c) {    // 64 values of the row's part: a box
                        const uint8_t* src = (c < 4 ? q0 : q1) + (c & 3) * kPgBlockBytes;
                        uint32_t word[16];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint2 x = *reinterpret_cast<const uint2*>(src + at8[k]);
                            word[2 * k] = x.x;
                            word[2 * k + 1] = x.y;
                        }
                        tmem_st16(trow + kPgColQ + 16 * c, word);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                fence_proxy_async_smem();            // the slots' next loads come after these writes
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }
            const int done = item - 1, t = t_prev;
            const bool whole = whole_prev, first = done == 0;
            t_prev = w.t;
            whole_prev = more && w.k0 == 0 && n == pg_tiles(p, w.t);
            const int any = teams_prev;          // the softmax teams that had tiles of the item before
            teams_prev = teams_next;
            w.next(n);
            if (done < 0) {
                if (!more) break;                // a CTA without a tile
                continue;
            }
            // the output of the item before, once the next one's q is in place
            ok = pg_wait_warp(&sh.o_full, uint32_t(done) & 1u, ab, &sh.status);
            if (!ok) break;
            tc_fence_after();
            const int st = done & 1;
            float* fin = sh.fin[quarter];
            const int part_at = int(blockIdx.x) * 2 + (first ? 0 : 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = lane + 32 * j;
                if (h >= heads) continue;
                // sums are in units of 2^(reference - bias)
                const float ma = any & 1 ? sh.ref[st][0][h] : -INFINITY, mb = any & 2 ? sh.ref[st][1][h] : -INFINITY;
                const float la = any & 1 ? sh.l[st][0][h] : 0.f, lb = any & 2 ? sh.l[st][1][h] : 0.f;
                // references only rise within an item: the larger is the accumulator's
                const float mu = fmaxf(ma, mb);
                const float m2 = mu == -INFINITY ? 0.f : mu - kPgBias;
                const float sum_l = (la == 0.f || ma == mu ? la : mul_ex2(la, ma - mu)) +
                                    (lb == 0.f || mb == mu ? lb : mul_ex2(lb, mb - mu));
                const float l = sum_l == 0.f ? 0.f : sum_l + sh.qodd[done & 3][h];
                if (whole) {
                    const float sink = sinks[j];
                    // a NaN sum stays one; a sum of zero leaves the sink alone
                    const float top = l == 0.f ? sink : fmaxf(m2, sink);
                    const float base = top == -INFINITY ? 0.f : top;
                    const float sum = mul_ex2(l, m2 - base) + (p.sink ? ex2_approx(sink - base) : 0.f);
                    fin[h] = sum == 0.f ? 0.f : ex2_approx(m2 - base) / sum;
                    if (quarter == 0)
                        p.lse[int64_t(t) * p.H + head0 + h] =
                            sum == 0.f ? -INFINITY : base * kPgLn2 + logf(sum);
                } else {
                    if (quarter == 0)
                        p.part_ml[int64_t(part_at) * p.group_heads + h] = make_float2(l == 0.f ? -INFINITY : m2, l);
                }
            }
            __syncwarp();
            // 16 heads x 32 columns of D at a time, the next ones read from TMEM while these are
            // stored. A whole token's are read as matrix fragments (lane i: rows i / 4 of eight
            // columns, heads 2 (i % 4) and the next), turned by stmatrix in shared memory and stored
            // 16 bytes a lane; a part's are stored four heads of a column at a time.
            auto read = [&](int k, uint32_t (&x)[16]) {
                const uint32_t src = trow + kPgColO + 64 * (k & 3) + 16 * (k >> 2);
                if (whole) {
                    tmem_ld_frag16(src, x);
                    tmem_ld_frag16(src + (16u << 16), x + 8);
                } else {
                    tmem_ld16(src, x);
                }
            };
            auto store = [&](int k, const uint32_t (&x)[16]) {
                const int h = (k >> 2) * 16, d = 128 * (k & 3) + 32 * quarter;
                if (whole) {
                    uint8_t* at = stage + 1024 * (k & 1);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {            // heads 0-7, 8-15
                        const float2 f = *reinterpret_cast<const float2*>(fin + h + 8 * e + 2 * (lane & 3));
                        uint32_t m[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {        // rows 8r .. 8r + 7
                            const int i = 8 * (r >> 1) + 4 * e + 2 * (r & 1);
                            m[r] = pack_bf16x2(__uint_as_float(x[i]) * f.x, __uint_as_float(x[i + 1]) * f.y);
                        }
                        // 64-byte rows, pieces of 16 bytes swizzled
                        const int r = 8 * e + (lane & 7), c = lane >> 3;
                        stmatrix_x4_trans(at + r * 64 + ((c ^ ((r >> 1) & 3)) << 4), m);
                    }
                    __syncwarp();
                    uint4* dst = reinterpret_cast<uint4*>(p.o + (int64_t(t) * p.H + head0 + h) * kD + d);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * e + (lane >> 2), c = lane & 3;
                        dst[r * (kD / 8) + c] =
                            *reinterpret_cast<const uint4*>(at + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
                    }
                } else {
                    float4* dst = reinterpret_cast<float4*>(p.part_o) +
                                  (int64_t(part_at) * (p.group_heads / 4) + h / 4) * kD + d + lane;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e * kD] = make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                                                  __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3]));
                }
            };
            uint32_t v[2][16];
            read(0, v[0]);
            tmem_wait_ld();
            const int chunks = heads / 4;
#pragma unroll 1
            for (int k = 0; k < chunks; k += 2) {
                read(k + 1, v[1]);
                store(k, v[0]);
                tmem_wait_ld();
                if (k + 2 < chunks) {
                    read(k + 2, v[0]);
                } else {                         // all of the accumulator is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.o_empty);
                }
                store(k + 1, v[1]);
                tmem_wait_ld();
            }
            if (!more) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) p.cta_status[blockIdx.x] = sh.status;
    if (warp == kPgMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Joins the parts of a token that several CTAs shared, in a fixed order (so the result does not
// depend on the run): o = sum_i 2^(m_i - m) O_i / (sum_i 2^(m_i - m) l_i + 2^(sink - m)), in fp32.
// kSplit 0: block (c, y) joins the token that ends in CTA c, heads 4y .. 4y + 3 of its group; a
// thread has 512 / kThreads columns of all four. Else block (x, y, z) belongs to a token and group,
// x = t * groups + group, looks for the CTA that ends it, and has 512 / kSplit columns; kStep
// threads share a column, each with every kStep-th part, and their sums are added in order.
// One block also joins the CTAs' status bits.
// Bound: the latency of the first look-ups, then L2 (a part is 2 KB a head, written by the
// kernel before); 152 CTAs have at most two parts each. ~3 us after the kernel above at 128
// tokens of 64 heads, 10 us with cold caches.
template <int kThreads, int kSplit>
__global__ void __launch_bounds__(kThreads) combine_paged_kernel(const PgParams p) {
    constexpr bool kFew = kSplit > 0;
    constexpr int kWidth = kFew ? kD / kSplit : kD, kStep = kFew ? kThreads / kWidth : 1;     // columns, threads a column
    constexpr int kWarps = kThreads / 32, kCols = kFew ? 1 : kD / kThreads;
    constexpr int kRounds = (kPgMaxCtas + kThreads / 4 - 1) / (kThreads / 4);
    __shared__ float4 wgt[kPgMaxCtas];
    __shared__ float red[2][kWarps];
    __shared__ float4 inv_of;
    const int group = int(blockIdx.x) % p.groups;
    grid_dep_wait();
    grid_dep_launch();
    int4 end;
    if (kFew) {
        static_assert(!kFew || (kThreads >= kPgMaxCtas && kThreads % kWidth == 0), "a thread a CTA, whole columns");
        __shared__ int4 found;
        if (threadIdx.x == 0) found = make_int4(-1, 0, 0, 0);
        __syncthreads();
        if (int(threadIdx.x) < p.ctas) {
            int4 m = __ldcg(p.meta + threadIdx.x * p.groups + group);
            m.w = threadIdx.x;
            if (m.x == int(blockIdx.x) / p.groups) found = m;
        }
        __syncthreads();
        end = found;
    } else {
        end = __ldcg(p.meta + blockIdx.x);
        end.w = int(blockIdx.x) / p.groups;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) {
        unsigned bits = 0;
        for (int c = threadIdx.x; c < p.ctas * p.groups; c += 32) bits |= __ldcg(p.cta_status + c);
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (threadIdx.x == 0) *p.status = bits;
    }
    if (end.x < 0) return;
    const int h0 = 4 * int(blockIdx.y), head0 = group * p.group_heads + h0;
    if (head0 >= p.H) return;                            // (heads come in sixteens)
    const int n = end.w - end.y + 1;                     // parts, at most the CTAs of a group
    auto part_of = [&](int i) {
        return (int64_t(end.y + i) * p.groups + group) * 2 + (i == 0 ? end.z : 0);
    };
    // weights: a quarter of the threads a head
    const int k = threadIdx.x / (kThreads / 4), lane = threadIdx.x % (kThreads / 4);
    const float sink = p.sink ? __ldg(p.sink + head0 + k) * kPgLog2e : -INFINITY;
    float2 ml[kRounds];
    float top = sink;
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = lane + kThreads / 4 * j;
        ml[j] = i < n ? __ldcg(p.part_ml + part_of(i) * p.group_heads + h0 + k) : make_float2(-INFINITY, 0.f);
        if (ml[j].y != 0.f) top = fmaxf(top, ml[j].x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kWarps / 4; ++j) top = fmaxf(top, red[0][kWarps / 4 * k + j]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = lane + kThreads / 4 * j;
        const float w = ml[j].y == 0.f ? 0.f : ex2_approx(ml[j].x - base);
        if (i < n) reinterpret_cast<float*>(wgt + i)[k] = w;
        if (ml[j].y != 0.f) sum += mul_ex2(ml[j].y, ml[j].x - base);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((threadIdx.x & 31) == 0) red[1][threadIdx.x >> 5] = sum;
    __syncthreads();
    if (lane == 0) {                             // (blocks of the same heads write the same lse)
        sum = p.sink ? ex2_approx(sink - base) : 0.f;
#pragma unroll
        for (int j = 0; j < kWarps / 4; ++j) sum += red[1][kWarps / 4 * k + j];
        reinterpret_cast<float*>(&inv_of)[k] = sum == 0.f ? 0.f : 1.f / sum;
        p.lse[int64_t(end.x) * p.H + head0 + k] = sum == 0.f ? -INFINITY : base * kPgLn2 + logf(sum);
    }
    __syncthreads();
    const int col = kFew ? kWidth * int(blockIdx.z) + int(threadIdx.x) % kWidth : int(threadIdx.x);
    const int start = kFew ? int(threadIdx.x) / kWidth : 0;      // the thread's first part
    float4 acc[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t size = int64_t(p.group_heads / 4) * kD;        // float4s of a part
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + (h0 / 4) * kD + col;
    auto add = [&](const float4* at, int i) {
        const float4 w = wgt[i];
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float4 v = __ldcg(at + kThreads * j);
            acc[j].x = fmaf(w.x, v.x, acc[j].x);
            acc[j].y = fmaf(w.y, v.y, acc[j].y);
            acc[j].z = fmaf(w.z, v.z, acc[j].z);
            acc[j].w = fmaf(w.w, v.w, acc[j].w);
        }
    };
    if (start == 0) add(src + part_of(0) * size, 0);
    const float4* rest = src + part_of(1) * size;
#pragma unroll (8 / kCols)
    for (int i = start == 0 ? kStep : start; i < n; i += kStep) add(rest + (i - 1) * 2 * p.groups * size, i);
    if (kStep > 1) {
        __shared__ float4 part_sum[kStep > 1 ? kStep - 1 : 1][kWidth];
        if (start > 0) part_sum[start - 1][threadIdx.x % kWidth] = acc[0];
        __syncthreads();
        if (start > 0) return;
#pragma unroll
        for (int k = 0; k < kStep - 1; ++k) {
            const float4 v = part_sum[k][threadIdx.x];
            acc[0].x += v.x;
            acc[0].y += v.y;
            acc[0].z += v.z;
            acc[0].w += v.w;
        }
    }
    const float4 f = inv_of;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + (int64_t(end.x) * p.H + head0) * kD + col;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        __nv_bfloat16* to = dst + kThreads * j;
        to[0] = __float2bfloat16_rn(acc[j].x * f.x);
        to[kD] = __float2bfloat16_rn(acc[j].y * f.y);
        to[2 * kD] = __float2bfloat16_rn(acc[j].z * f.z);
        to[3 * kD] = __float2bfloat16_rn(acc[j].w * f.w);
    }
}

namespace {

struct PgPlan { int groups, group_heads; size_t status, meta, ml, o, bytes; };

PgPlan plan_paged(int H) {
    PgPlan x{};
    x.groups = (H + kPgHeads - 1) / kPgHeads;
    x.group_heads = (H / 16 + x.groups - 1) / x.groups * 16;
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes, 256); return o; };
    x.status = take(size_t(kPgMaxCtas) * 4);
    x.meta = take(size_t(kPgMaxCtas) * sizeof(int4));
    x.ml = take(size_t(kPgMaxCtas) * 2 * x.group_heads * sizeof(float2));
    x.o = take(size_t(kPgMaxCtas) * 2 * x.group_heads * kD * 4);
    x.bytes = off;
    return x;
}

}  // namespace

size_t paged_scratch_bytes(int T, int H) { return T > 0 ? plan_paged(H).bytes : 0; }

cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t s) {
    static bool attr_done[64] = {false};
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(fwd_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmem);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const PgPlan plan = plan_paged(a.H);
    const CacheView& c = a.cache;
    const uint64_t rows = uint64_t(c.num_pages) << c.page_shift;
    const uint32_t box = (1 << c.page_shift) < kPgTile ? uint32_t(1) << c.page_shift : uint32_t(kPgTile);
    CUtensorMap mq, mb;
    if (!make_tmap_bf16_2d(&mq, a.q, uint64_t(a.T) * a.H, kD, kD, plan.group_heads, 64, true) ||
        !make_tmap_u8_rows(&mb, c.pages, rows, box))
        return cudaErrorInvalidValue;
    PgParams p{};
    p.table = a.table; p.seq = a.seq; p.lens = a.lens; p.topk = a.topk;
    p.pages = c.pages; p.scales = c.scales; p.sink = a.sink; p.o = a.o; p.lse = a.lse;
    p.T = a.T; p.H = a.H; p.K = a.K; p.B = a.B; p.max_pages = a.max_pages;
    p.num_pages = c.num_pages; p.page_shift = c.page_shift; p.block_shift = c.block_shift;
    p.groups = plan.groups; p.group_heads = plan.group_heads;
    p.scale = a.scale; p.status = a.status;
    p.cta_status = reinterpret_cast<unsigned*>(a.scratch + plan.status);
    p.meta = reinterpret_cast<int4*>(a.scratch + plan.meta);
    p.part_ml = reinterpret_cast<float2*>(a.scratch + plan.ml);
    p.part_o = reinterpret_cast<float*>(a.scratch + plan.o);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int ctas = (sms < kPgMaxCtas ? sms : kPgMaxCtas) / plan.groups;
    p.ctas = ctas;
    // Programmatic launches: a kernel's blocks may start when the one before no longer needs the SMs,
    // and wait for its end (grid_dep_wait) before they read or write anything.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas * plan.groups);
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = kPgSmem;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fwd_paged_kernel, mq, mb, p);
    if (e != cudaSuccess) return e;
    // The join: few tokens have blocks of their own, with their columns split as far as the blocks stay
    // within 256 (more wait for one another, fewer leave the parts of a long token to few SMs); more
    // tokens have two or three parts each, and a block for each CTA and four heads, of 128 threads,
    // so that most are on the GPU at once. Device time of a call, us (T x positions, heads;
    // columns split in 8 / 4 / 2 / 1 / a block a CTA):
    //   1 x 81920, 64: 24.8 / 28.0 / 31.7 / 39.2 / 82.7     8 x 10000, 64: - / 30.3 / 27.4 / 28.3 / 35.5
    //   16 x 5000, 64: - / 34.3 / 30.7 / 27.8 / 31.4        31 x 2500, 128: - / 60.8 / 48.0 / 39.6 / 36.5
    const int64_t work = int64_t(a.T) * a.H;                 // four times the blocks of a split of 1
    const int split = work <= 128 ? 8 : work <= 256 ? 4 : work <= 512 ? 2 : work <= 1024 ? 1 : 0;
    cfg.gridDim = dim3((split ? a.T : ctas) * plan.groups, plan.group_heads / 4, split ? split : 1);
    cfg.blockDim = dim3(split ? 512 : 128);
    cfg.dynamicSmemBytes = 0;
    switch (split) {
        case 8: e = cudaLaunchKernelEx(&cfg, combine_paged_kernel<512, 8>, p); break;
        case 4: e = cudaLaunchKernelEx(&cfg, combine_paged_kernel<512, 4>, p); break;
        case 2: e = cudaLaunchKernelEx(&cfg, combine_paged_kernel<512, 2>, p); break;
        case 1: e = cudaLaunchKernelEx(&cfg, combine_paged_kernel<512, 1>, p); break;
        default: e = cudaLaunchKernelEx(&cfg, combine_paged_kernel<128, 0>, p);
    }
    if (e != cudaSuccess) return e;
    note_launch(2);
    return cudaGetLastError();
}

}  // namespace smla
