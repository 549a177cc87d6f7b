// k_beam_select.cu -- the next beams of each group: the n best of beams x vocabulary.
//
// Candidate (k, v) of a group scores scores[k] + logits[k,v] - logsumexp(logits[k,:]); a finished beam has the
// one candidate (k, eos) with scores[k]. Best first, ties by k, the logit, then v; scores that are not finite are never
// taken.
//
// A row's candidates rank as its logits do, so one pass over the logits gives both parts of the answer:
// beam_rows_kernel cuts a row into chunks, keeps the maxima of a chunk's vectors in registers, and writes its maximum, its
// sum of exponentials and its n best logits; beam_merge_kernel joins a row's sums and merges the lists of a group.
//
// Log-sums: a thread adds 64 exponentials (16-bit types: 128) in fp32, two vectors' as a tree, and scales its sum when its
// maximum rises; the threads of a CTA are joined in fp32 pairs (48 bits), chunks and rows in 64 bits. A value d below its row's
// maximum passes up to 13 additions, 8 scalings and 9 ex2.approx (2^-22 each), and its argument is off by up to 2.7 d 2^-24:
// 100 2^-24 at most, as sum_i w_i d_i <= log V; 2^-23 as a rule. 64-bit exponentials would take the fp64 units ms.
// Scores are compared in 64 bits. Sums do not depend on where a row starts: equal rows, equal sums.
//
// Bound: 256 rows of 128000 in bf16 (65.5 MB): 25 us, of which the rows take 13.4 (4.9 TB/s) and the merge 7 with its
// start behind them; 4 rows of 32000 in fp32: 11 us. Chunks of 64 KB in groups of two loads a thread, six CTAs an
// SM: 25.7 us; of four, four CTAs: 27.2; 512 threads: 28.7; chunks of 32 KB held in registers whole: 32, and of 16 KB 40.
// The merge: log-sums 3 us (64-bit exponentials and logarithms: latency), bound and ranks 3. Rows between 16-byte
// boundaries, of which a vector is cut from two loads: 256 of 128001 in bf16 32.5 us.
//
// A chunk's n best: a bound that n to 2n threads' largest values reach (bisection over their bits, a count and a
// barrier a step), so that at most 2 n threads' values pass it, then their exact ranks among those.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "smla_internal.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr int kBsThreads = 256;
constexpr int kBsVecs = 16, kBsGroup = 2;        // 16-byte vectors of a thread; on their way together
constexpr int kBsMergeThreads = 512;
constexpr int kBsEach = 4;                       // candidates of a thread of the merge
constexpr int kBsBatch = kBsMergeThreads * kBsEach;
static_assert(SMLA_MAX_VOCAB / (kBsThreads * kBsVecs * 4) <= kBsMergeThreads, "a row's chunks are joined in one part");
constexpr float kBsLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Two floats at a time.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
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

// What a type's 16-byte vectors hold; kNone: words of -inf.
template <int kType>
struct Logit;
template <>
struct Logit<SMLA_F32> {
    static constexpr int kSize = 4;
    static constexpr uint32_t kNone = 0xff800000u;
    static __device__ __forceinline__ void copy(uint4* to, int e, const uint8_t* row, int i, int V) {
        reinterpret_cast<uint32_t*>(to)[e] = i < V ? __ldg(reinterpret_cast<const uint32_t*>(row) + i) : kNone;
    }
    static __device__ __forceinline__ float top(const uint4& x) {
        return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)),
                     fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
    }
    static __device__ __forceinline__ void spread(const uint4& x, float* v) {
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
    }
};
template <>
struct Logit<SMLA_BF16> {
    static constexpr int kSize = 2;
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ void copy(uint4* to, int e, const uint8_t* row, int i, int V) {
        reinterpret_cast<uint16_t*>(to)[e] = i < V ? __ldg(reinterpret_cast<const uint16_t*>(row) + i) : 0xff80u;
    }
    static __device__ __forceinline__ float top(const uint4& x) {
        auto as = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(as(x.x), as(x.y)), __hmax2(as(x.z), as(x.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void spread(const uint4& x, float* v) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
    }
};
template <>
struct Logit<SMLA_F16> {
    static constexpr int kSize = 2;
    static constexpr uint32_t kNone = 0xfc00fc00u;
    static __device__ __forceinline__ void copy(uint4* to, int e, const uint8_t* row, int i, int V) {
        reinterpret_cast<uint16_t*>(to)[e] = i < V ? __ldg(reinterpret_cast<const uint16_t*>(row) + i) : 0xfc00u;
    }
    static __device__ __forceinline__ float top(const uint4& x) {
        auto as = [](uint32_t w) { return *reinterpret_cast<const __half2*>(&w); };
        const float2 m = __half22float2(__hmax2(__hmax2(as(x.x), as(x.y)), __hmax2(as(x.z), as(x.w))));
        return fmaxf(m.x, m.y);
    }
    static __device__ __forceinline__ void spread(const uint4& x, float* v) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x; v[2 * i + 1] = f.y;
        }
    }
};

constexpr int chunk_of(int type) { return kBsThreads * kBsVecs * (type == SMLA_F32 ? 4 : 8); }
// values that pass a chunk's bound at most: those of 2 n threads
constexpr size_t passing(int type, int n) { return size_t(2) * n * kBsVecs * (type == SMLA_F32 ? 4 : 8); }

// The 16 bytes from byte `off` of two vectors on; off is a multiple of kSize.
template <int kSize>
__device__ __forceinline__ uint4 cut(const uint4& lo, const uint4& hi, int off) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
    if (kSize < 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ bool out_of_play(const BeamArgs& a, int row) {
    const float s = __ldg(a.scores + row);
    return !(fabsf(s) < INFINITY) || (a.done && __ldg(a.done + row));
}

}  // namespace

// kShift: rows may start between 16-byte boundaries.
template <int kType, bool kShift>
__global__ void __launch_bounds__(kBsThreads, kShift ? 4 : 6)
beam_rows_kernel(const BeamArgs a) {
    constexpr int kSize = Logit<kType>::kSize, kEach = 16 / kSize;
    extern __shared__ __align__(16) unsigned long long best[];    // values that pass the bound
    __shared__ uint32_t warp_top[kBsThreads / 32], warp_low[kBsThreads / 32];
    __shared__ float2 warp_sum[kBsThreads / 32];
    __shared__ uint4 ends[3];
    __shared__ int count;
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = int(blockIdx.x), chunk = int(blockIdx.y);
    if (out_of_play(a, row)) return;             // (nobody looks at its lists)
    // Vector v of a row is its values from kEach * v on, wherever they lie: what is added to what goes by the values'
    // indices alone, and equal rows have equal sums. A vector between two boundaries is cut from two aligned ones.
    // [from, to) are the vectors that can be, without a look outside of the row; its others, at most one at its start and
    // two at its end, come value by value into `ends`.
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + int64_t(row) * a.stride * kSize;
    const int off = kShift ? int(reinterpret_cast<uintptr_t>(base) & 15) : 0;
    const int vecs = (a.V + kEach - 1) / kEach, from = off ? 1 : 0;
    const int to = max(from, kShift ? (a.V * kSize + off) / 16 - 1 : a.V / kEach);
    const int chunk0 = chunk * kBsThreads * kBsVecs, first = chunk0 + int(threadIdx.x);
    const uint4* src = reinterpret_cast<const uint4*>(base - off) + first;
    constexpr uint32_t kNone = Logit<kType>::kNone;
    const uint4 none4 = make_uint4(kNone, kNone, kNone, kNone);
    uint4 raw[2][kBsGroup][kShift ? 2 : 1];
    auto load = [&](int g) {
#pragma unroll
        for (int k = 0; k < kBsGroup; ++k) {
            const int at = (g * kBsGroup + k) * kBsThreads;
            const bool whole = first + at >= from && first + at < to;
#pragma unroll
            for (int h = 0; h < (kShift ? 2 : 1); ++h) raw[g & 1][k][h] = whole ? __ldg(src + at + h) : none4;
        }
    };
    load(0);
    uint32_t odd = 0;                            // which of the thread's vectors are in `ends`
    if (first < from) odd = 1;
#pragma unroll
    for (int i = 0; i < (kShift ? 2 : 1); ++i) {
        const int d = to + i - first;
        if (to + i < vecs && d >= 0 && d % kBsThreads == 0 && d < kBsThreads * kBsVecs) odd |= 1u << (d / kBsThreads);
    }
    auto slot = [&](int v) { return !kShift ? 1 : v < from ? 0 : 1 + v - to; };
    if (threadIdx.x < 3 * kEach) {
        const int i = threadIdx.x / kEach, e = threadIdx.x % kEach, v = i ? to + i - 1 : 0;
        if ((i || from) && v >= chunk0 && v < min(vecs, chunk0 + kBsThreads * kBsVecs))
            Logit<kType>::copy(ends + i, e, base, v * kEach + e, a.V);
    }
    __syncthreads();

    // A thread's largest value and its sum of exponentials relative to it, which follow each other from group to group
    // (two values at a time); the largest of each vector.
    const uint64_t log2e = pair_of(kBsLog2e, kBsLog2e);
    float tops[kBsVecs], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int g = 0; g < kBsVecs / kBsGroup; ++g) {
        uint4 now[kBsGroup];
        if (g + 1 < kBsVecs / kBsGroup) load(g + 1);
        float high = top;                        // (maxima pass over NaN)
#pragma unroll
        for (int k = 0; k < kBsGroup; ++k) {
            const int i = g * kBsGroup + k;
            now[k] = kShift ? cut<kSize>(raw[g & 1][k][0], raw[g & 1][k][kShift], off) : raw[g & 1][k][0];
            if ((odd >> i) & 1) now[k] = ends[slot(first + i * kBsThreads)];
            tops[g * kBsGroup + k] = Logit<kType>::top(now[k]);
            high = fmaxf(high, tops[g * kBsGroup + k]);
        }
        if (high > top) sum *= ex2_approx((top - high) * kBsLog2e);      // (top -inf: sum is 0)
        top = high;
        const float ref = top == -INFINITY ? 0.f : top;
        const uint64_t shift = pair_of(-ref, -ref);
        uint64_t part[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kBsGroup; ++k) {
            float v[kEach];
            Logit<kType>::spread(now[k], v);
#pragma unroll
            for (int e = 0; e < kEach; e += 2) {
                const float2 t = floats_of(mul2(add2(pair_of(v[e], v[e + 1]), shift), log2e));
                part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], pair_of(ex2_approx(t.x), ex2_approx(t.y)));
            }
        }
        const float2 both = floats_of(add2(part[0], part[1]));
        sum += both.x + both.y;
    }
    const uint32_t mine = order_of(top + 0.f);   // (both zeros alike)
    const uint32_t wt = __reduce_max_sync(0xffffffffu, mine), wl = __reduce_min_sync(0xffffffffu, mine);
    if (lane == 0) { warp_top[warp] = wt; warp_low[warp] = wl; }
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    uint32_t most = 0, least = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kBsThreads / 32; ++w) { most = max(most, warp_top[w]); least = min(least, warp_low[w]); }
    const uint32_t none = order_of(-INFINITY);
    const float peak = value_of(most), ref = most == none ? 0.f : peak;

    // The values of the thread's vectors that hold one of at least `from`, one after the other: few threads do this, so
    // the vectors are loaded again, in code that is short (the kernel waited for instructions most when it was not).
    auto look = [&](auto each, float from) {
        uint32_t which = 0;
#pragma unroll
        for (int k = 0; k < kBsVecs; ++k) which |= uint32_t(tops[k] >= from) << k;
#pragma unroll 1
        for (; which; which &= which - 1) {
            const int k = __ffs(which) - 1;
            const int at = k * kBsThreads;
            uint4 again;
            if ((odd >> k) & 1) again = ends[slot(first + at)];
            else again = kShift ? cut<kSize>(__ldg(src + at), __ldg(src + at + 1), off) : __ldg(src + at);
            float v[kEach];
            Logit<kType>::spread(again, v);
#pragma unroll
            for (int e = 0; e < kEach; ++e) each(v[e], (first + at) * kEach + e);
        }
    };
    // The bound: threads whose largest value reaches it number n to 2n. Where many threads' are equal to it, their
    // first places decide (`until`).
    const int n = a.n;
    uint32_t bound = least > none ? least : none + 1, above = most + 1;
    int until = INT32_MAX;
    int reached = __syncthreads_count(mine >= bound);
    if (reached > 2 * n) {
        while (above - bound > 1 && reached > 2 * n) {
            const uint32_t mid = bound + (above - bound) / 2;
            const int r = __syncthreads_count(mine >= mid);
            if (r >= n) { bound = mid; reached = r; } else above = mid;
        }
        if (reached > 2 * n) {
            const int over = __syncthreads_count(mine > bound);
            const float at = value_of(bound);
            int place = INT32_MAX;               // of the thread's first value that is equal
            if (mine == bound) look([&](float y, int i) { if (y == at) place = min(place, i); }, at);
            int lo = -1, hi = a.V - 1;           // too few up to lo, enough up to hi
            until = hi;
            while (hi - lo > 1 && reached > 2 * n) {
                const int mid = lo + (hi - lo) / 2;
                const int r = over + __syncthreads_count(mine == bound && place <= mid);
                if (r >= n) { hi = until = mid; reached = r; } else lo = mid;
            }
        }
    }
    if (mine >= bound) {
        auto pass = [&](float y, int i) {
            const uint32_t o = order_of(y + 0.f);
            if (y != y || !(o > bound || (o == bound && i <= until))) return;
            best[atomicAdd(&count, 1)] = (static_cast<unsigned long long>(o) << 32) | (0xffffffffu - uint32_t(i));
        };
        look(pass, value_of(bound));
    }
    // the threads' sums, relative to the chunk's largest, with what each addition rounds off beside them (64-bit
    // additions of a warp occupy their unit for 16 cycles each)
    if (top != peak) sum *= ex2_approx((top - ref) * kBsLog2e);
    float all = sum, rest = 0.f;
    auto add = [&](float y, float more) {
        const float both = all + y, z = both - all;
        rest += ((all - (both - z)) + (y - z)) + more;
        all = both;
    };
#pragma unroll
    for (int d = 16; d; d >>= 1)
        add(__shfl_xor_sync(0xffffffffu, all, d), __shfl_xor_sync(0xffffffffu, rest, d));
    if (lane == 0) warp_sum[warp] = make_float2(all, rest);
    __syncthreads();
    const int c = count;
    const int64_t part_at = int64_t(row) * a.chunks + chunk;
    for (int i = threadIdx.x; i < c; i += kBsThreads) {
        const unsigned long long key = best[i];
        int rank = 0;
        for (int j = 0; j < c; ++j) rank += best[j] > key;
        if (rank < n) a.lists[part_at * n + rank] = key;
    }
    for (int i = c + threadIdx.x; i < n; i += kBsThreads) a.lists[part_at * n + i] = 0;
    if (threadIdx.x == kBsThreads - 1) {
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kBsThreads / 32; ++w) total += double(warp_sum[w].x) + double(warp_sum[w].y);
        a.peaks[part_at] = peak;
        a.sums[part_at] = total;
    }
}

// A score a little below the one that a key stands for.
__device__ __forceinline__ float float_below(unsigned long long key) {
    return __double2float_rd(__longlong_as_double(key >> 63 ? key ^ (1ull << 63) : ~key));
}

// Where a candidate of beam k stands among those of equal scores: by beam, then by its logit (a score of a large size
// rounds off what tells a beam's logits apart), then by token.
__device__ __forceinline__ unsigned long long place_of(int k, uint32_t order, int v) {
    static_assert(SMLA_MAX_VOCAB == 1 << 22 && SMLA_MAX_BEAMS <= 1 << 10, "22 bits of token, 32 of logit, 10 of beam");
    return static_cast<unsigned long long>(k) << 54 | static_cast<unsigned long long>(~order) << 22 | uint32_t(v);
}

// A group's n best out of its rows' chunks' lists (each best first), 2048 candidates less the n best so far at a time:
// the n-th of a list has n - 1 better ones, so nothing below the best n-th matters; the rest rank by counting.
__global__ void __launch_bounds__(kBsMergeThreads)
beam_merge_kernel(const BeamArgs a) {
    __shared__ double lse[SMLA_MAX_BEAMS], before[SMLA_MAX_BEAMS];
    __shared__ int state[SMLA_MAX_BEAMS];        // 0: runs, 1: ended, 2: dead
    __shared__ float peaks[kBsMergeThreads], row_peak[SMLA_MAX_BEAMS];
    __shared__ double sums[kBsMergeThreads];
    __shared__ float warp_bar[kBsMergeThreads / 32];
    __shared__ unsigned long long keys[kBsBatch];
    __shared__ unsigned long long places[kBsBatch];
    __shared__ unsigned long long top_keys[SMLA_MAX_BEAMS];
    __shared__ unsigned long long top_places[SMLA_MAX_BEAMS];
    __shared__ int count;
    grid_dep_wait();
    const int b = int(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (b == 0 && threadIdx.x == 0) *a.status = 0;
    const int n = a.n, total = a.K * a.chunks * n;
    const int64_t row0 = int64_t(b) * a.K;
    // candidate j of the group: entry j % n of list j / n, read ahead of the sums
    const int batch = kBsBatch - n;
    unsigned long long raw[kBsEach];
    auto read = [&](int base) {
#pragma unroll
        for (int e = 0; e < kBsEach; ++e) {
            const int i = e * kBsMergeThreads + int(threadIdx.x), j = base + i;
            raw[e] = i < batch && j < total ? __ldcg(a.lists + row0 * a.chunks * n + j) : 0;
        }
    };
    read(0);
    // The rows' log-sums. 64-bit instructions are slow and cost a warp as much for one lane as for 32: exponentials
    // of many chunks a warp, logarithms of many rows.
    for (int k = threadIdx.x; k < a.K; k += kBsMergeThreads) {
        const float s = __ldg(a.scores + row0 + k);
        before[k] = s;
        state[k] = !(fabsf(s) < INFINITY) ? 2 : a.done && __ldg(a.done + row0 + k) ? 1 : 0;
    }
    const int lists = a.K * a.chunks;
    const int part = kBsMergeThreads / a.chunks * a.chunks;              // whole rows: all sums are made alike
    for (int l0 = 0; l0 < lists; l0 += part) {
        const int l = l0 + int(threadIdx.x), l1 = min(l0 + part, lists);
        if (l < l1) {
            peaks[threadIdx.x] = __ldcg(a.peaks + row0 * a.chunks + l);
            sums[threadIdx.x] = __ldcg(a.sums + row0 * a.chunks + l);
        }
        __syncthreads();
        const int k0 = l0 / a.chunks, i0 = int(threadIdx.x) * a.chunks;  // a row's peak and sum: a thread a row
        const bool mine = k0 + int(threadIdx.x) < l1 / a.chunks;
        if (mine) {
            float peak = -INFINITY;
            for (int i = i0; i < i0 + a.chunks; ++i) peak = fmaxf(peak, peaks[i]);
            row_peak[threadIdx.x] = peak;
        }
        __syncthreads();
        if (l < l1) {
            const float peak = peaks[threadIdx.x], most = row_peak[threadIdx.x / a.chunks];
            if (peak != most) sums[threadIdx.x] *= exp(double(peak) - double(most));
        }
        __syncthreads();
        if (mine) {
            double sum = 0.0;
            for (int i = i0; i < i0 + a.chunks; ++i) sum += sums[i];
            lse[k0 + threadIdx.x] = double(row_peak[threadIdx.x]) + log(sum);
        }
        __syncthreads();
    }
    int have = 0;                                // of the best so far
    for (int base = 0; base < total; base += batch) {
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        // In 32 bits first, with room for their rounding: what is below the bar for sure is never looked at in 64.
        float low[kBsEach], high[kBsEach], bar = have == n ? float_below(top_keys[n - 1]) : -INFINITY;
#pragma unroll
        for (int e = 0; e < kBsEach; ++e) {
            const int i = e * kBsMergeThreads + int(threadIdx.x), j = base + i;
            high[e] = __int_as_float(0x7fffffff);                        // NaN: no candidate
            if (i >= batch || j >= total) continue;
            const int list = j / n, at = j - list * n, k = list / a.chunks, st = state[k];
            if (st == 0 ? raw[e] == 0 : st == 2 || at > 0 || list != k * a.chunks) continue;
            const float s = float(before[k]), x = st ? 0.f : value_of(uint32_t(raw[e] >> 32)), l = st ? 0.f : float(lse[k]);
            const float sum = s + (x - l), room = 0x1p-21f * (fabsf(s) + fabsf(x) + fabsf(l)) + 0x1p-100f;
            // (where 32 bits overflow, nothing is for sure)
            high[e] = fabsf(sum) < INFINITY && room < INFINITY ? sum + room : INFINITY;
            low[e] = fabsf(sum) < INFINITY && room < INFINITY ? sum - room : -INFINITY;
            if (at == n - 1 && st == 0) bar = fmaxf(bar, low[e]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) bar = fmaxf(bar, __shfl_xor_sync(0xffffffffu, bar, d));
        if (lane == 0) warp_bar[warp] = bar;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kBsMergeThreads / 32; ++w) bar = fmaxf(bar, warp_bar[w]);
#pragma unroll
        for (int e = 0; e < kBsEach; ++e)
            if (high[e] >= bar) {
                const int at = atomicAdd(&count, 1);
                keys[at] = raw[e];
                places[at] = base + e * kBsMergeThreads + int(threadIdx.x);
            }
        if (base + batch < total) read(base + batch);
        __syncthreads();
        // those in 64 bits; one that is not finite is 0, below all
        for (int i = threadIdx.x; i < count; i += kBsMergeThreads) {
            const unsigned long long was = keys[i];
            const int list = int(places[i]) / n, k = list / a.chunks;
            const bool ended = state[k] != 0;
            const double s = ended ? before[k] : before[k] + (double(value_of(uint32_t(was >> 32))) - lse[k]);
            const long long bits = __double_as_longlong(s + 0.0);
            keys[i] = !(fabs(s) < INFINITY) ? 0 : bits < 0 ? ~bits : bits | (1ll << 63);
            places[i] = place_of(k, ended ? 0u : uint32_t(was >> 32), ended ? a.eos : int(0xffffffffu - uint32_t(was)));
        }
        __syncthreads();
        if (threadIdx.x < have) {
            const int at = atomicAdd(&count, 1);
            keys[at] = top_keys[threadIdx.x];
            places[at] = top_places[threadIdx.x];
        }
        __syncthreads();
        const int c = count;
        for (int i = threadIdx.x; i < c; i += kBsMergeThreads) {
            const unsigned long long mine = keys[i];
            const unsigned long long place = places[i];
            int rank = 0;
            for (int j = 0; j < c; ++j) rank += keys[j] > mine || (keys[j] == mine && places[j] < place);
            if (rank < n) { top_keys[rank] = mine; top_places[rank] = place; }
        }
        __syncthreads();
        have = c < n ? c : n;
        while (have > 0 && top_keys[have - 1] == 0) --have;
    }
    if (threadIdx.x < n) {
        const int64_t at = int64_t(b) * n + threadIdx.x;
        const bool any = threadIdx.x < have;
        const unsigned long long place = any ? top_places[threadIdx.x] : 0;
        const unsigned long long key = any ? top_keys[threadIdx.x] : 0;
        const double s = __longlong_as_double(key >> 63 ? key ^ (1ull << 63) : ~key);
        a.parents[at] = any ? int(row0) + int(place >> 54) : -1;
        a.tokens[at] = any ? int(place & (SMLA_MAX_VOCAB - 1)) : -1;
        a.new_scores[at] = any ? float(s) : -INFINITY;
    }
}

namespace {

struct BeamPlan { size_t peaks, sums, lists, bytes; int chunks; };

BeamPlan plan_beam(int64_t rows, int V, int n, int type) {
    BeamPlan p{};
    p.chunks = (V + chunk_of(type) - 1) / chunk_of(type);
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes, 256); return o; };
    p.peaks = take(size_t(rows) * p.chunks * 4);
    p.sums = take(size_t(rows) * p.chunks * 8);
    p.lists = take(size_t(rows) * p.chunks * n * 8);
    p.bytes = off;
    return p;
}

template <int kType, bool kShift>
cudaError_t launch_rows(const BeamArgs& a, cudaStream_t s) {
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(beam_rows_kernel<kType, kShift>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   int(passing(kType, SMLA_MAX_BEAMS) * 8));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    beam_rows_kernel<kType, kShift><<<dim3(unsigned(a.B) * a.K, a.chunks), kBsThreads, passing(kType, a.n) * 8, s>>>(a);
    return cudaGetLastError();
}

template <int kType>
cudaError_t launch_rows(const BeamArgs& a, cudaStream_t s) {
    const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                         (int64_t(a.B) * a.K == 1 || a.stride * Logit<kType>::kSize % 16 == 0);
    return aligned ? launch_rows<kType, false>(a, s) : launch_rows<kType, true>(a, s);
}

}  // namespace

// (of the type with the smaller chunks)
size_t beam_scratch_bytes(int B, int K, int V, int n) { return plan_beam(int64_t(B) * K, V, n, SMLA_F32).bytes; }
int beam_chunks(int V) { return plan_beam(1, V, 1, SMLA_F32).chunks; }

cudaError_t launch_beam_select(BeamArgs a, int type, char* scratch, cudaStream_t s) {
    const BeamPlan p = plan_beam(int64_t(a.B) * a.K, a.V, a.n, type);
    a.chunks = p.chunks;
    a.peaks = reinterpret_cast<float*>(scratch + p.peaks);
    a.sums = reinterpret_cast<double*>(scratch + p.sums);
    a.lists = reinterpret_cast<unsigned long long*>(scratch + p.lists);
    cudaError_t e = type == SMLA_F32    ? launch_rows<SMLA_F32>(a, s)
                    : type == SMLA_BF16 ? launch_rows<SMLA_BF16>(a, s)
                                        : launch_rows<SMLA_F16>(a, s);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.B));
    cfg.blockDim = dim3(kBsMergeThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    note_launch(2);
    return cudaLaunchKernelEx(&cfg, beam_merge_kernel, a);
}

}  // namespace smla
