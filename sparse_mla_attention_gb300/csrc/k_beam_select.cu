// k_beam_select.cu -- the next beams of each group: the n best of beams x vocabulary.
//
// Candidate (k, v) of a group scores scores[k] + logits[k,v] - logsumexp(logits[k,:]); a finished beam has the
// one candidate (k, eos) with scores[k]. Best first, ties by k, then v; scores that are not finite are never taken.
//
// A row's candidates rank as its logits do, so one pass over the logits gives both parts of the answer:
// beam_rows_kernel cuts a row into chunks, keeps a chunk's values in registers, and writes its maximum, its sum of
// exponentials and its n best logits; beam_merge_kernel joins a row's sums and merges the lists of a group.
// Which candidate comes first is decided in 64 bits: sums of 33 exponentials in 32 bits, the rest in 64.
//
// A chunk's n best: a bound that n to 2n threads' largest values reach (bisection over their bits, a count and a
// barrier a step), so that at most 66 n values pass it, then their exact ranks among those.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "smla_internal.cuh"
#include "sm100.cuh"

namespace smla {
using namespace sm100;

namespace {

constexpr int kBsThreads = 256;
constexpr int kBsPer = 32;                       // values of a thread, beside one at the row's ends
constexpr int kBsMergeThreads = 256;
constexpr float kBsLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <int kType>
struct Logit;
template <>
struct Logit<SMLA_F32> {
    static constexpr int kSize = 4;
    static __device__ __forceinline__ float one(const uint8_t* p) { return __ldg(reinterpret_cast<const float*>(p)); }
    static __device__ __forceinline__ void spread(const uint4& x, float* v) {
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
    }
};
template <>
struct Logit<SMLA_BF16> {
    static constexpr int kSize = 2;
    static __device__ __forceinline__ float one(const uint8_t* p) {
        return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p))) << 16);
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
    static __device__ __forceinline__ float one(const uint8_t* p) {
        return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const uint16_t*>(p))));
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

__device__ __forceinline__ bool out_of_play(const BeamArgs& a, int row) {
    const float s = __ldg(a.scores + row);
    return !(fabsf(s) < INFINITY) || (a.done && __ldg(a.done + row));
}

}  // namespace

template <int kType>
__global__ void __launch_bounds__(kBsThreads)
beam_rows_kernel(const BeamArgs a) {
    constexpr int kSize = Logit<kType>::kSize, kEach = 16 / kSize, kVecs = kBsPer / kEach;
    extern __shared__ __align__(16) unsigned long long best[];    // values that pass the bound: at most 66 n
    __shared__ uint32_t warp_top[kBsThreads / 32], warp_low[kBsThreads / 32];
    __shared__ double warp_sum[kBsThreads / 32];
    __shared__ int count;
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = int(blockIdx.x) / a.chunks, chunk = int(blockIdx.x) % a.chunks;
    if (out_of_play(a, row)) return;             // (nobody looks at its lists)
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + int64_t(row) * a.stride * kSize;
    // the row from its first 16-byte boundary on as vectors; threads of the first and the last chunk take what is
    // before and behind them, a value each
    int lead = int((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kSize;
    if (lead > a.V) lead = a.V;
    const int vecs = (a.V - lead) / kEach, tail = a.V - lead - vecs * kEach;
    float v[kBsPer], x = -INFINITY;
    int xi = -1;
    const int first = chunk * kBsThreads * kVecs + int(threadIdx.x);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int i = first + k * kBsThreads;
        if (i < vecs) {
            const uint4 raw = __ldg(reinterpret_cast<const uint4*>(base + lead * kSize) + i);
            Logit<kType>::spread(raw, v + k * kEach);
        } else {
#pragma unroll
            for (int e = 0; e < kEach; ++e) v[k * kEach + e] = -INFINITY;
        }
    }
    if (chunk == 0 && threadIdx.x < lead) xi = threadIdx.x;
    if (chunk == a.chunks - 1 && threadIdx.x >= kBsThreads - tail) xi = a.V - (kBsThreads - int(threadIdx.x));
    if (xi >= 0) x = Logit<kType>::one(base + int64_t(xi) * kSize);

    float top = x;                               // (fmaxf passes over NaN)
#pragma unroll
    for (int e = 0; e < kBsPer; ++e) top = fmaxf(top, v[e]);
    if (top != top) top = -INFINITY;
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
    float sum = ex2_approx((x - ref) * kBsLog2e);
#pragma unroll
    for (int e = 0; e < kBsPer; ++e) sum += ex2_approx((v[e] - ref) * kBsLog2e);
    double all = sum;
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    if (lane == 0) warp_sum[warp] = all;

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
            if (mine == bound) {
                if (x == at) place = xi;
#pragma unroll
                for (int e = 0; e < kBsPer; ++e)
                    if (v[e] == at) place = min(place, lead + (first + e / kEach * kBsThreads) * kEach + e % kEach);
            }
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
        if (xi >= 0) pass(x, xi);
#pragma unroll
        for (int e = 0; e < kBsPer; ++e) pass(v[e], lead + (first + e / kEach * kBsThreads) * kEach + e % kEach);
    }
    __syncthreads();
    const int c = count;
    const int64_t list = int64_t(blockIdx.x) * n;
    for (int i = threadIdx.x; i < c; i += kBsThreads) {
        const unsigned long long key = best[i];
        int rank = 0;
        for (int j = 0; j < c; ++j) rank += best[j] > key;
        if (rank < n) a.lists[list + rank] = key;
    }
    for (int i = c + threadIdx.x; i < n; i += kBsThreads) a.lists[list + i] = 0;
    if (threadIdx.x == 0) {
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kBsThreads / 32; ++w) total += warp_sum[w];
        a.peaks[blockIdx.x] = peak;
        a.sums[blockIdx.x] = total;
    }
}

__global__ void __launch_bounds__(kBsMergeThreads)
beam_merge_kernel(const BeamArgs a) {
    __shared__ double lse[SMLA_MAX_BEAMS];
    __shared__ double warp_score[2][kBsMergeThreads / 32];
    __shared__ int warp_flat[2][kBsMergeThreads / 32];
    extern __shared__ uint8_t taken[];           // of each list
    grid_dep_wait();
    const int b = int(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (b == 0 && threadIdx.x == 0) *a.status = 0;
    for (int k = warp; k < a.K; k += kBsMergeThreads / 32) {
        const int row = b * a.K + k;
        if (out_of_play(a, row)) continue;
        float peak = -INFINITY;
        for (int i = lane; i < a.chunks; i += 32) peak = fmaxf(peak, __ldcg(a.peaks + int64_t(row) * a.chunks + i));
#pragma unroll
        for (int d = 16; d; d >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, d));
        double sum = 0.0;
        for (int i = lane; i < a.chunks; i += 32)
            sum += __ldcg(a.sums + int64_t(row) * a.chunks + i) *
                   exp(double(__ldcg(a.peaks + int64_t(row) * a.chunks + i)) - double(peak));
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) lse[k] = double(peak) + log(sum);
    }
    const int lists = a.K * a.chunks;
    for (int i = threadIdx.x; i < lists; i += kBsMergeThreads) taken[i] = 0;
    __syncthreads();
    // the best head of this thread's lists
    double score = -INFINITY;
    int flat = INT32_MAX, from = -1;
    auto look = [&]() {
        score = -INFINITY;
        flat = INT32_MAX;
        from = -1;
        for (int i = threadIdx.x; i < lists; i += kBsMergeThreads) {
            const int k = i / a.chunks, row = b * a.K + k, at = taken[i];
            const float before = __ldg(a.scores + row);
            double s = -INFINITY;
            int f = 0;
            if (!out_of_play(a, row)) {
                const unsigned long long key =
                    at < a.n ? __ldcg(a.lists + (int64_t(row) * a.chunks + (i - k * a.chunks)) * a.n + at) : 0;
                if (key == 0) continue;
                s = double(before) + (double(value_of(uint32_t(key >> 32))) - lse[k]);
                f = k * a.V + int(0xffffffffu - uint32_t(key));
            } else if (a.done && __ldg(a.done + row) && i == k * a.chunks && at == 0) {
                s = before;
                f = k * a.V + a.eos;
            }
            if (!(fabs(s) < INFINITY)) continue;
            if (s > score || (s == score && f < flat)) { score = s; flat = f; from = i; }
        }
    };
    look();
    for (int r = 0; r < a.n; ++r) {
        double s = score;
        int f = flat;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double os = __shfl_xor_sync(0xffffffffu, s, d);
            const int of = __shfl_xor_sync(0xffffffffu, f, d);
            if (os > s || (os == s && of < f)) { s = os; f = of; }
        }
        if (lane == 0) { warp_score[r & 1][warp] = s; warp_flat[r & 1][warp] = f; }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kBsMergeThreads / 32; ++w) {
            const double os = warp_score[r & 1][w];
            const int of = warp_flat[r & 1][w];
            if (os > s || (os == s && of < f)) { s = os; f = of; }
        }
        if (threadIdx.x == 0) {
            const int64_t at = int64_t(b) * a.n + r;
            const bool any = f != INT32_MAX;
            a.parents[at] = any ? b * a.K + f / a.V : -1;
            a.tokens[at] = any ? f % a.V : -1;
            a.new_scores[at] = any ? float(s) : -INFINITY;
        }
        if (from >= 0 && f == flat) {            // (no two candidates have one place)
            ++taken[from];
            look();
        }
    }
}

namespace {

struct BeamPlan { size_t peaks, sums, lists, bytes; int chunks; };

BeamPlan plan_beam(int64_t rows, int V, int n) {
    BeamPlan p{};
    // 16-byte vectors hold 4 values at least
    p.chunks = (V + kBsThreads * kBsPer - 1) / (kBsThreads * kBsPer);
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes, 256); return o; };
    p.peaks = take(size_t(rows) * p.chunks * 4);
    p.sums = take(size_t(rows) * p.chunks * 8);
    p.lists = take(size_t(rows) * p.chunks * n * 8);
    p.bytes = off;
    return p;
}

template <int kType>
cudaError_t launch_rows(const BeamArgs& a, cudaStream_t s) {
    const size_t smem = size_t(a.n) * 2 * (kBsPer + 1) * 8;
    beam_rows_kernel<kType><<<unsigned(a.B) * a.K * a.chunks, kBsThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t beam_scratch_bytes(int B, int K, int V, int n) { return plan_beam(int64_t(B) * K, V, n).bytes; }
int beam_chunks(int V) { return plan_beam(1, V, 1).chunks; }

cudaError_t launch_beam_select(BeamArgs a, int type, char* scratch, cudaStream_t s) {
    const BeamPlan p = plan_beam(int64_t(a.B) * a.K, a.V, a.n);
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
    cfg.dynamicSmemBytes = size_t(a.K) * a.chunks;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    note_launch(2);
    return cudaLaunchKernelEx(&cfg, beam_merge_kernel, a);
}

}  // namespace smla
