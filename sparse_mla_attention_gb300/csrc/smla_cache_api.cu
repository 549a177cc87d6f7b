// smla_cache_api.cu -- the C ABI of serving (the paged 8-bit cache and beam search): argument
// validation and workspace carving; the kernels are in k_fwd_paged.cu, k_cache_write.cu,
// k_cache_pages.cu, k_cache_weights.cu, k_cache_evict.cu and k_beam_select.cu.
#include <cmath>

#include "smla_internal.cuh"

using namespace smla;

namespace {

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

int check_cache(const smla_cache* c) {
    if (!c || !c->pages || !c->scales) return SMLA_ERR_NULL;
    if (c->D != kD) return SMLA_ERR_D512;
    const int ps = c->page_size, sb = c->scale_block;
    const bool ps_ok = ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256;
    const bool sb_ok = (sb == 16 || sb == 32 || sb == 64) && sb <= ps;
    if (!ps_ok || !sb_ok || c->num_pages < 1 || int64_t(c->num_pages) * ps > int64_t(INT32_MAX))
        return SMLA_ERR_CACHE;
    return SMLA_OK;
}

// Sequences and children per call: grids and slot numbers stay within 32 bits.
constexpr int kMaxSeqs = 1 << 24;

// Rows of q of a call of accumulated weights: a pass over a sequence's takes 0.8 us for each 32 of them (1.2 at the lowest
// clocks under load), and the warp that loads the next pass's tiles waits that long, with a limit of 2 s.
constexpr int64_t kMaxWeightsRows = int64_t(1) << 25;

int check_table(const smla_cache& c, int B, int max_pages) {
    if (B < 0 || B > kMaxSeqs || max_pages < 1 || int64_t(max_pages) * c.page_size > int64_t(INT32_MAX))
        return SMLA_ERR_SHAPE;
    return SMLA_OK;
}

CacheView view(const smla_cache& c) {
    return CacheView{c.pages, c.scales, c.refcount, c.num_pages, log2_of(c.page_size),
                     log2_of(c.scale_block)};
}

size_t page_bytes(const smla_cache& c) { return size_t(c.num_pages) * c.page_size * kD; }
size_t scale_bytes(const smla_cache& c) {
    return size_t(c.num_pages) * (c.page_size / c.scale_block) * 4;
}
size_t count_bytes(const smla_cache& c) { return c.refcount ? size_t(c.num_pages) * 4 : 0; }

struct ScratchPlan {
    size_t need, tail, src, dst, map, bytes;
};

ScratchPlan plan_pages(const smla_cache& c, int64_t n) {
    ScratchPlan p{};
    size_t off = kStatusBytes + 256;        // the pair count follows the status word
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes > 0 ? bytes : 1, 256); return o; };
    const size_t list = size_t(n > c.num_pages ? n : c.num_pages) * 4;
    p.need = take(size_t(n) * 4);
    p.tail = take(size_t(n) * 4);
    p.src = take(list);
    p.dst = take(list);
    p.map = take(size_t(c.num_pages) * 4);
    p.bytes = off;
    return p;
}

PageScratch carve(char* ws, const ScratchPlan& p) {
    auto at = [ws](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
    return PageScratch{at(kStatusBytes), at(p.need), at(p.tail), at(p.src), at(p.dst), at(p.map)};
}

struct EvictPlan { size_t need, start, fresh, bytes; };

EvictPlan plan_evict(const smla_cache& c, int64_t B, int64_t keep) {
    EvictPlan p{};
    size_t off = kStatusBytes + 256;        // whether the pages were granted follows the status word
    auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes > 0 ? bytes : 1, 256); return o; };
    p.need = take(size_t(B) * 4);
    p.start = take(size_t(B) * 4);
    p.fresh = take(size_t(c.num_pages) * 4);
    p.bytes = off;
    return p;
}

struct ReorderPlan { size_t heir, spare, tail, need, src, dst, bytes; };

ReorderPlan plan_reorder(int64_t B, int64_t n) {
    ReorderPlan p{};
    size_t off = kStatusBytes + 256;        // the pair count follows the status word
    auto take = [&](int64_t items) { size_t o = off; off += align_up(size_t(items > 0 ? items : 1) * 4, 256); return o; };
    p.heir = take(B); p.spare = take(B);
    p.tail = take(n); p.need = take(n); p.src = take(n); p.dst = take(n);
    p.bytes = off;
    return p;
}

// Lists of candidates are counted in 32 bits, and a group's within shared memory.
int check_beams(int B, int K, int V, int n) {
    if (B < 0 || B > kMaxSeqs || K < 1 || K > SMLA_MAX_BEAMS || n < 1 || n > SMLA_MAX_BEAMS || V < 1 ||
        V > SMLA_MAX_VOCAB)
        return SMLA_ERR_SHAPE;
    if (int64_t(B) * K * beam_chunks(V) > int64_t(INT32_MAX) || int64_t(K) * V > int64_t(INT32_MAX) ||
        int64_t(B) * n > int64_t(INT32_MAX))
        return SMLA_ERR_SHAPE;
    return SMLA_OK;
}

int check_align(const void* const* ptrs, int n) {
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && !aligned16(ptrs[i])) return SMLA_ERR_ALIGN;
    return SMLA_OK;
}

int check_device(const void* const* ptrs, int n) {
    const int rc = check_arch();
    return rc ? rc : check_device_ptrs(ptrs, n);
}

// Arch and pointer checks, then the status word of the call is cleared.
int begin(const void* const* ptrs, int n, void* workspace, cudaStream_t s) {
    const int rc = check_device(ptrs, n);
    return rc ? rc : cuda_rc(cudaMemsetAsync(workspace, 0, sizeof(unsigned), s));
}

}  // namespace

extern "C" {

int smla_paged_workspace_size(const smla_paged_dims* d, size_t* bytes) {
    if (!d || !bytes) return SMLA_ERR_NULL;
    if (d->T < 0 || d->H < 16 || d->H > 128 || d->H % 16 != 0) return SMLA_ERR_SHAPE;
    *bytes = kStatusBytes + paged_scratch_bytes(d->T, d->H);
    return SMLA_OK;
}

int smla_fwd_paged(const uint16_t* q, const smla_cache* cache, const int32_t* table,
                   const int32_t* seq, const int32_t* lens, const int32_t* topk,
                   const float* sink, uint16_t* o, float* lse, const smla_paged_dims* dims,
                   void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (!dims) return SMLA_ERR_NULL;
    const smla_cache& c = *cache;
    const smla_paged_dims& d = *dims;
    if (d.D != kD) return SMLA_ERR_D512;
    if (d.T < 0 || d.topk < 0 || d.H < 16 || d.H > 128 || d.H % 16 != 0 || (d.T > 0 && d.B < 1)) return SMLA_ERR_SHAPE;
    if ((rc = check_table(c, d.B, d.max_pages))) return rc;
    if (int64_t(d.T) * d.topk > int64_t(INT32_MAX) || (!seq && d.T > d.B)) return SMLA_ERR_SHAPE;
    // tiles of 64 ranks are counted in 32 bits
    if (int64_t(d.T) * ((int64_t(d.max_pages) * c.page_size + 63) / 64) > int64_t(INT32_MAX)) return SMLA_ERR_SHAPE;
    if ((d.topk > 0) != (topk != nullptr) && d.T > 0) return SMLA_ERR_ARG;
    if (!std::isfinite(d.scale) || d.scale < 0.f) return SMLA_ERR_ARG;
    if (!workspace) return SMLA_ERR_NULL;
    if (d.T > 0 && (!q || !table || !lens || !o || !lse)) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, q, table, seq, lens, topk, sink, o, lse, workspace};
    if ((rc = check_align(ptrs, 11))) return rc;
    if (workspace_bytes < kStatusBytes + paged_scratch_bytes(d.T, d.H)) return SMLA_ERR_WORKSPACE;
    const size_t thd = size_t(d.T) * d.H * kD * 2;
    const Span ins[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {q, thd},
                        {table, size_t(d.B) * d.max_pages * 4}, {seq, seq ? size_t(d.T) * 4 : 0},
                        {lens, size_t(d.T) * 4}, {topk, size_t(d.T) * d.topk * 4},
                        {sink, sink ? size_t(d.H) * 4 : 0}};
    const Span outs[] = {{o, thd}, {lse, size_t(d.T) * d.H * 4}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 3, ins, 8))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d.T == 0) return begin(ptrs, 11, workspace, s);
    if ((rc = check_device(ptrs, 11))) return rc;        // (the kernels write the status word)
    PagedArgs a{};
    a.q = q; a.cache = view(c); a.table = table; a.seq = seq; a.lens = lens; a.topk = topk; a.sink = sink;
    a.o = o; a.lse = lse;
    a.T = d.T; a.H = d.H; a.K = d.topk; a.B = d.B; a.max_pages = d.max_pages;
    a.scale = d.scale > 0.f ? d.scale : 1.0f / std::sqrt(float(kD));
    a.status = static_cast<unsigned*>(workspace);
    a.scratch = static_cast<char*>(workspace) + kStatusBytes;
    return cuda_rc(launch_fwd_paged(a, s));
}

int smla_cache_write(const smla_cache* cache, const int32_t* table, const int32_t* start,
                     const int32_t* cu, const uint16_t* rows, int32_t B, int32_t max_pages,
                     int32_t n_rows, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (n_rows < 0) return SMLA_ERR_SHAPE;
    if (!workspace) return SMLA_ERR_NULL;
    const bool any = B > 0 && n_rows > 0;
    if (any && (!table || !start || !cu || !rows)) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, table, start, cu, rows, workspace};
    if ((rc = check_align(ptrs, 7))) return rc;
    if (workspace_bytes < kStatusBytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{table, size_t(B) * max_pages * 4}, {start, size_t(B) * 4},
                        {cu, size_t(B + 1) * 4}, {rows, size_t(n_rows) * kD * 2}};
    const Span outs[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 3, ins, 4))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) return begin(ptrs, 7, workspace, s);
    if ((rc = check_device(ptrs, 7))) return rc;         // (the kernel writes the status word)
    return cuda_rc(launch_cache_write(view(c), table, start, cu, rows, B, max_pages, n_rows,
                                      static_cast<unsigned*>(workspace), s));
}

int smla_cache_workspace_size(const smla_cache* cache, int32_t n, size_t* bytes) {
    if (!bytes) return SMLA_ERR_NULL;
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (n < 0) return SMLA_ERR_SHAPE;
    *bytes = plan_pages(*cache, n).bytes;
    return SMLA_OK;
}

int smla_cache_alloc(const smla_cache* cache, int32_t* table, const int32_t* lens, int32_t B,
                     int32_t max_pages, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (!c.refcount || !workspace || (B > 0 && (!table || !lens))) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, lens, workspace};
    if ((rc = check_align(ptrs, 6))) return rc;
    const ScratchPlan plan = plan_pages(c, B);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {lens, size_t(B) * 4}};
    const Span outs[] = {{table, size_t(B) * max_pages * 4}, {c.refcount, count_bytes(c)},
                         {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 3, ins, 3))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0) return begin(ptrs, 6, workspace, s);
    if ((rc = check_device(ptrs, 6))) return rc;         // (the kernel writes the status word)
    return cuda_rc(launch_cache_alloc(view(c), table, lens, B, max_pages,
                                      carve(static_cast<char*>(workspace), plan),
                                      static_cast<unsigned*>(workspace), s));
}

int smla_cache_fork(const smla_cache* cache, const int32_t* table, const int32_t* lens,
                    const int32_t* parents, int32_t* child_table, int32_t B, int32_t n,
                    int32_t max_pages, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (n < 0 || n > kMaxSeqs) return SMLA_ERR_SHAPE;
    if (!c.refcount || !workspace) return SMLA_ERR_NULL;
    if (n > 0 && (!parents || !child_table || (B > 0 && (!table || !lens)))) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, lens, parents, child_table, workspace};
    if ((rc = check_align(ptrs, 8))) return rc;
    const ScratchPlan plan = plan_pages(c, n);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{table, size_t(B) * max_pages * 4}, {lens, size_t(B) * 4}, {parents, size_t(n) * 4}};
    const Span outs[] = {{child_table, size_t(n) * max_pages * 4}, {c.pages, page_bytes(c)},
                         {c.scales, scale_bytes(c)}, {c.refcount, count_bytes(c)},
                         {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 5, ins, 3))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) return begin(ptrs, 8, workspace, s);
    if ((rc = check_device(ptrs, 8))) return rc;
    return cuda_rc(launch_cache_fork(view(c), table, lens, parents, child_table, B, n, max_pages,
                                     carve(static_cast<char*>(workspace), plan),
                                     static_cast<unsigned*>(workspace), s));
}

int smla_cache_free(const smla_cache* cache, int32_t* table, const int32_t* rows, int32_t B,
                    int32_t n, int32_t max_pages, void* workspace, size_t workspace_bytes,
                    void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (n < 0 || n > kMaxSeqs || (!rows && n != B && n != 0)) return SMLA_ERR_SHAPE;
    if (!c.refcount || !workspace || (n > 0 && B > 0 && !table)) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, rows, workspace};
    if ((rc = check_align(ptrs, 6))) return rc;
    if (workspace_bytes < kStatusBytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {rows, rows ? size_t(n) * 4 : 0}};
    const Span outs[] = {{table, size_t(B) * max_pages * 4}, {c.refcount, count_bytes(c)},
                         {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 3, ins, 3))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) return begin(ptrs, 6, workspace, s);
    if ((rc = check_device(ptrs, 6))) return rc;         // (the launch sees to the status word)
    return cuda_rc(launch_cache_free(view(c), table, rows, B, n, max_pages,
                                     static_cast<unsigned*>(workspace), s));
}

int smla_cache_compact(const smla_cache* cache, const int32_t* table, int32_t* new_table,
                       int32_t* new_refcount, int32_t B, int32_t max_pages, void* workspace,
                       size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (!c.refcount || !new_refcount || !workspace) return SMLA_ERR_NULL;
    if (B > 0 && (!table || !new_table)) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, new_table, new_refcount, workspace};
    if ((rc = check_align(ptrs, 7))) return rc;
    const ScratchPlan plan = plan_pages(c, 0);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{table, size_t(B) * max_pages * 4}, {c.refcount, count_bytes(c)}};
    const Span outs[] = {{new_table, size_t(B) * max_pages * 4}, {new_refcount, count_bytes(c)},
                         {c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 5, ins, 2))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rc = check_device(ptrs, 7))) return rc;
    return cuda_rc(launch_cache_compact(view(c), table, new_table, new_refcount, B, max_pages,
                                        carve(static_cast<char*>(workspace), plan),
                                        static_cast<unsigned*>(workspace), s));
}

int smla_cache_copy_pages(const smla_cache* cache, const int32_t* src, const int32_t* dst,
                          int32_t n, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if (n < 0) return SMLA_ERR_SHAPE;
    if (!workspace || (n > 0 && (!src || !dst))) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, src, dst, workspace};
    if ((rc = check_align(ptrs, 5))) return rc;
    const ScratchPlan plan = plan_pages(c, n);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const Span ins[] = {{src, size_t(n) * 4}, {dst, size_t(n) * 4}};
    const Span outs[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 3, ins, 2))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) return begin(ptrs, 5, workspace, s);
    if ((rc = check_device(ptrs, 5))) return rc;
    return cuda_rc(launch_cache_copy(view(c), src, dst, n, carve(static_cast<char*>(workspace), plan),
                                     static_cast<unsigned*>(workspace), s));
}

int smla_weights_workspace_size(const smla_paged_dims* d, size_t* bytes) {
    if (!d || !bytes) return SMLA_ERR_NULL;
    if (d->T < 0 || d->B < 0 || d->B > kMaxSeqs || d->H < 16 || d->H > 128 || d->H % 16 != 0 ||
        int64_t(d->T) * d->H > kMaxWeightsRows)
        return SMLA_ERR_SHAPE;
    *bytes = kStatusBytes + weights_scratch_bytes(d->T, d->H);
    return SMLA_OK;
}

int smla_cache_weights(const uint16_t* q, const smla_cache* cache, const int32_t* table, const int32_t* cu,
                       const int32_t* lens, const float* lse, const float* earlier, float decay, float* weights,
                       const smla_paged_dims* dims, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (!dims) return SMLA_ERR_NULL;
    const smla_cache& c = *cache;
    const smla_paged_dims& d = *dims;
    if (d.D != kD) return SMLA_ERR_D512;
    if (d.T < 0 || d.H < 16 || d.H > 128 || d.H % 16 != 0) return SMLA_ERR_SHAPE;
    if ((rc = check_table(c, d.B, d.max_pages))) return rc;
    if (int64_t(d.T) * d.H > kMaxWeightsRows || (!cu && d.T > d.B)) return SMLA_ERR_SHAPE;
    if (d.topk != 0 || !std::isfinite(d.scale) || d.scale < 0.f || !std::isfinite(decay)) return SMLA_ERR_ARG;
    if (!workspace) return SMLA_ERR_NULL;
    const bool any = d.B > 0 && d.T > 0;
    if (any && (!q || !table || !lens || !lse || !weights || (decay != 0.f && !earlier))) return SMLA_ERR_NULL;
    if (decay == 0.f) earlier = nullptr;
    const void* ptrs[] = {c.pages, c.scales, q, table, cu, lens, lse, earlier, weights, workspace};
    if ((rc = check_align(ptrs, 10))) return rc;
    if (workspace_bytes < kStatusBytes + weights_scratch_bytes(d.T, d.H)) return SMLA_ERR_WORKSPACE;
    const size_t sums = size_t(d.B) * d.max_pages * c.page_size * 4;
    const bool in_place = earlier == weights;
    const Span ins[] = {{c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {q, size_t(d.T) * d.H * kD * 2},
                        {table, size_t(d.B) * d.max_pages * 4}, {cu, cu ? size_t(d.B + 1) * 4 : 0},
                        {lens, size_t(d.T) * 4}, {lse, size_t(d.T) * d.H * 4},
                        {earlier, earlier && !in_place ? sums : 0}};
    const Span outs[] = {{weights, sums}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 2, ins, 8))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) return begin(ptrs, 10, workspace, s);
    if ((rc = check_device(ptrs, 10))) return rc;
    WeightsArgs a{};
    a.q = q; a.cache = view(c); a.table = table; a.cu = cu; a.lens = lens; a.lse = lse;
    a.earlier = earlier; a.weights = weights;
    a.T = d.T; a.H = d.H; a.B = d.B; a.max_pages = d.max_pages;
    a.scale = d.scale > 0.f ? d.scale : 1.0f / std::sqrt(float(kD));
    a.decay = decay;
    a.status = static_cast<unsigned*>(workspace);
    a.scratch = static_cast<char*>(workspace) + kStatusBytes;
    return cuda_rc(launch_cache_weights(a, s));
}

int smla_cache_evict_workspace_size(const smla_cache* cache, int32_t B, int32_t keep, size_t* bytes) {
    if (!bytes) return SMLA_ERR_NULL;
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0 || B > kMaxSeqs || keep < 1) return SMLA_ERR_SHAPE;
    *bytes = plan_evict(*cache, B, keep).bytes;
    return SMLA_OK;
}

int smla_cache_evict(const smla_cache* cache, const int32_t* table, const int32_t* lens, const float* weights,
                     int32_t* new_table, int32_t* new_lens, float* new_weights, int32_t* kept, int32_t B,
                     int32_t max_pages, int32_t keep, int32_t first, int32_t recent, void* workspace,
                     size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (keep < 1 || int64_t(keep) > int64_t(max_pages) * c.page_size) return SMLA_ERR_SHAPE;
    if (first < 0 || recent < 0 || int64_t(first) + recent > keep) return SMLA_ERR_ARG;
    if (!c.refcount || !workspace) return SMLA_ERR_NULL;
    if (B > 0 && (!table || !lens || !weights || !new_table || !new_lens || !new_weights || !kept)) return SMLA_ERR_NULL;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, lens, weights, new_table, new_lens, new_weights, kept,
                          workspace};
    if ((rc = check_align(ptrs, 11))) return rc;
    const EvictPlan plan = plan_evict(c, B, keep);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const size_t entries = size_t(B) * max_pages * 4, sums = entries * c.page_size;
    const Span ins[] = {{table, entries}, {lens, size_t(B) * 4}, {weights, sums}};
    const Span outs[] = {{new_table, entries}, {new_lens, size_t(B) * 4}, {new_weights, sums},
                         {kept, size_t(B) * keep * 4}, {c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)},
                         {c.refcount, count_bytes(c)}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 8, ins, 3))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0) return begin(ptrs, 11, workspace, s);
    if ((rc = check_device(ptrs, 11))) return rc;
    char* ws = static_cast<char*>(workspace);
    auto at = [ws](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
    EvictArgs a{};
    a.cache = view(c); a.table = table; a.lens = lens; a.weights = weights;
    a.new_table = new_table; a.new_lens = new_lens; a.new_weights = new_weights; a.kept = kept;
    a.B = B; a.max_pages = max_pages; a.keep = keep; a.first = first; a.recent = recent;
    a.granted = at(kStatusBytes); a.need = at(plan.need); a.start = at(plan.start); a.fresh = at(plan.fresh);
    a.status = static_cast<unsigned*>(workspace);
    return cuda_rc(launch_cache_evict(a, s));
}

int smla_cache_reorder_workspace_size(int32_t B, int32_t n, size_t* bytes) {
    if (!bytes) return SMLA_ERR_NULL;
    if (B < 0 || B > kMaxSeqs || n < 0 || n > kMaxSeqs) return SMLA_ERR_SHAPE;
    *bytes = plan_reorder(B, n).bytes;
    return SMLA_OK;
}

int smla_cache_reorder(const smla_cache* cache, const int32_t* table, const int32_t* lens, const int32_t* parents,
                       const float* weights, int32_t* new_table, int32_t* new_lens, float* new_weights, int32_t B,
                       int32_t n, int32_t max_pages, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    const smla_cache& c = *cache;
    if ((rc = check_table(c, B, max_pages))) return rc;
    if (n < 0 || n > kMaxSeqs) return SMLA_ERR_SHAPE;
    if (!c.refcount || !workspace) return SMLA_ERR_NULL;
    if ((B > 0 && (!table || !lens)) || (n > 0 && (!parents || !new_table || !new_lens))) return SMLA_ERR_NULL;
    if ((weights != nullptr) != (new_weights != nullptr) && B > 0 && n > 0) return SMLA_ERR_ARG;
    const void* ptrs[] = {c.pages, c.scales, c.refcount, table, lens, parents, weights, new_table, new_lens, new_weights,
                          workspace};
    if ((rc = check_align(ptrs, 11))) return rc;
    const ReorderPlan plan = plan_reorder(B, n);
    if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
    const size_t row = size_t(max_pages) * 4, sums = weights || new_weights ? row * c.page_size : 0;
    const Span ins[] = {{table, B * row}, {lens, size_t(B) * 4}, {parents, size_t(n) * 4},
                        {weights, weights ? B * sums : 0}};
    const Span outs[] = {{new_table, n * row}, {new_lens, size_t(n) * 4}, {new_weights, new_weights ? n * sums : 0},
                         {c.pages, page_bytes(c)}, {c.scales, scale_bytes(c)}, {c.refcount, count_bytes(c)},
                         {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 7, ins, 4))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 && n == 0) return begin(ptrs, 11, workspace, s);
    if ((rc = check_device(ptrs, 11))) return rc;
    char* ws = static_cast<char*>(workspace);
    auto at = [ws](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
    ReorderArgs a{};
    a.cache = view(c); a.table = table; a.lens = lens; a.parents = parents;
    a.weights = weights;
    a.new_table = new_table; a.new_lens = new_lens; a.new_weights = new_weights;
    a.B = B; a.n = n; a.max_pages = max_pages;
    a.count = at(kStatusBytes); a.heir = at(plan.heir); a.spare = at(plan.spare);
    a.tail = at(plan.tail); a.need = at(plan.need); a.src = at(plan.src); a.dst = at(plan.dst);
    a.status = static_cast<unsigned*>(workspace);
    return cuda_rc(launch_cache_reorder(a, s));
}

int smla_beam_workspace_size(int32_t B, int32_t K, int32_t V, int32_t n, size_t* bytes) {
    if (!bytes) return SMLA_ERR_NULL;
    const int rc = check_beams(B, K, V, n);
    if (rc) return rc;
    *bytes = kStatusBytes + beam_scratch_bytes(B, K, V, n);
    return SMLA_OK;
}

int smla_beam_select(const void* logits, int32_t type, int64_t row_stride, const float* scores, const uint8_t* done,
                     int32_t eos, int32_t* parents, int32_t* tokens, float* new_scores, int32_t B, int32_t K,
                     int32_t V, int32_t n, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_beams(B, K, V, n);
    if (rc) return rc;
    if (type != SMLA_F32 && type != SMLA_BF16 && type != SMLA_F16) return SMLA_ERR_ARG;
    const int64_t size = type == SMLA_F32 ? 4 : 2, rows = int64_t(B) * K;
    if (row_stride < 0 || (rows > 1 && row_stride > (int64_t(1) << 60) / rows)) return SMLA_ERR_SHAPE;
    if (done && (eos < 0 || eos >= V)) return SMLA_ERR_ARG;
    if (!workspace) return SMLA_ERR_NULL;
    if (B > 0 && (!logits || !scores || !parents || !tokens || !new_scores)) return SMLA_ERR_NULL;
    // values need no more than their own alignment: rows of an odd width start anywhere
    const void* ptrs[] = {logits, scores, done, parents, tokens, new_scores, workspace};
    if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(logits) % size != 0) return SMLA_ERR_ALIGN;
    for (int i : {1, 3, 4, 5})
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % 4 != 0) return SMLA_ERR_ALIGN;
    if (workspace_bytes < kStatusBytes + beam_scratch_bytes(B, K, V, n)) return SMLA_ERR_WORKSPACE;
    const size_t picks = size_t(B) * n * 4;
    const Span ins[] = {{logits, rows > 0 ? size_t(((rows - 1) * row_stride + V) * size) : 0},
                        {scores, size_t(rows) * 4}, {done, done ? size_t(rows) : 0}};
    const Span outs[] = {{parents, picks}, {tokens, picks}, {new_scores, picks}, {workspace, workspace_bytes}};
    if ((rc = check_overlap(outs, 4, ins, 3))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0) return begin(ptrs, 7, workspace, s);
    if ((rc = check_device(ptrs, 7))) return rc;
    BeamArgs a{};
    a.logits = logits; a.stride = row_stride; a.scores = scores; a.done = done;
    a.parents = parents; a.tokens = tokens; a.new_scores = new_scores;
    a.B = B; a.K = K; a.V = V; a.n = n; a.eos = eos;
    a.status = static_cast<unsigned*>(workspace);
    return cuda_rc(launch_beam_select(a, type, static_cast<char*>(workspace) + kStatusBytes, s));
}

}  // extern "C"
