// sv_cache.hip -- lengths, pages and slots of a paged cache: what a decode
// loop needs before the forward pass (pages, block tables, slot maps) and
// after the verify step (lengths, pages given back), from lengths that are
// on the GPU already, so that the loop never waits for them on the host.
//
// Both calls are a prefix sum over the sequences followed by independent work
// per token (page).  One workgroup scans: there are at most a few thousand
// sequences, and a second workgroup would need a hand-off that costs more
// than their loads.  Few tokens follow in the same workgroup, so that a
// decode step is one launch; many get a launch of their own.
#include <algorithm>

#include "specdecode.h"
#include "sv_internal.h"

namespace sv {

constexpr int kPlan = 1024;             // threads of the scanning workgroup
constexpr int kPlanWaves = kPlan / 64;
constexpr int kFusedTokens = 8192;      // at most so many tokens in the scanning workgroup
constexpr int kFusedPages = 65536;      // the same for pages that can come back
constexpr int kMaxCacheSeqs = 1 << 20;

struct CacheArgs {
    const int32_t *seq_len, *counts, *accepted, *finished;  // counts: new_len, or reserved
    int32_t *table;
    int32_t *free_list;
    const int32_t *free_count;
    int32_t *free_count_out, *seq_len_out;
    int64_t *slots;
    int32_t *positions, *seq_ids, *query_start, *granted, *page_start;
    int32_t *error_word;
    int32_t extra, B, max_blocks, page_size, num_pages, max_tokens;
};

__device__ __forceinline__ int64_t wave_scan(int64_t v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t w = __shfl_up(v, d);
        if (lane >= d) v += w;
    }
    return v;
}

// Exclusive prefix sums of two counts over the workgroup, and their totals.
struct Sums {
    int64_t a, b, all_a, all_b;
};

__device__ __forceinline__ Sums plan_scan(int64_t a, int64_t b, int64_t *lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t ia = wave_scan(a), ib = wave_scan(b);
    if (lane == 63) {
        lds[wave] = ia;
        lds[kPlanWaves + wave] = ib;
    }
    __syncthreads();
    Sums s = {ia - a, ib - b, 0, 0};
    for (int w = 0; w < kPlanWaves; ++w) {
        const int64_t x = lds[w], y = lds[kPlanWaves + w];
        if (w < wave) {
            s.a += x;
            s.b += y;
        }
        s.all_a += x;
        s.all_b += y;
    }
    __syncthreads();
    return s;
}

__device__ __forceinline__ void cache_error(const CacheArgs &a, int bit)
{
    if (a.error_word) atomicOr(a.error_word, bit);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size)
{
    return tokens / page_size + (tokens % page_size ? 1 : 0);
}

// The free list's length, held within the list.
__device__ __forceinline__ int free_pages(const CacheArgs &a)
{
    const int f = *a.free_count;
    const int held = min(max(f, 0), a.num_pages);
    if (held != f && threadIdx.x == 0) cache_error(a, SV_ERR_PAGES);
    return held;
}

// The last i in [lo, hi) with start[i] <= t (start[lo] <= t).
__device__ __forceinline__ int find_run(const int32_t *start, int lo, int hi, int t)
{
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// Extend.

struct NewTokens {
    int len, n, need;  // held, new, pages taken
};

__device__ __forceinline__ NewTokens new_tokens(const CacheArgs &a, int b, bool &bad)
{
    NewTokens x;
    x.len = a.seq_len[b];
    const int64_t n = (int64_t)(a.counts ? a.counts[b] : 0) + a.extra;
    const int64_t most = (int64_t)a.max_blocks * a.page_size;
    bad = x.len < 0 || n < 0 || x.len + n > most;
    x.n = bad ? 0 : (int)n;
    x.need = bad ? 0 : pages_of(x.len + x.n, a.page_size) - pages_of(x.len, a.page_size);
    return x;
}

// Token t (of `total`) of the call; `free` is the free list's length before it.
__device__ __forceinline__ void place_token(const CacheArgs &a, int t, int total, int lo, int hi, int free)
{
    int64_t slot = -1;
    int at = 0, b = -1;
    if (t < total) {
        b = find_run(a.query_start, lo, hi, t);
        const int len = a.seq_len[b], i = t - a.query_start[b];
        at = len + i;
        if (a.granted[b]) {
            const int block = at / a.page_size, off = at - block * a.page_size;
            const int first = pages_of(len, a.page_size);
            int32_t *entry = a.table + (int64_t)b * a.max_blocks + block;
            int page;
            if (block >= first) {
                page = a.free_list[free - 1 - (a.page_start[b] + block - first)];
                if (off == 0) *entry = page;  // a new page's first token is at its start
            } else {
                page = *entry;
            }
            if (page >= 0 && page < a.num_pages) slot = (int64_t)page * a.page_size + off;
            else cache_error(a, SV_ERR_PAGE);
        }
    }
    a.slots[t] = slot;
    a.positions[t] = at;
    a.seq_ids[t] = b;
}

template <bool FUSED>
__global__ __launch_bounds__(kPlan) void extend_plan_kernel(const CacheArgs a)
{
    __shared__ int64_t lds[2 * kPlanWaves];
    __shared__ int used;
    const int tid = threadIdx.x;
    const int run = (a.B + kPlan - 1) / kPlan;  // sequences per thread
    const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
    const int free = free_pages(a);
    if (tid == 0) used = 0;
    int64_t n = 0, need = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const NewTokens x = new_tokens(a, b, bad);
        any_bad |= bad;
        n += x.n;
        need += x.need;
    }
    const Sums s = plan_scan(n, need, lds);  // its barriers order `used` too
    int64_t q = s.a, p = s.b;
    int taken = 0;
    bool lack = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const NewTokens x = new_tokens(a, b, bad);
        const bool room = q + x.n <= a.max_tokens;
        const bool fits = room && (x.need == 0 || p + x.need <= free);
        any_bad |= !room;
        lack |= room && !fits;
        a.query_start[b] = (int32_t)min(q, (int64_t)a.max_tokens);
        a.page_start[b] = (int32_t)min(p, (int64_t)free);
        a.granted[b] = fits ? x.n : 0;
        q += x.n;
        p += x.need;
        if (fits && x.need) taken = (int)p;
    }
    if (taken) atomicMax(&used, taken);
    if (any_bad) cache_error(a, SV_ERR_LENGTH);
    if (lack) cache_error(a, SV_ERR_PAGES);
    __syncthreads();
    const int total = (int)min(s.all_a, (int64_t)a.max_tokens);
    // behind the sequences that got theirs nothing is taken
    for (int b = b0; b < b1; ++b)
        if (a.page_start[b] > used) a.page_start[b] = used;
    if (tid == 0) {
        a.query_start[a.B] = total;
        a.page_start[a.B] = used;
        *a.free_count_out = free - used;
    }
    if (FUSED) {
        __syncthreads();
        for (int t = tid; t < a.max_tokens; t += kPlan) place_token(a, t, total, 0, a.B, free);
    }
}

__global__ __launch_bounds__(kBlock) void extend_tokens_kernel(const CacheArgs a)
{
    const int t = blockIdx.x * kBlock + threadIdx.x;
    if (t >= a.max_tokens) return;
    place_token(a, t, a.query_start[a.B], 0, a.B, *a.free_count_out + a.page_start[a.B]);
}

// ---------------------------------------------------------------------------
// Commit.

struct Kept {
    int len, first, back;  // new length, first block given back, blocks given back
};

__device__ __forceinline__ Kept kept_tokens(const CacheArgs &a, int b, bool &bad)
{
    const int len = a.seq_len[b], held = a.counts[b];
    const bool ended = a.finished && a.finished[b];
    Kept k = {ended ? 0 : len, 0, 0};
    bad = len < 0 || held < 0 || (int64_t)len + held > (int64_t)a.max_blocks * a.page_size;
    if (bad) return k;
    const int64_t want = (int64_t)a.accepted[b] + a.extra;
    const int keep = (int)min(max(want, (int64_t)0), (int64_t)held);
    if (!ended) {
        bad = want != keep;
        k.len = len + keep;
    }
    k.first = pages_of(k.len, a.page_size);
    k.back = pages_of(len + held, a.page_size) - k.first;
    return k;
}

// Page i of the `total` that come back; the list held `free` before.
__device__ __forceinline__ void give_page(const CacheArgs &a, int i, int total, int free)
{
    const int b = find_run(a.page_start, 0, a.B, i);
    const int block = pages_of(a.seq_len_out[b], a.page_size) + i - a.page_start[b];
    int page = a.table[(int64_t)b * a.max_blocks + block];
    if (page < 0 || page >= a.num_pages) {
        cache_error(a, SV_ERR_PAGE);
        page = -1;
    }
    a.free_list[free + total - 1 - i] = page;
}

template <bool FUSED>
__global__ __launch_bounds__(kPlan) void commit_plan_kernel(const CacheArgs a)
{
    __shared__ int64_t lds[2 * kPlanWaves];
    const int tid = threadIdx.x;
    const int run = (a.B + kPlan - 1) / kPlan;
    const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
    const int free = free_pages(a);
    int64_t back = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        back += kept_tokens(a, b, bad).back;
        any_bad |= bad;
    }
    const Sums s = plan_scan(back, 0, lds);
    const int room = a.num_pages - free;
    const int total = (int)min(s.all_a, (int64_t)room);
    int64_t p = s.a;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const Kept k = kept_tokens(a, b, bad);
        a.page_start[b] = (int32_t)min(p, (int64_t)room);
        a.seq_len_out[b] = k.len;
        p += k.back;
    }
    if (any_bad) cache_error(a, SV_ERR_LENGTH);
    if (tid == 0) {
        if (s.all_a > room) cache_error(a, SV_ERR_PAGES);
        a.page_start[a.B] = total;
        *a.free_count_out = free + total;
    }
    if (FUSED) {
        __syncthreads();
        for (int i = tid; i < total; i += kPlan) give_page(a, i, total, free);
    }
}

__global__ __launch_bounds__(kBlock) void commit_pages_kernel(const CacheArgs a)
{
    const int total = a.page_start[a.B], free = *a.free_count_out - total;
    for (int i = blockIdx.x * kBlock + threadIdx.x; i < total; i += gridDim.x * kBlock) give_page(a, i, total, free);
}

static bool cache_ok(int32_t B, int32_t max_blocks, int32_t page_size, int32_t num_pages)
{
    return B >= 0 && B <= kMaxCacheSeqs && max_blocks >= 1 && page_size >= 1 && num_pages >= 0 &&
           (int64_t)max_blocks * page_size < ((int64_t)1 << 31) && num_pages < 1 << 30;
}

}  // namespace sv

extern "C" {

int32_t spec_cache_extend(const int32_t *seq_len, const int32_t *new_len, int32_t extra, int32_t B,
                          int32_t *block_table, int32_t max_blocks, int32_t page_size, const int32_t *free_list,
                          int32_t num_pages, const int32_t *free_count, int32_t *free_count_out,
                          int32_t max_tokens, int64_t *slots, int32_t *positions, int32_t *seq_ids,
                          int32_t *query_start, int32_t *granted, int32_t *page_start, int32_t *error_word,
                          void *stream)
{
    if (!sv::cache_ok(B, max_blocks, page_size, num_pages) || max_tokens < 0) return SV_EINVAL;
    if (B == 0) return SV_OK;
    if (!seq_len || !block_table || !free_list || !free_count || !free_count_out || !query_start || !granted ||
        !page_start || (max_tokens > 0 && (!slots || !positions || !seq_ids)))
        return SV_EINVAL;
    sv::CacheArgs a = {};
    a.seq_len = seq_len;
    a.counts = new_len;
    a.extra = extra;
    a.B = B;
    a.table = block_table;
    a.max_blocks = max_blocks;
    a.page_size = page_size;
    a.free_list = const_cast<int32_t *>(free_list);
    a.num_pages = num_pages;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.max_tokens = max_tokens;
    a.slots = slots;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.query_start = query_start;
    a.granted = granted;
    a.page_start = page_start;
    a.error_word = error_word;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (max_tokens <= sv::kFusedTokens) {
        sv::extend_plan_kernel<true><<<1, sv::kPlan, 0, s>>>(a);
    } else {
        sv::extend_plan_kernel<false><<<1, sv::kPlan, 0, s>>>(a);
        sv::extend_tokens_kernel<<<(unsigned)(((int64_t)max_tokens + sv::kBlock - 1) / sv::kBlock), sv::kBlock, 0, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

int32_t spec_cache_commit(const int32_t *seq_len, const int32_t *reserved, const int32_t *accepted_len,
                          int32_t extra, const int32_t *finished, int32_t B, const int32_t *block_table,
                          int32_t max_blocks, int32_t page_size, int32_t *free_list, int32_t num_pages,
                          const int32_t *free_count, int32_t *free_count_out, int32_t *seq_len_out,
                          int32_t *page_start, int32_t *error_word, void *stream)
{
    if (!sv::cache_ok(B, max_blocks, page_size, num_pages)) return SV_EINVAL;
    if (B == 0) return SV_OK;
    if (!seq_len || !reserved || !accepted_len || !block_table || !free_list || !free_count || !free_count_out ||
        !seq_len_out || !page_start)
        return SV_EINVAL;
    sv::CacheArgs a = {};
    a.seq_len = seq_len;
    a.counts = reserved;
    a.accepted = accepted_len;
    a.extra = extra;
    a.finished = finished;
    a.B = B;
    a.table = const_cast<int32_t *>(block_table);
    a.max_blocks = max_blocks;
    a.page_size = page_size;
    a.free_list = free_list;
    a.num_pages = num_pages;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.seq_len_out = seq_len_out;
    a.page_start = page_start;
    a.error_word = error_word;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!finished || (int64_t)B * max_blocks <= sv::kFusedPages) {
        sv::commit_plan_kernel<true><<<1, sv::kPlan, 0, s>>>(a);
    } else {
        sv::commit_plan_kernel<false><<<1, sv::kPlan, 0, s>>>(a);
        const int64_t most = std::min<int64_t>((int64_t)B * max_blocks, num_pages);
        const unsigned grid = (unsigned)std::min<int64_t>((most + sv::kBlock - 1) / sv::kBlock, 1024);
        if (grid) sv::commit_pages_kernel<<<grid, sv::kBlock, 0, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
