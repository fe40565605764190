// sv_cache.hip -- lengths, pages and slots of a paged cache: what a decode
// loop needs before the forward pass (pages, block tables, slot maps) and
// after the verify step (lengths, pages given back), from lengths that are
// on the GPU already, so that the loop never waits for them on the host.
//
// Both calls are a prefix sum over the sequences followed by independent work
// per token (page).  One workgroup scans: there are at most a few thousand
// sequences, and a second workgroup would need a hand-off that costs more
// than their loads.  Few tokens follow in the same workgroup, so that a
// decode step is one launch; many get a launch of their own.  What bounds a
// step is dependent memory round trips: lengths, then pages.  Up to kPlan
// sequences have a thread each, their sums stay in LDS, and then every
// sequence gets as many lanes as there are to spare for its tokens, so that
// nothing searches and no trip is added.  64 sequences: extend by 6 tokens
// 3.7 us of kernel, commit 2.9 us, where an empty launch takes 3.5 us from one
// to the next; 256 sequences with up to 4096 new tokens each 4.4 us for the
// scan and 9.5 us for a million tokens' places; the end of a step of 2000
// sequences, 100 of them giving all their pages back, 5.0 and 5.1 us.
#include <algorithm>

#include "specdecode.h"
#include "sv_internal.h"

namespace sv {

constexpr int kPlan = 1024;             // threads of the scanning workgroup
constexpr int kPlanWaves = kPlan / 64;
// At most so many tokens are placed by the scanning workgroup (64 sequences:
// 384 tokens 4.7 us, with a launch of their own 7.5; 4096 8.0 and 9.7; 8192 9.6
// and 9.9; 512 sequences, 8192 tokens 17.8 and 11.9).
constexpr int kFusedTokens = 4096;
// The same for pages that could come back when sequences end, which few do in
// a step (64 sequences of up to 512 blocks: none ends 4.3 us, with a launch of
// their own 7.1; a tenth 5.3 to 8.7 and 7.2; all of them 34 and 7.2).
constexpr int kFusedPages = 65536;
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
    uint32_t page_mul, page_shift;  // page_of
};

// Exclusive prefix sums of two counts over the workgroup, and their totals.
// Sums stay below 2^20 2^31, which doubles hold exactly.
struct Sums {
    int64_t a, b, all_a, all_b;
};

__device__ __forceinline__ Sums plan_scan(int64_t a, int64_t b, double *lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const double ia = wave_inclusive_scan((double)a), ib = wave_inclusive_scan((double)b);
    if (lane == 63) {
        lds[wave] = ia;
        lds[kPlanWaves + wave] = ib;
    }
    __syncthreads();
    double xa = ia, xb = ib, all_a = 0.0, all_b = 0.0;
    for (int w = 0; w < waves; ++w) {
        const double x = lds[w], y = lds[kPlanWaves + w];
        if (w < wave) {
            xa += x;
            xb += y;
        }
        all_a += x;
        all_b += y;
    }
    __syncthreads();
    return {(int64_t)xa - a, (int64_t)xb - b, (int64_t)all_a, (int64_t)all_b};
}

__device__ __forceinline__ void cache_error(const CacheArgs &a, int bit)
{
    if (a.error_word) atomicOr(a.error_word, bit);
}

// n / page_size for 0 <= n < 2^31 by a product: with 2^(s-1) < page_size <=
// 2^s and mul = ceil(2^(31+s) / page_size), n mul >> (31 + s).
__device__ __forceinline__ int page_of(const CacheArgs &a, int n)
{
    return (int)(__umulhi(2u * (uint32_t)n, a.page_mul) >> a.page_shift);
}

__device__ __forceinline__ int pages_of(const CacheArgs &a, int tokens)
{
    const int full = page_of(a, tokens);
    return full + (tokens != full * a.page_size ? 1 : 0);
}

// The free list's length, held within the list.
__device__ __forceinline__ int free_pages(const CacheArgs &a)
{
    const int f = *a.free_count;
    const int held = min(max(f, 0), a.num_pages);
    if (held != f && threadIdx.x == 0) cache_error(a, SV_ERR_PAGES);
    return held;
}

// Tokens per thread where they have a launch of their own (1, 2, 8: 15.2, 13.9
// and 16.7 us against 13.7 for a million).
constexpr int kTokens = 4;
constexpr int kStaged = 2048;  // sequences whose numbers a workgroup of it copies to LDS (64: 9.9 us against 11.0)

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
    x.need = bad ? 0 : pages_of(a, x.len + x.n) - pages_of(a, x.len);
    return x;
}

// Token i of sequence b (len tokens held, query_start q, page_start p) into
// place t of the call; `free` is the free list's length before the call.
__device__ __forceinline__ void place_token(const CacheArgs &a, int t, int b, int i, int len, bool granted, int p,
                                            int free)
{
    const int at = len + i;
    int64_t slot = -1;
    if (granted) {
        const int block = page_of(a, at), off = at - block * a.page_size;
        const int first = pages_of(a, len);
        int32_t *entry = a.table + (int64_t)b * a.max_blocks + block;
        const bool fresh = block >= first;
        const int page = *(fresh ? a.free_list + (free - 1 - (p + block - first)) : entry);
        if (fresh && off == 0) *entry = page;  // a new page's first token is at its start
        if (page >= 0 && page < a.num_pages) slot = (int64_t)page * a.page_size + off;
        else cache_error(a, SV_ERR_PAGE);
    }
    a.slots[t] = slot;
    a.positions[t] = at;
    a.seq_ids[t] = b;
}

__device__ __forceinline__ void no_token(const CacheArgs &a, int t)
{
    a.slots[t] = -1;
    a.positions[t] = 0;
    a.seq_ids[t] = -1;
}

// What a sequence with x new tokens before q and p gets.
struct Grant {
    bool room, fits;
};

__device__ __forceinline__ Grant grant(const CacheArgs &a, const NewTokens &x, int64_t q, int64_t p, int free)
{
    const bool room = q + x.n <= a.max_tokens;
    return {room, room && (x.need == 0 || p + x.need <= free)};
}

// Sequences a workgroup's width at a time, one per thread, the next ones
// requested while these are scanned; FUSED (one round of them): their tokens too.
template <bool FUSED>
__global__ __launch_bounds__(kPlan) void extend_plan_kernel(const CacheArgs a)
{
    __shared__ double lds[2 * kPlanWaves];
    __shared__ int4 seqs[FUSED ? kPlan : 1];  // len, query_start, tokens (negative: not granted), page_start
    __shared__ int used;
    const int tid = threadIdx.x;
    NewTokens x = {0, 0, 0};
    bool bad = false;
    if (tid < a.B) x = new_tokens(a, tid, bad);
    const int free = free_pages(a);
    if (tid == 0) used = 0;
    int64_t q0 = 0, p0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        NewTokens next = {0, 0, 0};
        bool next_bad = false;
        if (!FUSED && b + (int)blockDim.x < a.B) next = new_tokens(a, b + blockDim.x, next_bad);
        const Sums s = plan_scan(x.n, x.need, lds);  // its barriers order `used` too
        const int64_t qs = q0 + s.a, ps = p0 + s.b;
        const Grant g = grant(a, x, qs, ps, free);
        if (b < a.B) {
            if (g.fits && x.need) atomicMax(&used, (int)(ps + x.need));
            if (bad || !g.room) cache_error(a, SV_ERR_LENGTH);
            if (g.room && !g.fits) cache_error(a, SV_ERR_PAGES);
        }
        __syncthreads();
        if (b < a.B) {
            // behind the sequences that got theirs nothing is taken, so that
            // `used` is final for whoever it cuts off
            const int q = (int)min(qs, (int64_t)a.max_tokens), p = (int)min(ps, (int64_t)used);
            a.query_start[b] = q;
            a.page_start[b] = p;
            a.granted[b] = g.fits ? x.n : 0;
            if (FUSED) {
                const int here = min(x.n, a.max_tokens - q);
                seqs[b] = make_int4(x.len, q, g.fits ? here : -here, p);
            }
        }
        q0 += s.all_a;
        p0 += s.all_b;
        x = next;
        bad = next_bad;
    }
    const int total = (int)min(q0, (int64_t)a.max_tokens);
    if (tid == 0) {
        a.query_start[a.B] = total;
        a.page_start[a.B] = used;
        *a.free_count_out = free - used;
    }
    if (!FUSED) return;
    __syncthreads();
    int lanes = 1;  // per sequence
    while (2 * lanes * a.B <= (int)blockDim.x) lanes *= 2;
    const int b = tid / lanes;
    if (b < a.B) {
        const int4 v = seqs[b];
        for (int i = tid % lanes; i < abs(v.z); i += lanes) place_token(a, v.y + i, b, i, v.x, v.z > 0, v.w, free);
    }
    for (int t = total + tid; t < a.max_tokens; t += blockDim.x) no_token(a, t);
}

// kTokens tokens per thread, a workgroup apart, every step for all of them at
// once: their sequences, their pages, the stores.  The sequences' numbers are
// searched and read in LDS where they fit (STAGED): one memory round trip for
// them all instead of one per step of the search.
template <bool STAGED>
__global__ __launch_bounds__(kBlock) void extend_tokens_kernel(const CacheArgs a)
{
    __shared__ int32_t lds[STAGED ? 4 : 1][STAGED ? kStaged : 1];
    if (STAGED) {
        for (int i = threadIdx.x; i < a.B; i += kBlock) {
            lds[0][i] = a.query_start[i];
            lds[1][i] = a.seq_len[i];
            lds[2][i] = a.page_start[i];
            lds[3][i] = a.granted[i];
        }
    }
    const int total = a.query_start[a.B], free = *a.free_count_out + a.page_start[a.B];
    __syncthreads();
    const int32_t *start = STAGED ? lds[0] : a.query_start, *lens = STAGED ? lds[1] : a.seq_len;
    const int32_t *taken = STAGED ? lds[2] : a.page_start, *granted = STAGED ? lds[3] : a.granted;
    const int64_t t0 = (int64_t)blockIdx.x * (kTokens * kBlock) + threadIdx.x;
    int t[kTokens], b[kTokens], at[kTokens], off[kTokens], first[kTokens], p[kTokens], page[kTokens];
    int32_t *entry[kTokens];
    bool some[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        t[j] = (int)min(t0 + j * kBlock, (int64_t)a.max_tokens);
        some[j] = t[j] < total;
        b[j] = 0;
    }
    for (int step = 1 << (31 - __clz(a.B)); step; step >>= 1)
#pragma unroll
        for (int j = 0; j < kTokens; ++j)
            if (b[j] + step < a.B && start[b[j] + step] <= t[j]) b[j] += step;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        const int len = lens[b[j]];
        at[j] = len + t[j] - start[b[j]];
        first[j] = pages_of(a, len);
        p[j] = taken[b[j]];
        some[j] = some[j] && granted[b[j]] > 0;
    }
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        const int block = page_of(a, at[j]);
        off[j] = at[j] - block * a.page_size;
        const bool fresh = block >= first[j];
        entry[j] = fresh && off[j] == 0 ? a.table + (int64_t)b[j] * a.max_blocks + block : nullptr;
        const int32_t *from = fresh ? a.free_list + (free - 1 - (p[j] + block - first[j]))
                                    : a.table + (int64_t)b[j] * a.max_blocks + block;
        page[j] = *(some[j] ? from : a.query_start);
    }
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        if (t[j] >= a.max_tokens) continue;
        if (t[j] >= total) {
            no_token(a, t[j]);
            continue;
        }
        int64_t slot = -1;
        if (some[j]) {
            if (entry[j]) *entry[j] = page[j];
            if (page[j] >= 0 && page[j] < a.num_pages)
                slot = (int64_t)page[j] * a.page_size + off[j];
            else
                cache_error(a, SV_ERR_PAGE);
        }
        a.slots[t[j]] = slot;
        a.positions[t[j]] = at[j];
        a.seq_ids[t[j]] = b[j];
    }
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
        bad = want != keep && held > 0;  // what got no pages keeps nothing
        k.len = len + keep;
    }
    k.first = pages_of(a, k.len);
    k.back = pages_of(a, len + held) - k.first;
    return k;
}

// Number i of the `total` pages that come back; the list held `free` before.
__device__ __forceinline__ void put_page(const CacheArgs &a, int page, int i, int total, int free)
{
    if (page < 0 || page >= a.num_pages) {
        cache_error(a, SV_ERR_PAGE);
        page = -1;
    }
    a.free_list[free + total - 1 - i] = page;
}

__device__ __forceinline__ void give_page(const CacheArgs &a, int b, int block, int i, int total, int free)
{
    put_page(a, a.table[(int64_t)b * a.max_blocks + block], i, total, free);
}

// As extend_plan_kernel; FUSED (one round of sequences): their pages too.
template <bool FUSED>
__global__ __launch_bounds__(kPlan) void commit_plan_kernel(const CacheArgs a)
{
    __shared__ double lds[2 * kPlanWaves];
    __shared__ int4 seqs[FUSED ? kPlan : 1];  // first block given back, blocks, page_start
    const int tid = threadIdx.x;
    Kept k = {0, 0, 0};
    bool bad = false;
    if (tid < a.B) k = kept_tokens(a, tid, bad);
    const int free = free_pages(a), room = a.num_pages - free, most = k.back;
    int64_t p0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        Kept next = {0, 0, 0};
        bool next_bad = false;
        if (!FUSED && b + (int)blockDim.x < a.B) next = kept_tokens(a, b + blockDim.x, next_bad);
        const Sums s = plan_scan(k.back, 0, lds);
        const int p = (int)min(p0 + s.a, (int64_t)room);
        if (b < a.B) {
            a.page_start[b] = p;
            a.seq_len_out[b] = k.len;
            if (FUSED) seqs[b] = make_int4(k.first, min(k.back, room - p), p, 0);
            if (bad) cache_error(a, SV_ERR_LENGTH);
        }
        p0 += s.all_a;
        k = next;
        bad = next_bad;
    }
    const int total = (int)min(p0, (int64_t)room);
    if (tid == 0) {
        if (p0 > room) cache_error(a, SV_ERR_PAGES);
        a.page_start[a.B] = total;
        *a.free_count_out = free + total;
    }
    if (!FUSED) return;
    int lanes = 1;  // per sequence
    while (2 * lanes * a.B <= (int)blockDim.x) lanes *= 2;
    // a sequence that gives back many pages (its end, usually) has everyone at
    // work on all of them, each searching for its own
    if (__syncthreads_or(most > 4 * lanes)) {
        constexpr int kAtOnce = 4;
        for (int i0 = tid; i0 < total; i0 += kAtOnce * blockDim.x) {
            int lo[kAtOnce] = {};
            for (int step = 1 << (31 - __clz(a.B)); step; step >>= 1)
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    if (lo[j] + step < a.B && seqs[lo[j] + step].z <= i0 + j * (int)blockDim.x) lo[j] += step;
            int page[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = min(i0 + j * (int)blockDim.x, total - 1), block = seqs[lo[j]].x + i - seqs[lo[j]].z;
                page[j] = a.table[(int64_t)lo[j] * a.max_blocks + block];
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (i0 + j * (int)blockDim.x < total) put_page(a, page[j], i0 + j * (int)blockDim.x, total, free);
        }
        return;
    }
    const int b = tid / lanes;
    if (b < a.B) {
        const int4 v = seqs[b];
        for (int i = tid % lanes; i < v.y; i += lanes) give_page(a, b, v.x + i, v.z + i, total, free);
    }
}

template <bool STAGED>
__global__ __launch_bounds__(kBlock) void commit_pages_kernel(const CacheArgs a)
{
    __shared__ int32_t lds[STAGED ? 2 : 1][STAGED ? kStaged : 1];
    const int total = a.page_start[a.B], free = *a.free_count_out - total;
    if ((int64_t)blockIdx.x * kBlock >= total) return;
    if (STAGED) {
        for (int i = threadIdx.x; i < a.B; i += kBlock) {
            lds[0][i] = a.page_start[i];
            lds[1][i] = a.seq_len_out[i];
        }
    }
    __syncthreads();
    const int32_t *start = STAGED ? lds[0] : a.page_start, *lens = STAGED ? lds[1] : a.seq_len_out;
    for (int i = blockIdx.x * kBlock + threadIdx.x; i < total; i += gridDim.x * kBlock) {
        const int b = find_run(start, 0, a.B, i);
        give_page(a, b, pages_of(a, lens[b]) + i - start[b], i, total, free);
    }
}

// Threads of the scanning workgroup: one per sequence, and enough for `work`.
static unsigned plan_threads(int32_t B, int64_t work)
{
    unsigned n = 256;
    while (n < (unsigned)kPlan && (n < (unsigned)B || n < work)) n *= 2;
    return n;
}

static void set_page_size(CacheArgs &a, int32_t page_size)
{
    a.page_size = page_size;
    a.page_shift = 0;
    while (((int64_t)1 << a.page_shift) < page_size) ++a.page_shift;
    a.page_mul = (uint32_t)((((uint64_t)1 << (31 + a.page_shift)) + page_size - 1) / page_size);
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
    sv::set_page_size(a, page_size);
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
    const bool fused = B <= sv::kPlan && max_tokens <= sv::kFusedTokens;
    if (fused) sv::extend_plan_kernel<true><<<1, sv::plan_threads(B, max_tokens), 0, s>>>(a);
    else sv::extend_plan_kernel<false><<<1, sv::plan_threads(B, 0), 0, s>>>(a);
    if (!fused && max_tokens > 0) {
        const int64_t per = sv::kBlock * sv::kTokens;
        const unsigned grid = (unsigned)((max_tokens + per - 1) / per);
        if (B <= sv::kStaged) sv::extend_tokens_kernel<true><<<grid, sv::kBlock, 0, s>>>(a);
        else sv::extend_tokens_kernel<false><<<grid, sv::kBlock, 0, s>>>(a);
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
    sv::set_page_size(a, page_size);
    a.free_list = free_list;
    a.num_pages = num_pages;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.seq_len_out = seq_len_out;
    a.page_start = page_start;
    a.error_word = error_word;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool fused = B <= sv::kPlan && (!finished || (int64_t)B * max_blocks <= sv::kFusedPages);
    if (fused) sv::commit_plan_kernel<true><<<1, sv::plan_threads(B, B), 0, s>>>(a);
    else sv::commit_plan_kernel<false><<<1, sv::plan_threads(B, 0), 0, s>>>(a);
    if (!fused) {
        const int64_t most = std::min<int64_t>((int64_t)B * max_blocks, num_pages);
        const unsigned grid = (unsigned)std::min<int64_t>((most + sv::kBlock - 1) / sv::kBlock, 1024);
        if (grid && B <= sv::kStaged) sv::commit_pages_kernel<true><<<grid, sv::kBlock, 0, s>>>(a);
        else if (grid) sv::commit_pages_kernel<false><<<grid, sv::kBlock, 0, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
