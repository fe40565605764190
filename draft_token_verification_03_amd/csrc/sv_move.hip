// sv_move.hip -- rows of caches that change places: the beams of a beam
// search (dense caches and block tables) and the accepted path of a token
// tree.  Copies bound by memory, done in place without a second buffer: one
// thread owns one vector column of all rows that exchange contents, so it
// has read every source before it writes, and no two threads touch the same
// bytes.  Each source that another beam takes over is read once, each beam
// with another parent written once; nontemporal, since a cache is larger than
// L2 and read next by other kernels (165 -> 151 us for 0.7 GB).  With every
// beam moving, bf16: dense W = 4 5.9 TB/s, 8 5.8, 16 5.3, 32 4.9; paged 5.6,
// 5.5, 5.5, 3.9 (at 32 the columns in registers leave two waves per SIMD); a
// plain copy of this card's memory runs at 5.1 TB/s.
#include <algorithm>

#include "specdecode.h"
#include "sv_internal.h"

namespace sv {

constexpr int kMovePools = 128;  // pools per launch: their addresses travel as kernel arguments

struct MoveArgs {
    char *pool[kMovePools];
    const int32_t *table;     // block tables, or null for dense caches
    const int32_t *parent;    // reorder
    const int32_t *start, *length;
    const int32_t *path, *accepted;  // compact
    int32_t *error_word;
    int32_t B, W, G, S;       // S: positions per beam (dense) or per page
    int32_t row_vecs;         // vectors per row
    int32_t num_pages, max_blocks, max_length;
    int32_t N, first;
    int32_t chunks;           // workgroups per (pool, sequence, group), or per sequence
    int32_t pools;            // of this launch
};

__device__ __forceinline__ void move_error(const MoveArgs &a, int bit)
{
    if (a.error_word) atomicOr(a.error_word, bit);
}

// ---------------------------------------------------------------------------
// Reordering of beams: beam j <- beam parent[j].  Lane j of each wave holds
// parent[j]; the destinations of source s are one ballot.

template <int WM>
struct BeamMoves {
    uint32_t to[WM];  // beams that take over beam s, itself aside
};

template <int WM>
__device__ __forceinline__ BeamMoves<WM> beam_moves(const MoveArgs &a, int b)
{
    const int lane = threadIdx.x & 63;
    int p = -1;
    if (lane < a.W) p = a.parent[(int64_t)b * a.W + lane];
    if (p >= a.W) {
        move_error(a, SV_ERR_PARENT);
        p = -1;
    }
    BeamMoves<WM> m;
#pragma unroll
    for (int s = 0; s < WM; ++s) m.to[s] = (uint32_t)__ballot(p == s && lane != s);
    return m;
}

// NV vectors of each beam per thread, so that W NV are in flight: with W = 4
// 2, 4 and 8 of them take 364, 365 and 381 us for 1.07 GB moved.
template <class T, int WM, int NV>
__global__ __launch_bounds__(kBlock) void reorder_dense_kernel(const MoveArgs a)
{
    int blk = blockIdx.x;
    const int chunk = blk % a.chunks;
    blk /= a.chunks;
    const int g = blk % a.G;
    blk /= a.G;
    const int b = blk % a.B, pool = blk / a.B;
    int len = a.S;
    if (a.length) {
        len = a.length[b];
        if (len < 0 || len > a.S) {
            if (threadIdx.x == 0) move_error(a, SV_ERR_LENGTH);
            return;
        }
    }
    const int64_t n = (int64_t)len * a.row_vecs;
    const int64_t v0 = (int64_t)chunk * (kBlock * NV);
    if (v0 >= n) return;
    const BeamMoves<WM> m = beam_moves<WM>(a, b);
    const int64_t beam = (int64_t)a.G * a.S * a.row_vecs;  // vectors from beam to beam
    T *base = reinterpret_cast<T *>(a.pool[pool]) + (int64_t)b * a.W * beam + (int64_t)g * a.S * a.row_vecs;
    T x[WM][NV];
#pragma unroll
    for (int s = 0; s < WM; ++s)
        if (m.to[s])
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t v = v0 + i * kBlock + threadIdx.x;
                if (v < n) x[s][i] = __builtin_nontemporal_load(&base[s * beam + v]);
            }
#pragma unroll
    for (int s = 0; s < WM; ++s)
        for (uint32_t to = m.to[s]; to; to &= to - 1) {
            const int j = __ffs(to) - 1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t v = v0 + i * kBlock + threadIdx.x;
                if (v < n) __builtin_nontemporal_store(x[s][i], &base[j * beam + v]);
            }
        }
}

template <class T, int WM>
__global__ __launch_bounds__(kBlock) void reorder_paged_kernel(const MoveArgs a)
{
    int blk = blockIdx.x;
    const int chunk = blk % a.chunks;
    blk /= a.chunks;
    const int g = blk % a.G;
    blk /= a.G;
    const int b = blk % a.B, pool = blk / a.B;
    int len = a.length[b];
    const int from = a.start ? a.start[b] : 0;
    const int most = a.max_blocks * a.S;
    if (from < 0 || len < 0 || len > most || from > most) {
        if (threadIdx.x == 0) move_error(a, SV_ERR_LENGTH);
        return;
    }
    if (len > a.max_length) {
        if (threadIdx.x == 0) move_error(a, SV_ERR_LENGTH);
        len = a.max_length;
    }
    const int64_t v = (int64_t)chunk * kBlock + threadIdx.x;
    const int64_t n = (int64_t)(len - from) * a.row_vecs;
    if ((int64_t)chunk * kBlock >= n) return;
    const BeamMoves<WM> m = beam_moves<WM>(a, b);  // every lane still here
    if (v >= n) return;
    const int r = (int)(v / a.row_vecs);
    const int at = from + r, block = at / a.S;
    const int64_t inside = ((int64_t)g * a.S + at % a.S) * a.row_vecs + (v - (int64_t)r * a.row_vecs);
    const int64_t page_vecs = (int64_t)a.G * a.S * a.row_vecs;
    const int32_t *table = a.table + (int64_t)b * a.W * a.max_blocks + block;
    T *base = reinterpret_cast<T *>(a.pool[pool]) + inside;
    int page[WM];
    T x[WM];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < WM; ++s) page[s] = m.to[s] ? table[(int64_t)s * a.max_blocks] : -1;
#pragma unroll
    for (int s = 0; s < WM; ++s) {
        if (!m.to[s]) continue;
        if (page[s] < 0 || page[s] >= a.num_pages) {
            bad = true;
            page[s] = -1;
        } else {
            x[s] = __builtin_nontemporal_load(&base[page[s] * page_vecs]);
        }
    }
#pragma unroll
    for (int s = 0; s < WM; ++s) {
        if (page[s] < 0) continue;
        for (uint32_t to = m.to[s]; to; to &= to - 1) {
            const int p = table[(int64_t)(__ffs(to) - 1) * a.max_blocks];
            if (p < 0 || p >= a.num_pages) bad = true;
            else if (p != page[s]) __builtin_nontemporal_store(x[s], &base[p * page_vecs]);
        }
    }
    if (bad) move_error(a, SV_ERR_PAGE);
}

// ---------------------------------------------------------------------------
// The accepted path of a tree: row first + path[i] -> row first + i, i
// ascending.  path[i] >= i, and a later source lies above every earlier
// destination, so a thread that reads ahead of its writes reads what was
// there before the call.

constexpr int kMaxPath = 128;
constexpr int kPathAhead = 8;  // rows read before the first of them is written

// A workgroup takes kBlock vectors of one position of one sequence, of all
// pools behind each other.  Its first threads turn the path into row offsets
// (one round trip for the path, one for the tables), the rest is copies: 8.5
// us for 34 MB (64 sequences, 32 pools of 2 KB rows), against 16.6 with the
// offsets formed by every thread and a workgroup per pool; 4.7 us for four
// sequences, a launch's time.
template <class T>
__global__ __launch_bounds__(kBlock) void compact_kernel(const MoveArgs a)
{
    __shared__ int64_t from[kMaxPath], to[kMaxPath];  // vectors from a column's start; to < 0: stays
    __shared__ int errors;
    const int chunk = blockIdx.x % a.chunks, b = blockIdx.x / a.chunks, tid = threadIdx.x;
    const int d = a.accepted[b];
    if (d <= 0) return;
    if (d > a.N) {
        if (tid == 0) move_error(a, SV_ERR_TREE);
        return;
    }
    if (tid == 0) errors = 0;
    __syncthreads();
    const int64_t page_vecs = (int64_t)a.G * a.S * a.row_vecs;
    if (tid < d) {
        const int32_t *path = a.path + (int64_t)b * a.N, *table = a.table + (int64_t)b * a.max_blocks;
        const int p = path[tid], before = tid ? path[tid - 1] : -1, len = a.length[b];
        const int64_t base = (int64_t)len + a.first, most = (int64_t)a.max_blocks * a.S;
        int bad = p >= a.N || p <= before ? SV_ERR_TREE : len < 0 || base + p >= most ? SV_ERR_LENGTH : 0;
        if (bad) atomicOr(&errors, bad);
        from[tid] = 0;
        to[tid] = -1;
        if (!bad && p != tid && base + tid < most) {
            const int at = (int)base + p, dest = (int)base + tid;
            const int pf = table[at / a.S], pd = table[dest / a.S];
            if (pf < 0 || pf >= a.num_pages || pd < 0 || pd >= a.num_pages) {
                move_error(a, SV_ERR_PAGE);
            } else {
                from[tid] = pf * page_vecs + (int64_t)(at % a.S) * a.row_vecs;
                to[tid] = pd * page_vecs + (int64_t)(dest % a.S) * a.row_vecs;
            }
        }
    }
    __syncthreads();
    if (errors) {  // the sequence stays as it is
        if (tid == 0) move_error(a, errors);
        return;
    }
    const int64_t v = (int64_t)chunk * kBlock + tid;
    const int cols = a.G * a.row_vecs, pool = (int)(v / cols);
    if (pool >= a.pools) return;
    const int c = (int)(v - (int64_t)pool * cols), g = c / a.row_vecs;
    T *col = reinterpret_cast<T *>(a.pool[pool]) + (int64_t)g * a.S * a.row_vecs + (c - g * a.row_vecs);
    for (int i0 = 0; i0 < d; i0 += kPathAhead) {
        // all loads of a batch are in flight together; a row that stays reads its pool's first
        T x[kPathAhead];
#pragma unroll
        for (int k = 0; k < kPathAhead; ++k) x[k] = col[from[min(i0 + k, d - 1)]];
#pragma unroll
        for (int k = 0; k < kPathAhead; ++k)
            if (i0 + k < d && to[i0 + k] >= 0) col[to[i0 + k]] = x[k];
    }
}

// ---------------------------------------------------------------------------

// Bytes per vector that every row of every pool allows.
static int move_vector(void *const *pools, int32_t n, int64_t row_bytes)
{
    uintptr_t bits = (uintptr_t)row_bytes;
    for (int32_t i = 0; i < n; ++i) bits |= (uintptr_t)pools[i];
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
}

static bool pools_ok(void *const *pools, int32_t n)
{
    if (n > 0 && !pools) return false;
    for (int32_t i = 0; i < n; ++i)
        if (!pools[i]) return false;
    return true;
}

template <class T>
static void launch_reorder(const MoveArgs &a, int n, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)n * a.B * a.G * a.chunks);
    if (a.table) {
        if (a.W <= 4) reorder_paged_kernel<T, 4><<<grid, kBlock, 0, s>>>(a);
        else if (a.W <= 8) reorder_paged_kernel<T, 8><<<grid, kBlock, 0, s>>>(a);
        else if (a.W <= 16) reorder_paged_kernel<T, 16><<<grid, kBlock, 0, s>>>(a);
        else reorder_paged_kernel<T, 32><<<grid, kBlock, 0, s>>>(a);
    } else {
        if (a.W <= 4) reorder_dense_kernel<T, 4, 4><<<grid, kBlock, 0, s>>>(a);
        else if (a.W <= 8) reorder_dense_kernel<T, 8, 2><<<grid, kBlock, 0, s>>>(a);
        else if (a.W <= 16) reorder_dense_kernel<T, 16, 1><<<grid, kBlock, 0, s>>>(a);
        else reorder_dense_kernel<T, 32, 1><<<grid, kBlock, 0, s>>>(a);
    }
}

template <class T>
static void launch_compact(const MoveArgs &a, hipStream_t s)
{
    compact_kernel<T><<<(unsigned)((int64_t)a.B * a.chunks), kBlock, 0, s>>>(a);
}

enum Move { kReorder, kCompact };

static int32_t move_launch(MoveArgs &a, Move what, void *const *pools, int32_t n_pools, int64_t row_bytes,
                           int64_t positions, hipStream_t s)
{
    const int vb = move_vector(pools, n_pools, row_bytes);
    a.row_vecs = (int32_t)(row_bytes / vb);
    const int64_t most = ((int64_t)1 << 31) - kBlock;
    // workgroups: per (pool, sequence, group) for the positions of a beam, or
    // per sequence for the vectors of a position in all pools
    const int nv = what == kReorder && !a.table ? (a.W <= 4 ? 4 : a.W <= 8 ? 2 : 1) : 1;
    const int64_t each = what == kReorder ? positions * a.row_vecs : (int64_t)a.G * a.row_vecs;
    if (what == kCompact && each >= most) return SV_EINVAL;
    for (int32_t p0 = 0; p0 < n_pools; p0 += kMovePools) {
        a.pools = std::min(kMovePools, n_pools - p0);
        const int64_t vecs = what == kReorder ? each : each * a.pools, per = (int64_t)kBlock * nv;
        const int64_t chunks = std::max<int64_t>(1, (vecs + per - 1) / per);
        if (chunks > most / a.B / (what == kReorder ? a.pools * (int64_t)a.G : 1)) return SV_EINVAL;
        a.chunks = (int32_t)chunks;
        for (int i = 0; i < a.pools; ++i) a.pool[i] = static_cast<char *>(pools[p0 + i]);
        if (what == kReorder) {
            if (vb == 16) launch_reorder<u32x4>(a, a.pools, s);
            else if (vb == 4) launch_reorder<uint32_t>(a, a.pools, s);
            else launch_reorder<uint8_t>(a, a.pools, s);
        } else {
            if (vb == 16) launch_compact<u32x4>(a, s);
            else if (vb == 4) launch_compact<uint32_t>(a, s);
            else launch_compact<uint8_t>(a, s);
        }
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

static bool paged_ok(int32_t G, int32_t page_size, int64_t row_bytes, int32_t num_pages, int32_t max_blocks)
{
    return G >= 1 && page_size >= 1 && row_bytes >= 1 && num_pages >= 1 && max_blocks >= 1 &&
           (int64_t)max_blocks * page_size < ((int64_t)1 << 31) && row_bytes < ((int64_t)1 << 31) &&
           (double)num_pages * G * page_size * (double)row_bytes < 0x1p62;
}

}  // namespace sv

extern "C" {

int32_t spec_beam_reorder(void *const *pools, int32_t n_pools, int32_t B, int32_t W, int32_t G, int32_t S,
                          int64_t row_bytes, const int32_t *parent, const int32_t *length, int32_t *error_word,
                          void *stream)
{
    if (n_pools < 0 || n_pools > SV_MAX_POOLS || B < 0 || W < 1 || W > SV_MAX_BEAMS || G < 1 || S < 0 ||
        row_bytes < 1 || row_bytes >= ((int64_t)1 << 31) ||
        (double)B * W * G * S * (double)row_bytes >= 0x1p62)
        return SV_EINVAL;
    if (B == 0 || n_pools == 0 || S == 0) return SV_OK;
    if (!sv::pools_ok(pools, n_pools) || !parent) return SV_EINVAL;
    sv::MoveArgs a = {};
    a.parent = parent;
    a.length = length;
    a.error_word = error_word;
    a.B = B;
    a.W = W;
    a.G = G;
    a.S = S;
    return sv::move_launch(a, sv::kReorder, pools, n_pools, row_bytes, S, static_cast<hipStream_t>(stream));
}

int32_t spec_beam_reorder_paged(void *const *pools, int32_t n_pools, int32_t B, int32_t W, int32_t G,
                                int32_t page_size, int64_t row_bytes, int32_t num_pages,
                                const int32_t *block_table, int32_t max_blocks, const int32_t *parent,
                                const int32_t *start, const int32_t *length, int32_t max_length,
                                int32_t *error_word, void *stream)
{
    if (n_pools < 0 || n_pools > SV_MAX_POOLS || B < 0 || W < 1 || W > SV_MAX_BEAMS || max_length < 0 ||
        !sv::paged_ok(G, page_size, row_bytes, num_pages, max_blocks) ||
        (int64_t)max_length > (int64_t)max_blocks * page_size)
        return SV_EINVAL;
    if (B == 0 || n_pools == 0 || max_length == 0) return SV_OK;
    if (!sv::pools_ok(pools, n_pools) || !parent || !length || !block_table) return SV_EINVAL;
    sv::MoveArgs a = {};
    a.table = block_table;
    a.parent = parent;
    a.start = start;
    a.length = length;
    a.error_word = error_word;
    a.B = B;
    a.W = W;
    a.G = G;
    a.S = page_size;
    a.num_pages = num_pages;
    a.max_blocks = max_blocks;
    a.max_length = max_length;
    return sv::move_launch(a, sv::kReorder, pools, n_pools, row_bytes, max_length,
                           static_cast<hipStream_t>(stream));
}

int32_t spec_cache_compact(void *const *pools, int32_t n_pools, int32_t B, int32_t G, int32_t page_size,
                           int64_t row_bytes, int32_t num_pages, const int32_t *block_table, int32_t max_blocks,
                           const int32_t *seq_len, int32_t first, const int32_t *path,
                           const int32_t *accepted_len, int32_t N, int32_t *error_word, void *stream)
{
    if (n_pools < 0 || n_pools > SV_MAX_POOLS || B < 0 || N < 0 || N > sv::kMaxPath || first < 0 ||
        !sv::paged_ok(G, page_size, row_bytes, num_pages, max_blocks))
        return SV_EINVAL;
    if (B == 0 || n_pools == 0 || N == 0) return SV_OK;
    if (!sv::pools_ok(pools, n_pools) || !block_table || !seq_len || !path || !accepted_len) return SV_EINVAL;
    sv::MoveArgs a = {};
    a.table = block_table;
    a.length = seq_len;
    a.first = first;
    a.path = path;
    a.accepted = accepted_len;
    a.N = N;
    a.error_word = error_word;
    a.B = B;
    a.W = 1;
    a.G = G;
    a.S = page_size;
    a.num_pages = num_pages;
    a.max_blocks = max_blocks;
    return sv::move_launch(a, sv::kCompact, pools, n_pools, row_bytes, 1, static_cast<hipStream_t>(stream));
}

}  // extern "C"
