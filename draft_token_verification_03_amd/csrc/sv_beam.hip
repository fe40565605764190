// sv_beam.hip -- beam search's selection over beams and vocabulary.
//
//   c(w, v) = s_w + z_w(v) / T - ln sum_u exp(z_w(u) / T)
//
//   1. beam_rows_kernel   one workgroup per (row, chunk): one pass over the
//                         logits for the maximum and the sum of exponentials.
//   2. beam_merge_kernel  one workgroup per sequence: the rows' normalisers
//                         and the best M candidates.
//
// The pass is bound by reading the logits, and on bf16 nearly by its
// exponentials (eight per 16 bytes), so it keeps no lists: beside the sums it
// leaves only the maxima of `cols` columns of its chunk (column l: vectors l,
// l + cols, ...), which its lanes hold anyway.  c rises with z within a beam,
// so the merge turns the maxima into c and takes the M-th largest over all
// columns of the sequence as a floor: M columns hold a candidate at least as
// large each, so no smaller one is among the best M.  Only the columns whose
// maximum reaches the floor, about M, are read again, all at once, and of a
// long one only the tile that held its maximum where the pass saw that no
// other tile of it reaches the floor; what reaches the floor there is ranked by
// counting.  A sequence has between 1024 and 2048 columns (fewer for short
// rows): the merge holds eight a thread, and more leave less to read again.
#include <algorithm>
#include <cfloat>

#include "specdecode.h"
#include "sv_internal.h"
#include "sv_sort.h"
#include "sv_stream.h"
#include "sv_tile.h"

namespace sv {

constexpr double kLn2 = 0.6931471805599453;
constexpr int kBeamLoads = 4;        // 16-byte vectors per thread per tile
// Workgroups the streaming grid aims for: two per CU.  (32 x 8 x 128256 bf16
// 23.3 us, with 768 24.9, with 1536 24.6; no difference beyond 1 us elsewhere.)
constexpr int kBeamFill = 512;
constexpr int kBeamMaxChunks = 64;   // chunks per row: the merge gives each a lane
constexpr int kBeamRowChunks = 256;  // W * chunks at most: with lanes to spare, one thread each in the merge
constexpr int kBeamPre = 8;          // column maxima per thread of the merge
constexpr int kMerge = 1024;         // threads of the merge: 256 hold columns, all of them read columns again
constexpr int kBeamAgain = 2;        // vectors each requests at once
constexpr int kBeamHits = 256;       // columns read again
// Vectors from which on a column is read again by its hint, which costs a
// round trip: at 63 vectors a column 22.1 us with and 23.7 without (32 x 8 x
// 128256 bf16), at 32 12.5 with and 12.1 without (4 x 4 x 128256 bf16).
constexpr int kBeamLong = 40;
constexpr int kBeamKeep = 512;       // candidates ranked at once
constexpr int kBeamRound = 256;      // vectors the slow path takes at once
constexpr int kBeamCut = 704;        // keys its cuts leave at most: of kBeamSlow, 11 from each of 64 threads
constexpr int kBeamSlow = kBeamRound * 8 + kBeamCut;
static_assert((kBeamSlow + kBlock - 1) / kBlock * SV_MAX_CANDIDATES <= kBeamCut, "a cut leaves M threads' keys");
constexpr int kBeamRowKeep = 192;    // keys a row's last cut leaves: of kBeamCut, 3 from each of 64 threads
static_assert((kBeamCut + kBlock - 1) / kBlock * SV_MAX_CANDIDATES <= kBeamRowKeep &&
                  kBeamRowKeep + SV_MAX_CANDIDATES <= kBeamKeep, "a row's keys and the best so far");

struct BeamPart {
    float m;     // chunk maximum
    int32_t pad;
    double s;    // sum of exp2(z c - offset(m)) over the chunk; NaN for NaN or +inf logits
};

// Of a column: the vector at which its maximum's tile starts for the lane that
// had it (kBeamLoads vectors, kBlock apart), and the maximum of its other tiles.
struct BeamHint {
    float other;
    int32_t q;
};

struct BeamArgs {
    const char *logits;
    const float *scores, *temperature;
    const int32_t *finished;
    int64_t seq_bytes, beam_bytes;
    int32_t B, W, V, M, eos, nvec, nc, cvec, cols_log, aligned;
    int32_t per, g_log;  // the merge: columns per thread, 1 << g_log >= nc lanes per row
    int32_t nv, hinted;  // vectors per column; whether they are enough for hints
    BeamPart *part;     // [B][W][nc]
    float *cols;        // [B][W][nc][1 << cols_log] column maxima
    BeamHint *hints;    // the same
    float *out_score;
    int32_t *out_parent, *out_token, *out_finished, *error_word;
};

struct BeamPlan {
    int32_t nvec, nc, cvec, cols_log, per, g_log;
    size_t off_cols, off_hints, bytes;
};

static bool make_beam_plan(int32_t B, int32_t W, int32_t V, int32_t dtype, int32_t M, BeamPlan *p)
{
    if (B < 0 || W < 1 || W > SV_MAX_BEAMS || V < 1 || M < 1 || M > SV_MAX_CANDIDATES ||
        (dtype != SV_F32 && dtype != SV_BF16) || (int64_t)W * V >= ((int64_t)1 << 31))
        return false;
    const int vec = dtype == SV_F32 ? 4 : 8;
    p->nvec = (int32_t)(((int64_t)V + vec - 1) / vec);
    const int64_t rows = (int64_t)std::max(B, 1) * W;
    int64_t nc = (kBeamFill + rows - 1) / rows;
    nc = std::min<int64_t>(nc, std::max(1, p->nvec / kBlock));
    nc = std::min<int64_t>(nc, std::min(kBeamMaxChunks, std::max(1, kBeamRowChunks / W)));
    p->cvec = (int32_t)((p->nvec + nc - 1) / nc);
    p->nc = (p->nvec + p->cvec - 1) / p->cvec;
    p->cols_log = 8;  // W * nc <= 256, so at least 8 columns
    while (((int64_t)W * p->nc) << p->cols_log > kBeamPre * kBlock) --p->cols_log;
    if ((rows * p->nc) << p->cols_log >= ((int64_t)1 << 31)) return false;
    p->per = 1;
    while (p->per * kBlock < (W * p->nc) << p->cols_log) p->per <<= 1;
    p->g_log = 0;
    while (1 << p->g_log < p->nc) ++p->g_log;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    p->off_cols = align(sizeof(BeamPart) * (size_t)(rows * p->nc));
    p->off_hints = align(p->off_cols + sizeof(float) * (size_t)((rows * p->nc) << p->cols_log));
    p->bytes = align(p->off_hints + sizeof(BeamHint) * (size_t)((rows * p->nc) << p->cols_log));
    return true;
}

// ---------------------------------------------------------------------------
// Exponentials relative to a row's offset, in base 2 with c = fp32(log2 e /
// T).  For |m c| < 2^30 the offset is fp32(m c) and one fma forms x c -
// offset; the fp32 number is used as it is everywhere, so its own rounding
// costs nothing.  Beyond (a row whose logits are all a huge negative mask)
// that rounding would exceed the exponent's range, and (x - m) c is taken
// instead, which makes the offset m c exactly.

__device__ __forceinline__ bool beam_wide(float m, const ExpScale &e)
{
    return !(fabsf(m * e.c) < 0x1p30f);
}

__device__ __forceinline__ double beam_offset(float m, const ExpScale &e)
{
    return beam_wide(m, e) ? (double)m * e.c64 : (double)(m * e.c);
}

// A sum taken against the offset of m, against that of M >= m.
__device__ __forceinline__ double beam_rebase(double s, float m, float M, const ExpScale &e)
{
    return m == -INFINITY ? s : s * exp2(beam_offset(m, e) - beam_offset(M, e));
}

struct BeamRun {
    float m;      // wave-uniform running maximum
    float o;      // its offset where !wide
    bool wide;
    double s;     // this lane's sum
};

template <int DT>
__device__ __forceinline__ float vec_sum_exp_wide(uint4 r, float m, const ExpScale &e)
{
    constexpr int VEC = Elt<DT>::kVec;
    float x[VEC], sum = 0.f;
    Elt<DT>::unpack(r, x);
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum += __builtin_amdgcn_exp2f((x[k] - m) * e.c);
    return sum;
}

// A tile's exponentials; returns the lane's maximum of the tile.  A lane
// maximum ignores NaN, so a NaN shows in the sum alone, also before any
// finite logit.
template <int DT, int U>
__device__ __forceinline__ float beam_tile(const uint4 (&r)[U], const ExpScale &e, BeamRun &run)
{
    constexpr int VEC = Elt<DT>::kVec;
    const float lm = tile_lane_max<DT, U>(r);
    if (__ballot(lm > run.m) != 0ull) {
        const float mw = wave_max(lm);
        if (run.s != 0.0) run.s *= exp2(beam_offset(run.m, e) - beam_offset(mw, e));
        run.m = mw;
        run.o = mw * e.c;
        run.wide = beam_wide(mw, e);
    }
    if (run.m == -INFINITY) {
        bool bad = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[VEC];
            Elt<DT>::unpack(r[u], x);
#pragma unroll
            for (int k = 0; k < VEC; ++k) bad |= x[k] != x[k];
        }
        if (bad) run.s = NAN;
    } else if (!run.wide) {
#pragma unroll
        for (int u = 0; u < U; ++u) run.s += (double)vec_sum_exp<DT>(r[u], run.o, e);
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) run.s += (double)vec_sum_exp_wide<DT>(r[u], run.m, e);
    }
    return lm;
}

struct BeamColumn {
    float best, other;
    int q;
    __device__ __forceinline__ void join(float b, float o, int at)
    {
        other = fmaxf(fmaxf(other, o), fminf(best, b));
        q = b > best ? at : q;
        best = fmaxf(best, b);
    }
    template <int MASK>
    __device__ __forceinline__ void join_lane()
    {
        join(lane_xor<MASK>(best), lane_xor<MASK>(other), lane_xor<MASK>(q));
    }
};

__device__ __forceinline__ const char *beam_row(const BeamArgs &a, int b, int w)
{
    return a.logits + b * a.seq_bytes + w * a.beam_bytes;
}

__device__ __forceinline__ bool beam_temperature_ok(float T) { return T > 0.f && T < INFINITY; }

// Rows are read for beams in the running: a finite score, not finished.
__device__ __forceinline__ bool beam_live(const BeamArgs &a, int slot)
{
    const float s = a.scores[slot];
    return s > -INFINITY && s < INFINITY && !(a.finished && a.finished[slot]);
}

// The first tile is requested before the beam's score and temperature are
// known, so the stream starts a round trip earlier; a dead beam wastes it.
// Bound by reading: 27 us for 156 MB of bf16 (64 x 8 x 152064, 5.8 TB/s), 41 us
// for 263 MB of fp32 (128 x 4 x 128256, 6.4 TB/s), 3 to 4 us for one request.
// Lists kept while streaming (an earlier form) took 47 us for the former.
template <int DT, bool ALIGNED>
__global__ __launch_bounds__(kBlock) void beam_rows_kernel(const BeamArgs a)
{
    constexpr int U = kBeamLoads;
    __shared__ float lds_best[kBlock], lds_other[kBlock], lds_m[kWaves];
    __shared__ int lds_q[kBlock];
    __shared__ double lds_s[kWaves];
    const int slot = blockIdx.x / a.nc, chunk = blockIdx.x % a.nc;
    const int b = slot / a.W, w = slot % a.W, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const char *row = beam_row(a, b, w);
    const int q0 = chunk * a.cvec, q1 = min(a.nvec, q0 + a.cvec);
    PairTileU<U> ra;
    issue_pair<DT, ALIGNED, false>(row, nullptr, q0, q1, a.V, ra);
    const float T = a.temperature ? a.temperature[b] : 1.f;
    if (!beam_temperature_ok(T) || !beam_live(a, slot)) return;
    const ExpScale e = make_scale(T);
    BeamRun run = {-INFINITY, -INFINITY, false, 0.0};
    BeamColumn col = {-INFINITY, -INFINITY, q0};
    stream_pair<DT, ALIGNED, false>(row, nullptr, q0, q1, a.V, ra, [&](const PairTileU<U> &r, int qb) {
        col.join(beam_tile<DT, U>(r.t, e, run), -INFINITY, qb);
    });
    col.q += tid;
    const double s = wave_sum(run.s);  // against the wave's maximum
    // column l of C: threads l, l + C, ...
    const int C = 1 << a.cols_log;
    if (a.hinted) {
        if (C < 64) col.join_lane<32>();
        if (C < 32) col.join_lane<16>();
        if (C < 16) col.join_lane<8>();
        lds_other[tid] = col.other;
        lds_q[tid] = col.q;
    } else {
        if (C < 64) col.best = fmaxf(col.best, lane_xor<32>(col.best));
        if (C < 32) col.best = fmaxf(col.best, lane_xor<16>(col.best));
        if (C < 16) col.best = fmaxf(col.best, lane_xor<8>(col.best));
    }
    lds_best[tid] = col.best;
    if (lane == 0) {
        lds_m[wave] = run.m;
        lds_s[wave] = s;
    }
    __syncthreads();
    const size_t at = (size_t)slot * a.nc + chunk;
    if (tid < C) {
        for (int i = tid + max(C, 64); i < kBlock; i += max(C, 64)) {
            if (a.hinted) col.join(lds_best[i], lds_other[i], lds_q[i]);
            else col.best = fmaxf(col.best, lds_best[i]);
        }
        a.cols[(at << a.cols_log) + tid] = col.best;
        if (a.hinted) a.hints[(at << a.cols_log) + tid] = {col.other, col.q};
    }
    if (wave != 0) return;
    const float top = fmaxf(fmaxf(lds_m[0], lds_m[1]), fmaxf(lds_m[2], lds_m[3]));
    double sum = 0.0;
    if (lane < kWaves) sum = beam_rebase(lds_s[lane], lds_m[lane], top, e);
    sum += dpp_double<kDppQuadXor1>(sum);
    sum += dpp_double<kDppQuadXor2>(sum);
    if (lane == 0) a.part[at] = {top, 0, sum};
}

// ---------------------------------------------------------------------------
// The merge.

// Doubles in order as whole numbers, none of them 0.
__device__ __forceinline__ uint64_t double_order(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | (1ull << 63));
}

__device__ __forceinline__ double order_double(uint64_t o)
{
    return __longlong_as_double((long long)((o >> 63) ? (o & ~(1ull << 63)) : ~o));
}

// A candidate: c's order (0 = none), its row key (logit, then lower token) and beam.
struct BeamCand {
    uint64_t c, key;
    int w;
};

__device__ __forceinline__ bool ahead(const BeamCand &x, const BeamCand &y)
{
    return x.c > y.c || (x.c == y.c && (x.w < y.w || (x.w == y.w && x.key > y.key)));
}

struct __align__(16) BeamRow {
    double base;  // s_w - ln sum_u exp((z(u) - m) / T)
    float m;
    int state;    // 0: no candidate, 1: its row's, 2: finished
};

// c of logit x of a row in the running.
__device__ __forceinline__ double beam_c(const BeamRow &r, float x, double inv_t)
{
    return r.base + ((double)x - (double)r.m) * inv_t;
}

// c rounded to fp32 for floors, where order may be lost but not reversed, and
// held above -inf, which stands for no candidate.
__device__ __forceinline__ float beam_rough(double c) { return fmaxf((float)c, -FLT_MAX); }

// Sum and maximum over aligned groups of G lanes (a power of two up to 64).
template <class T, class Op>
__device__ __forceinline__ T group_reduce(T v, int G, Op op)
{
    if (G > 1) v = op(v, lane_xor<1>(v));
    if (G > 2) v = op(v, lane_xor<2>(v));
    if (G > 4) v = op(v, lane_xor<4>(v));
    if (G > 8) v = op(v, lane_xor<8>(v));
    if (G > 16) v = op(v, lane_xor<16>(v));
    if (G > 32) v = op(v, lane_xor<32>(v));
    return v;
}

// Vector q of a row with elements at or beyond V as -inf (for the slow path).
template <int DT>
__device__ __forceinline__ uint4 beam_vector(const BeamArgs &a, const char *row, int q)
{
    constexpr int VEC = Elt<DT>::kVec;
    const char *p = row + (size_t)q * 16;
    const int valid = min(VEC, a.V - q * VEC);
    uint4 r;
    if (a.aligned) r = *reinterpret_cast<const uint4 *>(p);
    else r = load16_unaligned(p, ((uint32_t)((uintptr_t)p & 15)) + (uint32_t)valid * Elt<DT>::kBytes > 16u);
    if (valid < VEC) mask_raw<DT>(r, valid);
    return r;
}

// ---------------------------------------------------------------------------
// When more candidates reach the floor than are ranked at once (many equal
// ones, or the best all in neighbouring columns), row by row: vectors in index
// order, kBeamRound at a time, those keys collected that beat a floor under the
// row's M-th best so far.  A row ends early when that floor's logit is the
// row's maximum: whatever follows has a larger index.  (64 x 8 x 152064 bf16:
// all logits equal 0.1 ms, a cut at many equal ones below the best 0.7 ms.)

// Raises the floor: the M-th largest of 256 threads' largest keys, which
// leaves the keys of M threads in buf[0, n); returns how many.
__device__ __forceinline__ int beam_cut(uint64_t *buf, int n, int M, uint64_t &floor, int *cnt, uint64_t *lds_k)
{
    constexpr int kOwn = (kBeamSlow + kBlock - 1) / kBlock;
    uint64_t own[kOwn], best = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int i = threadIdx.x + j * kBlock;
        own[j] = (int)threadIdx.x < kBlock && i < n ? buf[i] : 0;
        best = larger(best, own[j]);
    }
    if (threadIdx.x == 0) *cnt = 0;
    floor = larger(floor, block_kth(best, M, lds_k));
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (own[j] && own[j] >= floor) buf[atomicAdd(cnt, 1)] = own[j];
    __syncthreads();
    n = *cnt;
    __syncthreads();
    return n;
}

template <int DT>
__device__ __forceinline__ int beam_row_slow(const BeamArgs &a, const BeamRow &r, const char *row, float floor_c,
                                          double inv_t, uint64_t *buf, int *cnt, uint64_t *lds_k)
{
    constexpr int VEC = Elt<DT>::kVec;
    uint64_t floor = 0;
    if (threadIdx.x == 0) *cnt = 0;
    __syncthreads();
    int n = 0;
    for (int qb = 0; qb < a.nvec; qb += kBeamRound) {
        const int q = qb + (int)threadIdx.x;
        if ((int)threadIdx.x < kBeamRound && q < a.nvec) {
            float x[VEC];
            Elt<DT>::unpack(beam_vector<DT>(a, row, q), x);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                if (!(x[k] > -INFINITY) || beam_rough(beam_c(r, x[k], inv_t)) < floor_c) continue;
                const uint64_t key = top_key(x[k], q * VEC + k);
                if (key > floor) buf[atomicAdd(cnt, 1)] = key;
            }
        }
        __syncthreads();
        n = *cnt;
        __syncthreads();
        if (n > kBeamCut) {
            n = beam_cut(buf, n, a.M, floor, cnt, lds_k);
            if (key_value(floor) == r.m) break;
        }
    }
    while (n > kBeamRowKeep) n = beam_cut(buf, n, a.M, floor, cnt, lds_k);
    return n;
}

// The best M into cand[0, n) in order; returns n.
template <int DT>
__device__ __forceinline__ int beam_slow(const BeamArgs &a, const BeamRow *rows, int b, float floor_c, double inv_t,
                                      BeamCand *cand, uint64_t *buf, int *cnt, uint64_t *lds_k)
{
    int n = 0;
    for (int w = 0; w < a.W; ++w) {
        const BeamRow r = rows[w];
        // base is c of the row's best; a later beam loses a tie
        if (r.state == 0 || beam_rough(r.base) < floor_c || (n == a.M && double_order(r.base) <= cand[n - 1].c))
            continue;
        int k = 1;
        if (r.state == 1) k = beam_row_slow<DT>(a, r, beam_row(a, b, w), floor_c, inv_t, buf, cnt, lds_k);
        __syncthreads();
        for (int i = threadIdx.x; i < k; i += kMerge) {
            const uint64_t key = r.state == 2 ? top_key(0.f, a.eos) : buf[i];
            const double c = r.state == 2 ? r.base : beam_c(r, key_value(key), inv_t);
            cand[n + i] = {double_order(c), key, w};
        }
        __syncthreads();
        BeamCand own = {0, 0, 0};
        int rank = a.M;
        if ((int)threadIdx.x < n + k) {
            own = cand[threadIdx.x];
            rank = 0;
            for (int j = 0; j < n + k; ++j) rank += ahead(cand[j], own);
        }
        __syncthreads();
        if (rank < a.M) cand[rank] = own;
        n = min(n + k, a.M);
        __syncthreads();
    }
    return n;
}

// A 16-byte vector requested now and put together later: of an unaligned
// address the two aligned blocks that hold its `valid` elements (the first
// one twice where it holds them all).
template <int DT, bool ALIGNED>
struct BeamLoad {
    u32x4 x, y;
    uint32_t sh;
    __device__ __forceinline__ void issue(const char *p, int valid)
    {
        sh = ALIGNED ? 0u : (uint32_t)((uintptr_t)p & 15);
        const u32x4 *blk = reinterpret_cast<const u32x4 *>(p - sh);
        x = blk[0];
        if (!ALIGNED) y = blk[sh + (uint32_t)valid * Elt<DT>::kBytes > 16u ? 1 : 0];
    }
    __device__ __forceinline__ uint4 vector() const
    {
        if (ALIGNED) return make_uint4(x.x, x.y, x.z, x.w);
        // words sh / 4 + 0..4 of the eight
        const bool one = sh & 4u, two = sh & 8u;
        const uint32_t a0 = one ? x.y : x.x, a1 = one ? x.z : x.y, a2 = one ? x.w : x.z, a3 = one ? y.x : x.w;
        const uint32_t a4 = one ? y.y : y.x, a5 = one ? y.z : y.y, a6 = one ? y.w : y.z;
        const uint32_t f0 = two ? a2 : a0, f1 = two ? a3 : a1, f2 = two ? a4 : a2, f3 = two ? a5 : a3;
        const uint32_t f4 = two ? a6 : a4, r = sh & 3u;
        return make_uint4(funnel_bytes(f0, f1, r), funnel_bytes(f1, f2, r), funnel_bytes(f2, f3, r),
                          funnel_bytes(f3, f4, r));
    }
};

// The merge is a chain of memory round trips (inputs, columns read again) and
// barriers, 7 to 10 us, hardly depending on the sizes: 1.3 us until the inputs
// are there, 1.3 the normalisers in fp64, 0.9 the floor's sorts, 0.8 the
// columns that reach it, 1.2 to 1.8 reading them again, 0.6 the ranks.  Its
// code is kept short, each step once, since a step runs once per call and
// fetching its instructions counts (checks unrolled over 64 elements took 4
// us more).
static_assert(2 * kBeamRowChunks <= kMerge, "a thread for each chunk of a sequence, a power of two a row");

template <int DT, bool ALIGNED, bool HINTS>
__global__ __launch_bounds__(kMerge) void beam_merge_kernel(const BeamArgs a)
{
    __shared__ BeamRow rows[SV_MAX_BEAMS];
    __shared__ float low[SV_MAX_BEAMS];  // no smaller logit of the row reaches the floor
    __shared__ __align__(16) char lds[kBeamSlow * 8];
    __shared__ BeamCand cand[kBeamKeep];
    __shared__ int hits[kBeamHits], near[kBeamHits];
    __shared__ uint64_t lds_k[kBlock + 1];
    __shared__ int n_hits, n_cand, any_far, errors;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n_cols = (a.W * a.nc) << a.cols_log;
    // everything the normalisers and the floor need is requested at once: a
    // barrier waits for the loads before it
    const float *cols = a.cols + (size_t)b * n_cols;
    // (this thread's columns follow each other, so they are one row's)
    const int per = a.per;
    const int col0 = min(tid * per, n_cols - per);
    const bool mine = tid < kBlock && tid * per < n_cols;
    float x[kBeamPre];
#pragma unroll
    for (int j = 0; j < kBeamPre; ++j) x[j] = cols[col0 + min(j, per - 1)];
    // G lanes to a row, one per chunk; W G <= 2 W nc, so each thread has one
    const int G = 1 << a.g_log;
    const int w = min(tid >> a.g_log, a.W - 1), chunk = tid & (G - 1), slot = b * a.W + w;
    const float s = a.scores[slot];
    BeamPart p = a.part[(size_t)slot * a.nc + min(chunk, a.nc - 1)];
    const bool ended = a.finished && a.finished[slot];
    const float T = a.temperature ? a.temperature[b] : 1.f;
    if (tid == 0) n_hits = n_cand = any_far = errors = 0;
    __syncthreads();
    const bool good_t = beam_temperature_ok(T);
    const ExpScale e = make_scale(good_t ? T : 1.f);
    if (!good_t && tid == 0) errors = SV_ERR_TEMPERATURE;
    if (chunk >= a.nc) p = {-INFINITY, 0, 0.0};
    const float m = group_reduce(p.m, G, [](float u, float v) { return fmaxf(u, v); });
    const double sum = group_reduce(beam_rebase(p.s, p.m, m, e), G, [](double u, double v) { return u + v; });
    if (chunk == 0 && tid < a.W * G) {
        int state = 0, bad = 0;
        double base = (double)s;
        if (!(s < INFINITY)) {
            bad = SV_ERR_SCORE;
        } else if (s > -INFINITY && ended) {
            state = 2;
        } else if (s > -INFINITY) {
            if (!(sum < INFINITY)) {  // NaN
                bad = SV_ERR_ROW;
            } else if (m > -INFINITY) {
                state = 1;
                // ln 2 (log2 sum + offset - m c): the offset's rounding comes off again
                base -= (log2(sum) + (beam_offset(m, e) - (double)m * e.c64)) * kLn2;
            }
        }
        if (bad && good_t) atomicOr(&errors, bad);
        rows[w] = {base, m, state};
    }
    __syncthreads();
    float *out_score = a.out_score + (size_t)b * a.M;
    int32_t *out_parent = a.out_parent + (size_t)b * a.M, *out_token = a.out_token + (size_t)b * a.M;
    int32_t *out_finished = a.out_finished ? a.out_finished + (size_t)b * a.M : nullptr;
    int found = 0;
    auto put = [&](int r, const BeamCand &c) {
        const int token = key_index(c.key);
        out_score[r] = (float)order_double(c.c);
        out_parent[r] = c.w;
        out_token[r] = token;
        if (out_finished) out_finished[r] = (rows[c.w].state == 2 || token == a.eos) ? 1 : 0;
    };
    if (errors) {
        if (tid == 0 && a.error_word) atomicOr(a.error_word, errors);
    } else {
        const double inv_t = 1.0 / (double)T;
        // the columns' best candidates, roughly; i / nc for i < 256, nc <= 64 by a product
        const uint32_t inv_nc = 65536u / (uint32_t)a.nc + 1u;
        auto row_of = [&](int chunk) { return (int)((uint32_t)chunk * inv_nc >> 16); };
        const int own = row_of(col0 >> a.cols_log);
        const BeamRow r = rows[own];
        const bool alone = r.state == 2 && col0 == (own * a.nc) << a.cols_log;
        float best = -INFINITY;
        if (mine && r.state == 1) {
            float top = x[0];
#pragma unroll
            for (int j = 1; j < kBeamPre; ++j) top = fmaxf(top, x[j]);
            if (top > -INFINITY) best = beam_rough(beam_c(r, top, inv_t));
        } else if (mine && alone) {
            best = beam_rough(r.base);
        }
        float *lds_f = reinterpret_cast<float *>(lds_k);
        const float tau = fmaxf(block_kth(best, a.M, lds_f), -FLT_MAX);
        // the floor as a logit of a row, held low enough for every rounding on
        // the way: that of the floor itself (half a step of |tau|, in units of T
        // as a logit), and those of m, the difference and the result
        auto floor_of = [&](const BeamRow &r) {
            if (tau == -FLT_MAX) return -INFINITY;  // no floor, or one that rounding held up
            const double m = (double)r.m, d = ((double)tau - r.base) * (double)T;
            return (float)(m + d - 0x1p-20 * (fabs(m) + fabs(d) + fabs((double)tau) * (double)T));
        };
        auto keep = [&](double c, uint64_t key, int w) {
            const int at = atomicAdd(&n_cand, 1);
            if (at < kBeamKeep) cand[at] = {double_order(c), key, w};
        };
        constexpr int VEC = Elt<DT>::kVec;
        const int C = 1 << a.cols_log;
        if (best >= tau) {
            const float least = floor_of(r);
            if (alone) keep(r.base, top_key(0.f, a.eos), own);
#pragma unroll
            for (int j = 0; j < kBeamPre; ++j) {
                if (alone || j >= per || !(x[j] >= least && x[j] > -INFINITY)) continue;
                const int at = atomicAdd(&n_hits, 1);
                if (at < kBeamHits) hits[at] = col0 + j;
            }
        }
        if (tid < a.W) low[tid] = floor_of(rows[tid]);
        __syncthreads();
        const int nh = min(n_hits, kBeamHits);
        // a long column is read again only at its maximum's tile when its other
        // tiles stay below the floor, which almost all do
        if (HINTS) {
            if (tid < nh) {
                const BeamHint h = a.hints[(size_t)b * n_cols + hits[tid]];
                near[tid] = h.other < low[row_of(hits[tid] >> a.cols_log)] ? h.q : -1;
                if (near[tid] < 0) any_far = 1;
            }
            __syncthreads();
        }
        for (int far = HINTS ? 0 : 1; far < (HINTS && !any_far ? 1 : 2); ++far) {
            const int each = far ? a.nv : kBeamLoads;
            for (int i0 = tid; i0 < nh * each; i0 += kBeamAgain * kMerge) {
                // every load of a batch is unconditional (the maxima stand in
                // where there is no vector), so that all are in flight at once
                BeamLoad<DT, ALIGNED> in[kBeamAgain];
                int q[kBeamAgain], w[kBeamAgain];
#pragma unroll
                for (int j = 0; j < kBeamAgain; ++j) {
                    const int i = i0 + j * kMerge, h = min(i / each, nh - 1), v = i - h * each;
                    const int col = hits[h], chunk = col >> a.cols_log, from = HINTS ? near[h] : -1;
                    w[j] = row_of(chunk);
                    const int q0 = (chunk - w[j] * a.nc) * a.cvec;
                    q[j] = far ? q0 + (col & (C - 1)) + (v << a.cols_log) : from + v * kBlock;
                    if (i >= nh * each || (from < 0) == !far || q[j] >= min(a.nvec, q0 + a.cvec)) q[j] = -1;
                    const bool some = q[j] >= 0;
                    in[j].issue(some ? beam_row(a, b, w[j]) + (size_t)q[j] * 16 : reinterpret_cast<const char *>(cols),
                                some ? min(VEC, a.V - q[j] * VEC) : 1);
                }
#pragma unroll
                for (int j = 0; j < kBeamAgain; ++j) {
                    if (q[j] < 0) continue;
                    const uint4 vec = in[j].vector();
                    float z[VEC];
                    Elt<DT>::unpack(vec, z);
                    const float least = low[w[j]];
                    uint32_t at = 0;  // elements that may reach the floor
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        at |= (z[e] >= least && z[e] != -INFINITY && q[j] * VEC + e < a.V) ? 1u << e : 0u;
                    // (no more once there are too many)
                    if (at && *const_cast<volatile int *>(&n_cand) > kBeamKeep) at = 0;
                    for (; at; at &= at - 1) {
                        const int e = __ffs(at) - 1;
                        const float ze = elt_of<DT>(vec, e);
                        const double c = beam_c(rows[w[j]], ze, inv_t);
                        if (beam_rough(c) >= tau) keep(c, top_key(ze, q[j] * VEC + e), w[j]);
                    }
                }
            }
        }
        __syncthreads();
        const int k = n_cand;
        const bool whole = n_hits <= kBeamHits && k <= kBeamKeep;
        __syncthreads();  // the slow path counts with n_cand too
        if (whole) {
            // distinct candidates: a place is the number of better ones
            // (eight lanes to a candidate)
            for (int i0 = 0; i0 < k; i0 += kMerge / 8) {
                const int i = i0 + tid / 8;
                const BeamCand c = cand[min(i, k - 1)];
                int rank = 0;
                for (int j = tid % 8; j < k; j += 8) rank += ahead(cand[j], c);
                rank += lane_xor<1>(rank);
                rank += lane_xor<2>(rank);
                rank += lane_xor<4>(rank);
                if (tid % 8 == 0 && i < k && rank < a.M) put(rank, c);
            }
            found = min(k, a.M);
        } else {
            // the candidates found so far may give a higher floor
            float mine = -INFINITY;
            if (tid < kBlock)
                for (int i = tid; i < min(k, kBeamKeep); i += kBlock)
                    mine = fmaxf(mine, beam_rough(order_double(cand[i].c)));
            const float floor_c = fmaxf(tau, block_kth(mine, a.M, lds_f));
            found = beam_slow<DT>(a, rows, b, floor_c, inv_t, cand, reinterpret_cast<uint64_t *>(lds), &n_cand, lds_k);
            for (int i = tid; i < found; i += kMerge) put(i, cand[i]);
        }
    }
    for (int r = found + tid; r < a.M; r += kMerge) {
        out_score[r] = -INFINITY;
        out_parent[r] = -1;
        out_token[r] = -1;
        if (out_finished) out_finished[r] = 0;
    }
}

template <int DT>
static void launch_beam(const BeamArgs &a, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)a.B * a.W * a.nc);
    if (a.aligned) {
        beam_rows_kernel<DT, true><<<grid, kBlock, 0, s>>>(a);
        if (a.hinted) beam_merge_kernel<DT, true, true><<<(unsigned)a.B, kMerge, 0, s>>>(a);
        else beam_merge_kernel<DT, true, false><<<(unsigned)a.B, kMerge, 0, s>>>(a);
    } else {
        beam_rows_kernel<DT, false><<<grid, kBlock, 0, s>>>(a);
        if (a.hinted) beam_merge_kernel<DT, false, true><<<(unsigned)a.B, kMerge, 0, s>>>(a);
        else beam_merge_kernel<DT, false, false><<<(unsigned)a.B, kMerge, 0, s>>>(a);
    }
}

}  // namespace sv

extern "C" {

size_t spec_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t dtype, int32_t M)
{
    sv::BeamPlan p;
    return sv::make_beam_plan(B, W, V, dtype, M, &p) ? p.bytes : 0;
}

int32_t spec_beam_select(const void *logits, int32_t B, int32_t W, int32_t V, int32_t dtype, int64_t seq_stride,
                         int64_t beam_stride, const float *scores, const float *temperature,
                         const int32_t *finished, int32_t eos, int32_t M, float *out_score, int32_t *out_parent,
                         int32_t *out_token, int32_t *out_finished, int32_t *error_word, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    sv::BeamPlan p;
    if (!sv::make_beam_plan(B, W, V, dtype, M, &p)) return SV_EINVAL;
    if (seq_stride < 0 || beam_stride < 0 || eos < -1 || eos >= V || (finished && eos < 0)) return SV_EINVAL;
    if (B == 0) return SV_OK;
    if (!logits || !scores || !out_score || !out_parent || !out_token) return SV_EINVAL;
    const int64_t elt = dtype == SV_F32 ? 4 : 2;
    if ((uintptr_t)logits % (uintptr_t)elt || (int64_t)B * seq_stride + (int64_t)W * beam_stride > ((int64_t)1 << 40))
        return SV_EINVAL;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < p.bytes) return SV_EWORKSPACE;
    sv::BeamArgs a = {};
    a.logits = static_cast<const char *>(logits);
    a.scores = scores;
    a.temperature = temperature;
    a.finished = finished;
    a.seq_bytes = seq_stride * elt;
    a.beam_bytes = beam_stride * elt;
    a.B = B;
    a.W = W;
    a.V = V;
    a.M = M;
    a.eos = eos;
    a.nvec = p.nvec;
    a.nc = p.nc;
    a.cvec = p.cvec;
    a.cols_log = p.cols_log;
    a.per = p.per;
    a.nv = (p.cvec + (1 << p.cols_log) - 1) >> p.cols_log;
    a.hinted = a.nv >= sv::kBeamLong;
    a.g_log = p.g_log;
    a.part = static_cast<sv::BeamPart *>(workspace);
    a.cols = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.off_cols);
    a.hints = reinterpret_cast<sv::BeamHint *>(static_cast<char *>(workspace) + p.off_hints);
    a.out_score = out_score;
    a.out_parent = out_parent;
    a.out_token = out_token;
    a.out_finished = out_finished;
    a.error_word = error_word;
    a.aligned = ((uintptr_t)logits | (uintptr_t)a.seq_bytes | (uintptr_t)a.beam_bytes) % 16 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SV_F32) sv::launch_beam<0>(a, s);
    else sv::launch_beam<1>(a, s);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
