// sv_beam.hip -- beam search's selection over beams and vocabulary.
//
//   c(w, v) = s_w + z_w(v) / T - ln sum_u exp(z_w(u) / T)
//
// Within a beam c rises with z, so a beam's best M candidates are its M
// largest logits, and the best M of a sequence are among the W beams' lists:
//   1. beam_rows_kernel   one workgroup per (row, chunk): one pass over the
//                         logits for the running maximum and the sum of
//                         exponentials, and the chunk's M largest logits.
//   2. beam_merge_kernel  one workgroup per sequence: the rows' normalisers,
//                         c in fp64 for W * chunks * M candidates, the best M.
//
// The pass is bound by reading the logits, and on bf16 nearly by its
// exponentials (eight per 16 bytes), so it may not spend VALU on keeping
// lists.  While it streams it keeps only maxima: of each lane over the chunk
// and of each lane over groups of tiles (LDS, at most kGroups a lane).  The
// M-th largest of the 256 lanes' maxima is a floor under the chunk's M-th
// largest logit, since M lanes hold one at least as large each.  Few logits
// reach it (M ln-like: the best k fall on 256 lanes at random, so ~M (1 +
// M/512)), and they lie in the groups whose maximum does, which their lanes
// read again; the survivors are ranked by counting.
#include <algorithm>
#include <climits>

#include "specdecode.h"
#include "sv_internal.h"
#include "sv_sort.h"
#include "sv_stream.h"
#include "sv_tile.h"

namespace sv {

constexpr int kBeamLoads = 4;        // 16-byte vectors per thread per tile
constexpr int kBeamGroups = 16;      // groups of tiles per lane with a maximum of their own
constexpr int kBeamFill = 768;       // workgroups the streaming grid aims for
constexpr int kBeamMaxChunks = 64;   // chunks per row: one per lane when the merge reads them
constexpr int kBeamLists = 8192;     // W * chunks * M at most: the merge's candidates per sequence
constexpr int kBeamKeep = 512;       // survivors ranked at once
constexpr int kBeamRound = kBlock * 8;  // most survivors of one vector per thread
constexpr int kBeamSlow = kBeamRound + SV_MAX_CANDIDATES;

struct BeamPart {
    float m;     // chunk maximum
    int32_t pad;
    double s;    // sum of exp2(z c - offset(m)) over the chunk; NaN for NaN or +inf logits
};

struct BeamArgs {
    const char *logits;
    const float *scores, *temperature;
    const int32_t *finished;
    int64_t seq_bytes, beam_bytes;
    int32_t B, W, V, M, eos, nvec, nc, cvec, gt;  // gt: tiles per group
    BeamPart *part;     // [B][W][nc]
    uint64_t *keys;     // [B][W][nc][M] descending, 0 = none
    float *out_score;
    int32_t *out_parent, *out_token, *out_finished, *error_word;
};

struct BeamPlan {
    int32_t nvec, nc, cvec, gt;
    size_t off_keys, bytes;
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
    nc = std::min<int64_t>(nc, std::min(kBeamMaxChunks, std::max(1, kBeamLists / (W * M))));
    p->cvec = (int32_t)((p->nvec + nc - 1) / nc);
    p->nc = (p->nvec + p->cvec - 1) / p->cvec;
    const int32_t tiles = (p->cvec + kBlock * kBeamLoads - 1) / (kBlock * kBeamLoads);
    p->gt = (tiles + kBeamGroups - 1) / kBeamGroups;
    if (rows * p->nc * M >= ((int64_t)1 << 31)) return false;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    p->off_keys = align(sizeof(BeamPart) * (size_t)(rows * p->nc));
    p->bytes = align(p->off_keys + sizeof(uint64_t) * (size_t)(rows * p->nc * M));
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

// ---------------------------------------------------------------------------
// The chunk's M largest logits when more than kBeamKeep reach the floor (many
// equal ones): vectors in index order, one per thread a round, those that
// beat the best M so far collected and cut back to M.  Ends early when the
// M-th best equals the chunk's maximum: whatever follows has a larger index.

// The best M of buf[0, n), n >= M, moved to its front (unordered): the M-th
// largest key by its bits from the top, counting.
__device__ __forceinline__ uint64_t beam_cut(uint64_t *buf, int n, int M, int *cnt, int *ldsi)
{
    uint64_t kth = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const uint64_t c = kth | (1ull << bit);
        int k = 0;
        for (int i = threadIdx.x; i < n; i += kBlock) k += buf[i] >= c;
        k = wave_sum_int(k);
        if ((threadIdx.x & 63) == 0) ldsi[threadIdx.x >> 6] = k;
        __syncthreads();
        k = ldsi[0] + ldsi[1] + ldsi[2] + ldsi[3];
        __syncthreads();
        if (k >= M) kth = c;
    }
    // keys are distinct: M of them are >= kth
    constexpr int kOwn = (kBeamSlow + kBlock - 1) / kBlock;
    uint64_t own[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int i = threadIdx.x + j * kBlock;
        own[j] = i < n ? buf[i] : 0;
    }
    if (threadIdx.x == 0) *cnt = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (own[j] >= kth) buf[atomicAdd(cnt, 1)] = own[j];
    __syncthreads();
    return kth;
}

template <int DT, bool ALIGNED>
__device__ __noinline__ int beam_collect_slow(const char *row, int q0, int q1, int V, float tau, float top, int M,
                                              uint64_t *buf, int *cnt, int *ldsi)
{
    constexpr int VEC = Elt<DT>::kVec;
    uint64_t floor = 0;
    if (threadIdx.x == 0) *cnt = 0;
    __syncthreads();
    int n = 0;
    for (int qb = q0; qb < q1; qb += kBlock) {
        PairTileU<1> r;
        issue_pair<DT, ALIGNED, false>(row, nullptr, qb, q1, V, r);
        fix_pair<DT, false>(qb, q1, V, r);
        float x[VEC];
        Elt<DT>::unpack(r.t[0], x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const uint64_t key = top_key(x[k], elem_index(qb, 0, k, VEC));
            if (x[k] >= tau && x[k] > -INFINITY && key > floor) buf[atomicAdd(cnt, 1)] = key;
        }
        __syncthreads();
        n = *cnt;
        __syncthreads();
        if (n > SV_MAX_CANDIDATES) {
            floor = beam_cut(buf, n, M, cnt, ldsi);
            n = M;
            if (key_value(floor) == top) break;
        }
    }
    return n;
}

template <int DT, bool ALIGNED>
__device__ __forceinline__ void beam_chunk(const BeamArgs &a, const char *row, int slot, int chunk, float T)
{
    constexpr int VEC = Elt<DT>::kVec;
    constexpr int U = kBeamLoads, kStep = kBlock * kBeamLoads;
    __shared__ __align__(16) char lds[kBeamGroups * kBlock * 4 + kBeamKeep * 8];
    static_assert(sizeof(lds) >= kBeamSlow * 8, "the slow path's buffer");
    __shared__ float lds_k[kBlock + 1];
    __shared__ double lds_d[kWaves];
    __shared__ int lds_i[kWaves], cnt;
    float *gm = reinterpret_cast<float *>(lds);
    uint64_t *buf = reinterpret_cast<uint64_t *>(lds + kBeamGroups * kBlock * 4);
    const int tid = threadIdx.x;
    const int q0 = chunk * a.cvec, q1 = min(a.nvec, q0 + a.cvec);
    PairTileU<U> ra;
    issue_pair<DT, ALIGNED, false>(row, nullptr, q0, q1, a.V, ra);
    const ExpScale e = make_scale(T);
    BeamRun run = {-INFINITY, -INFINITY, false, 0.0};
    float best = -INFINITY, gmax = -INFINITY;
    int t = 0, g = 0;
    stream_pair<DT, ALIGNED, false>(row, nullptr, q0, q1, a.V, ra, [&](const PairTileU<U> &r, int) {
        const float lm = beam_tile<DT, U>(r.t, e, run);
        best = fmaxf(best, lm);
        gmax = fmaxf(gmax, lm);
        if (++t == a.gt) {
            gm[g * kBlock + tid] = gmax;
            gmax = -INFINITY;
            t = 0;
            ++g;
        }
    });
    if (t) gm[g++ * kBlock + tid] = gmax;
    // normaliser of the chunk
    const float top = block_max(run.m, lds_k);
    const double sc = run.m == -INFINITY ? run.s : run.s * exp2(beam_offset(run.m, e) - beam_offset(top, e));
    const double sum = block_sum(sc, lds_d);
    if (tid == 0) {
        a.part[(size_t)slot * a.nc + chunk] = {top, 0, sum};
        cnt = 0;
    }
    // candidates
    const float tau = block_kth(best, a.M, lds_k);
    if (best >= tau && best > -INFINITY) {
        for (int h = 0; h < g; ++h) {
            if (!(gm[h * kBlock + tid] >= tau)) continue;
            for (int i = 0; i < a.gt; ++i) {
                const int qb = q0 + (h * a.gt + i) * kStep;
                if (qb >= q1) break;
                PairTileU<U> r;
                issue_pair<DT, ALIGNED, false>(row, nullptr, qb, q1, a.V, r);
                fix_pair<DT, false>(qb, q1, a.V, r);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[VEC];
                    Elt<DT>::unpack(r.t[u], x);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        if (x[k] >= tau && x[k] > -INFINITY) {
                            const int at = atomicAdd(&cnt, 1);
                            if (at < kBeamKeep) buf[at] = top_key(x[k], elem_index(qb, u, k, VEC));
                        }
                }
            }
        }
    }
    __syncthreads();
    int n = cnt;
    if (n > kBeamKeep) {
        __syncthreads();
        buf = reinterpret_cast<uint64_t *>(lds);
        n = beam_collect_slow<DT, ALIGNED>(row, q0, q1, a.V, tau, top, a.M, buf, &cnt, lds_i);
    }
    // distinct keys: a key's place is the number of larger ones
    uint64_t *out = a.keys + ((size_t)slot * a.nc + chunk) * a.M;
    for (int i = tid; i < n; i += kBlock) {
        const uint64_t k = buf[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += buf[j] > k;
        if (rank < a.M) out[rank] = k;
    }
    for (int i = n + tid; i < a.M; i += kBlock) out[i] = 0;
}

__device__ __forceinline__ bool beam_temperature_ok(float T) { return T > 0.f && T < INFINITY; }

// Rows are read for beams in the running: a finite score, not finished.
__device__ __forceinline__ bool beam_live(const BeamArgs &a, int slot)
{
    const float s = a.scores[slot];
    return s > -INFINITY && s < INFINITY && !(a.finished && a.finished[slot]);
}

template <int DT, bool ALIGNED>
__global__ __launch_bounds__(kBlock) void beam_rows_kernel(const BeamArgs a)
{
    const int slot = blockIdx.x / a.nc, chunk = blockIdx.x % a.nc;
    const int b = slot / a.W, w = slot % a.W;
    const float T = a.temperature ? a.temperature[b] : 1.f;
    if (!beam_temperature_ok(T) || !beam_live(a, slot)) return;
    beam_chunk<DT, ALIGNED>(a, a.logits + b * a.seq_bytes + w * a.beam_bytes, slot, chunk, T);
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

struct BeamRows {
    double base[SV_MAX_BEAMS];  // s_w - ln sum_u exp((z(u) - m) / T)
    float m[SV_MAX_BEAMS];
    int state[SV_MAX_BEAMS];    // 0: no candidate, 1: its row's, 2: finished
};

__device__ __forceinline__ BeamCand beam_candidate(const BeamArgs &a, const BeamRows &r, const uint64_t *keys,
                                                   int i, double inv_t)
{
    const int per = a.nc * a.M, w = i / per;
    BeamCand c = {0, 0, w};
    if (r.state[w] == 1) {
        c.key = keys[i];
        if (c.key) c.c = double_order(r.base[w] + ((double)key_value(c.key) - (double)r.m[w]) * inv_t);
    } else if (r.state[w] == 2 && i == w * per) {
        c.key = top_key(0.f, a.eos);
        c.c = double_order(r.base[w]);
    }
    return c;
}

__global__ __launch_bounds__(kBlock) void beam_merge_kernel(const BeamArgs a)
{
    __shared__ BeamRows rows;
    __shared__ BeamCand cand[kBeamKeep];
    __shared__ uint64_t lds_k[kBlock + 1];
    __shared__ int cnt, errors;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) {
        cnt = 0;
        errors = 0;
    }
    __syncthreads();
    const float T = a.temperature ? a.temperature[b] : 1.f;
    const bool good_t = beam_temperature_ok(T);
    if (!good_t && tid == 0) errors = SV_ERR_TEMPERATURE;
    const ExpScale e = make_scale(good_t ? T : 1.f);
    for (int w = wave; w < a.W && good_t; w += kWaves) {
        const int slot = b * a.W + w;
        const float s = a.scores[slot];
        const bool ended = a.finished && a.finished[slot];
        int state = 0;
        double base = (double)s;
        float m = -INFINITY;
        if (!(s < INFINITY)) {
            if (lane == 0) atomicOr(&errors, SV_ERR_SCORE);
        } else if (s > -INFINITY && ended) {
            state = 2;
        } else if (s > -INFINITY) {
            BeamPart p = {-INFINITY, 0, 0.0};
            if (lane < a.nc) p = a.part[(size_t)slot * a.nc + lane];
            m = wave_max(p.m);
            const double off = beam_offset(m, e);
            const double sum = wave_sum(p.m == -INFINITY ? p.s : p.s * exp2(beam_offset(p.m, e) - off));
            if (!(sum < INFINITY)) {  // NaN
                if (lane == 0) atomicOr(&errors, SV_ERR_ROW);
            } else if (m > -INFINITY) {
                state = 1;
                // ln 2 (log2 sum + off - m c): the offset's rounding comes off again
                base -= (log2(sum) + (off - (double)m * e.c64)) / kLog2e;
            }
        }
        if (lane == 0) {
            rows.state[w] = state;
            rows.base[w] = base;
            rows.m[w] = m;
        }
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
        if (out_finished) out_finished[r] = (rows.state[c.w] == 2 || token == a.eos) ? 1 : 0;
    };
    if (errors) {
        if (tid == 0 && a.error_word) atomicOr(a.error_word, errors);
    } else {
        const uint64_t *keys = a.keys + (size_t)b * a.W * a.nc * a.M;
        const int n = a.W * a.nc * a.M;
        const double inv_t = 1.0 / (double)T;
        uint64_t best = 0;
        for (int i = tid; i < n; i += kBlock) best = larger(best, beam_candidate(a, rows, keys, i, inv_t).c);
        const uint64_t tau = larger(block_kth(best, a.M, lds_k), (uint64_t)1);
        if (best >= tau)
            for (int i = tid; i < n; i += kBlock) {
                const BeamCand c = beam_candidate(a, rows, keys, i, inv_t);
                if (c.c < tau) continue;
                const int at = atomicAdd(&cnt, 1);
                if (at < kBeamKeep) cand[at] = c;
            }
        __syncthreads();
        const int k = cnt;
        if (k <= kBeamKeep) {
            for (int i = tid; i < k; i += kBlock) {
                const BeamCand c = cand[i];
                int rank = 0;
                for (int j = 0; j < k; ++j) rank += ahead(cand[j], c);
                if (rank < a.M) put(rank, c);
            }
            found = min(k, a.M);
        } else {
            // more equal ones than fit: the best behind the last, M times
            __syncthreads();
            BeamCand last = {~0ull, ~0ull, -1};
            for (; found < a.M; ++found) {
                BeamCand top = {0, 0, INT_MAX};
                for (int i = tid; i < n; i += kBlock) {
                    const BeamCand c = beam_candidate(a, rows, keys, i, inv_t);
                    if (c.c && ahead(last, c) && ahead(c, top)) top = c;
                }
                cand[tid] = top;
                __syncthreads();
                for (int h = kBlock / 2; h > 0; h >>= 1) {
                    if (tid < h && ahead(cand[tid + h], cand[tid])) cand[tid] = cand[tid + h];
                    __syncthreads();
                }
                last = cand[0];
                __syncthreads();
                if (!last.c) break;
                if (tid == 0) put(found, last);
            }
        }
    }
    for (int r = found + tid; r < a.M; r += kBlock) {
        out_score[r] = -INFINITY;
        out_parent[r] = -1;
        out_token[r] = -1;
        if (out_finished) out_finished[r] = 0;
    }
}

template <int DT>
static void launch_beam(const BeamArgs &a, bool aligned, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)a.B * a.W * a.nc);
    if (aligned) beam_rows_kernel<DT, true><<<grid, kBlock, 0, s>>>(a);
    else beam_rows_kernel<DT, false><<<grid, kBlock, 0, s>>>(a);
    beam_merge_kernel<<<(unsigned)a.B, kBlock, 0, s>>>(a);
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
    a.gt = p.gt;
    a.part = static_cast<sv::BeamPart *>(workspace);
    a.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + p.off_keys);
    a.out_score = out_score;
    a.out_parent = out_parent;
    a.out_token = out_token;
    a.out_finished = out_finished;
    a.error_word = error_word;
    const bool aligned = ((uintptr_t)logits | (uintptr_t)a.seq_bytes | (uintptr_t)a.beam_bytes) % 16 == 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SV_F32) sv::launch_beam<0>(a, aligned, s);
    else sv::launch_beam<1>(a, aligned, s);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
