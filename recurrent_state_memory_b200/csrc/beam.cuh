// beam.cuh -- kernels of the beam selection and of the state reorder.
//
// Selection.  Within a beam the order of the candidates is the order of its logits, so the M best
// of a beam need no sum; across beams the scores score + (logit - lse) are compared in 64 bits.
//
//   1. beam_row_kernel: a block per (beam, piece of the vocabulary) reads its piece once into
//      registers and leaves the piece's maximum, its sum of exp(x - maximum) and its M best
//      (logit, token) pairs.  The M-th largest of the maxima of groups of
//      lanes is reached by at least M elements, and for logits in no particular
//      order by few more, so one sweep over the registers collects them all and a count of the
//      larger ones ranks them.
//   2. beam_group_kernel: a block per group merges its beams' pieces the same way.  Its sums hold
//      fp32 exponentials, so two scores of different beams within TOL of each other may be in the
//      wrong order.  Only candidates down to TOL below the M-th can belong to the M best; where one
//      of the M has one of another beam that near, itself among the M or not, both beams' sums are
//      formed again from the logits in 64 bits and the merge is repeated.  What stays in fp32 lies
//      further than TOL from everything that it could change places with, so the order is the
//      64-bit one.  (The beams that are summed again go one after another through one block: 300 us
//      where all of 32 x 8 x 32000 are, 1.4 ms for 1 x 16 x 262144; 13 and 17 us where none is.)
//
// Bound: the read of the logits (one exponential and about ten instructions each); for one small
// group the latency of the two launches.
#pragma once

#include "common.cuh"

namespace gdr {
namespace bms {

constexpr int NT = 256;
constexpr int WARPS = NT / 32;
constexpr int MOST = 64;                // of K and M
constexpr int LIST = 1024;              // candidates that reach the mark; more (many equal, or a mark of -inf): M rounds of the largest

struct BeamParams {
    int G, K, V, M;
    long long row;
    int eos, pieces, piece;             // pieces of a row, elements of a piece
    const void* logits;
    const float* scores;
    const unsigned char* finished;
    float* out_scores;
    int* out_parent;
    int* out_token;
    float2* sums;                       // [G*K, pieces] maximum, sum of exp(x - maximum)
    float* best;                        // [G*K, pieces, M] logits
    int* token;                         // their tokens, -1: none
};

// Unsigned keys in the order of the values, above zero; NaN (which drops its beam out) like -inf,
// both zeros alike.
__device__ __forceinline__ unsigned key_of(float x) {
    x = x != x ? -INFINITY : x + 0.f;
    const unsigned u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A mark that at least `want` of a block's keys reach, and few more of keys in no particular order:
// the want-th largest of the maxima of groups of lanes.  group_lanes: the largest groups of which
// the `active` first threads make at least 2 * want (so at most 4 * want, unless a group is one
// lane).  0 when there are not that many; it then lets everything through.
constexpr int MARKS = 4 * (MOST + 2);
__device__ __forceinline__ int group_lanes(int active, int want) {
    int l = 32;
    while (l > 1 && active < 2 * want * l) l >>= 1;
    return l;
}
__device__ __forceinline__ void put_marks(unsigned key, int lanes, int active, unsigned* marks) {
    for (int o = 1; o < lanes; o <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
    if ((threadIdx.x & (lanes - 1)) == 0 && (int)threadIdx.x < active) marks[threadIdx.x / lanes] = key;
    if (threadIdx.x < 4) marks[(active + lanes - 1) / lanes + threadIdx.x] = 0;      // to a whole four
}
// Behind a barrier; *mark was set to 0 before it.  Each warp compares 32 of the n marks with all.
template <int WARPS_> __device__ __forceinline__ void find_mark(const unsigned* marks, int n, int want, unsigned* mark) {
    const int lane = threadIdx.x & 31;
    for (int i0 = (threadIdx.x >> 5) * 32; i0 < n; i0 += WARPS_ * 32) {
        const int i = i0 + lane;
        const unsigned k = i < n ? marks[i] : 0u;
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; j += 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(marks + j);
            rank += (q.x > k || (q.x == k && j < i)) + (q.y > k || (q.y == k && j + 1 < i)) +
                    (q.z > k || (q.z == k && j + 2 < i)) + (q.w > k || (q.w == k && j + 3 < i));
        }
        if (i < n && rank == want - 1) *mark = k;
    }
}

// Sum over the 8 lanes that share a candidate.
__device__ __forceinline__ int sum8(int v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// E elements of one thread as they lie in memory: two of 16 bits a register, element 2 j + h in half h
// of word j.
template <typename XT, int E> struct Held;
template <int E> struct Held<float, E> {
    float v[E];
    __device__ __forceinline__ void set(int j, unsigned w) { v[j] = __uint_as_float(w); }
    __device__ __forceinline__ void one(int i, float x) { v[i] = x; }
    __device__ __forceinline__ float top() const {                   // passes NaN over
        float t = v[0];
#pragma unroll
        for (int i = 1; i < E; ++i) t = fmaxf(t, v[i]);
        return t;
    }
    __device__ __forceinline__ Pair two(int j) const { return pair(v[2 * j], v[2 * j + 1]); }
    // a bit for every element that is at least x
    __device__ __forceinline__ unsigned reach(float x) const {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) m |= v[i] >= x ? 1u << i : 0u;
        return m;
    }
    static __device__ __forceinline__ unsigned every() { return (unsigned)((1ull << E) - 1); }
    static __device__ __forceinline__ int element(int bit) { return bit; }
};
template <int E> struct Held<__nv_bfloat16, E> {
    __nv_bfloat162 v[E / 2];
    __device__ __forceinline__ void set(int j, unsigned w) { v[j] = *reinterpret_cast<__nv_bfloat162*>(&w); }
    __device__ __forceinline__ void one(int i, float x) { (i & 1 ? v[i / 2].y : v[i / 2].x) = __float2bfloat16_rn(x); }
    __device__ __forceinline__ float top() const {
        __nv_bfloat162 t = v[0];
#pragma unroll
        for (int i = 1; i < E / 2; ++i) t = __hmax2(t, v[i]);
        return fmaxf(__low2float(t), __high2float(t));
    }
    __device__ __forceinline__ Pair two(int j) const {
        const unsigned w = *reinterpret_cast<const unsigned*>(&v[j]);
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ unsigned reach(float x) const {       // x is one of the values: exact in 16 bits
        const __nv_bfloat162 x2 = __float2bfloat162_rn(x);
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < E / 2; ++j) m |= (__hge2_mask(v[j], x2) & 0x00010001u) << j;
        return m;
    }
    static __device__ __forceinline__ unsigned every() { return ((1u << (E / 2)) - 1) * 0x00010001u; }
    static __device__ __forceinline__ int element(int bit) { return 2 * (bit & 15) + (bit >> 4); }
};

// E elements per thread: 16-byte loads (VEC) or one by one.
template <typename XT, int E, bool VEC>
__global__ void __launch_bounds__(NT, E > 8 && sizeof(XT) == 4 ? 4 : 6) beam_row_kernel(BeamParams p) {
    __shared__ __align__(16) unsigned marks[MARKS];
    __shared__ unsigned the_mark;
    __shared__ float2 sums[WARPS];
    __shared__ int count;
    __shared__ unsigned long long pick[WARPS];
    __shared__ unsigned long long list[LIST];       // key, then the token's complement: larger is better
    // unsigned: the last rows' grid reaches past 2^31 where G * K comes near it
    const unsigned row = blockIdx.z * gridDim.y + blockIdx.y;
    const int piece = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (row >= (unsigned)p.G * (unsigned)p.K) return;
    asm volatile("griddepcontrol.launch_dependents;");               // the groups' blocks may come; they wait
    const int v0 = piece * p.piece, n = min(p.piece, p.V - v0);      // this block's tokens
    const XT* x = static_cast<const XT*>(p.logits) + (size_t)row * p.row + v0;
    constexpr int W = VEC ? 16 / (int)sizeof(XT) : 1;                // elements of a load
    // element i of this thread: load i / W at (i / W * NT + thread) * W
    auto at = [&](int i) { return (i / W * NT + (int)threadIdx.x) * W + i % W; };
    Held<XT, E> v;
#pragma unroll
    for (int j = 0; j < E / W; ++j) {
        const int o = (j * NT + (int)threadIdx.x) * W;
        if constexpr (VEC) {
            if (o + W <= n && GDR_INB(v0 + o + W <= p.V, 1001)) {
                const uint4 q = *reinterpret_cast<const uint4*>(x + o);
                v.set(4 * j, q.x); v.set(4 * j + 1, q.y); v.set(4 * j + 2, q.z); v.set(4 * j + 3, q.w);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v.one(j * W + i, o + i < n && GDR_INB(v0 + o + i < p.V, 1002) ? ld_f32(x + o + i) : -INFINITY);
            }
        } else {
            v.one(j, o < n && GDR_INB(v0 + o < p.V, 1004) ? ld_f32(x + o) : -INFINITY);
        }
    }
    if (threadIdx.x == 0) { count = 0; the_mark = 0; }
    const float top = v.top();
    const int active = min((n + W - 1) / W, NT), lanes = group_lanes(active, p.M);
    const unsigned key = at(0) < n ? key_of(top) : 0u, top_key = __reduce_max_sync(0xffffffffu, key);
    put_marks(key, lanes, active, marks);
    // exp(x - maximum); all masked (maximum -inf): nothing but NaN counts.  +inf gives NaN: the beam
    // drops out.
    const float big = top_key ? value_of(top_key) : -INFINITY, base = big == -INFINITY ? 0.f : big;
    const Pair off = pair(-base, -base), log2e = pair(1.44269502f, 1.44269502f);
    Pair s2 = pair(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const Pair d = (v.two(j) + off) * log2e;
        float e0, e1;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(lo(d)));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(hi(d)));
        s2 = s2 + pair(e0, e1);
    }
    float s = lo(s2) + hi(s2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[warp] = make_float2(big, s);
    __syncthreads();
    find_mark<WARPS>(marks, (active + lanes - 1) / lanes, p.M, &the_mark);
    __syncthreads();
    const size_t out = (size_t)row * p.pieces + piece;
    const unsigned mark = the_mark;
    // this thread's elements that reach the mark; a mark of -inf or less lets everything through
    unsigned hits = mark > key_of(-INFINITY) ? v.reach(value_of(mark)) : v.every();
    auto element = [&](int i) { return (unsigned long long)key_of(ld_f32(x + at(i))) << 32 | (unsigned)~at(i); };
    while (hits) {                                                   // few: read them again
        const int i = v.element(__ffs(hits) - 1);
        hits &= hits - 1;
        if (at(i) >= n) continue;
        const unsigned long long c = element(i);
        if ((unsigned)(c >> 32) < mark) continue;
        const int slot = atomicAdd(&count, 1);
        if (slot < LIST) list[slot] = c;
    }
    __syncthreads();
    const int have = count;
    float* best = p.best + out * p.M;
    int* token = p.token + out * p.M;
    if (threadIdx.x == 0) {
        float m = sums[0].x;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sums[w].x);
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            // a masked warp adds nothing, unless it holds a NaN
            if (sums[w].x > -INFINITY || sums[w].y != sums[w].y) t += sums[w].y * expf(sums[w].x - m);
        }
        p.sums[out] = make_float2(m, t);
    }
    if (have <= LIST) {
        // the rank of a candidate is the number of larger ones (all differ), counted by 8 lanes
        for (int i0 = 0; i0 < have; i0 += NT / 8) {
            const int i = i0 + (int)threadIdx.x / 8;
            const unsigned long long c = i < have ? list[i] : 0;
            int rank = 0;
            for (int j = threadIdx.x & 7; j < have; j += 8) rank += list[j] > c;
            rank = sum8(rank);
            if (i < have && (threadIdx.x & 7) == 0 && rank < p.M && GDR_INB(rank >= 0 && piece < p.pieces, 1003)) {
                best[rank] = value_of((unsigned)(c >> 32));
                token[rank] = v0 + (int)~(unsigned)c;
            }
        }
        for (int i = have + threadIdx.x; i < p.M; i += NT) {
            best[i] = -INFINITY;
            token[i] = -1;
        }
    } else {
        // too many for the list (equal ones, or all of a piece whose mark is -inf): the largest, M times
        unsigned long long last = ~0ull;
        for (int m = 0; m < p.M; ++m) {
            unsigned long long c = 0;
#pragma unroll 1
            for (int i = 0; i < E; ++i) {
                if (at(i) >= n) continue;
                const unsigned long long k = element(i);
                if (k < last && k > c) c = k;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) { const unsigned long long k = __shfl_xor_sync(0xffffffffu, c, o); c = k > c ? k : c; }
            if (lane == 0) pick[warp] = c;
            __syncthreads();
            c = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) c = pick[w] > c ? pick[w] : c;
            __syncthreads();
            last = c;
            if (threadIdx.x == 0) {
                best[m] = value_of((unsigned)(c >> 32));
                token[m] = v0 + (int)~(unsigned)c;
            }
        }
    }
}

// Candidates of a group: the larger score, of equal ones the lower k * V + v, goes first.
struct Cand { double s; int at, beam; };
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) { return a.s > b.s || (a.s == b.s && a.at < b.at); }
// A key of 32 bits that never orders two scores the other way round (it may merge near ones).
__device__ __forceinline__ unsigned key_of_score(double s) { return key_of(__double2float_rd(s)); }

// How far two scores may be from their 64-bit values together, u = 2^-24: an exponent d = x - maximum
// and its product with the rounded log2(e) are off by 2.25 u |d|, |d| weighted by e^d is at most
// log V <= 22: 50 u; the exponential 3 u; 17 sums in a thread, 5 in its warp, 8 across the block, 6
// across the pieces (each lane adds its own in 64 bits) and the factors of warps and pieces (4 u
// each) 44 u: together 97 u of the sum, as much in its logarithm, whose rounding adds 17 u (it is at
// most 22).  114 u = 6.8e-6, twice that for two beams.
constexpr double TOL = 1.4e-5;
constexpr float BELOW = 1.5e-5f;        // more than TOL

constexpr int HELD = 2;                 // candidates of a thread that stay in registers

// The 64-bit sum over one beam's logits.
template <typename XT, int GNT>
__device__ double exact_lse(const BeamParams& p, int row, double big, double* red) {
    const XT* x = static_cast<const XT*>(p.logits) + (size_t)row * p.row;
    double s = 0.0;
    for (int v = threadIdx.x; v < p.V; v += GNT) s += exp((double)ld_f32(x + v) - big);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int i = 0; i < GNT / 32; ++i) s += red[i];
    __syncthreads();
    return big + log(s);
}

// GNT threads: as many as there are candidates for, 256 or 1024.  FEW: all of them stay in registers.
template <typename XT, int GNT, bool FEW>
__global__ void __launch_bounds__(GNT) beam_group_kernel(BeamParams p) {
    constexpr int GWARPS = GNT / 32;
    __shared__ __align__(16) unsigned marks[MARKS];
    __shared__ unsigned the_mark;
    __shared__ int count;
    __shared__ Cand list[LIST];
    __shared__ Cand first[MOST];                    // the best in order
    __shared__ double lse[MOST], top[MOST], red[GWARPS];
    __shared__ float score[MOST];
    __shared__ unsigned char kind[MOST], redo[MOST];
    enum { LIVE, ENDED, OUT };                      // a beam that goes on, that has one candidate, that has none
    const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = p.pieces * p.M, n = p.K * per;
    float sc = 0.f;                                 // of beam `warp`: older than the rows' launch
    bool ended = false;
    if (warp < p.K) { sc = p.scores[(size_t)g * p.K + warp]; ended = p.finished && p.finished[(size_t)g * p.K + warp]; }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    float2 mine = make_float2(-INFINITY, 0.f);      // of beam `warp`, its piece `lane`
    if (warp < p.K && lane < p.pieces) mine = p.sums[((size_t)g * p.K + warp) * p.pieces + lane];
    // this thread's candidates: beam, position in its lists, logit and token.  Few of them: a warp's
    // lanes lie evenly over all beams and pieces, so that every warp has some of the best; many: one
    // behind the other, so that every thread has some of every beam.
    const int span = (n + 31) / 32;
    auto index = [&](int u) {
        if (!FEW) return (int)threadIdx.x + u * GNT;
        const int j = warp + u * GWARPS;
        return j < span ? lane * span + j : n;
    };
    int hk[HELD], hj[HELD], ht[HELD];
    float hx[HELD];
#pragma unroll
    for (int u = 0; u < HELD; ++u) {
        const int i = index(u);
        hk[u] = i / per;
        hj[u] = i - hk[u] * per;
        if (i < n && GDR_INB(i >= 0 && hk[u] < p.K && g < p.G, 1012)) {
            const size_t at = (size_t)g * n + i;
            ht[u] = p.token[at];
            hx[u] = p.best[at];
        }
    }
    for (int k = warp; k < p.K; k += GWARPS) {      // a warp per beam, lanes along its pieces
        const size_t row = (size_t)g * p.K + k;
        const float2* sums = p.sums + row * p.pieces;
        if (k != warp) {
            sc = p.scores[row];
            ended = p.finished && p.finished[row];
            mine = lane < p.pieces ? sums[lane] : make_float2(-INFINITY, 0.f);
        }
        float big = mine.x;
        for (int i = lane + 32; i < p.pieces; i += 32) big = fmaxf(big, sums[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        double s = 0.0;
        auto add = [&](float2 e) {
            // an all-masked piece adds nothing, unless it holds a NaN
            if (e.x > -INFINITY) s += (double)(e.y * expf(e.x - big));
            else if (e.y != e.y) s = e.y;
        };
        add(mine);
        for (int i = lane + 32; i < p.pieces; i += 32) add(sums[i]);
        float total = (float)s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) {
            const bool no_score = !(sc < INFINITY) || sc == -INFINITY;
            score[k] = sc;
            top[k] = big;
            lse[k] = (double)big + (double)logf(total);
            kind[k] = no_score ? OUT : ended ? ENDED : !(big > -INFINITY && big < INFINITY && total == total) ? OUT : LIVE;
            redo[k] = 0;
        }
    }
    __syncthreads();

    auto score_of = [&](int k, int j, int t, float x, Cand& c) -> bool {
        c.beam = k;
        if (kind[k] == LIVE) {
            c.s = (double)score[k] + ((double)x - lse[k]);
            c.at = k * p.V + t;
            return t >= 0;
        }
        // without logits of its own: the lowest tokens at -inf, behind `eos` of a finished beam
        if (kind[k] == ENDED) {
            c.s = j == 0 ? (double)score[k] : -INFINITY;
            c.at = k * p.V + (j == 0 ? p.eos : j - 1 < p.eos ? j - 1 : j);
        } else {
            c.s = -INFINITY;
            c.at = k * p.V + j;
        }
        return j < p.M && j < p.V;
    };
    // f(candidate) for this thread's candidates
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            Cand c;
            if (index(u) < n && score_of(hk[u], hj[u], ht[u], hx[u], c)) f(c);
        }
        for (int i0 = threadIdx.x + HELD * GNT; !FEW && i0 < n; i0 += 4 * GNT) {
            int t[4];
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {           // four loads in flight
                const int i = i0 + u * GNT;
                if (i < n && GDR_INB(i >= 0 && g < p.G, 1013)) { t[u] = p.token[(size_t)g * n + i]; x[u] = p.best[(size_t)g * n + i]; }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * GNT;
                Cand c;
                if (i < n && score_of(i / per, i % per, t[u], x[u], c)) f(c);
            }
        }
    };
    const int want = p.M;                           // at most K * V
    for (int turn = 0; turn < 2; ++turn) {
        unsigned mine = 0;
        each([&](const Cand& c) { mine = max(mine, key_of_score(c.s)); });
        const int active = FEW ? 32 * min(GWARPS, span) : GNT, lanes = group_lanes(active, want);
        put_marks(mine, lanes, active, marks);
        if (threadIdx.x == 0) { count = 0; the_mark = 0; }
        if (threadIdx.x < p.M) first[threadIdx.x] = Cand{-INFINITY, -1, 0};
        __syncthreads();
        find_mark<GWARPS>(marks, active / lanes, want, &the_mark);
        __syncthreads();
        // and down to TOL below it: the list also holds what may belong before its M-th
        const unsigned mark = the_mark ? key_of(__fsub_rd(value_of(the_mark), BELOW)) : 0u;
        each([&](const Cand& c) {
            if (key_of_score(c.s) < mark) return;
            const int slot = atomicAdd(&count, 1);
            if (slot < LIST) list[slot] = c;
        });
        __syncthreads();
        const int have = count;
        bool near = have > LIST;                    // a pair to look at: unknown of a list that overflowed
        if (have <= LIST) {
            for (int i0 = 0; i0 < have; i0 += GNT / 8) {
                const int i = i0 + (int)threadIdx.x / 8;
                const Cand c = i < have ? list[i] : Cand{0.0, 0, 0};
                int rank = 0;
                bool close = false;
                for (int j = threadIdx.x & 7; j < have; j += 8) {
                    const Cand o = list[j];
                    rank += before(o, c);
                    close |= o.beam != c.beam && fabs(o.s - c.s) <= TOL;
                }
                rank = sum8(rank);
                near |= close && i < have && rank < want;
                if (i < have && (threadIdx.x & 7) == 0 && rank < want) first[rank] = c;
            }
            __syncthreads();
        } else {
            // too many equal ones for the list: the best, want times
            Cand last = {INFINITY, -1, 0};
            for (int m = 0; m < want; ++m) {
                Cand b = {-INFINITY, INT32_MAX, 0};
                each([&](const Cand& c) { if (before(last, c) && before(c, b)) b = c; });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const Cand c = {__shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.at, o),
                                    __shfl_xor_sync(0xffffffffu, b.beam, o)};
                    if (before(c, b)) b = c;
                }
                if (lane == 0) list[warp] = b;
                __syncthreads();
                b = list[0];
                for (int w = 1; w < GWARPS; ++w) if (before(list[w], b)) b = list[w];
                if (threadIdx.x == 0) first[m] = b;
                last = b;
                __syncthreads();
            }
        }
        if (turn == 1) break;
        // pairs of different beams that the fp32 sums cannot order, one of them among the M
        if (!__syncthreads_or(near)) break;
        bool again = false;
        for (int m = 0; m < want; ++m) {
            const Cand a = first[m];
            each([&](const Cand& c) {
                if (c.beam == a.beam || !(fabs(c.s - a.s) <= TOL)) return;
                if (kind[a.beam] == LIVE) { redo[a.beam] = 1; again = true; }
                if (kind[c.beam] == LIVE) { redo[c.beam] = 1; again = true; }
            });
        }
        if (!__syncthreads_or(again)) break;
        for (int k = 0; k < p.K; ++k) {
            if (!redo[k]) continue;
            const double l = exact_lse<XT, GNT>(p, g * p.K + k, top[k], red);
            if (threadIdx.x == 0) lse[k] = l;
        }
        __syncthreads();
    }
    for (int m = threadIdx.x; m < p.M; m += GNT) {
        const size_t at = (size_t)g * p.M + m;
        const Cand c = first[m];
        if (!GDR_INB(c.at >= 0 && c.at < (long long)p.K * p.V, 1011)) continue;
        p.out_scores[at] = (float)c.s;
        p.out_parent[at] = c.beam;
        p.out_token[at] = c.at - c.beam * p.V;
    }
}

// ---------------------------------------------------------------- reorder ----

struct ReorderParams {
    int G, K;
    int first;              // layer * G + group of the grid's first
    size_t n;               // elements (of the kernel's width) of one state
    char* S;
    const int* parent;
};

// One thread owns one position of the K states of a group: it reads what every moving beam takes
// over, and only then writes, so that the exchange needs no second buffer and no other thread.
template <typename VT, int KMAX>
__global__ void __launch_bounds__(NT) reorder_kernel(ReorderParams p) {
    const int g = (p.first + blockIdx.y) % p.G;
    const int* parent = p.parent + (size_t)g * p.K;
    VT* S = reinterpret_cast<VT*>(p.S) + (size_t)blockIdx.y * p.K * p.n;
    if (blockIdx.x == 0 && p.first + (int)blockIdx.y < p.G && threadIdx.x < p.K) {
        const int q = parent[threadIdx.x];
        if (q < 0 || q >= p.K) atomicOr(&g_device_status, STATUS_INDEX);
    }
    for (size_t i = (size_t)blockIdx.x * NT + threadIdx.x; i < p.n; i += (size_t)gridDim.x * NT) {
        VT v[KMAX];
        bool moves[KMAX];
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            const int q = j < p.K ? parent[j] : j;
            moves[j] = q != j && q >= 0 && q < p.K && GDR_INB(j < p.K && i < p.n, 1021);
            if (moves[j]) v[j] = S[(size_t)q * p.n + i];
        }
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
            if (moves[j]) S[(size_t)j * p.n + i] = v[j];
    }
}

}  // namespace bms
}  // namespace gdr
