// beam.cuh -- kernels of the beam selection and of the state reorder.
//
// Selection.  Within a beam the order of the candidates is the order of its logits, so the M best
// of a beam need no sum; across beams the scores score + (logit - lse) are compared in 64 bits.
//
//   1. beam_row_kernel: a block per (beam, piece of the vocabulary) reads its piece once into
//      registers and leaves the piece's maximum, its sum of exp(x - maximum) and its M best
//      (logit, token) pairs, unordered.  Every warp takes the q-th largest of its lanes' own maxima,
//      q = M / warps rounded up; at least M elements reach the smallest of these marks, and for
//      logits in no particular order only a few more do, so one sweep over the registers collects
//      them all and a count of the larger ones ranks them.
//   2. beam_group_kernel: a block per group merges its beams' pieces the same way.  Its sums hold
//      fp32 exponentials; where two neighbours of the list from different beams are closer than
//      those allow (TOL), the beams' sums are formed again from the logits in 64 bits and the
//      merge is repeated, so that the order is the 64-bit one.
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
constexpr int LIST = 1024;              // candidates that reach the mark; more: M rounds of the largest

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

// The q-th largest of the lanes' keys (equal ones count one by one); 0 when fewer are above zero.
__device__ __forceinline__ unsigned warp_mark(unsigned key, int q) {
    unsigned m = 0;
    for (int i = 0; i < q; ++i) {
        m = __reduce_max_sync(0xffffffffu, key);
        const unsigned who = __ballot_sync(0xffffffffu, key == m);
        if ((int)(threadIdx.x & 31) == __ffs(who) - 1) key = 0;
    }
    return m;
}

struct BlockSmem {
    unsigned mark[WARPS];
    float red[WARPS];
    int count;
    unsigned long long pick[WARPS];
};

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) v = fmaxf(v, red[i]);
    __syncthreads();
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v += red[i];
    __syncthreads();
    return v;
}

// E elements per thread: 16-byte loads (VEC) or one by one.
template <typename XT, int E, bool VEC>
__global__ void __launch_bounds__(NT) beam_row_kernel(BeamParams p) {
    __shared__ BlockSmem sm;
    __shared__ unsigned long long list[LIST];       // key, then the token's complement: larger is better
    const int row = blockIdx.y, piece = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int v0 = piece * p.piece, n = min(p.piece, p.V - v0);      // this block's tokens
    const XT* x = static_cast<const XT*>(p.logits) + (size_t)row * p.row + v0;
    constexpr int W = VEC ? 16 / (int)sizeof(XT) : 1;                // elements of a load
    // element i of this thread: load i / W at (i / W * NT + thread) * W
    auto at = [&](int i) { return (i / W * NT + (int)threadIdx.x) * W + i % W; };
    float v[E];
#pragma unroll
    for (int j = 0; j < E / W; ++j) {
        const int o = (j * NT + (int)threadIdx.x) * W;
        if constexpr (VEC) {
            if (o + W <= n) {
                const uint4 q = *reinterpret_cast<const uint4*>(x + o);
                const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if constexpr (sizeof(XT) == 4) v[j * W + i] = __uint_as_float(w[i]);
                    else v[j * W + i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[j * W + i] = o + i < n ? ld_f32(x + o + i) : -INFINITY;
            }
        } else {
            v[j] = o < n ? ld_f32(x + o) : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < E; ++i) top = fmaxf(top, v[i]);              // passes NaN over
    const unsigned mine = at(0) < n ? key_of(top) : 0u;
    // the marks of the warps all of whose lanes hold elements (a short piece fills the first ones)
    const int full = min((n + W - 1) / W, NT) / 32, q = full ? (p.M + full - 1) / full : 33;
    const unsigned mark_w = q <= 32 && warp < full ? warp_mark(mine, q) : 0u;
    if (lane == 0) sm.mark[warp] = mark_w;
    if (threadIdx.x == 0) sm.count = 0;
    const float big = block_max(top, sm.red);
    // exp(x - big); all masked (big = -inf): nothing but NaN counts.  +inf gives NaN: the beam drops out.
    const float base = big == -INFINITY ? 0.f : big;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((v[i] - base) * 1.44269502f));
        s += e;
    }
    s = block_sum(s, sm.red);
    const size_t out = (size_t)row * p.pieces + piece;
    if (threadIdx.x == 0) p.sums[out] = make_float2(big, s);

    unsigned mark = sm.mark[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mark = w < full ? min(mark, sm.mark[w]) : mark;
    const float least = value_of(max(mark, 1u));                     // a zero mark lets everything through
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (v[i] >= least || mark <= key_of(-INFINITY)) {
            if (at(i) < n && key_of(v[i]) >= mark) {
                const int slot = atomicAdd(&sm.count, 1);
                if (slot < LIST) list[slot] = (unsigned long long)key_of(v[i]) << 32 | (unsigned)~at(i);
            }
        }
    }
    __syncthreads();
    const int have = sm.count;
    float* best = p.best + out * p.M;
    int* token = p.token + out * p.M;
    if (have <= LIST) {
        // the rank of a candidate is the number of larger ones: all differ
        for (int i = threadIdx.x; i < max(have, p.M); i += NT) {
            if (i >= have) {
                best[i] = -INFINITY;
                token[i] = -1;
                continue;
            }
            const unsigned long long c = list[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += list[j] > c;
            if (rank < p.M && GDR_INB(rank >= 0, 1001)) {
                best[rank] = value_of((unsigned)(c >> 32));
                token[rank] = v0 + (int)~(unsigned)c;
            }
        }
    } else {
        // too many equal ones for the list: the largest, M times
        unsigned long long last = ~0ull;
        for (int m = 0; m < p.M; ++m) {
            unsigned long long c = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (at(i) >= n) continue;
                const unsigned long long k = (unsigned long long)key_of(v[i]) << 32 | (unsigned)~at(i);
                if (k < last && k > c) c = k;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) { const unsigned long long k = __shfl_xor_sync(0xffffffffu, c, o); c = k > c ? k : c; }
            if (lane == 0) sm.pick[warp] = c;
            __syncthreads();
            c = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) c = sm.pick[w] > c ? sm.pick[w] : c;
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
struct Cand { double s; int at; };
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) { return a.s > b.s || (a.s == b.s && a.at < b.at); }
// A key of 32 bits that never orders two scores the other way round (it may merge near ones).
__device__ __forceinline__ unsigned key_of_score(double s) { return key_of(__double2float_rd(s)); }

// How far two scores may be from their 64-bit values together, u = 2^-24: an exponent d = x - maximum
// and its product with the rounded log2(e) are off by 2.25 u |d|, |d| weighted by e^d is at most
// log V <= 22: 50 u; the exponential 3 u; 32 sums in a thread and 16 across the block 48 u.  101 u =
// 6.1e-6 of the sum, twice that for two beams.
constexpr double TOL = 1.25e-5;

template <typename XT>
__device__ double exact_lse(const BeamParams& p, int row, double big, double* red) {
    const XT* x = static_cast<const XT*>(p.logits) + (size_t)row * p.row;
    double s = 0.0;
    for (int v = threadIdx.x; v < p.V; v += NT) s += exp((double)ld_f32(x + v) - big);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) s += red[i];
    __syncthreads();
    return big + log(s);
}

template <typename XT>
__global__ void __launch_bounds__(NT) beam_group_kernel(BeamParams p) {
    __shared__ BlockSmem sm;
    __shared__ Cand list[LIST];
    __shared__ Cand first[MOST + 1];                // the best in order, and the one behind
    __shared__ double lse[MOST], top[MOST], red[WARPS];
    __shared__ float score[MOST];
    __shared__ unsigned char kind[MOST], redo[MOST];
    enum { LIVE, ENDED, OUT };                      // a beam that goes on, that has one candidate, that has none
    const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = threadIdx.x; k < p.K; k += NT) {
        const size_t row = (size_t)g * p.K + k;
        float big = -INFINITY;
        for (int i = 0; i < p.pieces; ++i) big = fmaxf(big, p.sums[row * p.pieces + i].x);
        double s = 0.0;
        for (int i = 0; i < p.pieces; ++i) {
            const float2 e = p.sums[row * p.pieces + i];
            // an all-masked piece adds nothing, unless it holds a NaN
            s += e.x == -INFINITY ? (e.y != e.y ? (double)e.y : 0.0) : (double)e.y * exp((double)e.x - (double)big);
        }
        const float sc = p.scores[row];
        const bool no_score = !(sc < INFINITY) || sc == -INFINITY;
        const bool ended = p.finished && p.finished[row];
        score[k] = sc;
        top[k] = big;
        lse[k] = (double)big + log(s);
        kind[k] = no_score ? OUT : ended ? ENDED : !(big > -INFINITY && big < INFINITY && s == s) ? OUT : LIVE;
        redo[k] = 0;
    }
    __syncthreads();

    const int per = p.pieces * p.M, n = p.K * per;
    auto cand = [&](int i, Cand& c) -> bool {
        const int k = i / per, j = i % per;
        if (kind[k] == LIVE) {
            const size_t at = ((size_t)g * p.K + k) * per + j;
            const int t = p.token[at];
            if (t < 0) return false;
            c.s = (double)score[k] + ((double)p.best[at] - lse[k]);
            c.at = k * p.V + t;
            return true;
        }
        // without logits of its own: the lowest tokens at -inf, behind `eos` of a finished beam
        if (j >= p.M || j >= p.V) return false;
        if (kind[k] == ENDED) {
            c.s = j == 0 ? (double)score[k] : -INFINITY;
            c.at = k * p.V + (j == 0 ? p.eos : j - 1 < p.eos ? j - 1 : j);
        } else {
            c.s = -INFINITY;
            c.at = k * p.V + j;
        }
        return true;
    };
    // one more than asked for: the candidate behind the last may be too near to it
    const long long all = (long long)p.K * p.V;
    const int want = (int)(all < p.M + 1 ? all : p.M + 1);
    for (int turn = 0; turn < 2; ++turn) {
        unsigned mine = 0;
        for (int i = threadIdx.x; i < n; i += NT) {
            Cand c;
            if (cand(i, c)) mine = max(mine, key_of_score(c.s));
        }
        const unsigned mark_w = warp_mark(mine, (want + WARPS - 1) / WARPS);
        if (lane == 0) sm.mark[warp] = mark_w;
        if (threadIdx.x == 0) sm.count = 0;
        if (threadIdx.x <= p.M) first[threadIdx.x] = Cand{-INFINITY, -1};
        __syncthreads();
        unsigned mark = sm.mark[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) mark = min(mark, sm.mark[w]);
        for (int i = threadIdx.x; i < n; i += NT) {
            Cand c;
            if (cand(i, c) && key_of_score(c.s) >= mark) {
                const int slot = atomicAdd(&sm.count, 1);
                if (slot < LIST) list[slot] = c;
            }
        }
        __syncthreads();
        const int have = sm.count;
        if (have <= LIST) {
            for (int i = threadIdx.x; i < have; i += NT) {
                const Cand c = list[i];
                int rank = 0;
                for (int j = 0; j < have; ++j) rank += before(list[j], c);
                if (rank < want) first[rank] = c;
            }
            __syncthreads();
        } else {
            Cand last = {INFINITY, -1};
            for (int m = 0; m < want; ++m) {
                Cand b = {-INFINITY, INT32_MAX};
                for (int i = threadIdx.x; i < n; i += NT) {
                    Cand c;
                    if (cand(i, c) && before(last, c) && before(c, b)) b = c;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const Cand c = {__shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.at, o)};
                    if (before(c, b)) b = c;
                }
                if (lane == 0) list[warp] = b;
                __syncthreads();
                b = list[0];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) if (before(list[w], b)) b = list[w];
                if (threadIdx.x == 0) first[m] = b;
                last = b;
                __syncthreads();
            }
        }
        if (turn == 1) break;
        // neighbours of different beams that the fp32 sums cannot order
        bool near = false;
        if ((int)threadIdx.x + 1 < want) {
            const Cand a = first[threadIdx.x], b = first[threadIdx.x + 1];
            if (b.at >= 0 && b.s > -INFINITY && a.s - b.s <= TOL) {
                const int ka = a.at / p.V, kb = b.at / p.V;
                if (ka != kb) {
                    if (kind[ka] == LIVE) { redo[ka] = 1; near = true; }
                    if (kind[kb] == LIVE) { redo[kb] = 1; near = true; }
                }
            }
        }
        if (!__syncthreads_or(near)) break;
        for (int k = 0; k < p.K; ++k) {
            if (!redo[k]) continue;
            const double l = exact_lse<XT>(p, g * p.K + k, top[k], red);
            if (threadIdx.x == 0) lse[k] = l;
        }
        __syncthreads();
    }
    for (int m = threadIdx.x; m < p.M; m += NT) {
        const size_t at = (size_t)g * p.M + m;
        const Cand c = first[m];
        if (!GDR_INB(c.at >= 0 && (long long)c.at < all, 1011)) continue;
        p.out_scores[at] = (float)c.s;
        p.out_parent[at] = c.at / p.V;
        p.out_token[at] = c.at % p.V;
    }
}

// ---------------------------------------------------------------- reorder ----

struct ReorderParams {
    int G, K;
    size_t n;               // elements (of the kernel's width) of one state
    char* S;
    const int* parent;
};

// One thread owns one position of the K states of a group: it reads what every moving beam takes
// over, and only then writes, so that the exchange needs no second buffer and no other thread.
template <typename VT, int KMAX>
__global__ void __launch_bounds__(NT) reorder_kernel(ReorderParams p) {
    const int g = blockIdx.y % p.G;
    const int* parent = p.parent + (size_t)g * p.K;
    VT* S = reinterpret_cast<VT*>(p.S) + (size_t)blockIdx.y * p.K * p.n;
    if (blockIdx.x == 0 && blockIdx.y < p.G && threadIdx.x < p.K) {
        const int q = parent[threadIdx.x];
        if (q < 0 || q >= p.K) atomicOr(&g_device_status, STATUS_INDEX);
    }
    for (size_t i = (size_t)blockIdx.x * NT + threadIdx.x; i < p.n; i += (size_t)gridDim.x * NT) {
        VT v[KMAX];
        bool moves[KMAX];
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            const int q = j < p.K ? parent[j] : j;
            moves[j] = q != j && q >= 0 && q < p.K;
            if (moves[j]) v[j] = S[(size_t)q * p.n + i];
        }
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
            if (moves[j]) S[(size_t)j * p.n + i] = v[j];
    }
}

}  // namespace bms
}  // namespace gdr
