// scan.cuh -- kernels of the per-channel gated linear recurrence h_t = a_t h_{t-1} + b_t.
//
// Mathematics.  A run of tokens maps the state before it to the state after it by s -> A s + H,
// with A the product of its decays and H its end state from zero; two neighbouring runs compose
// to (A2 A1, A2 H1 + H2).  So a tile of tokens is cut into short runs, one per thread; each
// thread forms its run's (A, H) in registers, the runs' start states come from composing what
// lies before them, and a second sweep over the same registers gives every h_t.  x and g are
// read once.  The backward adds the state's gradient, which runs the same way from the end:
// mu_t = a_t (dh_t + mu_{t+1}), with the same A and an M in place of H.
//
// Bound: HBM (a forward moves 6 to 12 bytes per element for about 20 instructions).
//
// Split.  A block of 8 warps owns CH = 32 or 16 channels x TOK tokens per turn and walks the sequence
// in turns.  Where the channels alone do not fill the GPU, a cluster of up to 16 blocks takes that
// many neighbouring tiles per turn: the blocks send one another their tiles' (A, H) by
// asynchronous stores into distributed shared memory, which an mbarrier counts (a cluster barrier
// per turn would also wait for the turn's output stores: 96 against 90 us); every block folds them
// in the same order, so the result does not depend on timing, and there is neither a workspace nor
// a wait on a block outside the cluster.  The next turns' tiles come by tensor-map copies (TMA)
// into a ring of shared-memory stages while the current one is computed (per-thread cp.async
// spent a quarter of the time in issuing).
#pragma once

#include <type_traits>

#include <cuda.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace gdr {
namespace scn {

struct ScanParams {
    int B, T, D;
    long long x_row, g_row;
    int gate_mode, tied;
    const void* x;
    const void* g;
    const float* h0;
    const int* lengths;
    void* h;
    float* h_T;
    float* ckpt;
    const void* dh;
    const float* dh_T;
    void* dx;
    void* dg;
    float* dh0;
    long long covered;                  // V = 1: rows (of B * T) that the tensor maps reach
};

constexpr int CKPT = GDR_SCAN_CKPT;
constexpr int NT = 256;
constexpr int WT = NT / 32;             // warps, along the tokens
constexpr int BOX_ROWS = 256;           // of one tensor copy at most
constexpr int MAX_CLUSTER = 16;
constexpr int STAGES = 2;

__device__ __forceinline__ int seq_len(const ScanParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// f(mode, tied) with the call's gate mode and form as compile-time constants: the branch is taken
// once per sweep instead of once per element.
template <typename F> __device__ __forceinline__ void with_mode(const ScanParams& p, F f) {
    if (p.gate_mode == 1) {
        if (p.tied) f(std::integral_constant<int, 1>(), std::true_type()); else f(std::integral_constant<int, 1>(), std::false_type());
    } else {
        if (p.tied) f(std::integral_constant<int, 0>(), std::true_type()); else f(std::integral_constant<int, 0>(), std::false_type());
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// V values of one thread as stored: loads from global or shared memory, and the rounding store.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void get(const Raw& r, float (&v)[4]) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
    static __device__ __forceinline__ Raw put(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Pack<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void get(const Raw& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw put(const float (&v)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        return make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
    }
};
template <typename T> struct Pack<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ void get(const Raw& r, float (&v)[1]) { v[0] = ld_f32(&r); }
    static __device__ __forceinline__ Raw put(const float (&v)[1]) { Raw r; st_from_f32(&r, v[0]); return r; }
};

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ uint32_t cluster_size() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without ordering memory (it does not wait for stores on their way).
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Store to the same shared-memory place of block `rank` of the cluster; the 8 bytes count towards
// the phase of that block's barrier.
__device__ __forceinline__ void store_peer(float2* p, float2 v, uint64_t* bar, uint32_t rank) {
    uint32_t a, m;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(smem_addr(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
                 ::"r"(a), "f"(v.x), "f"(v.y), "r"(m) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// Wait for a phase, for at most 2 s; false (and the status word's timeout bit) when it did not come.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
    if (phase_done(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!phase_done(bar, parity))
        if (tc::globaltimer_ns() - t0 > 2000000000ull) { atomicOr(&g_device_status, STATUS_TIMEOUT); return false; }
    return true;
}

// How a block's threads lie over its tile of CH channels: lanes of V = 4 channels, or of one (rows that
// start on no 16 bytes), the warp's other lanes along the tokens.
template <int V, int ELEMS, int CH> struct Tile {
    static constexpr int LC = CH / V;           // lanes along the channels
    static constexpr int TL = 32 / LC;          // runs in a warp
    static constexpr int R = ELEMS / V;         // tokens of a run
    static constexpr int TOK = WT * TL * R;     // tokens of a block
    int warp, lane_t, c;                        // warp, run in the warp, first channel in the block
    __device__ __forceinline__ Tile() : warp(threadIdx.x >> 5), lane_t((threadIdx.x & 31) / LC),
                                        c(((threadIdx.x & 31) % LC) * V) {}
    __device__ __forceinline__ int first_token() const { return (warp * TL + lane_t) * R; }
};

// Tiles whose rows start anywhere.  A tensor copy starts on 16 bytes, a row of odd length does not;
// but every P-th row has the same offset from 16 bytes, P = 16 / sizeof(T).  So the map takes P rows
// as one long row, and a tile comes in P copies, one for the tokens of each offset, each a few
// elements wider than the channels and started at the 16 bytes before them: slot q holds the
// tile's tokens q, q + P, .. .  The last B * T mod 8 rows, which no whole long row holds, are
// read from global memory.
template <typename T, int TOK, int CH> struct Phases {
    static constexpr int P = 16 / (int)sizeof(T), W = CH + P, ROWS = TOK / P;
    alignas(128) T v[P][ROWS][W];
    static __device__ __forceinline__ int lead(const void* base) { return (int)(reinterpret_cast<uintptr_t>(base) % 16 / sizeof(T)); }
    // Elements from the map's start to the first channel of the tile's token q (its row n0 + q).
    static __device__ __forceinline__ long long start(const void* base, long long row, int c0, long long n0, int q) {
        return lead(base) + (long long)((n0 + q) % P) * row + c0;
    }
    __device__ __forceinline__ void copy(int q, const void* base, long long row, int c0, long long n0,
                                         const CUtensorMap* map, uint64_t* bar) {
        const long long e = start(base, row, c0, n0, q);
        tc::tma_load_4d(smem_addr(v[q]), map, (int)(e - e % P), 0, (int)((n0 + q) / P), 0, bar);
    }
};
// R tokens of one lane's channel: tile tokens i0 .. (a multiple of P), row n0 of the tensor first.
// skew[q]: where slot q's rows hold the lane's channel.
template <typename T, int TOK, int CH, int R>
__device__ __forceinline__ void read_run(const Phases<T, TOK, CH>& ph, const int (&skew)[16 / sizeof(T)], int i0, float (&v)[R][1]) {
    constexpr int P = Phases<T, TOK, CH>::P;
#pragma unroll
    for (int r = 0; r < R; ++r) v[r][0] = ld_f32(&ph.v[r % P][(i0 + r) / P][skew[r % P]]);
}
template <typename T, int TOK, int CH>
__device__ __forceinline__ void skews(const Phases<T, TOK, CH>& ph, const void* base, long long row, int c0, long long n0,
                                      int c, int (&skew)[16 / sizeof(T)]) {
#pragma unroll
    for (int q = 0; q < ph.P; ++q) skew[q] = (int)(ph.start(base, row, c0, n0, q) % ph.P) + c;
}
template <typename T, int R>
__device__ __forceinline__ void read_run_global(const T* src, long long row, int have, int limit, float (&v)[R][1]) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r][0] = r < have && GDR_INB(r < limit, 804) ? ld_f32(src + r * row) : 0.f;
}

// Compose a warp's runs: in (A, H) of this thread's run; out the composition of the runs before
// it (ex_*) and, in the warp's last run's lanes, of all of them (A, H).  UP = false: from the end.
template <int V, int LC, int TL, bool UP>
__device__ __forceinline__ void warp_runs(float (&A)[V], float (&H)[V], float (&exA)[V], float (&exH)[V], int lane_t) {
    const int at = UP ? lane_t : TL - 1 - lane_t;
#pragma unroll
    for (int o = 1; o < TL; o <<= 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = UP ? __shfl_up_sync(0xffffffffu, A[i], o * LC) : __shfl_down_sync(0xffffffffu, A[i], o * LC);
            const float h = UP ? __shfl_up_sync(0xffffffffu, H[i], o * LC) : __shfl_down_sync(0xffffffffu, H[i], o * LC);
            if (at >= o) { H[i] = fmaf(A[i], h, H[i]); A[i] *= a; }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (TL > 1) {
            const float a = UP ? __shfl_up_sync(0xffffffffu, A[i], LC) : __shfl_down_sync(0xffffffffu, A[i], LC);
            const float h = UP ? __shfl_up_sync(0xffffffffu, H[i], LC) : __shfl_down_sync(0xffffffffu, H[i], LC);
            exA[i] = at > 0 ? a : 1.f;
            exH[i] = at > 0 ? h : 0.f;
        } else {
            exA[i] = 1.f; exH[i] = 0.f;
        }
    }
}

// The state before every warp's runs, along the scan's direction, by one warp (lane = channel).
// agg: the block's warps' (A, H); carry: the state at the cluster's turn start, which every block
// holds alike and moves on by the turn.  xch and bars hold two turns' worth: a block sends turn
// k + 2's only when it has turn k + 1's from every peer, each of which sent it behind its last
// read of turn k's.  lost: a wait ran out (status word); the block goes on without waiting.
template <bool UP, int CH>
__device__ __forceinline__ void warp_starts(const float2 (*agg)[CH], float2 (*xch)[CH], uint64_t* bars,
                                            float (*start)[CH], float& carry, bool& lost, int k, int rank, int ncl) {
    const int c = threadIdx.x & 31;
    if (CH < 32 && c >= CH) return;
    float2 e[WT];
#pragma unroll
    for (int w = 0; w < WT; ++w) e[w] = agg[UP ? w : WT - 1 - w][c];
    float s = carry;
    if (ncl > 1) {
        float A = 1.f, H = 0.f;
#pragma unroll
        for (int w = 0; w < WT; ++w) { H = fmaf(e[w].x, H, e[w].y); A *= e[w].x; }
        xch += (k & 1) * ncl;
        uint64_t* bar = bars + (k & 1);
        if (c == 0) expect_bytes(bar, (uint32_t)(ncl * CH * sizeof(float2)));
        for (int r = 0; r < ncl; ++r) store_peer(&xch[rank][c], make_float2(A, H), bar, r);
        if (!lost) lost = !wait_phase(bar, (uint32_t)(k >> 1) & 1u);
        float all = carry;
        for (int i = 0; i < ncl; ++i) {
            const int r = UP ? i : ncl - 1 - i;
            if (r == rank) s = all;
            const float2 x = xch[r][c];
            all = fmaf(x.x, all, x.y);
        }
        carry = all;
    }
#pragma unroll
    for (int w = 0; w < WT; ++w) {
        start[UP ? w : WT - 1 - w][c] = s;
        s = fmaf(e[w].x, s, e[w].y);
    }
    if (ncl == 1) carry = s;
}

// Before the first turn: the barriers (n of them), and the peers' shared memory exists.
__device__ __forceinline__ void barriers_begin(uint64_t* bars, int n, int ncl) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < n; ++i) tc::mbar_init(&bars[i], 1);
        tc::fence_mbar_init();
    }
    if (ncl > 1) cluster_sync();
    else __syncthreads();
}

// The state before this thread's run: its warp's start through the runs before it.
template <int V>
__device__ __forceinline__ void run_start(const float* start, const float (&exA)[V], const float (&exH)[V], float (&s)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = fmaf(exA[i], start[i], exH[i]);
}

// A tile in shared memory.
template <typename T, int TOK, int CH> struct Rows {
    alignas(128) T v[TOK][CH];
    __device__ __forceinline__ void copy(const CUtensorMap* map, int c0, int t, int b, uint64_t* bar) {
#pragma unroll
        for (int r = 0; r < TOK; r += BOX_ROWS) tc::tma_load_4d(smem_addr(v[r]), map, c0, 0, t + r, b, bar);
    }
};
template <typename T, int V, int TOK, int CH> using TileOf = std::conditional_t<(V > 1), Rows<T, TOK, CH>, Phases<T, TOK, CH>>;

// The tensor maps of a call.
struct ScanMaps { CUtensorMap x, g, dh; };

template <int V> constexpr int fwd_elems() { return V > 1 ? 32 : 16; }  // of a thread: 2 registers each
constexpr int BWD_ELEMS = 16;                                           // 5 registers each

template <typename XT, typename GT, int V, int CH> struct FwdSmem {
    static constexpr int TOK = Tile<V, fwd_elems<V>(), CH>::TOK;
    TileOf<GT, V, TOK, CH> g[STAGES];
    TileOf<XT, V, TOK, CH> x[STAGES];
    float2 agg[WT][CH];
    float start[WT][CH];
    uint64_t bars[2 + STAGES];          // the exchange's, the stages'
};
// Behind it: xch [2][cluster][CH].

template <typename XT, typename GT, typename OT, int V, int CH>
__global__ void __launch_bounds__(NT, V > 1 ? 2 : 3) scan_fwd_kernel(ScanParams p, const __grid_constant__ ScanMaps maps) {
    using L = Tile<V, fwd_elems<V>(), CH>;
    using S = FwdSmem<XT, GT, V, CH>;
    constexpr int R = L::R;
    extern __shared__ __align__(128) unsigned char raw[];
    const L l;
    const int rank = (int)cluster_rank(), ncl = (int)cluster_size();
    S& sm = *reinterpret_cast<S*>(raw);
    float2 (*const xch)[CH] = reinterpret_cast<float2 (*)[CH]>(&sm + 1);
    const int b = blockIdx.x / ncl, c0 = blockIdx.y * CH, c = c0 + l.c;
    const bool on = c < p.D;                              // V divides D, or V = 1
    const int len = seq_len(p, b), nck = (p.T + CKPT - 1) / CKPT;
    const XT* x = static_cast<const XT*>(p.x) + (size_t)b * p.T * p.x_row + c;
    const GT* g = static_cast<const GT*>(p.g) + (size_t)b * p.T * p.g_row + c;
    OT* h = static_cast<OT*>(p.h) + (size_t)b * p.T * p.D + c;
    const int turn = L::TOK * ncl, turns = (p.T + turn - 1) / turn;
    const int tile = rank * L::TOK, first = tile + l.first_token();     // of turn 0: this block's, this thread's
    bool lost = false;

    barriers_begin(sm.bars, 2 + STAGES, ncl);
    auto fetch = [&](int k) {                             // turn k's tile, unless it lies behind the sequence
        const int t = k * turn + tile, st = k % STAGES;
        if (l.warp != 0 || k >= turns || t >= len) return;
        uint64_t* bar = &sm.bars[2 + st];
        const int lane = threadIdx.x & 31;
        if constexpr (V > 1) {
            if (lane != 0) return;
            expect_bytes(bar, sizeof(sm.g[0]) + sizeof(sm.x[0]));
            sm.g[st].copy(&maps.g, c0, t, b, bar);
            sm.x[st].copy(&maps.x, c0, t, b, bar);
        } else if (p.covered > 0) {
            if (lane == 0) expect_bytes(bar, sizeof(sm.g[0]) + sizeof(sm.x[0]));
            __syncwarp();
            const long long n0 = (long long)b * p.T + t;
            if (lane < sm.g[0].P) sm.g[st].copy(lane, p.g, p.g_row, c0, n0, &maps.g, bar);
            else if (lane >= 16 && lane - 16 < sm.x[0].P) sm.x[st].copy(lane - 16, p.x, p.x_row, c0, n0, &maps.x, bar);
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch(k);

    int skew_g[V > 1 ? 1 : 16 / sizeof(GT)], skew_x[V > 1 ? 1 : 16 / sizeof(XT)];
    if constexpr (V == 1) {
        const long long n0 = (long long)b * p.T;          // tiles start a multiple of P tokens later
        skews(sm.g[0], p.g, p.g_row, c0, n0, l.c, skew_g);
        skews(sm.x[0], p.x, p.x_row, c0, n0, l.c, skew_x);
    }
    // of warp 0: the state at the turn's start, of the lane's channel
    const int lane_c = c0 + (int)(threadIdx.x & 31);
    const bool lane_on = l.warp == 0 && (int)(threadIdx.x & 31) < CH && lane_c < p.D;
    float carry = 0.f;
    if (lane_on && p.h0) carry = p.h0[(size_t)b * p.D + lane_c];

    for (int k = 0; k < turns; ++k) {
        const int t0 = k * turn + first;
        float a[R][V], bb[R][V], A[V], H[V], exA[V], exH[V];
        if (k * turn + tile < len) {
            const int st = k % STAGES;
            if ((V > 1 || p.covered > 0) && !lost) lost = !wait_phase(&sm.bars[2 + st], (uint32_t)(k / STAGES) & 1u);
            if constexpr (V > 1) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int t = l.first_token() + r;
                    Pack<GT, V>::get(*reinterpret_cast<const typename Pack<GT, V>::Raw*>(&sm.g[st].v[t][l.c]), a[r]);
                    Pack<XT, V>::get(*reinterpret_cast<const typename Pack<XT, V>::Raw*>(&sm.x[st].v[t][l.c]), bb[r]);
                }
            } else if ((long long)b * p.T + t0 + R <= p.covered) {
                read_run(sm.g[st], skew_g, l.first_token(), a);
                read_run(sm.x[st], skew_x, l.first_token(), bb);
            } else {
                read_run_global(g + t0 * p.g_row, p.g_row, on ? len - t0 : 0, p.T - t0, a);
                read_run_global(x + t0 * p.x_row, p.x_row, on ? len - t0 : 0, p.T - t0, bb);
            }
        }
        with_mode(p, [&](auto mode, auto tied) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float rest = 1.f;
                    decay_pair<mode.value, tied.value>(a[r][i], a[r][i], rest);
                    if (tied.value) bb[r][i] *= rest;
                }
            }
        });
        const bool whole = t0 + R <= len;
        if (!whole) {                                     // tokens behind the end keep the state
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (t0 + r >= len) { a[r][i] = 1.f; bb[r][i] = 0.f; }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) { A[i] = a[0][i]; H[i] = bb[0][i]; }
#pragma unroll
        for (int r = 1; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                H[i] = fmaf(a[r][i], H[i], bb[r][i]);
                A[i] *= a[r][i];
            }
        }
        warp_runs<V, L::LC, L::TL, true>(A, H, exA, exH, l.lane_t);
        if (l.lane_t == L::TL - 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) sm.agg[l.warp][l.c + i] = make_float2(A[i], H[i]);
        }
        __syncthreads();
        fetch(k + STAGES);                           // the stage of turn k is in registers
        if (l.warp == 0) warp_starts<true, CH>(sm.agg, xch, sm.bars, sm.start, carry, lost, k, rank, ncl);
        __syncthreads();
        float s[V];
        run_start<V>(&sm.start[l.warp][l.c], exA, exH, s);
        if (on && p.ckpt && t0 % CKPT == 0 && t0 < p.T) {
            float* ck = p.ckpt + ((size_t)b * nck + t0 / CKPT) * p.D + c;
            if (GDR_INB(t0 / CKPT < nck && c + V <= p.D, 801))
                *reinterpret_cast<typename Pack<float, V>::Raw*>(ck) = Pack<float, V>::put(s);
        }
        OT* out = h + (size_t)t0 * p.D;
        if (on && whole) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = fmaf(a[r][i], s[i], bb[r][i]);
                if (GDR_INB(t0 + r < p.T && c + V <= p.D, 802))
                    *reinterpret_cast<typename Pack<OT, V>::Raw*>(out) = Pack<OT, V>::put(s);
                out += p.D;
            }
        } else if (on) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = fmaf(a[r][i], s[i], bb[r][i]);
                    o[i] = t0 + r < len ? s[i] : 0.f;
                }
                if (t0 + r < p.T && GDR_INB(c + V <= p.D, 803))
                    *reinterpret_cast<typename Pack<OT, V>::Raw*>(out) = Pack<OT, V>::put(o);
                out += p.D;
            }
        }
    }
    if (ncl > 1) cluster_sync_relaxed();                  // no peer still sends here
    if (p.h_T && rank == 0 && lane_on) p.h_T[(size_t)b * p.D + lane_c] = carry;
}

template <typename XT, typename GT, typename OT, int V, int CH> struct BwdSmem {
    static constexpr int TOK = Tile<V, BWD_ELEMS, CH>::TOK;
    TileOf<GT, V, TOK, CH> g[STAGES];
    TileOf<XT, V, TOK, CH> x[STAGES];
    TileOf<OT, V, TOK, CH> dh[STAGES];
    float2 up[WT][CH];
    float2 down[WT][CH];
    float before[WT][CH];
    float start[WT][CH];
    uint64_t bars[2 + STAGES];
};

// The states inside a tile come from the checkpoint at its first token (a tile is a whole number of
// CKPT tokens), so only the gradient's direction goes through the cluster.
template <typename XT, typename GT, typename OT, int V, int CH>
__global__ void __launch_bounds__(NT, 2) scan_bwd_kernel(ScanParams p, const __grid_constant__ ScanMaps maps) {
    using L = Tile<V, BWD_ELEMS, CH>;
    using S = BwdSmem<XT, GT, OT, V, CH>;
    constexpr int R = L::R;
    static_assert(L::TOK % CKPT == 0, "a tile starts at a checkpoint");
    extern __shared__ __align__(128) unsigned char raw[];
    const L l;
    const int rank = (int)cluster_rank(), ncl = (int)cluster_size();
    S& sm = *reinterpret_cast<S*>(raw);
    float2 (*const xch)[CH] = reinterpret_cast<float2 (*)[CH]>(&sm + 1);
    const int b = blockIdx.x / ncl, c0 = blockIdx.y * CH, c = c0 + l.c;
    const bool on = c < p.D;
    const int len = seq_len(p, b), nck = (p.T + CKPT - 1) / CKPT;
    const XT* x = static_cast<const XT*>(p.x) + (size_t)b * p.T * p.x_row + c;
    const GT* g = static_cast<const GT*>(p.g) + (size_t)b * p.T * p.g_row + c;
    const OT* dh = static_cast<const OT*>(p.dh) + (size_t)b * p.T * p.D + c;
    XT* dx = static_cast<XT*>(p.dx) + (size_t)b * p.T * p.D + c;
    GT* dg = static_cast<GT*>(p.dg) + (size_t)b * p.T * p.D + c;
    const int turn = L::TOK * ncl, turns = (p.T + turn - 1) / turn;
    const int tile = rank * L::TOK, first = tile + l.first_token();
    const bool with_dh = p.dh != nullptr;
    bool lost = false;

    barriers_begin(sm.bars, 2 + STAGES, ncl);
    // turn k walks from the end: its tokens start at (turns - 1 - k) * turn.  Tiles behind the
    // sequence are not fetched, so the stages count the fetched ones, from turn `skip` on.
    const int live = (len - tile + turn - 1) / turn;      // turns of this block with tokens (len > tile), else <= 0
    const int skip = turns - max(live, 0);
    auto fetch = [&](int k) {
        if (l.warp != 0 || k < skip || k >= turns) return;
        const int t = (turns - 1 - k) * turn + tile, st = (k - skip) % STAGES, lane = threadIdx.x & 31;
        uint64_t* bar = &sm.bars[2 + st];
        const uint32_t bytes = sizeof(sm.g[0]) + sizeof(sm.x[0]) + (with_dh ? sizeof(sm.dh[0]) : 0);
        if constexpr (V > 1) {
            if (lane != 0) return;
            expect_bytes(bar, bytes);
            sm.g[st].copy(&maps.g, c0, t, b, bar);
            sm.x[st].copy(&maps.x, c0, t, b, bar);
            if (with_dh) sm.dh[st].copy(&maps.dh, c0, t, b, bar);
        } else if (p.covered > 0) {
            if (lane == 0) expect_bytes(bar, bytes);
            __syncwarp();
            const long long n0 = (long long)b * p.T + t;
            if (lane < sm.g[0].P) sm.g[st].copy(lane, p.g, p.g_row, c0, n0, &maps.g, bar);
            else if (lane >= 8 && lane - 8 < sm.x[0].P) sm.x[st].copy(lane - 8, p.x, p.x_row, c0, n0, &maps.x, bar);
            else if (with_dh && lane >= 16 && lane - 16 < sm.dh[0].P) sm.dh[st].copy(lane - 16, p.dh, p.D, c0, n0, &maps.dh, bar);
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch(skip + k);

    int skew_g[V > 1 ? 1 : 16 / sizeof(GT)], skew_x[V > 1 ? 1 : 16 / sizeof(XT)],
        skew_d[V > 1 ? 1 : 16 / sizeof(OT)];
    if constexpr (V == 1) {
        const long long n0 = (long long)b * p.T;
        skews(sm.g[0], p.g, p.g_row, c0, n0, l.c, skew_g);
        skews(sm.x[0], p.x, p.x_row, c0, n0, l.c, skew_x);
        skews(sm.dh[0], p.dh, p.D, c0, n0, l.c, skew_d);
    }
    // of warp 0: a_{t+1} lam_{t+1} behind the turn, of the lane's channel
    const int lane_c = c0 + (int)(threadIdx.x & 31);
    const bool lane_on = l.warp == 0 && (int)(threadIdx.x & 31) < CH && lane_c < p.D;
    float carry = 0.f;
    if (lane_on && p.dh_T) carry = p.dh_T[(size_t)b * p.D + lane_c];

    for (int k = 0; k < turns; ++k) {
        const int base = (turns - 1 - k) * turn, t0 = base + first;
        // of warp 1: the state before the tile
        float state = 0.f;
        if (l.warp == 1) {
            const int j = (base + tile) / CKPT;
            if (j < nck && lane_c < p.D && GDR_INB(j >= 0 && b < p.B, 812)) state = p.ckpt[((size_t)b * nck + j) * p.D + lane_c];
        }
        float a[R][V], rest[R][V], xv[R][V], d[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) d[r][i] = 0.f;
        if (k >= skip) {
            const int st = (k - skip) % STAGES;
            if ((V > 1 || p.covered > 0) && !lost) lost = !wait_phase(&sm.bars[2 + st], (uint32_t)((k - skip) / STAGES) & 1u);
            if constexpr (V > 1) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int t = l.first_token() + r;
                    Pack<GT, V>::get(*reinterpret_cast<const typename Pack<GT, V>::Raw*>(&sm.g[st].v[t][l.c]), a[r]);
                    Pack<XT, V>::get(*reinterpret_cast<const typename Pack<XT, V>::Raw*>(&sm.x[st].v[t][l.c]), xv[r]);
                    if (with_dh) Pack<OT, V>::get(*reinterpret_cast<const typename Pack<OT, V>::Raw*>(&sm.dh[st].v[t][l.c]), d[r]);
                }
            } else if ((long long)b * p.T + t0 + R <= p.covered) {
                read_run(sm.g[st], skew_g, l.first_token(), a);
                read_run(sm.x[st], skew_x, l.first_token(), xv);
                if (with_dh) read_run(sm.dh[st], skew_d, l.first_token(), d);
            } else {
                const int have = on ? len - t0 : 0;
                read_run_global(g + t0 * p.g_row, p.g_row, have, p.T - t0, a);
                read_run_global(x + t0 * p.x_row, p.x_row, have, p.T - t0, xv);
                if (with_dh) read_run_global(dh + (size_t)t0 * p.D, p.D, have, p.T - t0, d);
            }
        }
        float A[V], H[V], M[V], dA[V], exA[V], exH[V], exD[V], exM[V];
        // rest: 1 - a
        with_mode(p, [&](auto mode, auto tied) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    rest[r][i] = 0.f;
                    decay_pair<mode.value, mode.value == 1 || tied.value>(a[r][i], a[r][i], rest[r][i]);
                }
            }
        });
        const bool whole = t0 + R <= len;
        if (!whole) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (t0 + r >= len) { a[r][i] = 1.f; rest[r][i] = 0.f; xv[r][i] = 0.f; d[r][i] = 0.f; }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) { A[i] = 1.f; H[i] = 0.f; M[i] = 0.f; }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                H[i] = fmaf(a[r][i], H[i], p.tied ? rest[r][i] * xv[r][i] : xv[r][i]);
                A[i] *= a[r][i];
            }
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
#pragma unroll
            for (int i = 0; i < V; ++i) M[i] = a[r][i] * (d[r][i] + M[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) dA[i] = A[i];
        warp_runs<V, L::LC, L::TL, true>(A, H, exA, exH, l.lane_t);
        warp_runs<V, L::LC, L::TL, false>(dA, M, exD, exM, l.lane_t);
        if (l.lane_t == L::TL - 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) sm.up[l.warp][l.c + i] = make_float2(A[i], H[i]);
        }
        if (l.lane_t == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) sm.down[l.warp][l.c + i] = make_float2(dA[i], M[i]);
        }
        __syncthreads();
        if (k >= skip) fetch(k + STAGES);            // the stage of turn k is in registers
        if (l.warp == 0) warp_starts<false, CH>(sm.down, xch, sm.bars, sm.start, carry, lost, k, rank, ncl);
        else if (l.warp == 1) warp_starts<true, CH>(sm.up, nullptr, nullptr, sm.before, state, lost, k, 0, 1);
        __syncthreads();
        float s[V], m[V], before[R][V];
        run_start<V>(&sm.before[l.warp][l.c], exA, exH, s);
        run_start<V>(&sm.start[l.warp][l.c], exD, exM, m);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                before[r][i] = s[i];
                s[i] = fmaf(a[r][i], s[i], p.tied ? rest[r][i] * xv[r][i] : xv[r][i]);
            }
        }
        // the gradient of the gate: lam (h_{t-1} - [tied] x) a', a' = a or -a (1 - a)
        XT* out_x = dx + (size_t)(t0 + R - 1) * p.D;
        GT* out_g = dg + (size_t)(t0 + R - 1) * p.D;
        with_mode(p, [&](auto mode, auto tied) {
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                float ox[V], og[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float lam = d[r][i] + m[i];
                    m[i] = a[r][i] * lam;
                    ox[i] = tied.value ? rest[r][i] * lam : lam;
                    const float da = m[i] * (tied.value ? before[r][i] - xv[r][i] : before[r][i]);
                    og[i] = mode.value == 1 ? -da * rest[r][i] : da;
                }
                if (!whole && t0 + r >= len) {
#pragma unroll
                    for (int i = 0; i < V; ++i) ox[i] = og[i] = 0.f;
                }
                if (on && t0 + r < p.T && GDR_INB(c + V <= p.D, 811)) {
                    *reinterpret_cast<typename Pack<XT, V>::Raw*>(out_x) = Pack<XT, V>::put(ox);
                    *reinterpret_cast<typename Pack<GT, V>::Raw*>(out_g) = Pack<GT, V>::put(og);
                }
                out_x -= p.D;
                out_g -= p.D;
            }
        });
    }
    if (ncl > 1) cluster_sync_relaxed();
    if (p.dh0 && rank == 0 && lane_on) p.dh0[(size_t)b * p.D + lane_c] = carry;
}

// One token per sequence: elementwise, V channels per thread.
template <typename XT, typename GT, typename OT, int V>
__global__ void __launch_bounds__(NT) scan_step_kernel(ScanParams p) {
    const int per = p.D / V;                              // V divides D
    const size_t n = (size_t)p.B * per;
    for (size_t i = (size_t)blockIdx.x * NT + threadIdx.x; i < n; i += (size_t)gridDim.x * NT) {
        const size_t b = i / per, c = (i % per) * V;
        float a[V], x[V], s[V];
        Pack<GT, V>::get(*reinterpret_cast<const typename Pack<GT, V>::Raw*>(static_cast<const GT*>(p.g) + b * p.g_row + c), a);
        Pack<XT, V>::get(*reinterpret_cast<const typename Pack<XT, V>::Raw*>(static_cast<const XT*>(p.x) + b * p.x_row + c), x);
        typename Pack<float, V>::Raw* h = reinterpret_cast<typename Pack<float, V>::Raw*>(p.h_T + b * p.D + c);
        if (!GDR_INB(b < (size_t)p.B && c + V <= (size_t)p.D, 821)) break;
        Pack<float, V>::get(*h, s);
        with_mode(p, [&](auto mode, auto tied) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float dec, rest = 1.f;
                decay_pair<mode.value, tied.value>(a[j], dec, rest);
                s[j] = fmaf(dec, s[j], tied.value ? rest * x[j] : x[j]);
            }
        });
        *h = Pack<float, V>::put(s);
        if (p.h) *reinterpret_cast<typename Pack<OT, V>::Raw*>(static_cast<OT*>(p.h) + b * p.D + c) = Pack<OT, V>::put(s);
    }
}

}  // namespace scn
}  // namespace gdr
