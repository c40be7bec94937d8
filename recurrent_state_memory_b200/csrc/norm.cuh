// norm.cuh -- layer norm kernels.
//
// Mathematics.  Forward: mean, then the variance of the centred values (two sums over registers,
// so that rows far from zero lose nothing), y = (x - mean) rstd w + b.  Backward, with
// xh = (x - mean) rstd: dx = rstd (w dy - c1 - xh c2), c1 = mean(w dy), c2 = mean(w dy xh);
// dweight = sum over rows of dy xh, dbias of dy.
//
// Bound: HBM; x (and dy) are read once and y (dx) written once.
//
// Split.  A row belongs to a group of lanes that holds all of it in registers, 16 bytes a lane and
// load: G = 1 .. 32 lanes of a warp (several rows per warp), or a whole block of 64 to 1024 threads
// for rows longer than a warp's registers.  Groups walk the rows with the grid's stride, and the grid
// is what the GPU holds at once; the next row's loads are in flight while a row is reduced.  Rows
// that do not start on 16 bytes are taken in the tensor's 16-byte chunks or one by one (a pointer
// off, or where the dispatch measured that better).  Rows beyond a block's registers are read again
// from L2 instead.
//
// The gradients of weight and bias: a lane's columns are the same for all of its rows, so it sums
// them in registers; a block adds its groups' sums in a fixed order and writes one partial row,
// and a second launch adds the partial rows, again in a fixed order (no atomics: the same bits
// every time).
#pragma once

#include "common.cuh"

namespace gdr {
namespace lnm {

struct NormParams {
    long long rows;
    int D;
    float eps;
    const void* x;
    const void* dy;
    const void* weight;
    const void* bias;
    void* y;
    void* dx;
    float* mean;
    float* rstd;
    float* part_w;          // [parts, D] each block's share of dweight / dbias
    float* part_b;
    float* dweight;
    float* dbias;
    int parts;
    int w_bf16;             // weight and bias are bf16 (else fp32)
};

// A lane's V elements: pairs, or one value.
template <int V> struct Vals {
    static constexpr int H = V / 2;
    Pair v[H];
    __device__ __forceinline__ void all(float x) {
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = pair(x, x);
    }
    __device__ __forceinline__ float total() const {
        Pair s = v[0];
#pragma unroll
        for (int i = 1; i < H; ++i) s = s + v[i];
        return lo(s) + hi(s);
    }
    __device__ __forceinline__ void set(int i, float x) { v[i / 2] = i & 1 ? pair(lo(v[i / 2]), x) : pair(x, hi(v[i / 2])); }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? hi(v[i / 2]) : lo(v[i / 2]); }
};
template <> struct Vals<1> {
    float v;
    __device__ __forceinline__ void all(float x) { v = x; }
    __device__ __forceinline__ float total() const { return v; }
    __device__ __forceinline__ void set(int, float x) { v = x; }
    __device__ __forceinline__ float get(int) const { return v; }
};
template <int V> __device__ __forceinline__ Vals<V> operator+(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> d;
    if constexpr (V == 1) d.v = a.v + b.v;
    else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) d.v[i] = a.v[i] + b.v[i];
    }
    return d;
}
template <int V> __device__ __forceinline__ Vals<V> operator*(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> d;
    if constexpr (V == 1) d.v = a.v * b.v;
    else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) d.v[i] = a.v[i] * b.v[i];
    }
    return d;
}
template <int V> __device__ __forceinline__ Vals<V> fma(const Vals<V>& a, const Vals<V>& b, const Vals<V>& c) {
    Vals<V> d;
    if constexpr (V == 1) d.v = fmaf(a.v, b.v, c.v);
    else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) d.v[i] = fma(a.v[i], b.v[i], c.v[i]);
    }
    return d;
}

// V consecutive elements as they lie in memory (one access of 16 bytes or less, or two), and as fp32.
template <typename T, int V> struct Raw {
    static constexpr int BYTES = V * (int)sizeof(T), WORDS = BYTES < 4 ? 1 : BYTES / 4;
    unsigned w[WORDS];
    // ONCE: streamed (evicted first), for rows that are read once: 2 to 8 % of the kernels' time.
    template <bool ONCE = true> __device__ __forceinline__ void load(const T* p) {
        auto get = [](const auto* q) { return ONCE ? __ldcs(q) : *q; };
        if constexpr (BYTES == 32) {
            const uint4 a = get(reinterpret_cast<const uint4*>(p)), b = get(reinterpret_cast<const uint4*>(p) + 1);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        } else if constexpr (BYTES == 16) {
            const uint4 a = get(reinterpret_cast<const uint4*>(p));
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else if constexpr (BYTES == 8) {
            const uint2 a = get(reinterpret_cast<const uint2*>(p));
            w[0] = a.x; w[1] = a.y;
        } else if constexpr (BYTES == 4) {
            w[0] = get(reinterpret_cast<const unsigned*>(p));
        } else {
            w[0] = get(reinterpret_cast<const unsigned short*>(p));
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void ones(int c, int D) {                // ones where column c + i is in the row
        zero();
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((unsigned)(c + i) < (unsigned)D) w[i * (int)sizeof(T) / 4] |= sizeof(T) == 4 ? 0xffffffffu : i & 1 ? 0xffff0000u : 0xffffu;
    }
    __device__ __forceinline__ void operator&=(const Raw& m) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] &= m.w[i];
    }
    __device__ __forceinline__ void load_part(const T* p, int n) {      // the first n elements; the others 0
        zero();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= n) continue;
            if constexpr (sizeof(T) == 4) w[i] = *reinterpret_cast<const unsigned*>(p + i);
            else w[i / 2] |= (unsigned)*reinterpret_cast<const unsigned short*>(p + i) << (i & 1 ? 16 : 0);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ Vals<V> vals() const {
        Vals<V> x;
        if constexpr (V == 1) x.v = get(0);
        else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) x.v[i] = pair(get(2 * i), get(2 * i + 1));
        }
        return x;
    }
};
// V weights or biases from column c on.
template <typename WT, int V> __device__ __forceinline__ Vals<V> load_w(const void* p, int c) {
    Raw<WT, V> r;
    r.template load<false>(static_cast<const WT*>(p) + c);
    return r.vals();
}
// f(a value of the weights' type): the branch is taken once, not once a load.
template <typename F> __device__ __forceinline__ void with_weights(const NormParams& p, F f) {
    if (p.w_bf16) f(__nv_bfloat16());
    else f(0.f);
}
template <typename T, int V> __device__ __forceinline__ void store_v(T* p, const Vals<V>& v) {
    if constexpr (V == 1) {
        st_from_f32(p, v.v);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(v.get(i), v.get(i + 1), v.get(i + 2), v.get(i + 3));
    } else {
        unsigned w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v.get(2 * i), v.get(2 * i + 1));
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// Sums over a row's group of G lanes, n values at once: of a warp (G <= 32), or a block of G
// threads (sm: two sets of warp sums used in turn, so that one barrier a sum is enough).
template <int G, int MOST> struct Group {
    static constexpr int WARPS = G > 32 ? G / 32 : 1;
    float (*sm)[WARPS][MOST];           // [2]
    int turn;
    template <int n> __device__ __forceinline__ void sum(float (&v)[n]) {
        static_assert(n <= MOST, "values");
        if constexpr (G <= 32) {
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        } else {
            // four values: each exchange halves what a lane still adds, so that 6 exchanges do
            // the work of 20; lane l ends with value l & 3
            const int lane = threadIdx.x & 31;
            float (*s)[MOST] = sm[turn];
            turn ^= 1;
            if constexpr (n == 4) {
                const bool b0 = lane & 1, b1 = lane & 2;
                const float x0 = b0 ? v[0] : v[1], x1 = b0 ? v[2] : v[3];       // what the neighbour keeps
                float y0 = b0 ? v[1] : v[0], y1 = b0 ? v[3] : v[2];
                y0 += __shfl_xor_sync(0xffffffffu, x0, 1);
                y1 += __shfl_xor_sync(0xffffffffu, x1, 1);
                float z = b1 ? y1 : y0;
                z += __shfl_xor_sync(0xffffffffu, b1 ? y0 : y1, 2);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                if (lane < 4) s[threadIdx.x >> 5][lane] = z;
            } else {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < n; ++i) s[threadIdx.x >> 5][i] = v[i];
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
#pragma unroll
                for (int i = 0; i < n; ++i) v[i] += s[w][i];
        }
    }
};

constexpr int WARP_NT = 256;            // threads of a block of the warp kernels

// Threads of a block whose rows belong to G lanes each.
template <int G> constexpr int threads() { return G > 32 ? G : WARP_NT; }

// Blocks on an SM (and of the grid, which walks the rows): forward 1024 threads of 64 registers, 768
// of 80 where rows are shifted or two loads of pairs are held, 512 of 128 where a lane holds 16
// elements; backward 512 of 128.
template <bool SHIFT> __host__ __device__ constexpr int fwd_blocks(int V, int N, int threads) {
    const int most = V * N > 8 ? (threads <= 192 && !SHIFT ? 576 : 512) : SHIFT || (V > 1 && N > 1) ? 768 : 1024;
    return threads <= most ? most / threads : 1;
}
__host__ __device__ constexpr int bwd_blocks(int threads) { return threads <= 256 ? 512 / threads : 1; }

// Where this thread stands: its lane in its row's group, its (first) row in the first turn, the
// distance of a group's U rows of a turn, the rows of a turn of the grid, and the thread's first
// column.  Shifted: rows that do not start on 16 bytes.  Rows V apart start alike, so a group whose
// rows are multiples of V apart (the host makes the grid's groups one) still has columns of its own:
// its chunks are the tensor's 16-byte chunks, and the row begins and ends inside one.
template <int V, int G, int U, bool SHIFT> struct Place {
    static constexpr int PER = threads<G>() / G;      // groups of a block
    int lane, c0;
    long long row, dist, step;
    __device__ __forceinline__ Place(int D)
        : lane(threadIdx.x % G), row((long long)blockIdx.x * (SHIFT ? PER : PER * U) + threadIdx.x / G),
          dist(SHIFT ? (long long)gridDim.x * PER : PER), step((long long)gridDim.x * (PER * U)) {
        c0 = lane * V - (SHIFT ? (int)((unsigned long long)row * (unsigned)D % V) : 0);
    }
};
// A chunk with columns outside of the row.
template <int V, bool SHIFT> __device__ __forceinline__ bool ragged(int c, int D) { return SHIFT && (c < 0 || c + V > D); }
template <int V> __device__ __forceinline__ void only_row(Vals<V>& v, int c, int D) {
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((unsigned)(c + i) >= (unsigned)D) v.set(i, 0.f);
}
// Debug build: n elements from column c of row r on lie in the tensor; a chunk that begins there, in a
// shifted row perhaps outside of it, holds some of the row.
__device__ __forceinline__ bool in_tensor(const NormParams& p, long long r, int c, int n) {
    return r >= 0 && r < p.rows && r * p.D + c >= 0 && r * p.D + c + n <= p.rows * p.D;
}
template <int V, bool SHIFT> __device__ __forceinline__ bool in_row(const NormParams& p, long long r, int c) {
    return r >= 0 && r < p.rows && (SHIFT ? c + V > 0 && c < p.D : c >= 0 && c + V <= p.D);
}
// A row's last chunk at the tensor's end: left out of the loads ahead (a load within a branch would
// wait there), read by elements where it is used.  Elsewhere a chunk is read whole; its other
// columns are the neighbouring rows'.
template <int V, bool SHIFT> __device__ __forceinline__ bool at_end(int c, int D, bool last) { return SHIFT && last && c + V > D; }
template <bool SHIFT, typename T, int V> __device__ __forceinline__ void store_chunk(T* p, const Vals<V>& v, int c, int D) {
    if (ragged<V, SHIFT>(c, D)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((unsigned)(c + i) < (unsigned)D) st_from_f32(p + i, v.get(i));
    } else {
        store_v<T, V>(p, v);
    }
}
// Sums: the partial rows' starts are not shifted, so a shifted chunk has no alignment there.
template <bool SHIFT, int V> __device__ __forceinline__ void store_part(float* p, const Vals<V>& v, int c, int D) {
    if constexpr (SHIFT) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((unsigned)(c + i) < (unsigned)D) p[i] = v.get(i);
    } else {
        store_v<float, V>(p, v);
    }
}
// Weights or biases of a chunk; outside of the row: 0.
template <typename WT, int V, bool SHIFT> __device__ __forceinline__ Vals<V> load_chunk_w(const void* p, int c, int D) {
    if constexpr (SHIFT) {
        Vals<V> v;
#pragma unroll
        for (int i = 0; i < V; ++i) v.set(i, (unsigned)(c + i) < (unsigned)D ? load_w<WT, 1>(p, c + i).v : 0.f);
        return v;
    } else {
        return load_w<WT, V>(p, c);
    }
}

// Rows that a group takes per turn: two while a row is few registers, so that more loads are in
// flight and, in a block, two rows share a barrier.
template <int V, int N, int G> constexpr int rows_at_once() { return V * N <= (V == 1 ? 4 : 8) && G < 768 ? 2 : 1; }

// N loads of V elements per lane and row.
template <typename XT, typename YT, int V, int N, int G, bool SHIFT>
__global__ void __launch_bounds__(threads<G>(), fwd_blocks<SHIFT>(V, N, threads<G>())) norm_fwd_kernel(NormParams p) {
    constexpr int U = rows_at_once<V, N, G>();
    __shared__ __align__(16) float sm[2][G > 32 ? G / 32 : 1][U];
    const Place<V, G, U, SHIFT> at(p.D);
    Group<G, U> grp{sm, 0};
    const float inv = 1.f / (float)p.D;
    const int c0 = at.c0;                             // this lane's columns: c0 + j * G * V ..
    constexpr bool KEEP = V * N <= 16 && G < 1024;    // weights stay in registers
    Vals<V> w[KEEP ? N : 1], bi[KEEP ? N : 1];
    auto weights = [&](auto type, int j, Vals<V>& wv, Vals<V>& bv) {
        const int c = c0 + j * G * V;
        wv.all(1.f);
        bv.all(0.f);
        if (c < p.D) {
            if (p.weight) wv = load_chunk_w<decltype(type), V, SHIFT>(p.weight, c, p.D);
            if (p.bias) bv = load_chunk_w<decltype(type), V, SHIFT>(p.bias, c, p.D);
        }
    };
    if constexpr (KEEP) {
        with_weights(p, [&](auto type) {
#pragma unroll
            for (int j = 0; j < N; ++j) weights(type, j, w[j], bi[j]);
        });
    }
    const size_t jump = (size_t)at.step * p.D, next = (size_t)at.dist * p.D;
    const XT* x = static_cast<const XT*>(p.x) + (size_t)at.row * p.D + c0;      // the rows to fetch next
    YT* y = static_cast<YT*>(p.y) + (size_t)at.row * p.D + c0;
    Raw<XT, V> raw[U][N];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = c0 + j * G * V;
                if (r + u * at.dist < p.rows && c < p.D && !at_end<V, SHIFT>(c, p.D, r + u * at.dist == p.rows - 1)
                    GDR_AND_INB(in_tensor(p, r + u * at.dist, c, V), 902))
                    raw[u][j].load(x + u * next + j * G * V);
                else raw[u][j].zero();
            }
        x += jump;
    };
    // the chunks' elements that are the row's, as bits of the raw words and as ones of the values
    constexpr bool ONES = SHIFT && V * N <= 8;
    Raw<XT, V> mx[SHIFT ? N : 1];
    Vals<V> ones[ONES ? N : 1];
    if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            mx[j].ones(c0 + j * G * V, p.D);
            if constexpr (ONES) {
                ones[j].all(1.f);
                only_row(ones[j], c0 + j * G * V, p.D);
            }
        }
    }
    fetch(at.row);
    // every lane of a warp makes the same number of turns (the sums are warp-wide)
    const long long ahead = G > 32 ? 0 : (threadIdx.x & 31) / G;
    for (long long r = at.row; r - ahead < p.rows; r += at.step) {
        Vals<V> v[U][N], s;
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if constexpr (SHIFT) {
                    const int c = c0 + j * G * V;
                    if (c < p.D && at_end<V, SHIFT>(c, p.D, r + u * at.dist == p.rows - 1)
                        GDR_AND_INB(in_tensor(p, r + u * at.dist, c, p.D - c), 903))
                        raw[u][j].load_part(x - jump + u * next + j * G * V, p.D - c);
                    raw[u][j] &= mx[j];
                }
                v[u][j] = raw[u][j].vals();
                s = j ? s + v[u][j] : v[u][j];
            }
            mean[u] = s.total();
        }
        fetch(r + at.step);
        grp.sum(mean);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] *= inv;
            Vals<V> off;
            off.all(-mean[u]);
            s.all(0.f);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if constexpr (ONES) {
                    v[u][j] = fma(ones[j], off, v[u][j]);
                } else {
                    v[u][j] = v[u][j] + off;
                    if (ragged<V, SHIFT>(c0 + j * G * V, p.D)) only_row(v[u][j], c0 + j * G * V, p.D);
                }
                if (c0 + j * G * V < p.D) s = fma(v[u][j], v[u][j], s);
            }
            rstd[u] = s.total();
        }
        grp.sum(rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + u * at.dist >= p.rows) continue;
            rstd[u] = rsqrtf(rstd[u] * inv + p.eps);
            Vals<V> rs;
            rs.all(rstd[u]);
            auto put = [&](int j, const Vals<V>& wv, const Vals<V>& bv) {
                const Vals<V> o = fma(v[u][j] * rs, wv, bv);
                if (c0 + j * G * V < p.D && GDR_INB((in_row<V, SHIFT>(p, r + u * at.dist, c0 + j * G * V)), 901))
                    store_chunk<SHIFT>(y + u * next + j * G * V, o, c0 + j * G * V, p.D);
            };
            if constexpr (KEEP) {
#pragma unroll
                for (int j = 0; j < N; ++j) put(j, w[j], bi[j]);
            } else {
                with_weights(p, [&](auto type) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        Vals<V> wv, bv;
                        weights(type, j, wv, bv);
                        put(j, wv, bv);
                    }
                });
            }
            if (at.lane == 0) {
                if (p.mean) p.mean[r + u * at.dist] = mean[u];
                if (p.rstd) p.rstd[r + u * at.dist] = rstd[u];
            }
        }
        y += jump;
    }
}

// Backward: dx, and the block's share of dweight and dbias.
template <typename XT, typename YT, int V, int N, int G, bool SHIFT>
__global__ void __launch_bounds__(threads<G>(), bwd_blocks(threads<G>())) norm_bwd_kernel(NormParams p) {
    constexpr int U = rows_at_once<V, N, G>();
    extern __shared__ float part[];                   // G <= 32: the groups' sums [PER][D], in turn
    __shared__ __align__(16) float sm[2][G > 32 ? G / 32 : 1][2 * U];
    const Place<V, G, U, SHIFT> at(p.D);
    Group<G, 2 * U> grp{sm, 0};
    const float inv = 1.f / (float)p.D;
    const int c0 = at.c0;
    static_assert(V * N <= 8, "weights, rows and sums in registers");
    Vals<V> w[N];
    with_weights(p, [&](auto type) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            w[j].all(1.f);
            if (c0 + j * G * V < p.D && p.weight)
                w[j] = load_chunk_w<decltype(type), V, SHIFT>(p.weight, c0 + j * G * V, p.D);
        }
    });
    Vals<V> sw[N], sb[N];
#pragma unroll
    for (int j = 0; j < N; ++j) { sw[j].all(0.f); sb[j].all(0.f); }
    const size_t jump = (size_t)at.step * p.D, next = (size_t)at.dist * p.D, start = (size_t)at.row * p.D + c0;
    const XT* x = static_cast<const XT*>(p.x) + start;
    const YT* dy = static_cast<const YT*>(p.dy) + start;
    XT* dx = static_cast<XT*>(p.dx) + start;
    Raw<XT, V> rx[U][N];
    Raw<YT, V> rd[U][N];
    float mean[U], rstd[U];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = r + u * at.dist < p.rows;
            mean[u] = in ? p.mean[r + u * at.dist] : 0.f;
            rstd[u] = in ? p.rstd[r + u * at.dist] : 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = c0 + j * G * V;
                if (in && c < p.D && !at_end<V, SHIFT>(c, p.D, r + u * at.dist == p.rows - 1)
                    GDR_AND_INB(in_tensor(p, r + u * at.dist, c, V), 913)) {
                    rx[u][j].load(x + u * next + j * G * V);
                    rd[u][j].load(dy + u * next + j * G * V);
                } else { rx[u][j].zero(); rd[u][j].zero(); }
            }
        }
        x += jump;
        dy += jump;
    };
    Raw<XT, V> mx[SHIFT ? N : 1];                      // the chunks' elements that are the row's
    Raw<YT, V> my[SHIFT ? N : 1];
    if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            mx[j].ones(c0 + j * G * V, p.D);
            my[j].ones(c0 + j * G * V, p.D);
        }
    }
    fetch(at.row);
    const long long ahead = G > 32 ? 0 : (threadIdx.x & 31) / G;
    for (long long r = at.row; r - ahead < p.rows; r += at.step) {
        Vals<V> xh[U][N], d[U][N];
        float here[U], c[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Vals<V> s1, s2, rs, off;
            here[u] = rstd[u];
            rs.all(rstd[u]);
            off.all(-mean[u]);
#pragma unroll
            for (int j = 0; j < N; ++j) {             // columns behind D: dy is zero
                if constexpr (SHIFT) {
                    const int c = c0 + j * G * V;
                    if (c < p.D && at_end<V, SHIFT>(c, p.D, r + u * at.dist == p.rows - 1)
                        GDR_AND_INB(in_tensor(p, r + u * at.dist, c, p.D - c), 914)) {
                        rx[u][j].load_part(x - jump + u * next + j * G * V, p.D - c);
                        rd[u][j].load_part(dy - jump + u * next + j * G * V, p.D - c);
                    }
                    rx[u][j] &= mx[j];
                    rd[u][j] &= my[j];
                }
                xh[u][j] = (rx[u][j].vals() + off) * rs;
                d[u][j] = rd[u][j].vals();
                sw[j] = fma(d[u][j], xh[u][j], sw[j]);
                sb[j] = sb[j] + d[u][j];
                d[u][j] = d[u][j] * w[j];
                s1 = j ? s1 + d[u][j] : d[u][j];
                s2 = j ? fma(d[u][j], xh[u][j], s2) : d[u][j] * xh[u][j];
            }
            c[2 * u] = s1.total();
            c[2 * u + 1] = s2.total();
        }
        fetch(r + at.step);
        if (p.dx) {
            grp.sum(c);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u * at.dist >= p.rows) continue;
                Vals<V> m1, m2, rs;
                rs.all(here[u]);
                m1.all(-c[2 * u] * inv);
                m2.all(-c[2 * u + 1] * inv);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const Vals<V> o = (d[u][j] + fma(xh[u][j], m2, m1)) * rs;
                    if (c0 + j * G * V < p.D && GDR_INB((in_row<V, SHIFT>(p, r + u * at.dist, c0 + j * G * V)), 911))
                        store_chunk<SHIFT>(dx + u * next + j * G * V, o, c0 + j * G * V, p.D);
                }
            }
            dx += jump;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");  // the sum's blocks may come; they wait for these stores
    const size_t base = (size_t)blockIdx.x * p.D;
    if constexpr (G > 32) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = c0 + j * G * V;
            if (!(c < p.D GDR_AND_INB((int)blockIdx.x < p.parts && (SHIFT || c + V <= p.D), 915))) continue;
            if (p.part_w) store_part<SHIFT>(p.part_w + base + c, sw[j], c, p.D);
            if (p.part_b) store_part<SHIFT>(p.part_b + base + c, sb[j], c, p.D);
        }
    } else {
        // the block's groups, added column by column in the groups' order
        const int g = threadIdx.x / G;
        for (int which = 0; which < 2; ++which) {
            float* to = which ? p.part_b : p.part_w;
            if (!to) continue;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = c0 + j * G * V;
                if (c < p.D GDR_AND_INB(g < at.PER && (SHIFT || c + V <= p.D), 916)) store_part<SHIFT>(part + (size_t)g * p.D + c, which ? sb[j] : sw[j], c, p.D);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.D; c += WARP_NT) {
                float s = 0.f;
                for (int i = 0; i < at.PER; ++i) s += part[(size_t)i * p.D + c];
                if (GDR_INB((int)blockIdx.x < p.parts, 917)) to[base + c] = s;
            }
        }
    }
}

// Backward of rows of up to 16384 elements by a block of 1024 threads: x and dy stay as they lie in
// memory in registers (64 a thread), the sums of dweight and dbias in shared memory, each thread's
// columns its own, and x hat and w dy are formed twice.  The next row is on its way into L2
// meanwhile.  (2048 rows of 16384 bf16: 83 us; by the three passes below 137.)
constexpr int WIDE_NT = 1024;
template <typename XT, typename YT, int V, int N>
__global__ void __launch_bounds__(WIDE_NT) norm_bwd_wide_kernel(NormParams p) {
    extern __shared__ __align__(16) float part[];      // the sums: dweight, then dbias, four of a thread at a time
    __shared__ __align__(16) float sm[2][WIDE_NT / 32][2];
    Group<WIDE_NT, 2> grp{sm, 0};
    const float inv = 1.f / (float)p.D;
    const int c0 = threadIdx.x * V;
    const bool sums = p.part_w || p.part_b;
    auto at = [&](int which, int j) { return part + ((which * N + j) * (V / 4) * WIDE_NT + threadIdx.x) * 4; };
    auto get = [&](int which, int j) {
        Vals<V> v;
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const float4 a = *reinterpret_cast<const float4*>(at(which, j) + h * WIDE_NT * 4);
            v.v[2 * h] = pair(a.x, a.y);
            v.v[2 * h + 1] = pair(a.z, a.w);
        }
        return v;
    };
    auto put = [&](int which, int j, const Vals<V>& v) {
#pragma unroll
        for (int h = 0; h < V / 4; ++h)
            *reinterpret_cast<float4*>(at(which, j) + h * WIDE_NT * 4) =
                make_float4(v.get(4 * h), v.get(4 * h + 1), v.get(4 * h + 2), v.get(4 * h + 3));
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c0 + j * WIDE_NT * V < p.D) f(j, j * WIDE_NT * V);
    };
    if (sums) {
        Vals<V> z;
        z.all(0.f);
        each([&](int j, int) { put(0, j, z); put(1, j, z); });
    }
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D + c0;
        const YT* dy = static_cast<const YT*>(p.dy) + (size_t)r * p.D + c0;
        const float mean = p.mean[r], rstd = p.rstd[r];
        Raw<XT, V> rx[N];
        Raw<YT, V> rd[N];
        each([&](int j, int c) { if (GDR_INB(c0 + c + V <= p.D, 918)) { rx[j].load(x + c); rd[j].load(dy + c); } });
        if (r + gridDim.x < p.rows) {
            const size_t next = (size_t)gridDim.x * p.D;
            each([&](int, int c) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(x + next + c));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(dy + next + c));
            });
        }
        Vals<V> off, rs, s1, s2;
        off.all(-mean);
        rs.all(rstd);
        s1.all(0.f);
        s2.all(0.f);
        with_weights(p, [&](auto type) {
            each([&](int j, int c) {
                const Vals<V> xh = (rx[j].vals() + off) * rs;
                Vals<V> d = rd[j].vals();
                if (sums) {
                    put(0, j, fma(d, xh, get(0, j)));
                    put(1, j, get(1, j) + d);
                }
                if (p.weight) d = d * load_w<decltype(type), V>(p.weight, c0 + c);
                s1 = s1 + d;
                s2 = fma(d, xh, s2);
            });
        });
        if (!p.dx) continue;
        float c12[2] = {s1.total(), s2.total()};
        grp.sum(c12);
        Vals<V> m1, m2;
        m1.all(-c12[0] * inv);
        m2.all(-c12[1] * inv);
        XT* dx = static_cast<XT*>(p.dx) + (size_t)r * p.D + c0;
        with_weights(p, [&](auto type) {
            each([&](int j, int c) {
                const Vals<V> xh = (rx[j].vals() + off) * rs;
                Vals<V> d = rd[j].vals();
                if (p.weight) d = d * load_w<decltype(type), V>(p.weight, c0 + c);
                if (GDR_INB(c0 + c + V <= p.D, 912)) store_v<XT, V>(dx + c, (d + fma(xh, m2, m1)) * rs);
            });
        });
    }
    asm volatile("griddepcontrol.launch_dependents;");
    const size_t base = (size_t)blockIdx.x * p.D + c0;
    each([&](int j, int c) {
        if (!GDR_INB((int)blockIdx.x < p.parts && c0 + c + V <= p.D, 919)) return;
        if (p.part_w) store_v<float, V>(p.part_w + base + c, get(0, j));
        if (p.part_b) store_v<float, V>(p.part_b + base + c, get(1, j));
    });
}

// Rows beyond a block's registers: three passes over the row, two of them from L2.
constexpr int LONG_NT = 1024;
template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_NT) norm_fwd_long_kernel(NormParams p) {
    __shared__ __align__(16) float sm[2][LONG_NT / 32][2];
    Group<LONG_NT, 2> grp{sm, 0};
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        YT* y = static_cast<YT*>(p.y) + (size_t)r * p.D;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) s[0] += ld_f32(x + c);
        grp.sum(s);
        const float mean = s[0] * inv;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) { const float v = ld_f32(x + c) - mean; s[0] = fmaf(v, v, s[0]); }
        grp.sum(s);
        const float rstd = rsqrtf(s[0] * inv + p.eps);
        with_weights(p, [&](auto type) {
            for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
                const float w = p.weight ? load_w<decltype(type), 1>(p.weight, c).v : 1.f;
                const float b = p.bias ? load_w<decltype(type), 1>(p.bias, c).v : 0.f;
                st_from_f32(y + c, fmaf((ld_f32(x + c) - mean) * rstd, w, b));
            }
        });
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}
template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_NT) norm_dx_long_kernel(NormParams p) {
    __shared__ __align__(16) float sm[2][LONG_NT / 32][2];
    Group<LONG_NT, 2> grp{sm, 0};
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        const YT* dy = static_cast<const YT*>(p.dy) + (size_t)r * p.D;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s[2] = {0.f, 0.f};
        with_weights(p, [&](auto type) {
            for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
                const float w = p.weight ? load_w<decltype(type), 1>(p.weight, c).v : 1.f;
                const float wd = w * ld_f32(dy + c);
                s[0] += wd;
                s[1] = fmaf(wd, (ld_f32(x + c) - mean) * rstd, s[1]);
            }
        });
        grp.sum(s);
        const float s1 = s[0] * inv, s2 = s[1] * inv;
        XT* dx = static_cast<XT*>(p.dx) + (size_t)r * p.D;
        with_weights(p, [&](auto type) {
            for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
                const float w = p.weight ? load_w<decltype(type), 1>(p.weight, c).v : 1.f;
                const float xh = (ld_f32(x + c) - mean) * rstd;
                st_from_f32(dx + c, rstd * (w * ld_f32(dy + c) - s1 - xh * s2));
            }
        });
    }
}
// The shares of dweight and dbias: rows part, part + parts, .. of one column per thread.
template <typename XT, typename YT>
__global__ void __launch_bounds__(256) norm_part_long_kernel(NormParams p) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.D) return;
    float w = 0.f, b = 0.f;
    for (long long r = blockIdx.y; r < p.rows; r += p.parts) {
        const float dy = ld_f32(static_cast<const YT*>(p.dy) + (size_t)r * p.D + c);
        w = fmaf(dy, (ld_f32(static_cast<const XT*>(p.x) + (size_t)r * p.D + c) - p.mean[r]) * p.rstd[r], w);
        b += dy;
    }
    if (!GDR_INB((int)blockIdx.y < p.parts, 920)) return;
    if (p.part_w) p.part_w[(size_t)blockIdx.y * p.D + c] = w;
    if (p.part_b) p.part_b[(size_t)blockIdx.y * p.D + c] = b;
}

// The partial rows' sum: 32 columns per block, its 32 warps each every 32nd partial row.
constexpr int SUM_NT = 1024;
__global__ void __launch_bounds__(SUM_NT) norm_sum_kernel(NormParams p) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cols = (p.D + 31) / 32, which = blockIdx.x / cols, c = (blockIdx.x % cols) * 32 + lane;
    const bool weights = p.part_w && which == 0;
    const float* from = weights ? p.part_w : p.part_b;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead of the partial rows' end
    float s = 0.f;
    if (c < p.D) {
        for (int i0 = warp; i0 < p.parts; i0 += 32 * 10) {     // ten loads at once: 296 partial rows in one turn
            float v[10];
#pragma unroll
            for (int u = 0; u < 10; ++u) v[u] = i0 + 32 * u < p.parts ? from[(size_t)(i0 + 32 * u) * p.D + c] : 0.f;
#pragma unroll
            for (int u = 0; u < 10; ++u) s += v[u];
        }
    }
    sm[warp][lane] = s;
    __syncthreads();
    s = sm[lane][warp];                               // lane: partial; warp: column
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int cc = (blockIdx.x % cols) * 32 + warp;
    if (lane == 0 && cc < p.D) (weights ? p.dweight : p.dbias)[cc] = s;
}

}  // namespace lnm
}  // namespace gdr
