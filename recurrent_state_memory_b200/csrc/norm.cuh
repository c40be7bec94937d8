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
// load: G = 1 .. 32 lanes of a warp (several rows per warp), or a whole block for rows longer than
// a warp's registers.  Groups walk the rows with the grid's stride; the next row's loads are in
// flight while a row is reduced.  Rows that 16-byte access does not fit (D or a pointer off) take
// one element per lane and load.  Rows beyond a block's registers are read again from L2 instead.
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
    int group;              // lanes of a row (warp kernels): 1, 2, .. 32
};

// V consecutive elements as they lie in memory (one access of 16 bytes or less, or two), and as fp32.
template <typename T, int V> struct Raw {
    static constexpr int BYTES = V * (int)sizeof(T), WORDS = BYTES < 4 ? 1 : BYTES / 4;
    unsigned w[WORDS];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (BYTES == 32) {
            const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        } else if constexpr (BYTES == 16) {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else if constexpr (BYTES == 8) {
            const uint2 a = *reinterpret_cast<const uint2*>(p);
            w[0] = a.x; w[1] = a.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const unsigned*>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short*>(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
// V weights or biases from column c on, of either type.
template <int V> __device__ __forceinline__ void load_w(const void* p, int bf16, int c, float (&v)[V]) {
    if (bf16) {
        Raw<__nv_bfloat16, V> r;
        r.load(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = r.get(i);
    } else {
        Raw<float, V> r;
        r.load(static_cast<const float*>(p) + c);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = r.get(i);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        st_from_f32(p, v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        unsigned w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// The sum over a row's group: lanes of a warp (n lanes), or the block (BLOCK threads; sm: two
// sets of warp sums used in turn, so that one barrier a sum is enough).
template <int BLOCK> struct Group {
    float* sm;
    int n, turn;
    __device__ __forceinline__ float sum(float v) {
        if constexpr (BLOCK == 0) {
            for (int o = n >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            float* s = sm + turn * (BLOCK / 32);
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
            __syncthreads();
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < BLOCK / 32; ++i) t += s[i];
            return t;
        }
    }
    __device__ __forceinline__ void sum2(float& a, float& b) {
        if constexpr (BLOCK == 0) {
            for (int o = n >> 1; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
            float2* s = reinterpret_cast<float2*>(sm) + turn * (BLOCK / 32);
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
            __syncthreads();
            a = b = 0.f;
#pragma unroll
            for (int i = 0; i < BLOCK / 32; ++i) { a += s[i].x; b += s[i].y; }
        }
    }
};

constexpr int WARP_NT = 256;            // threads of a block of the warp kernels

// Threads of a block: BLOCK, or WARP_NT where a row is a warp's lanes.
template <int BLOCK> constexpr int threads() { return BLOCK ? BLOCK : WARP_NT; }

// Where this thread's group stands: its first row, the stride to its next, its lane, its lanes.
template <int BLOCK> struct Place {
    long long row, step;
    int lane, lanes;
    __device__ __forceinline__ explicit Place(const NormParams& p) {
        if constexpr (BLOCK == 0) {
            const int per = WARP_NT / p.group;
            lane = threadIdx.x & (p.group - 1);
            lanes = p.group;
            row = (long long)blockIdx.x * per + threadIdx.x / p.group;
            step = (long long)gridDim.x * per;
        } else {
            lane = threadIdx.x;
            lanes = BLOCK;
            row = blockIdx.x;
            step = gridDim.x;
        }
    }
};

// One row per group and turn, N loads of V elements per lane.
template <typename XT, typename YT, int V, int N, int BLOCK>
__global__ void __launch_bounds__(threads<BLOCK>()) norm_fwd_kernel(NormParams p) {
    __shared__ float2 sm[2 * (BLOCK ? BLOCK / 32 : 1)];
    const Place<BLOCK> at(p);
    Group<BLOCK> grp{reinterpret_cast<float*>(sm), at.lanes, 0};
    const float inv = 1.f / (float)p.D;
    const XT* x = static_cast<const XT*>(p.x);
    YT* y = static_cast<YT*>(p.y);
    constexpr bool KEEP = V * N <= 16;                // weights stay in registers
    float w[KEEP ? N : 1][V], bi[KEEP ? N : 1][V];
    auto weights = [&](int j, float (&wv)[V], float (&bv)[V]) {
        const int c = (j * at.lanes + at.lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) { wv[i] = 1.f; bv[i] = 0.f; }
        if (c < p.D) {
            if (p.weight) load_w<V>(p.weight, p.w_bf16, c, wv);
            if (p.bias) load_w<V>(p.bias, p.w_bf16, c, bv);
        }
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < N; ++j) weights(j, w[j], bi[j]);
    }
    Raw<XT, V> raw[N];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * at.lanes + at.lane) * V;
            if (r < p.rows && c < p.D) raw[j].load(x + (size_t)r * p.D + c);
            else raw[j].zero();
        }
    };
    // every lane of a warp makes the same number of turns (the sums are warp-wide)
    const long long first = BLOCK ? at.row : at.row - (threadIdx.x & 31) / at.lanes;
    fetch(at.row);
    for (long long r0 = first; r0 < p.rows; r0 += at.step) {
        const long long r = r0 + (at.row - first);
        float v[N][V], s = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) { v[j][i] = raw[j].get(i); s += v[j][i]; }
        fetch(r + at.step);
        const float mean = grp.sum(s) * inv;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if ((j * at.lanes + at.lane) * V < p.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) { v[j][i] -= mean; s = fmaf(v[j][i], v[j][i], s); }
            }
        }
        const float rstd = 1.f / sqrtf(grp.sum(s) * inv + p.eps);
        if (r < p.rows) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = (j * at.lanes + at.lane) * V;
                if (c >= p.D) continue;
                float o[V];
                if constexpr (KEEP) {
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = fmaf(v[j][i] * rstd, w[j][i], bi[j][i]);
                } else {
                    float wv[V], bv[V];
                    weights(j, wv, bv);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = fmaf(v[j][i] * rstd, wv[i], bv[i]);
                }
                if (GDR_INB(c + V <= p.D, 901)) store_v<YT, V>(y + (size_t)r * p.D + c, o);
            }
            if (at.lane == 0) {
                if (p.mean) p.mean[r] = mean;
                if (p.rstd) p.rstd[r] = rstd;
            }
        }
    }
}

// Backward: dx, and the block's share of dweight and dbias.
template <typename XT, typename YT, int V, int N, int BLOCK>
__global__ void __launch_bounds__(threads<BLOCK>()) norm_bwd_kernel(NormParams p) {
    extern __shared__ float part[];                   // warp kernels: the groups' sums [NT / lanes][D], in turn
    __shared__ float2 sm[2 * (BLOCK ? BLOCK / 32 : 1)];
    const Place<BLOCK> at(p);
    Group<BLOCK> grp{reinterpret_cast<float*>(sm), at.lanes, 0};
    const float inv = 1.f / (float)p.D;
    const XT* x = static_cast<const XT*>(p.x);
    const YT* dy = static_cast<const YT*>(p.dy);
    XT* dx = static_cast<XT*>(p.dx);
    constexpr bool KEEP = V * N <= 8;
    float w[KEEP ? N : 1][V];
    auto weights = [&](int j, float (&wv)[V]) {
        const int c = (j * at.lanes + at.lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) wv[i] = 1.f;
        if (c < p.D && p.weight) load_w<V>(p.weight, p.w_bf16, c, wv);
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < N; ++j) weights(j, w[j]);
    }
    float sw[N][V], sb[N][V];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) sw[j][i] = sb[j][i] = 0.f;
    Raw<XT, V> rx[N];
    Raw<YT, V> rd[N];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r) {
        const bool in = r < p.rows;
        mean = in ? p.mean[r] : 0.f;
        rstd = in ? p.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * at.lanes + at.lane) * V;
            if (in && c < p.D) {
                rx[j].load(x + (size_t)r * p.D + c);
                rd[j].load(dy + (size_t)r * p.D + c);
            } else { rx[j].zero(); rd[j].zero(); }
        }
    };
    const long long first = BLOCK ? at.row : at.row - (threadIdx.x & 31) / at.lanes;
    fetch(at.row);
    for (long long r0 = first; r0 < p.rows; r0 += at.step) {
        const long long r = r0 + (at.row - first);
        float xh[N][V], d[N][V], c1 = 0.f, c2 = 0.f;
        const float here = rstd;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float wv[V];
            if constexpr (!KEEP) weights(j, wv);
#pragma unroll
            for (int i = 0; i < V; ++i) {             // columns behind D: dy is zero
                xh[j][i] = (rx[j].get(i) - mean) * rstd;
                d[j][i] = rd[j].get(i);
                sw[j][i] = fmaf(d[j][i], xh[j][i], sw[j][i]);
                sb[j][i] += d[j][i];
                d[j][i] *= KEEP ? w[KEEP ? j : 0][i] : wv[i];
                c1 += d[j][i];
                c2 = fmaf(d[j][i], xh[j][i], c2);
            }
        }
        fetch(r + at.step);
        if (!dx) continue;
        grp.sum2(c1, c2);
        c1 *= inv;
        c2 *= inv;
        if (r < p.rows) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = (j * at.lanes + at.lane) * V;
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = here * (d[j][i] - fmaf(xh[j][i], c2, c1));
                if (c < p.D && GDR_INB(c + V <= p.D, 911)) store_v<XT, V>(dx + (size_t)r * p.D + c, o);
            }
        }
    }
    const size_t base = (size_t)blockIdx.x * p.D;
    if constexpr (BLOCK != 0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * at.lanes + at.lane) * V;
            if (c >= p.D) continue;
            if (p.part_w) store_v<float, V>(p.part_w + base + c, sw[j]);
            if (p.part_b) store_v<float, V>(p.part_b + base + c, sb[j]);
        }
    } else {
        // the block's groups, added column by column in the groups' order
        const int per = WARP_NT / at.lanes, g = threadIdx.x / at.lanes;
        for (int which = 0; which < 2; ++which) {
            float* to = which ? p.part_b : p.part_w;
            if (!to) continue;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = (j * at.lanes + at.lane) * V;
                if (c < p.D) store_v<float, V>(part + (size_t)g * p.D + c, which ? sb[j] : sw[j]);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.D; c += WARP_NT) {
                float s = 0.f;
                for (int i = 0; i < per; ++i) s += part[(size_t)i * p.D + c];
                to[base + c] = s;
            }
        }
    }
}

// Rows beyond a block's registers: three passes over the row, two of them from L2.
constexpr int LONG_NT = 1024;
template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_NT) norm_fwd_long_kernel(NormParams p) {
    __shared__ float2 sm[2 * LONG_NT / 32];
    Group<LONG_NT> grp{reinterpret_cast<float*>(sm), LONG_NT, 0};
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        YT* y = static_cast<YT*>(p.y) + (size_t)r * p.D;
        float s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) s += ld_f32(x + c);
        const float mean = grp.sum(s) * inv;
        s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) { const float v = ld_f32(x + c) - mean; s = fmaf(v, v, s); }
        const float rstd = 1.f / sqrtf(grp.sum(s) * inv + p.eps);
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
            float w[1] = {1.f}, b[1] = {0.f};
            if (p.weight) load_w<1>(p.weight, p.w_bf16, c, w);
            if (p.bias) load_w<1>(p.bias, p.w_bf16, c, b);
            st_from_f32(y + c, fmaf((ld_f32(x + c) - mean) * rstd, w[0], b[0]));
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}
template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_NT) norm_dx_long_kernel(NormParams p) {
    __shared__ float2 sm[2 * LONG_NT / 32];
    Group<LONG_NT> grp{reinterpret_cast<float*>(sm), LONG_NT, 0};
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        const YT* dy = static_cast<const YT*>(p.dy) + (size_t)r * p.D;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
            float w[1] = {1.f};
            if (p.weight) load_w<1>(p.weight, p.w_bf16, c, w);
            const float wd = w[0] * ld_f32(dy + c);
            s1 += wd;
            s2 = fmaf(wd, (ld_f32(x + c) - mean) * rstd, s2);
        }
        grp.sum2(s1, s2);
        s1 *= inv;
        s2 *= inv;
        XT* dx = static_cast<XT*>(p.dx) + (size_t)r * p.D;
        for (int c = threadIdx.x; c < p.D; c += LONG_NT) {
            float w[1] = {1.f};
            if (p.weight) load_w<1>(p.weight, p.w_bf16, c, w);
            const float xh = (ld_f32(x + c) - mean) * rstd;
            st_from_f32(dx + c, rstd * (w[0] * ld_f32(dy + c) - s1 - xh * s2));
        }
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
    float s = 0.f;
    if (c < p.D)
        for (int i = warp; i < p.parts; i += 32) s += from[(size_t)i * p.D + c];
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
