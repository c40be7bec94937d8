// beam.cu -- beam search in the decode loop: the best continuations of every group of beams
// (gdr_beam_select) and the states that follow them (gdr_state_reorder).
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
#include "common.cuh"

namespace gdr {
namespace bms {

constexpr int NT = 256;

struct BeamParams {
    int G, K, V, M;
    long long row;
    int eos;
    const void* logits;
    const float* scores;
    const unsigned char* finished;
    float* out_scores;
    int* out_parent;
    int* out_token;
    double* lse;            // [G*K]
};

// log sum exp of one beam's logits per block, in 64 bits.
template <typename XT>
__global__ void __launch_bounds__(NT) beam_lse_kernel(BeamParams p) {
    __shared__ double sm[NT];
    const XT* x = static_cast<const XT*>(p.logits) + (size_t)blockIdx.x * p.row;
    float top = -INFINITY;
    for (int v = threadIdx.x; v < p.V; v += NT) top = fmaxf(top, ld_f32(x + v));
    sm[threadIdx.x] = top;
    __syncthreads();
    for (int o = NT / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) sm[threadIdx.x] = fmax(sm[threadIdx.x], sm[threadIdx.x + o]);
        __syncthreads();
    }
    const double big = sm[0];
    __syncthreads();
    double s = 0.0;
    for (int v = threadIdx.x; v < p.V; v += NT) s += exp((double)ld_f32(x + v) - big);
    sm[threadIdx.x] = s;
    __syncthreads();
    for (int o = NT / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) sm[threadIdx.x] += sm[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) p.lse[blockIdx.x] = big + log(sm[0]);
}

struct Cand { double s; int at; };
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) { return a.s > b.s || (a.s == b.s && a.at < b.at); }

template <typename XT>
__device__ __forceinline__ double cand_score(const BeamParams& p, int g, int k, int v) {
    const size_t row = (size_t)g * p.K + k;
    const double sc = p.scores[row];
    double s;
    if (p.finished && p.finished[row]) s = v == p.eos ? sc : -INFINITY;
    else s = sc + ((double)ld_f32(static_cast<const XT*>(p.logits) + row * p.row + v) - p.lse[row]);
    return s != s || s == INFINITY ? -INFINITY : s;
}

// M rounds over a group's candidates: each takes the best one behind the last.
template <typename XT>
__global__ void __launch_bounds__(NT) beam_pick_kernel(BeamParams p) {
    __shared__ Cand sm[NT];
    const int g = blockIdx.x, n = p.K * p.V;
    Cand last = {INFINITY, -1};
    for (int m = 0; m < p.M; ++m) {
        Cand best = {-INFINITY, INT32_MAX};
        for (int i = threadIdx.x; i < n; i += NT) {
            const Cand c = {cand_score<XT>(p, g, i / p.V, i % p.V), i};
            if (before(last, c) && before(c, best)) best = c;
        }
        sm[threadIdx.x] = best;
        __syncthreads();
        for (int o = NT / 2; o > 0; o >>= 1) {
            if (threadIdx.x < o && before(sm[threadIdx.x + o], sm[threadIdx.x])) sm[threadIdx.x] = sm[threadIdx.x + o];
            __syncthreads();
        }
        last = sm[0];
        __syncthreads();
        if (threadIdx.x == 0) {
            const size_t at = (size_t)g * p.M + m;
            p.out_scores[at] = (float)last.s;
            p.out_parent[at] = last.at / p.V;
            p.out_token[at] = last.at % p.V;
        }
    }
}

template <typename XT>
static gdr_status launch_select(const BeamParams& p, cudaStream_t st) {
    beam_lse_kernel<XT><<<p.G * p.K, NT, 0, st>>>(p);
    beam_pick_kernel<XT><<<p.G, NT, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(beam selection)");
}

static gdr_status check_desc(const gdr_beam_desc* d) {
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->G < 0) return fail(GDR_ERR_INVALID_ARG, "G must be >= 0%s");
    if (d->K < 1 || d->K > 64 || d->M < 1 || d->M > 64) return fail(GDR_ERR_UNSUPPORTED, "K and M must be 1 .. 64%s");
    if (d->V < 1) return fail(GDR_ERR_INVALID_ARG, "V must be >= 1%s");
    const long long n = (long long)d->K * d->V;
    if (n > 0x7fffffffLL || (long long)d->G * d->K > 0x7fffffffLL)
        return fail(GDR_ERR_UNSUPPORTED, "K * V and G * K must be below 2^31%s");
    if (d->M > n) return fail(GDR_ERR_INVALID_ARG, "M must be at most K * V%s");
    if (d->row != 0 && d->row < d->V) return fail(GDR_ERR_INVALID_ARG, "row must be 0 or at least V%s");
    if (!dtype_ok(d->x_dtype)) return fail(GDR_ERR_INVALID_ARG, "bad dtype%s");
    return GDR_OK;
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

template <typename VT>
static gdr_status launch_reorder(int L, ReorderParams p, size_t bytes, cudaStream_t st) {
    p.n = bytes / sizeof(VT);
    const size_t blocks = (p.n + NT - 1) / NT;
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)((long long)L * p.G));
    if (p.K <= 4) reorder_kernel<VT, 4><<<grid, NT, 0, st>>>(p);
    else if (p.K <= 8) reorder_kernel<VT, 8><<<grid, NT, 0, st>>>(p);
    else if (p.K <= 16) reorder_kernel<VT, 16><<<grid, NT, 0, st>>>(p);
    else reorder_kernel<VT, 64><<<grid, NT, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(state reorder)");
}

}  // namespace bms

cudaError_t beam_take_status(unsigned int* word, unsigned int* site) { return take_status_here(word, site); }

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_beam_select_workspace_bytes(const gdr_beam_desc* d) {
    if (bms::check_desc(d) != GDR_OK) return 0;
    return (size_t)d->G * d->K * sizeof(double);
}

gdr_status gdr_beam_select(const gdr_beam_desc* d, const void* logits, const float* scores,
                           const unsigned char* finished, float* out_scores, int* out_parent, int* out_token,
                           void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = bms::check_desc(d);
    if (s != GDR_OK) return s;
    if (finished && (d->eos < 0 || d->eos >= d->V)) return fail(GDR_ERR_INVALID_ARG, "eos must be 0 .. V - 1%s");
    if (d->G == 0) return GDR_OK;
    if (!logits || !scores || !out_scores || !out_parent || !out_token)
        return fail(GDR_ERR_INVALID_ARG, "logits, scores and the outputs are required%s");
    for (const void* q : {(const void*)scores, (const void*)out_scores, (const void*)out_parent, (const void*)out_token})
        if (!aligned4(q)) return fail(GDR_ERR_INVALID_ARG, "scores and the outputs must be 4-byte aligned%s");
    if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned%s");
    if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(d->x_dtype) != 0)
        return fail(GDR_ERR_INVALID_ARG, "logits must be aligned to their elements%s");
    if (!workspace || workspace_bytes < gdr_beam_select_workspace_bytes(d))
        return fail(GDR_ERR_WORKSPACE, "workspace too small%s");
    bms::BeamParams p = {};
    p.G = d->G; p.K = d->K; p.V = d->V; p.M = d->M; p.row = d->row ? d->row : d->V; p.eos = d->eos;
    p.logits = logits; p.scores = scores; p.finished = finished;
    p.out_scores = out_scores; p.out_parent = out_parent; p.out_token = out_token;
    p.lse = static_cast<double*>(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return d->x_dtype == GDR_BF16 ? bms::launch_select<__nv_bfloat16>(p, st) : bms::launch_select<float>(p, st);
}

gdr_status gdr_state_reorder(const gdr_reorder_desc* d, void* S, const int* parent, gdr_stream_t stream) {
    t_detail[0] = 0;
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->L < 0 || d->G < 0) return fail(GDR_ERR_INVALID_ARG, "L and G must be >= 0%s");
    if (d->K < 1 || d->K > 64) return fail(GDR_ERR_UNSUPPORTED, "K must be 1 .. 64%s");
    if ((long long)d->L * d->G > 65535) return fail(GDR_ERR_UNSUPPORTED, "L * G must be at most 65535%s");
    if (d->L == 0 || d->G == 0 || d->state_bytes == 0) return GDR_OK;
    if (!S || !parent) return fail(GDR_ERR_INVALID_ARG, "S and parent are required%s");
    if (!aligned16(S) || !aligned4(parent))
        return fail(GDR_ERR_INVALID_ARG, "S must be 16-byte and parent 4-byte aligned%s");
    bms::ReorderParams p = {};
    p.G = d->G; p.K = d->K; p.S = static_cast<char*>(S); p.parent = parent;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t n = d->state_bytes;        // every state starts at a multiple of it
    if (n % 16 == 0 && d->K <= 16) return bms::launch_reorder<uint4>(d->L, p, n, st);
    if (n % 8 == 0 && d->K <= 16) return bms::launch_reorder<uint2>(d->L, p, n, st);
    if (n % 4 == 0) return bms::launch_reorder<unsigned int>(d->L, p, n, st);
    if (n % 2 == 0) return bms::launch_reorder<unsigned short>(d->L, p, n, st);
    return bms::launch_reorder<unsigned char>(d->L, p, n, st);
}

}  // extern "C"
