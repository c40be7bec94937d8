// beam.cu -- beam search in the decode loop: the best continuations of every group of beams
// (gdr_beam_select) and the states that follow them (gdr_state_reorder).
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
#include "common.cuh"
#include "beam.cuh"

namespace gdr {
namespace bms {

// Pieces of a row: 8192 elements (32 per thread) when the rows fill the GPU with them, 2048 (8 per
// thread) otherwise, so that a few beams still spread over the SMs.
static void plan_pieces(const gdr_beam_desc* d, int* piece, int* pieces) {
    const long long rows = (long long)d->G * d->K, big = (d->V + 8191) / 8192;
    *piece = rows * big >= 2LL * device_sm_count() ? 8192 : 2048;
    *pieces = (d->V + *piece - 1) / *piece;
}

// The workspace: the pieces' sums, their best logits and tokens.
static size_t workspace_of(const gdr_beam_desc* d, BeamParams* p, void* base) {
    int piece, pieces;
    plan_pieces(d, &piece, &pieces);
    const size_t n = (size_t)d->G * d->K * pieces;
    if (p) {
        p->piece = piece; p->pieces = pieces;
        p->sums = static_cast<float2*>(base);
        p->best = reinterpret_cast<float*>(p->sums + n);
        p->token = reinterpret_cast<int*>(p->best + n * d->M);
    }
    return n * (sizeof(float2) + (size_t)d->M * (sizeof(float) + sizeof(int)));
}

template <typename XT>
static gdr_status launch_select(const BeamParams& p, cudaStream_t st) {
    const unsigned rows = (unsigned)(p.G * p.K), y = rows < 65535 ? rows : 65535;
    const dim3 grid(p.pieces, y, (rows + y - 1) / y);
    // 16-byte loads where every row starts on them
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.row * sizeof(XT) % 16 == 0;
    if (p.piece == 8192) {
        if (vec) beam_row_kernel<XT, 32, true><<<grid, NT, 0, st>>>(p);
        else beam_row_kernel<XT, 32, false><<<grid, NT, 0, st>>>(p);
    } else {
        if (vec) beam_row_kernel<XT, 8, true><<<grid, NT, 0, st>>>(p);
        else beam_row_kernel<XT, 8, false><<<grid, NT, 0, st>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "launch(beam rows)");
    cudaLaunchConfig_t cfg = {};        // launched ahead of the rows' end, waits for it
    cfg.gridDim = dim3(p.G);
    const long long n = (long long)p.K * p.pieces * p.M;
    cfg.blockDim = dim3(n <= HELD * 256 ? 256 : 1024);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = n <= HELD * 256    ? cudaLaunchKernelEx(&cfg, beam_group_kernel<XT, 256, true>, p)
        : n <= HELD * 1024 ? cudaLaunchKernelEx(&cfg, beam_group_kernel<XT, 1024, true>, p)
                           : cudaLaunchKernelEx(&cfg, beam_group_kernel<XT, 1024, false>, p);
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(beam groups)");
}

static gdr_status check_desc(const gdr_beam_desc* d) {
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->G < 0) return fail(GDR_ERR_INVALID_ARG, "G must be >= 0%s");
    if (d->K < 1 || d->K > 64 || d->M < 1 || d->M > 64) return fail(GDR_ERR_UNSUPPORTED, "K and M must be 1 .. 64%s");
    if (d->V < 1) return fail(GDR_ERR_INVALID_ARG, "V must be >= 1%s");
    const long long n = (long long)d->K * d->V;
    if (n > 0x7fffffffLL) return fail(GDR_ERR_UNSUPPORTED, "K * V must be below 2^31%s");
    if ((long long)d->G * d->K > 0x7fffffffLL) return fail(GDR_ERR_UNSUPPORTED, "G * K must be below 2^31%s");
    if (d->M > n) return fail(GDR_ERR_INVALID_ARG, "M must be at most K * V%s");
    if (d->row != 0 && d->row < d->V) return fail(GDR_ERR_INVALID_ARG, "row must be 0 or at least V%s");
    if (!dtype_ok(d->x_dtype)) return fail(GDR_ERR_INVALID_ARG, "bad dtype%s");
    return GDR_OK;
}

template <typename VT>
static gdr_status launch_reorder(int L, ReorderParams p, size_t bytes, cudaStream_t st) {
    p.n = bytes / sizeof(VT);
    const size_t blocks = (p.n + NT - 1) / NT;
    // a group's positions first (61.6 us for the 256 x 16 decode states; groups first 63.5); as many
    // groups a launch as a grid's second dimension holds
    const long long all = (long long)L * p.G;
    for (long long first = 0; first < all; first += 65535) {
        const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)(all - first < 65535 ? all - first : 65535));
        p.first = (int)first;
        if (p.K <= 4) reorder_kernel<VT, 4><<<grid, NT, 0, st>>>(p);
        else if (p.K <= 8) reorder_kernel<VT, 8><<<grid, NT, 0, st>>>(p);
        else if (p.K <= 16) reorder_kernel<VT, 16><<<grid, NT, 0, st>>>(p);
        else if constexpr (sizeof(VT) <= 4) reorder_kernel<VT, 64><<<grid, NT, 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "launch(state reorder)");
        p.S += (size_t)65535 * p.K * bytes;
    }
    return GDR_OK;
}

}  // namespace bms

cudaError_t beam_status(StatusWords* w) { return status_here(w); }

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_beam_select_workspace_bytes(const gdr_beam_desc* d) {
    if (bms::check_desc(d) != GDR_OK) return 0;
    return bms::workspace_of(d, nullptr, nullptr);
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
    bms::workspace_of(d, &p, workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return d->x_dtype == GDR_BF16 ? bms::launch_select<__nv_bfloat16>(p, st) : bms::launch_select<float>(p, st);
}

gdr_status gdr_state_reorder(const gdr_reorder_desc* d, void* S, const int* parent, gdr_stream_t stream) {
    t_detail[0] = 0;
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->L < 0 || d->G < 0) return fail(GDR_ERR_INVALID_ARG, "L and G must be >= 0%s");
    if (d->K < 1 || d->K > 64) return fail(GDR_ERR_UNSUPPORTED, "K must be 1 .. 64%s");
    if ((long long)d->L * d->G > 0x7fffffffLL) return fail(GDR_ERR_UNSUPPORTED, "L * G must be below 2^31%s");
    if (d->L == 0 || d->G == 0 || d->state_bytes == 0) return GDR_OK;
    if (!S || !parent) return fail(GDR_ERR_INVALID_ARG, "S and parent are required%s");
    if (!aligned4(parent)) return fail(GDR_ERR_INVALID_ARG, "parent must be 4-byte aligned%s");
    bms::ReorderParams p = {};
    p.G = d->G; p.K = d->K; p.S = static_cast<char*>(S); p.parent = parent;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // the widest access that every state's start and size allow
    const size_t n = d->state_bytes | (reinterpret_cast<uintptr_t>(S) & 15u);
    if (n % 16 == 0 && d->K <= 16) return bms::launch_reorder<uint4>(d->L, p, d->state_bytes, st);
    if (n % 8 == 0 && d->K <= 16) return bms::launch_reorder<uint2>(d->L, p, d->state_bytes, st);
    if (n % 4 == 0) return bms::launch_reorder<unsigned int>(d->L, p, d->state_bytes, st);
    if (n % 2 == 0) return bms::launch_reorder<unsigned short>(d->L, p, d->state_bytes, st);
    return bms::launch_reorder<unsigned char>(d->L, p, d->state_bytes, st);
}

}  // extern "C"
