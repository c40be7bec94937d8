// scan.cu -- the per-channel gated linear recurrence (gdr_scan_fwd, gdr_scan_bwd, gdr_scan_step):
// argument checks, dispatch and kernels.
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
#include "common.cuh"
#include "scan.cuh"

namespace gdr {
namespace scn {

enum Pass { FWD, BWD, STEP };

// Blocks of a cluster (along the tokens): enough that the grid has about two blocks per SM, as far as
// the sequence has tiles for them.
static int cluster_of(long long tiles, int T, int tok, int sms) {
    int n = 1;
    while (n < MAX_CLUSTER && tiles * n * 2 <= 2LL * sms && n * tok < T) n *= 2;
    return n;
}
// Channels of a block: 16 where blocks of 32 and clusters of 8 would leave a block per SM at most (two
// blocks of an SM hide one another's turns: 36.0 against 45.2 us at B1 T32768 D512, its backward 60.7
// against 88.4), or where 32 would leave half of the lanes idle (17.8 against 28.9 us at B1 T20000
// D11); else 32, whose rows are longer (46.5 against 58.1 us at B4 T4096 D2048).
static int channels_of(const ScanParams& p, int sms) {
    const long long wide = (p.D + 31) / 32;
    return p.D <= 16 || wide * p.B * 8 <= sms ? 16 : 32;
}

template <typename KERN>
static gdr_status launch_clusters(KERN kern, const ScanParams& p, const ScanMaps& maps, int channels, int tok, size_t smem,
                                  cudaStream_t st) {
    const unsigned ct = (unsigned)((p.D + channels - 1) / channels);
    const int ncl = cluster_of((long long)ct * p.B, p.T, tok, device_sm_count());
    // the limit belongs to the kernel, not to the call: the same for every cluster, so that a call on
    // another host thread never finds it lower than it needs
    auto bytes = [&](int blocks) { return smem + (size_t)2 * blocks * channels * sizeof(float2); };
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(MAX_CLUSTER));
    if (e == cudaSuccess && ncl > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(scan)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ncl * p.B), ct);                // a sequence's cluster, its channels
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = bytes(ncl);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ncl; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p, maps);
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(scan)");
}

// A [B][T] tensor of rows `row` elements apart, the first D of each row: the map {D, 1, T, B} with
// boxes of `channels` x tok tokens.  What lies outside reads as zero.
template <typename T>
static gdr_status encode_rows(CUtensorMap* m, const void* base, const ScanParams& p, long long row, int channels, int tok) {
    EncodeTiledFn fn = nullptr;
    const gdr_status s = encode_fn(&fn);
    if (s != GDR_OK) return s;
    const cuuint64_t dims[4] = {(cuuint64_t)p.D, 1u, (cuuint64_t)p.T, (cuuint64_t)p.B};
    const cuuint64_t bytes = (cuuint64_t)row * sizeof(T);
    const cuuint64_t strides[3] = {bytes, bytes, bytes * (cuuint64_t)p.T};
    const cuuint32_t box[4] = {(cuuint32_t)channels, 1u, (cuuint32_t)(tok < BOX_ROWS ? tok : BOX_ROWS), 1u}, estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GDR_OK;
    snprintf(t_detail, sizeof(t_detail), "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return GDR_ERR_CUDA;
}

// The same tensor for rows that start anywhere (Phases in scan.cuh): P rows as one long row.
template <typename T>
static gdr_status encode_phases(CUtensorMap* m, const void* base, const ScanParams& p, long long row, int channels, int tok) {
    EncodeTiledFn fn = nullptr;
    const gdr_status s = encode_fn(&fn);
    if (s != GDR_OK) return s;
    constexpr int P = 16 / (int)sizeof(T);
    const uintptr_t at = reinterpret_cast<uintptr_t>(base), lead = at % 16 / sizeof(T);
    const cuuint64_t bytes = (cuuint64_t)P * row * sizeof(T), rows = (cuuint64_t)p.covered / P;
    const cuuint64_t dims[4] = {(cuuint64_t)(lead + (P - 1) * row + p.D), 1u, rows, 1u};
    const cuuint64_t strides[3] = {bytes, bytes, bytes * rows};
    const cuuint32_t box[4] = {(cuuint32_t)(channels + P), 1u, (cuuint32_t)(tok / P), 1u}, estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                          reinterpret_cast<void*>(at - at % 16), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GDR_OK;
    snprintf(t_detail, sizeof(t_detail), "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return GDR_ERR_CUDA;
}

template <typename T, int V>
static gdr_status encode(CUtensorMap* m, const void* base, const ScanParams& p, long long row, int channels, int tok) {
    return V > 1 ? encode_rows<T>(m, base, p, row, channels, tok) : encode_phases<T>(m, base, p, row, channels, tok);
}

template <typename XT, typename GT, typename OT, int V, int CH>
static gdr_status launch_sequences(Pass pass, ScanParams& p, cudaStream_t st) {
    const int tok = pass == FWD ? Tile<V, fwd_elems<V>(), CH>::TOK : Tile<V, BWD_ELEMS, CH>::TOK;
    ScanMaps maps = {};
    // V = 1: whole groups of 8 rows, where the copies' coordinates (of 8 rows in 16 bits, of 4 in 32) and
    // sizes fit their types
    const long long rows = (long long)p.B * p.T, wide = p.x_row > p.g_row ? p.x_row : p.g_row;
    auto inside = [&](const void* q, long long row, size_t el) {    // a long row does not reach into the next one
        const long long lead = (long long)(reinterpret_cast<uintptr_t>(q) % 16 / el);
        return lead == 0 || lead + p.D <= row;
    };
    const bool fits = rows / 4 < (1LL << 31) - 1 && wide < (1LL << 27) && rows * wide < (1LL << 37) &&
                      inside(p.x, p.x_row, sizeof(XT)) && inside(p.g, p.g_row, sizeof(GT)) &&
                      (pass != BWD || inside(p.dh, p.D, sizeof(OT)));
    p.covered = fits ? rows / 8 * 8 : 0;
    if (V > 1 || p.covered > 0) {
        gdr_status s = encode<XT, V>(&maps.x, p.x, p, p.x_row, CH, tok);
        if (s == GDR_OK) s = encode<GT, V>(&maps.g, p.g, p, p.g_row, CH, tok);
        if (s == GDR_OK && pass == BWD && p.dh) s = encode<OT, V>(&maps.dh, p.dh, p, p.D, CH, tok);
        if (s != GDR_OK) return s;
    }
    if (pass == FWD)
        return launch_clusters(scan_fwd_kernel<XT, GT, OT, V, CH>, p, maps, CH, tok, sizeof(FwdSmem<XT, GT, V, CH>), st);
    return launch_clusters(scan_bwd_kernel<XT, GT, OT, V, CH>, p, maps, CH, tok, sizeof(BwdSmem<XT, GT, OT, V, CH>), st);
}

template <typename XT, typename GT, typename OT, int V>
static gdr_status launch_v(Pass pass, ScanParams& p, cudaStream_t st) {
    if (pass == STEP) {
        const size_t blocks = ((size_t)p.B * (p.D / V) + NT - 1) / NT, cap = (size_t)device_sm_count() * 8;
        scan_step_kernel<XT, GT, OT, V><<<(unsigned)(blocks < cap ? blocks : cap), NT, 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(scan step)");
    }
    return channels_of(p, device_sm_count()) == 16 ? launch_sequences<XT, GT, OT, V, 16>(pass, p, st)
                                                   : launch_sequences<XT, GT, OT, V, 32>(pass, p, st);
}

// Four channels per thread (and tiles by TMA) where every row of every tensor starts on 16 bytes,
// one channel per thread otherwise.  The step only needs four elements' alignment.
template <typename XT, typename GT, typename OT>
static gdr_status launch(Pass pass, ScanParams& p, cudaStream_t st) {
    auto fits = [&](const void* q, long long row, size_t el) {
        const size_t by = pass == STEP ? 4 * el : 16;
        return reinterpret_cast<uintptr_t>(q) % by == 0 && row * el % by == 0 &&
               (unsigned long long)p.T * row * el < (1ull << 40);
    };
    const bool vec = p.D % 4 == 0 && fits(p.x, p.x_row, sizeof(XT)) && fits(p.g, p.g_row, sizeof(GT)) &&
                     (pass != BWD || fits(p.dh, p.D, sizeof(OT))) &&
                     (pass != STEP || (aligned16(p.h_T) && fits(p.h, p.D, sizeof(OT))));
    return vec ? launch_v<XT, GT, OT, 4>(pass, p, st) : launch_v<XT, GT, OT, 1>(pass, p, st);
}

template <typename XT, typename GT>
static gdr_status launch_o(const gdr_scan_desc* d, Pass pass, ScanParams& p, cudaStream_t st) {
    return d->out_dtype == GDR_BF16 ? launch<XT, GT, __nv_bfloat16>(pass, p, st) : launch<XT, GT, float>(pass, p, st);
}
static gdr_status dispatch(const gdr_scan_desc* d, Pass pass, ScanParams& p, cudaStream_t st) {
    const bool xb = d->x_dtype == GDR_BF16, gb = d->g_dtype == GDR_BF16;
    if (xb && gb) return launch_o<__nv_bfloat16, __nv_bfloat16>(d, pass, p, st);
    if (xb) return launch_o<__nv_bfloat16, float>(d, pass, p, st);
    if (gb) return launch_o<float, __nv_bfloat16>(d, pass, p, st);
    return launch_o<float, float>(d, pass, p, st);
}

static gdr_status check_desc(const gdr_scan_desc* d) {
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->B < 0 || d->T < 0 || d->D < 0) return fail(GDR_ERR_INVALID_ARG, "B, T, D must be >= 0%s");
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->g_dtype) || !dtype_ok(d->out_dtype))
        return fail(GDR_ERR_INVALID_ARG, "bad dtype%s");
    if (d->gate_mode != GDR_GATE_LOGDECAY && d->gate_mode != GDR_GATE_NEG_SOFTPLUS)
        return fail(GDR_ERR_INVALID_ARG, "bad gate_mode%s");
    if (d->tied != 0 && d->tied != 1) return fail(GDR_ERR_INVALID_ARG, "tied must be 0 or 1%s");
    if ((d->x_row != 0 && d->x_row < d->D) || (d->g_row != 0 && d->g_row < d->D))
        return fail(GDR_ERR_INVALID_ARG, "x_row and g_row must be 0 or at least D%s");
    return GDR_OK;
}

// What the grid and the tokens' 32-bit arithmetic of whole sequences hold.
static gdr_status check_sequences(const gdr_scan_desc* d) {
    const gdr_status s = check_desc(d);
    if (s != GDR_OK) return s;
    if (d->B > (1 << 26) || d->T > (1 << 30) || d->D > 65535 * 16)
        return fail(GDR_ERR_UNSUPPORTED, "B must be at most 2^26, T 2^30, D 1048560%s");
    return GDR_OK;
}

static ScanParams params(const gdr_scan_desc* d, const void* x, const void* g) {
    ScanParams p = {};
    p.B = d->B; p.T = d->T; p.D = d->D;
    p.x_row = d->x_row ? d->x_row : d->D;
    p.g_row = d->g_row ? d->g_row : d->D;
    p.gate_mode = (int)d->gate_mode; p.tied = d->tied;
    p.x = x; p.g = g;
    return p;
}

// dst = src, or zero where src is NULL
static gdr_status copy_state(float* dst, const float* src, size_t n, cudaStream_t st) {
    if (!dst || dst == src || n == 0) return GDR_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(dst, 0, n * sizeof(float), st);
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "copy(state)");
}

}  // namespace scn

cudaError_t scan_status(StatusWords* w) { return status_here(w); }

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_scan_fwd(const gdr_scan_desc* d, const void* x, const void* g, const float* h0, const int* lengths,
                        void* h, float* h_T, float* ckpt, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = scn::check_sequences(d);
    if (s != GDR_OK) return s;
    if (d->B == 0 || d->D == 0) return GDR_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!aligned16(h) || !aligned16(ckpt)) return fail(GDR_ERR_INVALID_ARG, "h and ckpt must be 16-byte aligned%s");
    if (!aligned4(lengths) || !aligned4(h0) || !aligned4(h_T))
        return fail(GDR_ERR_INVALID_ARG, "lengths, h0 and h_T must be 4-byte aligned%s");
    if (d->T == 0) return scn::copy_state(h_T, h0, (size_t)d->B * d->D, st);
    if (!x || !g || !h) return fail(GDR_ERR_INVALID_ARG, "x, g and h are required%s");
    if (!aligned_to(x, d->x_dtype) || !aligned_to(g, d->g_dtype))
        return fail(GDR_ERR_INVALID_ARG, "x and g must be aligned to their elements%s");
    scn::ScanParams p = scn::params(d, x, g);
    p.h0 = h0; p.lengths = lengths; p.h = h; p.h_T = h_T; p.ckpt = ckpt;
    return scn::dispatch(d, scn::FWD, p, st);
}

gdr_status gdr_scan_bwd(const gdr_scan_desc* d, const void* x, const void* g, const float* ckpt, const int* lengths,
                        const void* dh, const float* dh_T, void* dx, void* dg, float* dh0, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = scn::check_sequences(d);
    if (s != GDR_OK) return s;
    if (d->B == 0 || d->D == 0) return GDR_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!aligned16(dx) || !aligned16(dg)) return fail(GDR_ERR_INVALID_ARG, "dx and dg must be 16-byte aligned%s");
    if (!aligned4(lengths) || !aligned4(ckpt) || !aligned4(dh_T) || !aligned4(dh0) || !aligned_to(dh, d->out_dtype))
        return fail(GDR_ERR_INVALID_ARG, "lengths, ckpt, dh, dh_T and dh0 must be aligned to their elements%s");
    if (d->T == 0) return scn::copy_state(dh0, dh_T, (size_t)d->B * d->D, st);
    if (!x || !g || !ckpt || !dx || !dg) return fail(GDR_ERR_INVALID_ARG, "x, g, ckpt, dx and dg are required%s");
    if (!aligned_to(x, d->x_dtype) || !aligned_to(g, d->g_dtype))
        return fail(GDR_ERR_INVALID_ARG, "x and g must be aligned to their elements%s");
    scn::ScanParams p = scn::params(d, x, g);
    p.ckpt = const_cast<float*>(ckpt); p.lengths = lengths; p.dh = dh; p.dh_T = dh_T;
    p.dx = dx; p.dg = dg; p.dh0 = dh0;
    return scn::dispatch(d, scn::BWD, p, st);
}

gdr_status gdr_scan_step(const gdr_scan_desc* d, const void* x, const void* g, float* h, void* o,
                         gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = scn::check_desc(d);
    if (s != GDR_OK) return s;
    if (d->B == 0 || d->D == 0) return GDR_OK;
    if (!x || !g || !h) return fail(GDR_ERR_INVALID_ARG, "x, g and h are required%s");
    if (!aligned4(h) || !aligned_to(o, d->out_dtype))
        return fail(GDR_ERR_INVALID_ARG, "h and o must be aligned to their elements%s");
    if (!aligned_to(x, d->x_dtype) || !aligned_to(g, d->g_dtype))
        return fail(GDR_ERR_INVALID_ARG, "x and g must be aligned to their elements%s");
    scn::ScanParams p = scn::params(d, x, g);
    p.h_T = h; p.h = o;
    return scn::dispatch(d, scn::STEP, p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
