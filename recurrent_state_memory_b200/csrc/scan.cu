// scan.cu -- the per-channel gated linear recurrence (gdr_scan_fwd, gdr_scan_bwd, gdr_scan_step):
// argument checks, dispatch and kernels.
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
#include "common.cuh"

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
};

constexpr int CKPT = GDR_SCAN_CKPT;
constexpr int NT = 64;

__device__ __forceinline__ int seq_len(const ScanParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// One thread per channel walks the sequence.
template <typename XT, typename GT, typename OT>
__global__ void __launch_bounds__(NT) scan_fwd_kernel(ScanParams p) {
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y;
    if (c >= p.D) return;
    const int len = seq_len(p, b), nck = (p.T + CKPT - 1) / CKPT;
    const XT* x = static_cast<const XT*>(p.x) + (size_t)b * p.T * p.x_row + c;
    const GT* g = static_cast<const GT*>(p.g) + (size_t)b * p.T * p.g_row + c;
    OT* h = static_cast<OT*>(p.h) + (size_t)b * p.T * p.D + c;
    float s = p.h0 ? p.h0[(size_t)b * p.D + c] : 0.f;
    for (int t = 0; t < p.T; ++t) {
        if (p.ckpt && t % CKPT == 0) p.ckpt[((size_t)b * nck + t / CKPT) * p.D + c] = s;
        float out = 0.f;
        if (t < len) {
            float a, rest;
            decay_pair(ld_f32(g + (size_t)t * p.g_row), p.gate_mode, a, rest);
            const float xv = ld_f32(x + (size_t)t * p.x_row);
            s = fmaf(a, s, p.tied ? rest * xv : xv);
            out = s;
        }
        st_from_f32(h + (size_t)t * p.D, out);
    }
    if (p.h_T) p.h_T[(size_t)b * p.D + c] = s;
}

template <typename XT, typename GT, typename OT>
__global__ void __launch_bounds__(NT) scan_bwd_kernel(ScanParams p) {
    __shared__ float before[CKPT][NT];           // the states before the tokens of one piece
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y;
    if (c >= p.D) return;
    const int len = seq_len(p, b), nck = (p.T + CKPT - 1) / CKPT;
    const XT* x = static_cast<const XT*>(p.x) + (size_t)b * p.T * p.x_row + c;
    const GT* g = static_cast<const GT*>(p.g) + (size_t)b * p.T * p.g_row + c;
    const OT* dh = p.dh ? static_cast<const OT*>(p.dh) + (size_t)b * p.T * p.D + c : nullptr;
    XT* dx = static_cast<XT*>(p.dx) + (size_t)b * p.T * p.D + c;
    GT* dg = static_cast<GT*>(p.dg) + (size_t)b * p.T * p.D + c;
    float m = p.dh_T ? p.dh_T[(size_t)b * p.D + c] : 0.f;     // a_{t+1} lam_{t+1}
    for (int j = nck - 1; j >= 0; --j) {
        const int t0 = j * CKPT, t1 = min(t0 + CKPT, p.T);
        float s = p.ckpt[((size_t)b * nck + j) * p.D + c];
        for (int t = t0; t < min(t1, len); ++t) {
            before[t - t0][threadIdx.x] = s;
            float a, rest;
            decay_pair(ld_f32(g + (size_t)t * p.g_row), p.gate_mode, a, rest);
            const float xv = ld_f32(x + (size_t)t * p.x_row);
            s = fmaf(a, s, p.tied ? rest * xv : xv);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            float ox = 0.f, og = 0.f;
            if (t < len) {
                float a, rest;
                decay_pair(ld_f32(g + (size_t)t * p.g_row), p.gate_mode, a, rest);
                const float xv = ld_f32(x + (size_t)t * p.x_row);
                const float lam = m + (dh ? ld_f32(dh + (size_t)t * p.D) : 0.f);
                ox = p.tied ? rest * lam : lam;
                const float da = lam * (before[t - t0][threadIdx.x] - (p.tied ? xv : 0.f));
                og = p.gate_mode == 1 ? -da * (a * rest) : da * a;
                m = a * lam;
            }
            st_from_f32(dx + (size_t)t * p.D, ox);
            st_from_f32(dg + (size_t)t * p.D, og);
        }
    }
    if (p.dh0) p.dh0[(size_t)b * p.D + c] = m;
}

template <typename XT, typename GT, typename OT>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p) {
    const size_t n = (size_t)p.B * p.D;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        const size_t b = i / p.D, c = i % p.D;
        float a, rest;
        decay_pair(ld_f32(static_cast<const GT*>(p.g) + b * p.g_row + c), p.gate_mode, a, rest);
        const float xv = ld_f32(static_cast<const XT*>(p.x) + b * p.x_row + c);
        const float s = fmaf(a, p.h_T[i], p.tied ? rest * xv : xv);
        p.h_T[i] = s;
        if (p.h) st_from_f32(static_cast<OT*>(p.h) + i, s);
    }
}

enum Pass { FWD, BWD, STEP };

template <typename XT, typename GT, typename OT>
static gdr_status launch(Pass pass, const ScanParams& p, cudaStream_t st) {
    const dim3 grid((p.D + NT - 1) / NT, p.B);
    if (pass == FWD) scan_fwd_kernel<XT, GT, OT><<<grid, NT, 0, st>>>(p);
    else if (pass == BWD) scan_bwd_kernel<XT, GT, OT><<<grid, NT, 0, st>>>(p);
    else {
        const size_t blocks = ((size_t)p.B * p.D + 255) / 256, cap = (size_t)device_sm_count() * 8;
        scan_step_kernel<XT, GT, OT><<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, st>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(scan)");
}

template <typename XT, typename GT>
static gdr_status launch_o(const gdr_scan_desc* d, Pass pass, const ScanParams& p, cudaStream_t st) {
    return d->out_dtype == GDR_BF16 ? launch<XT, GT, __nv_bfloat16>(pass, p, st) : launch<XT, GT, float>(pass, p, st);
}
static gdr_status dispatch(const gdr_scan_desc* d, Pass pass, const ScanParams& p, cudaStream_t st) {
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
    if (d->B > 65535) return fail(GDR_ERR_UNSUPPORTED, "B must be at most 65535%s");
    return GDR_OK;
}

static bool aligned_to(const void* p, gdr_dtype t) { return reinterpret_cast<uintptr_t>(p) % dtype_bytes(t) == 0; }

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

cudaError_t scan_take_status(unsigned int* word, unsigned int* site) { return take_status_here(word, site); }

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_scan_fwd(const gdr_scan_desc* d, const void* x, const void* g, const float* h0, const int* lengths,
                        void* h, float* h_T, float* ckpt, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = scn::check_desc(d);
    if (s != GDR_OK) return s;
    if (d->B == 0 || d->D == 0) return GDR_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    for (const void* q : {(const void*)h0, (const void*)h, (const void*)h_T, (const void*)ckpt})
        if (q && !aligned16(q)) return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned%s");
    if (!aligned4(lengths)) return fail(GDR_ERR_INVALID_ARG, "lengths must be 4-byte aligned%s");
    if (d->T == 0) return scn::copy_state(h_T, h0, (size_t)d->B * d->D, st);
    if (!x || !g || !h) return fail(GDR_ERR_INVALID_ARG, "x, g and h are required%s");
    if (!scn::aligned_to(x, d->x_dtype) || !scn::aligned_to(g, d->g_dtype))
        return fail(GDR_ERR_INVALID_ARG, "x and g must be aligned to their elements%s");
    scn::ScanParams p = scn::params(d, x, g);
    p.h0 = h0; p.lengths = lengths; p.h = h; p.h_T = h_T; p.ckpt = ckpt;
    return scn::dispatch(d, scn::FWD, p, st);
}

gdr_status gdr_scan_bwd(const gdr_scan_desc* d, const void* x, const void* g, const float* ckpt, const int* lengths,
                        const void* dh, const float* dh_T, void* dx, void* dg, float* dh0, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = scn::check_desc(d);
    if (s != GDR_OK) return s;
    if (d->B == 0 || d->D == 0) return GDR_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    for (const void* q : {(const void*)ckpt, dh, (const void*)dh_T, (const void*)dx,
                          (const void*)dg, (const void*)dh0})
        if (q && !aligned16(q)) return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned%s");
    if (!aligned4(lengths)) return fail(GDR_ERR_INVALID_ARG, "lengths must be 4-byte aligned%s");
    if (d->T == 0) return scn::copy_state(dh0, dh_T, (size_t)d->B * d->D, st);
    if (!x || !g || !ckpt || !dx || !dg) return fail(GDR_ERR_INVALID_ARG, "x, g, ckpt, dx and dg are required%s");
    if (!scn::aligned_to(x, d->x_dtype) || !scn::aligned_to(g, d->g_dtype))
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
    if (!aligned16(h) || (o && !aligned16(o))) return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned%s");
    if (!scn::aligned_to(x, d->x_dtype) || !scn::aligned_to(g, d->g_dtype))
        return fail(GDR_ERR_INVALID_ARG, "x and g must be aligned to their elements%s");
    scn::ScanParams p = scn::params(d, x, g);
    p.h_T = h; p.h = o;
    return scn::dispatch(d, scn::STEP, p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
