// norm.cu -- layer norm forward and backward (gdr_layernorm_fwd, gdr_layernorm_bwd): argument
// checks, dispatch and kernels.
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
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
};

constexpr int NT = 256;
constexpr int PARTS = 296;

__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s += sm[i];
    return s;
}

// One block per row, three passes over it.
template <typename XT, typename YT, typename WT>
__global__ void __launch_bounds__(NT) norm_fwd_kernel(NormParams p) {
    __shared__ float sm[NT / 32];
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        YT* y = static_cast<YT*>(p.y) + (size_t)r * p.D;
        float s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += NT) s += ld_f32(x + c);
        const float mean = block_sum(s, sm) * inv;
        s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += NT) { const float v = ld_f32(x + c) - mean; s = fmaf(v, v, s); }
        const float rstd = 1.f / sqrtf(block_sum(s, sm) * inv + p.eps);
        for (int c = threadIdx.x; c < p.D; c += NT) {
            float v = (ld_f32(x + c) - mean) * rstd;
            if (p.weight) v *= ld_f32(static_cast<const WT*>(p.weight) + c);
            if (p.bias) v += ld_f32(static_cast<const WT*>(p.bias) + c);
            st_from_f32(y + c, v);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

template <typename XT, typename YT, typename WT>
__global__ void __launch_bounds__(NT) norm_dx_kernel(NormParams p) {
    __shared__ float sm[NT / 32];
    const float inv = 1.f / (float)p.D;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const XT* x = static_cast<const XT*>(p.x) + (size_t)r * p.D;
        const YT* dy = static_cast<const YT*>(p.dy) + (size_t)r * p.D;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.D; c += NT) {
            const float w = p.weight ? ld_f32(static_cast<const WT*>(p.weight) + c) : 1.f;
            const float wd = w * ld_f32(dy + c);
            s1 += wd;
            s2 = fmaf(wd, (ld_f32(x + c) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, sm) * inv;
        s2 = block_sum(s2, sm) * inv;
        XT* dx = static_cast<XT*>(p.dx) + (size_t)r * p.D;
        for (int c = threadIdx.x; c < p.D; c += NT) {
            const float w = p.weight ? ld_f32(static_cast<const WT*>(p.weight) + c) : 1.f;
            const float xh = (ld_f32(x + c) - mean) * rstd;
            st_from_f32(dx + c, rstd * (w * ld_f32(dy + c) - s1 - xh * s2));
        }
    }
}

// Rows part, part + parts, .. of one column per thread.
template <typename XT, typename YT>
__global__ void __launch_bounds__(NT) norm_part_kernel(NormParams p) {
    const int c = blockIdx.x * NT + threadIdx.x;
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

__global__ void __launch_bounds__(NT) norm_sum_kernel(NormParams p) {
    const int c = blockIdx.x * NT + threadIdx.x;
    if (c >= p.D) return;
    float w = 0.f, b = 0.f;
    for (int i = 0; i < p.parts; ++i) {
        if (p.part_w) w += p.part_w[(size_t)i * p.D + c];
        if (p.part_b) b += p.part_b[(size_t)i * p.D + c];
    }
    if (p.dweight) p.dweight[c] = w;
    if (p.dbias) p.dbias[c] = b;
}

static unsigned row_grid(const NormParams& p) {
    const long long cap = (long long)device_sm_count() * 8;
    return (unsigned)(p.rows < cap ? p.rows : cap);
}

template <typename XT, typename YT, typename WT>
static gdr_status launch(bool bwd, const NormParams& p, cudaStream_t st) {
    if (!bwd) norm_fwd_kernel<XT, YT, WT><<<row_grid(p), NT, 0, st>>>(p);
    else {
        if (p.dx && p.rows > 0) norm_dx_kernel<XT, YT, WT><<<row_grid(p), NT, 0, st>>>(p);
        if (p.dweight || p.dbias) {
            const unsigned cols = (unsigned)((p.D + NT - 1) / NT);
            norm_part_kernel<XT, YT><<<dim3(cols, p.parts), NT, 0, st>>>(p);
            norm_sum_kernel<<<cols, NT, 0, st>>>(p);
        }
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(layer norm)");
}
template <typename XT, typename YT>
static gdr_status launch_w(const gdr_norm_desc* d, bool bwd, const NormParams& p, cudaStream_t st) {
    return d->w_dtype == GDR_BF16 ? launch<XT, YT, __nv_bfloat16>(bwd, p, st) : launch<XT, YT, float>(bwd, p, st);
}
static gdr_status dispatch(const gdr_norm_desc* d, bool bwd, const NormParams& p, cudaStream_t st) {
    const bool xb = d->x_dtype == GDR_BF16, yb = d->y_dtype == GDR_BF16;
    if (xb && yb) return launch_w<__nv_bfloat16, __nv_bfloat16>(d, bwd, p, st);
    if (xb) return launch_w<__nv_bfloat16, float>(d, bwd, p, st);
    if (yb) return launch_w<float, __nv_bfloat16>(d, bwd, p, st);
    return launch_w<float, float>(d, bwd, p, st);
}

static gdr_status check_desc(const gdr_norm_desc* d) {
    if (!d) return fail(GDR_ERR_INVALID_ARG, "desc is NULL%s");
    if (d->rows < 0) return fail(GDR_ERR_INVALID_ARG, "rows must be >= 0%s");
    if (d->D < 1 || d->D > (1 << 20)) return fail(GDR_ERR_UNSUPPORTED, "D must be 1 .. 2^20%s");
    if (d->rows > (1LL << 40)) return fail(GDR_ERR_UNSUPPORTED, "rows must be at most 2^40%s");
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->y_dtype) || !dtype_ok(d->w_dtype))
        return fail(GDR_ERR_INVALID_ARG, "bad dtype%s");
    if (!(d->eps >= 0.f)) return fail(GDR_ERR_INVALID_ARG, "eps must be >= 0%s");
    return GDR_OK;
}

static int parts_of(const gdr_norm_desc* d) { return (int)(d->rows < PARTS ? (d->rows > 0 ? d->rows : 1) : PARTS); }

}  // namespace lnm

cudaError_t norm_take_status(unsigned int* word, unsigned int* site) { return take_status_here(word, site); }

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_layernorm_fwd(const gdr_norm_desc* d, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = lnm::check_desc(d);
    if (s != GDR_OK) return s;
    for (const void* q : {x, weight, bias, (const void*)y, (const void*)mean, (const void*)rstd})
        if (q && !aligned16(q)) return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned%s");
    if (d->rows == 0) return GDR_OK;
    if (!x || !y) return fail(GDR_ERR_INVALID_ARG, "x and y are required%s");
    lnm::NormParams p = {};
    p.rows = d->rows; p.D = d->D; p.eps = d->eps;
    p.x = x; p.weight = weight; p.bias = bias; p.y = y; p.mean = mean; p.rstd = rstd;
    return lnm::dispatch(d, false, p, reinterpret_cast<cudaStream_t>(stream));
}

size_t gdr_layernorm_bwd_workspace_bytes(const gdr_norm_desc* d, int with_dweight, int with_dbias) {
    if (lnm::check_desc(d) != GDR_OK) return 0;
    return (size_t)lnm::parts_of(d) * d->D * ((with_dweight ? 1 : 0) + (with_dbias ? 1 : 0)) * sizeof(float);
}

gdr_status gdr_layernorm_bwd(const gdr_norm_desc* d, const void* x, const void* dy, const void* weight,
                             const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                             void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = lnm::check_desc(d);
    if (s != GDR_OK) return s;
    for (const void* q : {x, dy, weight, (const void*)mean, (const void*)rstd, (const void*)dx, (const void*)dweight,
                          (const void*)dbias, (const void*)workspace})
        if (q && !aligned16(q)) return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned%s");
    if (!dx && !dweight && !dbias) return GDR_OK;
    if (d->rows > 0 && (!x || !dy || !mean || !rstd))
        return fail(GDR_ERR_INVALID_ARG, "x, dy, mean and rstd are required%s");
    const size_t need = gdr_layernorm_bwd_workspace_bytes(d, dweight != nullptr, dbias != nullptr);
    if (need > 0 && (!workspace || workspace_bytes < need)) return fail(GDR_ERR_WORKSPACE, "workspace too small%s");
    lnm::NormParams p = {};
    p.rows = d->rows; p.D = d->D; p.eps = d->eps;
    p.x = x; p.dy = dy; p.weight = weight; p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dx = dx; p.dweight = dweight; p.dbias = dbias;
    p.parts = lnm::parts_of(d);
    float* ws = static_cast<float*>(workspace);
    if (dweight) { p.part_w = ws; ws += (size_t)p.parts * d->D; }
    if (dbias) p.part_b = ws;
    return lnm::dispatch(d, true, p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
