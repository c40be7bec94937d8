// norm.cu -- layer norm forward and backward (gdr_layernorm_fwd, gdr_layernorm_bwd): argument
// checks, dispatch and kernels.
#include <initializer_list>

#include "gdr.h"
#include "host.cuh"
#include "common.cuh"
#include "norm.cuh"

namespace gdr {
namespace lnm {

// How a row of D elements is held: V elements a load, N loads a lane, G lanes (of a warp, or a block
// of G threads); N = 0: the row is too long for a block's registers.  Shifted: rows of V-element
// chunks that begin and end inside one.
struct Plan { int V, N, G; bool shift; };
// The backward of longer rows: in registers as they lie in memory, where 16-byte access fits.
static bool wide(int D, int V, bool bwd) { return bwd && V > 1 && D % V == 0 && D > 8 * 1024 && D <= 16 * 1024; }

// A warp while a lane holds at most 16 elements (one by one, and in the backward, which also holds
// dy, the weights and two sums: 8), then the block that holds the fewest elements beside the row.
// 33.5 M bf16 elements: rows of 1024 in 32 elements a lane of a warp 32.3 us forward, in 8 of 128
// threads 28.0; rows of 2560 in 16 of 192 27.8, of 256 37.7; backward, rows of 512 in 64 threads
// 39.7 us, in 128 54.2, rows of 6144 in 768 49.1, in 1024 56.6.
static Plan plan_of(int D, int V, bool bwd, bool shift) {
    Plan q{V, 0, 32, shift};
    const int nv = (D + (shift ? V - (D & -D) : 0) + V - 1) / V;     // loads of a row
    if (nv <= 32) {                             // one load a lane, as few lanes as hold the row
        q.N = 1;
        for (q.G = 1; q.G < nv; q.G *= 2) {}
        return q;
    }
    const int most = (bwd || V == 1 ? 8 : 16) / V;
    for (int n = 2; n <= most; n *= 2)
        if (nv <= 32 * n) { q.N = n; return q; }
    int held = 1 << 20;
    for (int g : {64, 96, 128, 192, 256, 384, 512, 768, 1024})
        for (int n = V == 1 || bwd ? most : 1; n <= most; n *= 2) {
            if (nv > g * n || g * n > held || (n < most && g > 128)) continue;
            held = g * n;
            q.G = g;
            q.N = n;
        }
    if (!bwd && V == 1 && !q.N && nv <= 16 * 1024) { q.G = 1024; q.N = 16; }
    return q;
}
// Rows of D elements where 16-byte access takes V of them.  Rows that are not multiples of it:
// shifted, where that holds no more elements than one by one, or takes few lanes; forward not by a
// whole warp a row of one load each, of fp32 only by less than a warp, and with weights in registers.
// (33.5 M bf16 elements, shifted against one by one: backward rows of 9 66 and 247 us, 14 83 and 161,
// 333 60 and 73, 5001 68 and 117; but 2047, in 384 threads, 64 and 55.  Forward 9 67 and 146, 14 80
// and 95, 5001 44 and 59, but 129 73 and 66; 16.8 M fp32, rows of 2047 64 and 23.)
static Plan plan(int D, int V, bool bwd) {
    if (D % V == 0) return plan_of(D, V, bwd, false);
    const Plan one = plan_of(D, 1, bwd, false), q = plan_of(D, V, bwd, true);
    const bool fits = q.N && (q.V * q.N * q.G <= (one.N ? one.N * one.G : 1 << 20) || q.G <= (bwd ? 16 : 4)) &&
                      (bwd || q.G < 32 || (V == 8 && q.N * q.G > 32 && q.G < 1024));
    return D > V && fits ? q : one;             // D > V: a chunk reaches into one neighbouring row at most
}
static int rows_of_block(const Plan& q) { return q.N && q.G <= 32 ? WARP_NT / q.G : 1; }
static int vector_of(const gdr_norm_desc* d) { return d->x_dtype == GDR_BF16 && d->y_dtype == GDR_BF16 ? 8 : 4; }

template <typename XT, typename YT, int V, int N, int G, bool BWD, bool SHIFT>
static gdr_status launch_one(const NormParams& p, cudaStream_t st) {
    constexpr int NTH = threads<G>(), per = NTH / G, U = rows_at_once<V, N, G>();
    if constexpr (!BWD) {
        constexpr int M = SHIFT && per % V ? V : 1;    // shifted: the grid's groups in multiples of V
        const long long blocks = (p.rows + per * U - 1) / (per * U), cap = (long long)device_sm_count() * fwd_blocks<SHIFT>(V, N, NTH);
        const long long grid = blocks + M - 1 < cap ? blocks + M - 1 : cap;
        norm_fwd_kernel<XT, YT, V, N, G, SHIFT><<<(unsigned)(grid < M ? M : grid / M * M), NTH, 0, st>>>(p);
    } else {
        // the groups' sums in turn: at most 256 threads x 16 columns
        const size_t smem = per == 1 || !(p.part_w || p.part_b) ? 0 : (size_t)per * p.D * sizeof(float);
        norm_bwd_kernel<XT, YT, V, N, G, SHIFT><<<p.parts, NTH, smem, st>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(layer norm)");
}

// The kernels that plan_of reaches.
template <typename XT, typename YT, int V, bool BWD, bool SHIFT>
static gdr_status launch_plan(const Plan& q, const NormParams& p, cudaStream_t st) {
#define GDR_NORM(n, g) if (q.N == n && q.G == g) return launch_one<XT, YT, V, n, g, BWD, SHIFT>(p, st)
    constexpr int MOST = (BWD || V == 1 ? 8 : 16) / V;
    if constexpr (!SHIFT) GDR_NORM(1, 1);
    GDR_NORM(1, 2); GDR_NORM(1, 4); GDR_NORM(1, 8); GDR_NORM(1, 16);
    if constexpr (BWD || !SHIFT) GDR_NORM(1, 32);
    if constexpr (BWD || V != 4 || !SHIFT) {
        if constexpr (MOST >= 2) GDR_NORM(2, 32);
        if constexpr (MOST >= 4) GDR_NORM(4, 32);
        if constexpr (MOST >= 8) GDR_NORM(8, 32);
        if constexpr (V == 8 && !BWD) { GDR_NORM(1, 96); GDR_NORM(1, 128); }
        if constexpr (V == 4 && !BWD) { GDR_NORM(2, 96); GDR_NORM(2, 128); }
        if constexpr (V == 1 || BWD) GDR_NORM(MOST, 64);
        GDR_NORM(MOST, 96); GDR_NORM(MOST, 128); GDR_NORM(MOST, 192); GDR_NORM(MOST, 256); GDR_NORM(MOST, 384);
        GDR_NORM(MOST, 512); GDR_NORM(MOST, 768);
        if constexpr (BWD || !SHIFT) GDR_NORM(MOST, 1024);
        if constexpr (V == 1 && !BWD) GDR_NORM(16, 1024);
    }
#undef GDR_NORM
    return fail(GDR_ERR_UNSUPPORTED, "layer norm: no kernel for this plan%s");
}

template <typename XT, typename YT, int V, bool BWD>
static gdr_status launch_width(const Plan& q, const NormParams& p, cudaStream_t st) {
    if (q.V == 1) return launch_plan<XT, YT, 1, BWD, false>(q, p, st);
    return q.shift ? launch_plan<XT, YT, V, BWD, true>(q, p, st) : launch_plan<XT, YT, V, BWD, false>(q, p, st);
}

template <typename XT, typename YT>
static gdr_status launch(const gdr_norm_desc* d, bool bwd, NormParams& p, cudaStream_t st) {
    constexpr int V = sizeof(XT) == 2 && sizeof(YT) == 2 ? 8 : 4;
    // one element a load where a tensor does not start on 16 bytes
    bool on16 = true;
    for (const void* a : {p.x, p.dy, p.weight, p.bias, (const void*)p.y, (const void*)p.dx}) on16 = on16 && aligned16(a);
    const Plan q = plan(p.D, on16 ? vector_of(d) : 1, bwd);
    p.w_bf16 = d->w_dtype == GDR_BF16;
    gdr_status s = GDR_OK;
    if (p.rows > 0) {
        if (q.N && bwd) s = launch_width<XT, YT, V, true>(q, p, st);
        else if (q.N) s = launch_width<XT, YT, V, false>(q, p, st);
        else if (wide(p.D, q.V, bwd)) {
            const auto kernel = norm_bwd_wide_kernel<XT, YT, V, 16 / V>;
            constexpr int SUMS = 2 * 16 * WIDE_NT * (int)sizeof(float);
            // the kernel's limit, which calls on other host threads share: always the largest
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SUMS);
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(layer norm)");
            kernel<<<p.parts, WIDE_NT, p.part_w || p.part_b ? SUMS : 0, st>>>(p);
        } else {
            const unsigned grid = (unsigned)(p.rows < 2 * device_sm_count() ? p.rows : 2 * device_sm_count());
            if (!bwd) norm_fwd_long_kernel<XT, YT><<<grid, LONG_NT, 0, st>>>(p);
            else {
                if (p.dx) norm_dx_long_kernel<XT, YT><<<grid, LONG_NT, 0, st>>>(p);
                if (p.part_w || p.part_b)
                    norm_part_long_kernel<XT, YT><<<dim3((unsigned)((p.D + 255) / 256), p.parts), 256, 0, st>>>(p);
            }
        }
    }
    if (s == GDR_OK && bwd && (p.dweight || p.dbias)) {
        if (p.rows > 0) {
            const unsigned cols = (unsigned)((p.D + 31) / 32);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(cols * ((p.dweight ? 1 : 0) + (p.dbias ? 1 : 0)));
            cfg.blockDim = dim3(SUM_NT);
            cfg.stream = st;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_sum_kernel, p);
            if (e != cudaSuccess) return cuda_fail(e, "launch(layer norm sums)");
        } else {
            cudaError_t e = cudaSuccess;
            for (float* q0 : {p.dweight, p.dbias})
                if (q0 && e == cudaSuccess) e = cudaMemsetAsync(q0, 0, (size_t)p.D * sizeof(float), st);
            if (e != cudaSuccess) return cuda_fail(e, "memset(dweight, dbias)");
        }
    }
    const cudaError_t e = cudaGetLastError();
    return s != GDR_OK ? s : e == cudaSuccess ? GDR_OK : cuda_fail(e, "launch(layer norm)");
}

// Blocks of the backward, each with a partial row of its own: 512 threads per SM, and at least
// eight rows for each of a block's groups, so that the partial rows stay few against the rows.
static int parts_of(const gdr_norm_desc* d) {
    const Plan q = plan(d->D, vector_of(d), true);
    const long long per = rows_of_block(q), n = (d->rows + 8 * per - 1) / (8 * per);
    const long long cap = (long long)device_sm_count() * (q.N ? bwd_blocks(q.G > 32 ? q.G : WARP_NT) : wide(d->D, q.V, true) ? 1 : 2);
    // shifted rows of a block: blocks in multiples of V, but no more than stay on the GPU
    const long long M = q.shift && per % q.V ? q.V : 1, parts = n < cap ? n + M - 1 : cap;
    return (int)(parts < M ? M : (parts < cap ? parts : cap) / M * M);
}

static gdr_status dispatch(const gdr_norm_desc* d, bool bwd, NormParams& p, cudaStream_t st) {
    const bool xb = d->x_dtype == GDR_BF16, yb = d->y_dtype == GDR_BF16;
    if (xb && yb) return launch<__nv_bfloat16, __nv_bfloat16>(d, bwd, p, st);
    if (xb) return launch<__nv_bfloat16, float>(d, bwd, p, st);
    if (yb) return launch<float, __nv_bfloat16>(d, bwd, p, st);
    return launch<float, float>(d, bwd, p, st);
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

}  // namespace lnm

cudaError_t norm_status(StatusWords* w) { return status_here(w); }

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_layernorm_fwd(const gdr_norm_desc* d, const void* x, const void* weight, const void* bias, void* y,
                             float* mean, float* rstd, gdr_stream_t stream) {
    t_detail[0] = 0;
    const gdr_status s = lnm::check_desc(d);
    if (s != GDR_OK) return s;
    if (!aligned_to(x, d->x_dtype) || !aligned_to(y, d->y_dtype) || !aligned_to(weight, d->w_dtype) ||
        !aligned_to(bias, d->w_dtype) || !aligned4(mean) || !aligned4(rstd))
        return fail(GDR_ERR_INVALID_ARG, "pointers must be aligned to their elements%s");
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
    if (!aligned_to(x, d->x_dtype) || !aligned_to(dx, d->x_dtype) || !aligned_to(dy, d->y_dtype) ||
        !aligned_to(weight, d->w_dtype) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias))
        return fail(GDR_ERR_INVALID_ARG, "pointers must be aligned to their elements%s");
    if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned%s");
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
