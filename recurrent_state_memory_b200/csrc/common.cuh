// common.cuh -- small device helpers shared by the gdr kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

// Device status word: kernels OR in a bit when a bounded wait gives up (bit 0) or a
// decay factor leaves the range of the factored tensor-core form (bit 1).  Read and
// cleared by gdr_query_device_status.  (Every translation unit has a word of its own.)
static __device__ unsigned int g_device_status = 0;

// Index checks of the debug build (compiled with -DGDR_BOUNDS_CHECK).  GDR_INB(cond, site)
// guards one global-memory access: when cond fails, the site number goes to g_bounds_site (the
// first failure is kept), bit 2 of the status word is set and the access is skipped.  In the
// default build the macro is the constant true and costs nothing.
constexpr unsigned STATUS_TIMEOUT = 1u;
constexpr unsigned STATUS_BOUNDS = 4u;
constexpr unsigned STATUS_INDEX = 8u;      // an index that the caller passed in device memory is out of range
static __device__ unsigned int g_bounds_site = 0;
#ifdef GDR_BOUNDS_CHECK
__device__ __forceinline__ bool in_bounds(bool c, unsigned site) {
    if (!c) {
        atomicCAS(&g_bounds_site, 0u, site);
        atomicOr(&g_device_status, STATUS_BOUNDS);
    }
    return c;
}
#define GDR_INB(cond, site) ::gdr::in_bounds((cond), (site))
#define GDR_AND_INB(cond, site) && ::gdr::in_bounds((cond), (site))
#else
#define GDR_INB(cond, site) true
#define GDR_AND_INB(cond, site)         // behind a condition whose code should not notice the mark
#endif

// Where this translation unit's status word and first bounds site are on the current device.
struct StatusWords { unsigned int *word, *site; };
static inline cudaError_t status_here(StatusWords* w) {
    const cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&w->word), g_device_status);
    return e == cudaSuccess ? cudaGetSymbolAddress(reinterpret_cast<void**>(&w->site), g_bounds_site) : e;
}

// Element loads/stores with the storage type chosen at compile time.
template <typename T> __device__ __forceinline__ float ld_f32(const T* p);
template <> __device__ __forceinline__ float ld_f32<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float ld_f32<__nv_bfloat16>(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
}

template <typename T> __device__ __forceinline__ void st_from_f32(T* p, float x);
template <> __device__ __forceinline__ void st_from_f32<float>(float* p, float x) { *p = x; }
template <> __device__ __forceinline__ void st_from_f32<__nv_bfloat16>(__nv_bfloat16* p, float x) {
    *p = __float2bfloat16_rn(x);
}

// Two fp32 values in one register pair: sm_100 adds, multiplies and fuses them in one instruction.
struct Pair { unsigned long long v; };
__device__ __forceinline__ Pair pair(float a, float b) { Pair p; asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b)); return p; }
__device__ __forceinline__ float lo(Pair p) { float a; asm("{\n\t.reg .f32 t;\n\tmov.b64 {%0, t}, %1;\n\t}" : "=f"(a) : "l"(p.v)); return a; }
__device__ __forceinline__ float hi(Pair p) { float b; asm("{\n\t.reg .f32 t;\n\tmov.b64 {t, %0}, %1;\n\t}" : "=f"(b) : "l"(p.v)); return b; }
__device__ __forceinline__ Pair operator+(Pair a, Pair b) { Pair d; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v)); return d; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) { Pair d; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v)); return d; }
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) { Pair d; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v)); return d; }

// Log-decay of one gate value.  gate_mode 1: g = -softplus(a) = -(max(a,0) + log1p(e^{-|a|})),
// the activation the workloads state; gate_mode 0: the value is g itself.
__device__ __forceinline__ float log_decay(float a, int gate_mode) {
    if (gate_mode == 1) return -(fmaxf(a, 0.f) + log1pf(expf(-fabsf(a))));
    return a;
}

// Multiplicative decay alpha = exp(g) of one gate value, computed without the
// log: for gate_mode 1, exp(-softplus(a)) = 1 / (1 + e^{a}) (a -> +inf gives 0).
__device__ __forceinline__ float decay_factor(float a, int gate_mode) {
    if (gate_mode == 1) return 1.f / (1.f + expf(a));
    return expf(a);
}

// The decay a = exp(g) of one gate value v, and 1 - a (REST) without taking a difference, which
// would lose it where a is near one.  Mode 1 with e = e^v: a = 1 / (1 + e), 1 - a = e a, and e is
// held at 2^126 where it would reach the product as infinity.  The product v log2(e) is rounded
// once and its error left in place: it moves the gate by 1.25 steps of 2^-24 of its own value, as
// storing the gate in fp32 does already.  NaN stays NaN.
template <int MODE, bool REST>
__device__ __forceinline__ void decay_pair(float v, float& a, float& rest) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * 1.44269502f));
    if constexpr (MODE == 1) {
        if constexpr (REST) asm("min.NaN.f32 %0, %1, %2;" : "=f"(e) : "f"(e), "f"(8.50705917e37f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.f + e));
        if constexpr (REST) rest = e * a;
    } else {
        a = e;
        if constexpr (REST) rest = -expm1f(v);
    }
}

// Reduce an angle to [-pi, pi] so that sums of many angles keep full accuracy.
__device__ __forceinline__ float wrap_angle(float x) {
    const float two_pi = 6.283185307179586f;
    return x - two_pi * rintf(x * (1.f / two_pi));
}

}  // namespace gdr
