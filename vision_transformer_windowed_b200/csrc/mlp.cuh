// Pieces shared by the kernels of the gated feed-forward block: matrix tiles by TMA, the
// activations.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace fswin {

namespace mlp {

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ unsigned long long pair_of(float x) { return pair(x, x); }

// act(g) and, for the gradient, act'(g) of two values.
// silu: g s, s (1 + g (1 - s)) with s = 1 / (1 + e^-g).
// gelu: g Phi(g), Phi(g) + g phi(g).  Phi(-x) = e^(-x^2 / 2) R(x) for x >= 0, R(x) the
// scaled complementary error function erfcx(x / sqrt 2) / 2 as t P(t), t = 1 / (1 + 0.31 x),
// P of degree 5, fitted for this file by reweighted least squares over 0 <= x <= 14: the
// relative error is below 4.7e-6, about 1e-5 with the fp32 steps, so that the tail too is
// right to the rounding of its bf16 result.  Phi(x) = 1 - Phi(-x).
// Four pairs at a time, step by step beside each other: one pair's steps depend on each
// other.
template <bool kSlope>
__device__ __forceinline__ void activate(const unsigned long long* g, int act, unsigned long long (&a)[4],
                                         unsigned long long (&slope)[4]) {
#define EACH _Pragma("unroll") for (int i = 0; i < 4; ++i)
    float x[4], y[4];
    if (act == 0) {
        EACH unpair(mul_pair(g[i], pair_of(-1.4426950408889634f)), x[i], y[i]);
        EACH unpair(add_pair(pair(ex2_approx(x[i]), ex2_approx(y[i])), pair_of(1.f)), x[i], y[i]);
        unsigned long long s[4];
        EACH s[i] = pair(rcp_approx(x[i]), rcp_approx(y[i]));
        EACH a[i] = mul_pair(g[i], s[i]);
        if (kSlope) EACH slope[i] = fma_pair(a[i], fma_pair(s[i], pair_of(-1.f), pair_of(1.f)), s[i]);
        return;
    }
    unsigned long long t[4], p[4], e[4], q[4];
    EACH unpair(fma_pair(g[i] & 0x7FFFFFFF7FFFFFFFull, pair_of(0.31f), pair_of(1.f)), x[i], y[i]);
    EACH t[i] = pair(rcp_approx(x[i]), rcp_approx(y[i]));
    EACH unpair(mul_pair(mul_pair(g[i], g[i]), pair_of(-0.72134752044448170f)), x[i], y[i]);
    EACH e[i] = pair(ex2_approx(x[i]), ex2_approx(y[i]));
    EACH p[i] = fma_pair(t[i], pair_of(-0.07392913f), pair_of(0.18045032f));
    EACH p[i] = fma_pair(p[i], t[i], pair_of(0.015744742f));
    EACH p[i] = fma_pair(p[i], t[i], pair_of(0.13342977f));
    EACH p[i] = fma_pair(p[i], t[i], pair_of(0.12044128f));
    EACH p[i] = fma_pair(p[i], t[i], pair_of(0.1238607f));
    EACH p[i] = mul_pair(mul_pair(p[i], t[i]), e[i]);             // Phi(-|g|)
    EACH q[i] = fma_pair(p[i], pair_of(-1.f), pair_of(1.f));      // Phi(|g|)
    EACH {
        float lo, hi, up_lo, up_hi;
        unpair(p[i], lo, hi);
        unpair(q[i], up_lo, up_hi);
        p[i] = pair(static_cast<int>(g[i]) < 0 ? lo : up_lo, static_cast<long long>(g[i]) < 0 ? hi : up_hi);  // by g's signs
    }
    EACH a[i] = mul_pair(g[i], p[i]);
    if (kSlope) EACH slope[i] = fma_pair(mul_pair(g[i], pair_of(0.39894228040143268f)), e[i], p[i]);
#undef EACH
}

// Columns c, c + 1, ... of a bias, 0 past its end or without one.
__device__ __forceinline__ float bias_at(const __nv_bfloat16* bias, int c, int n) {
    return bias && c < n ? __bfloat162float(bias[c]) : 0.f;
}

}  // namespace mlp

}  // namespace fswin
