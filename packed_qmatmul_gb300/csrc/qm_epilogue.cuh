// qm_epilogue.cuh -- what becomes of a product's float32 sums before their one
// rounding: bias, activation or gate, residual (qm_epilogue), shared by every
// product kernel.
//
// v / (1 + exp(-z)) is v times the reciprocal of 1 + 2^(-z log2 e), two special-function
// results and three products: exp2 is off by 2^-22 and, through its argument's rounding,
// by |z| 2^-23 relative, the reciprocal by 2^-23, both far below bf16's 2^-9. An
// exponential that overflows gives v times 0, and results below 2^-118 in size may
// come out as 0. tanh in gelu is the same: (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
//
// gelu's (1 + erf(v / sqrt 2)) / 2 is half of erfc(z) = exp(-z^2) g(z), z = |v| / sqrt 2, or 1 less
// that: g falls from 1 like 1 / z, and g(z) / t, t = 1 / (1 + 0.46 z), is a polynomial of
// degree 7 in t to 2^-20 of itself over z >= 0 (a least-squares fit reweighted towards its
// largest relative error), so that the tail keeps its relative precision.
#pragma once

#include "qm_device.cuh"
#include "qm_internal.h"

namespace qm {

QM_DEV float ex2_ftz(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
QM_DEV float rcp_ftz(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Maximum and minimum that keep a NaN.
QM_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
QM_DEV float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kLog2e = 1.44269504f;

QM_DEV float gelu_f(float v) {
    const float z = fabsf(v) * 0.70710678f, t = rcp_ftz(fmaf(0.46f, z, 1.0f));
    float g = 0.06773512f;
    g = fmaf(g, t, -0.22670604f);
    g = fmaf(g, t, 0.16930445f);
    g = fmaf(g, t, 0.05252517f);
    g = fmaf(g, t, 0.18688236f);
    g = fmaf(g, t, 0.23117466f);
    g = fmaf(g, t, 0.25955793f);
    g = fmaf(g, t, 0.25952703f);
    const float q = 0.5f * t * g * ex2_ftz(z * z * -kLog2e);
    return v * (v < 0.0f ? q : 1.0f - q);
}

// neg_alpha: -alpha log2 e.
template <int ACT>
QM_DEV float act_f(float v, float neg_alpha) {
    if constexpr (ACT == QM_ACT_RELU) return max_nan(v, 0.0f);
    if constexpr (ACT == QM_ACT_SILU) return v * rcp_ftz(1.0f + ex2_ftz(v * neg_alpha));
    if constexpr (ACT == QM_ACT_GELU) return gelu_f(v);
    if constexpr (ACT == QM_ACT_GELU_TANH)  // 2 sqrt(2 / pi) log2 e (v + 0.044715 v^3)
        return v * rcp_ftz(1.0f + ex2_ftz(v * fmaf(v * v, -0.10294324f, -2.3022082f)));
    return v;
}

// v[0], v[STEP], ... through the activation.
template <int STEP, int N>
QM_DEV void act_all(const Epi& e, float (&v)[N]) {
    const float neg_alpha = e.alpha * -kLog2e;
    switch (e.act) {
#define QM_ACT_CASE(A)                                                                      \
    case A:                                                                                 \
        _Pragma("unroll") for (int i = 0; i < N; i += STEP) v[i] = act_f<A>(v[i], neg_alpha); \
        break;
        QM_ACT_CASE(QM_ACT_RELU)
        QM_ACT_CASE(QM_ACT_SILU)
        QM_ACT_CASE(QM_ACT_GELU)
        QM_ACT_CASE(QM_ACT_GELU_TANH)
#undef QM_ACT_CASE
        default: break;
    }
}

QM_DEV float epi_act(const Epi& e, float v) {
    float a[1] = {v};
    act_all<1>(e, a);
    return a[0];
}

// A gate's argument and what stands beside it, clamped (NaN stays).
QM_DEV float clamp_gate(const Epi& e, float g) { return min_nan(g, e.limit); }
QM_DEV float clamp_up(const Epi& e, float u) { return max_nan(min_nan(u, e.limit), -e.limit) + e.up_offset; }

QM_DEV float epi_gate(const Epi& e, float g, float u) { return epi_act(e, clamp_gate(e, g)) * clamp_up(e, u); }

// Element `i` of the bias as its bits, and their value: apart, so that a load can be under way
// while something else is done.
QM_DEV uint32_t epi_bias_bits(const Epi& e, int64_t i) {
    if (e.bias_dtype == QM_F32) return __ldg(static_cast<const uint32_t*>(e.bias) + i);
    return __ldg(static_cast<const uint16_t*>(e.bias) + i);
}
QM_DEV float epi_bias_value(const Epi& e, uint32_t bits) {
    return e.bias_dtype == QM_F32 ? __uint_as_float(bits) : e.bias_dtype == QM_F16 ? f16_bits_to_f32(bits) : bf16_bits_to_f32(bits);
}

// Element `i` of the bias (0 without one).
QM_DEV float epi_bias(const Epi& e, int64_t i) { return e.bias ? epi_bias_value(e, epi_bias_bits(e, i)) : 0.0f; }

// The residual of result (row, col) (0 without one): a coherent load, since y may be
// the residual and an earlier kernel may just have written it.
QM_DEV float epi_residual(const Epi& e, int64_t row, int64_t col) {
    return e.residual ? bf16_bits_to_f32(__ldca(e.residual + row * e.residual_stride + col)) : 0.0f;
}

// Asks for the line at p, which a later load then finds in L1.
QM_DEV void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

QM_DEV uint16_t bf16_bits(float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&b);
}

// The activation of v, or of the gate v times u, both with their bias. Out of line and by
// value, for the kernels that finish few results to a thread: their loops keep their registers.
static __device__ __noinline__ float epi_value(int act, int gated, float alpha, float limit, float up_offset, float v, float u) {
    Epi e;
    e.act = act;
    e.alpha = alpha;
    e.limit = limit;
    e.up_offset = up_offset;
    return gated ? epi_gate(e, v, u) : epi_act(e, v);
}

// One result (row, col) from its sum v (gated: the gate's v and the sum u beside it), both with their bias.
QM_DEV uint16_t epi_result(const Epi& e, float v, float u, int64_t row, int64_t col) {
    const float r = epi_residual(e, row, col);
    return bf16_bits(epi_value(e.act, e.gated, e.alpha, e.limit, e.up_offset, v, u) + r);
}

// The same with bias elements from brow on still to be added.
QM_DEV uint16_t epi_finish(const Epi& e, float v, float u, int64_t brow, int64_t row, int64_t col) {
    return epi_result(e, v + epi_bias(e, brow), e.gated ? u + epi_bias(e, brow + 1) : 0.0f, row, col);
}

}  // namespace qm
