// qm_epilogue.cuh -- what becomes of a product's float32 sums before their one
// rounding: bias, activation or gate, residual (qm_epilogue), shared by every
// product kernel.
//
// sigmoid(z) is formed from t = exp(-|z|) <= 1, as 1 / (1 + t) or t / (1 + t), so
// that nothing overflows and small results keep their relative precision:
// exp2 of the scaled argument and the quotient are the fast forms, off by at most
// 2^-21 + |z| 2^-23 relative (the argument's rounding), far below bf16's 2^-9
// wherever the result is not itself below 1e-38. tanh in gelu is the same sigmoid,
// (1 + tanh z) / 2 = sigmoid(2 z), and 1 + erf is erfc, which keeps the tail.
#pragma once

#include "qm_device.cuh"
#include "qm_internal.h"

namespace qm {

QM_DEV float sigmoid_f(float z) {
    const float t = __expf(-fabsf(z));
    return __fdividef(z < 0.0f ? t : 1.0f, 1.0f + t);  // z NaN: t NaN
}

// Out of line: the one activation of more than a dozen instructions.
static __device__ __noinline__ float gelu_f(float v) { return 0.5f * v * erfcf(v * -0.70710678f); }

template <int ACT>
QM_DEV float act_f(float v, float alpha) {
    if constexpr (ACT == QM_ACT_RELU) return v < 0.0f ? 0.0f : v;  // NaN stays
    if constexpr (ACT == QM_ACT_SILU) return v * sigmoid_f(alpha * v);
    if constexpr (ACT == QM_ACT_GELU) return gelu_f(v);
    if constexpr (ACT == QM_ACT_GELU_TANH) return v * sigmoid_f(1.5957691f * fmaf(0.044715f * v * v, v, v));
    return v;
}

// v[0], v[STEP], ... through the activation.
template <int STEP, int N>
QM_DEV void act_all(const Epi& e, float (&v)[N]) {
    switch (e.act) {
#define QM_ACT_CASE(A)                                                                      \
    case A:                                                                                 \
        _Pragma("unroll") for (int i = 0; i < N; i += STEP) v[i] = act_f<A>(v[i], e.alpha); \
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
QM_DEV float clamp_gate(const Epi& e, float g) { return g > e.limit ? e.limit : g; }
QM_DEV float clamp_up(const Epi& e, float u) { return (u > e.limit ? e.limit : (u < -e.limit ? -e.limit : u)) + e.up_offset; }

QM_DEV float epi_gate(const Epi& e, float g, float u) { return epi_act(e, clamp_gate(e, g)) * clamp_up(e, u); }

// Element `i` of the bias (0 without one).
QM_DEV float epi_bias(const Epi& e, int64_t i) {
    if (!e.bias) return 0.0f;
    if (e.bias_dtype == QM_F32) return __ldg(static_cast<const float*>(e.bias) + i);
    const uint32_t h = __ldg(static_cast<const uint16_t*>(e.bias) + i);
    return e.bias_dtype == QM_F16 ? f16_bits_to_f32(h) : bf16_bits_to_f32(h);
}

// The residual of result (row, col) (0 without one): a coherent load, since y may be
// the residual and an earlier kernel may just have written it.
QM_DEV float epi_residual(const Epi& e, int64_t row, int64_t col) {
    return e.residual ? bf16_bits_to_f32(__ldca(e.residual + row * e.residual_stride + col)) : 0.0f;
}

QM_DEV uint16_t bf16_bits(float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&b);
}

// One result from its sum v (gated: the gate's v and the sum u beside it): bias
// elements from brow on, result (row, col). Out of line, for the kernels that finish
// few results to a thread: their loops keep their registers.
static __device__ __noinline__ uint16_t epi_finish(const Epi& e, float v, float u, int64_t brow, int64_t row, int64_t col) {
    v += epi_bias(e, brow);
    v = e.gated ? epi_gate(e, v, u + epi_bias(e, brow + 1)) : epi_act(e, v);
    return bf16_bits(v + epi_residual(e, row, col));
}

}  // namespace qm
