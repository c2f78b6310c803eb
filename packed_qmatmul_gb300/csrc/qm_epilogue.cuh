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
