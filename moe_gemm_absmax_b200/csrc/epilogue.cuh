// The fused output step of w8a8_linear_epilogue, shared by every GEMM path:
//
//   v = (float(acc) * sx[m]) * sw[n]          (the plain linear's fp32 value)
//   y[m, n] = bf16_rne( residual[m, n] + act( v + bias[n] ) )
//
// One fp32 rounding for each product and sum, the activation in fp32, one
// rounding to bf16 at the end.  What it saves: as separate elementwise passes
// bias, activation and residual read and write the [M, N] output once more
// each; here they cost one bf16 read of the residual.
#pragma once

#include "common.cuh"

namespace w8a8 {

struct EpiFused {
    const float* bias;     // [N] or null
    const uint16_t* res;   // bf16 [M, N], row stride ldr, or null; may be the output itself
    int64_t ldr, ldy;      // row strides of residual and output, elements (multiples of 8)
    int act;               // W8A8_ACT_*
};

// 1 / (1 + e^-t): ex2.approx and a division good to 2 ulp, which leaves the
// result within 2^-21 of its value, 1/4096 of a bf16 rounding step.  Far left
// e^-t overflows to infinity and the quotient is 0, the limit.
__device__ __forceinline__ float fast_sigmoid(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

// v * Phi(v).  With a = |v|, Phi(-a) = e^(-a^2 / 2) erfcx(a / sqrt 2) / 2, the
// scaled complementary error function as t times a polynomial of degree 6 in
// t = 1 / (1 + 0.375 a / sqrt 2), fitted to the least largest relative error
// over a / sqrt 2 in [0, 10.5] (6.4e-7): the left tail keeps its digits, which
// 1 + erf would lose to cancellation, at half the instructions of normcdff
// and without its branches.
__device__ __forceinline__ float gelu_erf(float v) {
    const float a = fabsf(v);
    const float t = __fdividef(1.0f, __fmaf_rn(a, 0.26516504294495535f, 1.0f));
    float p = -1.350962669e-01f;
    p = __fmaf_rn(p, t, 3.879391849e-01f);
    p = __fmaf_rn(p, t, -1.295993030e-01f);
    p = __fmaf_rn(p, t, 2.830630541e-01f);
    p = __fmaf_rn(p, t, 1.666639745e-01f);
    p = __fmaf_rn(p, t, 2.156893015e-01f);
    p = __fmaf_rn(p, t, 2.113394439e-01f);
    const float q = 0.5f * p * t * __expf(-0.5f * a * a);   // Phi(-a)
    return v * (v < 0.0f ? q : 1.0f - q);
}

__device__ __forceinline__ float act_apply(int act, float v) {
    switch (act) {
        case W8A8_ACT_RELU: return fmaxf(v, 0.0f);
        case W8A8_ACT_SILU: return v * fast_sigmoid(v);
        case W8A8_ACT_GELU: return gelu_erf(v);
        // (1 + tanh u) / 2 = sigmoid(2u)
        case W8A8_ACT_GELU_TANH:
            return v * fast_sigmoid(1.5957691216057308f * __fmaf_rn(0.044715f * v * v, v, v));
        default: return v;
    }
}

// Eight consecutive columns of one row: int32 accumulators, the columns'
// scales and biases (shared memory), the residual's 16 bytes -> 16 bytes of bf16.
__device__ __forceinline__ uint4 epi_fused8(const uint32_t* r, float sx, const float* sw8, const float* bias8,
                                            const uint4& res, int act) {
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 s = *reinterpret_cast<const float4*>(sw8 + 4 * h);
        const float4 b = *reinterpret_cast<const float4*>(bias8 + 4 * h);
        const float sv[4] = {s.x, s.y, s.z, s.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[4 * h + j] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * h + j]), sx), sv[j]), bv[j]);
    }
    // one branch a vector, uniform over the grid
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f(v[j]);
    };
    if (act == W8A8_ACT_SILU) each([](float t) { return act_apply(W8A8_ACT_SILU, t); });
    else if (act == W8A8_ACT_RELU) each([](float t) { return act_apply(W8A8_ACT_RELU, t); });
    else if (act == W8A8_ACT_GELU) each([](float t) { return act_apply(W8A8_ACT_GELU, t); });
    else if (act == W8A8_ACT_GELU_TANH) each([](float t) { return act_apply(W8A8_ACT_GELU_TANH, t); });
    const uint32_t rw[4] = {res.x, res.y, res.z, res.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(__fadd_rn(v[2 * j], __uint_as_float(rw[j] << 16)),
                           __fadd_rn(v[2 * j + 1], __uint_as_float(rw[j] & 0xffff0000u)));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// One output, for the kernels that hold single columns.
__device__ __forceinline__ uint16_t epi_fused1(int acc, float sx, float sw, const EpiFused& f, int64_t m, int n) {
    float v = __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
    if (f.bias) v = __fadd_rn(v, __ldg(f.bias + n));
    v = act_apply(f.act, v);
    if (f.res) v = __fadd_rn(v, bf16_bits_to_float(__ldcg(f.res + m * f.ldr + n)));
    return float_to_bf16_bits(v);
}

// 16 bytes of the residual: coherent (it may be the output), past L1 (read once).
__device__ __forceinline__ uint4 ld_residual16(const uint16_t* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }

}  // namespace w8a8
