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

// Activations on two values at a time (sm_100 adds and multiplies pairs of
// fp32 in one instruction).  1 / (1 + e^-t) from ex2.approx and rcp.approx,
// good to 2 ulp each; the exponent's roundings, 2^-24 of it each, come out as
// that part of e^-t times its size, so that the value is within 2^-19 of the
// true one for |t| < 8 and 2^-16 for |t| < 88, where e^-t leaves fp32.  (SiLU's
// t is v; GELU-tanh's is 1.6 v + 0.07 v^3 with four roundings, 49 at v = -8:
// 2^-16.5.)  All of that is far below bf16's half step, 2^-9.  Further left e^-t
// overflows to infinity and the quotient is 0, the limit.
__device__ __forceinline__ float epi_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float epi_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t f2_const(float c) { return f2_pack(c, c); }
__device__ __forceinline__ uint64_t f2_ex2(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(epi_ex2(a), epi_ex2(b));
}
__device__ __forceinline__ uint64_t f2_rcp(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(epi_rcp(a), epi_rcp(b));
}
// sigmoid(t) with t given times -log2 e
__device__ __forceinline__ uint64_t f2_sigmoid(uint64_t mt) { return f2_rcp(f2_add(f2_ex2(mt), f2_const(1.0f))); }

__device__ __forceinline__ uint64_t act_relu(uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    return f2_pack(fmax_nan(a, 0.0f), fmax_nan(b, 0.0f));   // NaN stays NaN
}
__device__ __forceinline__ uint64_t act_silu(uint64_t v) {
    return f2_mul(v, f2_sigmoid(f2_mul(v, f2_const(-1.4426950408889634f))));
}
// (1 + tanh u) / 2 = sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
__device__ __forceinline__ uint64_t act_gelu_tanh(uint64_t v) {
    const uint64_t w = f2_fma(f2_mul(f2_mul(v, v), f2_const(0.044715f)), v, v);
    return f2_mul(v, f2_sigmoid(f2_mul(w, f2_const(-2.302208198f))));   // -2 sqrt(2/pi) log2 e
}
// v * Phi(v).  With a = |v|, Phi(-a) = e^(-a^2 / 2) erfcx(a / sqrt 2) / 2, the
// scaled complementary error function as t times a polynomial of degree 6 in
// t = 1 / (1 + 0.375 a / sqrt 2), fitted to the least largest relative error
// over a / sqrt 2 in [0, 10.5] (6.4e-7): the left tail keeps its digits, which
// 1 + erf would lose to cancellation, without normcdff's branches (M = 4096,
// K = 5120, N = 17408: 360 us with normcdff).
__device__ __forceinline__ uint64_t act_gelu(uint64_t v) {
    float v0, v1;
    f2_unpack(v, v0, v1);
    const uint64_t a = f2_pack(fabsf(v0), fabsf(v1));
    const uint64_t t = f2_rcp(f2_fma(a, f2_const(0.26516504294495535f), f2_const(1.0f)));
    uint64_t p = f2_fma(f2_const(-0.135096266866f), t, f2_const(0.387939184904f));
    p = f2_fma(p, t, f2_const(-0.129599303007f));
    p = f2_fma(p, t, f2_const(0.283063054085f));
    p = f2_fma(p, t, f2_const(0.166663974524f));
    p = f2_fma(p, t, f2_const(0.215689301491f));
    p = f2_fma(p, t, f2_const(0.211339443922f));
    const uint64_t e = f2_ex2(f2_mul(f2_mul(a, a), f2_const(-0.7213475204444817f)));
    float q0, q1;
    f2_unpack(f2_mul(f2_mul(p, f2_mul(t, f2_const(0.5f))), e), q0, q1);   // Phi(-a)
    return f2_mul(v, f2_pack(v0 < 0.0f ? q0 : 1.0f - q0, v1 < 0.0f ? q1 : 1.0f - q1));
}

// One branch for all of them, uniform over the grid.
template <int N>
__device__ __forceinline__ void act_apply(int act, uint64_t (&v)[N]) {
    if (act == W8A8_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_silu(v[j]);
    } else if (act == W8A8_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_relu(v[j]);
    } else if (act == W8A8_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_gelu(v[j]);
    } else if (act == W8A8_ACT_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_gelu_tanh(v[j]);
    }
}

// v + residual (two bf16), to two bf16.
__device__ __forceinline__ uint32_t epi_out2(uint64_t v, uint32_t res) {
    float a, b;
    f2_unpack(v, a, b);
    return cvt_bf16x2(__fadd_rn(a, __uint_as_float(res << 16)), __fadd_rn(b, __uint_as_float(res & 0xffff0000u)));
}

// Bias after the two products, each rounded by itself: one fp32 at a time, as
// mul.f32x2 followed by add.f32x2 came out with the single rounding of an fma
// on sm_100a.
__device__ __forceinline__ uint64_t epi_bias2(uint64_t v, float b0, float b1) {
    float x, y;
    f2_unpack(v, x, y);
    return f2_pack(__fadd_rn(x, b0), __fadd_rn(y, b1));
}

// Four consecutive columns of one row: int32 accumulators, the columns' scales
// and biases, the residual's 8 bytes -> 8 bytes of bf16.
__device__ __forceinline__ uint2 epi_fused4(const int4& acc, float sx, const float4& sw, const float4& bias,
                                            const uint2& res, int act) {
    const uint64_t sx2 = f2_pack(sx, sx);
    uint64_t v[2] = {f2_pack(__int2float_rn(acc.x), __int2float_rn(acc.y)), f2_pack(__int2float_rn(acc.z), __int2float_rn(acc.w))};
    v[0] = epi_bias2(f2_mul(f2_mul(v[0], sx2), f2_pack(sw.x, sw.y)), bias.x, bias.y);
    v[1] = epi_bias2(f2_mul(f2_mul(v[1], sx2), f2_pack(sw.z, sw.w)), bias.z, bias.w);
    act_apply<2>(act, v);
    return make_uint2(epi_out2(v[0], res.x), epi_out2(v[1], res.y));
}

// Eight, with scales and biases in shared memory and 16 bytes of residual.
__device__ __forceinline__ uint4 epi_fused8(const uint32_t* r, float sx, const float* sw8, const float* bias8,
                                            const uint4& res, int act) {
    const uint64_t sx2 = f2_pack(sx, sx);
    uint64_t v[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 s = *reinterpret_cast<const float4*>(sw8 + 4 * h);
        const float4 b = *reinterpret_cast<const float4*>(bias8 + 4 * h);
        const uint64_t a0 = f2_pack(__int2float_rn((int)r[4 * h]), __int2float_rn((int)r[4 * h + 1]));
        const uint64_t a1 = f2_pack(__int2float_rn((int)r[4 * h + 2]), __int2float_rn((int)r[4 * h + 3]));
        v[2 * h] = epi_bias2(f2_mul(f2_mul(a0, sx2), f2_pack(s.x, s.y)), b.x, b.y);
        v[2 * h + 1] = epi_bias2(f2_mul(f2_mul(a1, sx2), f2_pack(s.z, s.w)), b.z, b.w);
    }
    act_apply<4>(act, v);
    return make_uint4(epi_out2(v[0], res.x), epi_out2(v[1], res.y), epi_out2(v[2], res.z), epi_out2(v[3], res.w));
}

// One output, for the kernels that hold single columns.
__device__ __forceinline__ uint16_t epi_fused1(int acc, float sx, float sw, const EpiFused& f, int64_t m, int n) {
    float x = __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
    if (f.bias) x = __fadd_rn(x, __ldg(f.bias + n));
    uint64_t v[1] = {f2_pack(x, x)};
    act_apply<1>(f.act, v);
    float a, b;
    f2_unpack(v[0], a, b);
    if (f.res) a = __fadd_rn(a, bf16_bits_to_float(__ldcg(f.res + m * f.ldr + n)));
    return float_to_bf16_bits(a);
}

}  // namespace w8a8
