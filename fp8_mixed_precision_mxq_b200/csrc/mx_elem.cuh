// mx_elem.cuh -- device helpers of the MX element formats shared by the quantizer and
// the GEMM epilogue that quantizes its output: packed bf16 abs-max, the E8M0 scale of a
// block, and the hardware conversions to E2M1 / E4M3 (round to nearest even,
// saturating, sign of a zero result kept); and the exact bf16 GELU of the fused FFN
// epilogue (a shared-memory table and closed forms).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "mxq.h"

namespace mxq {

// Packed max of |a| and |b| over two bf16 lanes (sign of the result is the xor of the
// signs, which the caller masks off); a NaN in either input yields NaN.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight fp32 -> one word of eight E2M1 codes (v[i] in nibble i).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Two fp32 -> two E4M3 codes in a 16-bit word (first argument in the low byte).
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

// E8M0 scale code of a block from the bf16 bit pattern of its absolute maximum: bf16
// and E8M0 share the exponent bias 127, so floor(log2 amax) + 127 is the exponent
// field; code = field - emax, clamped at 0 (zero and subnormal maxima), and 255 for a
// block holding Inf or NaN (exponent field 255).
template <uint32_t kEmax>
__device__ __forceinline__ uint32_t e8m0_code(uint32_t amax_bits)
{
    const uint32_t eb = (amax_bits & 0x7FFFu) >> 7;
    return eb == 255u ? 255u : (eb > kEmax ? eb - kEmax : 0u);
}

// 2^(127 - code) as fp32, the exact reciprocal of the scale.  Finite blocks give codes
// <= 252 (bf16 exponent fields stop at 254); for 255, a non-finite block, the caller
// forces the element codes to zero, so the clamp only keeps the value finite.
__device__ __forceinline__ float e8m0_inverse(uint32_t code)
{
    return __uint_as_float((254u - min(code, 253u)) << 23);
}

// Byte offset of the four scale bytes of row r, k-blocks 4*atom ... 4*atom + 3, in the tiled
// layout (one aligned 32-bit word).
__device__ __forceinline__ size_t sf_word(int64_t r, uint32_t atom, uint32_t atoms_k)
{
    return (static_cast<size_t>(r >> 7) * atoms_k + atom) * 512u + static_cast<uint32_t>(r & 31) * 16u +
           static_cast<uint32_t>((r >> 5) & 3) * 4u;
}

// ---- GELU of bf16 values ---------------------------------------------------------------
// h = bf16(GELU(x)) for a bf16 x, GELU(x) = x/2 erfc(-x / sqrt 2) (the plain erf form) rounded
// once to bf16, nearest with ties to even: what a bf16 network's GELU gives when computed
// exactly.  For 2^-10 <= |x| < 16 (14 binades of 128 significands, both signs: 3584 values)
// the result comes from a table that the kernel using it builds in shared memory from the
// fp64 erfc.  Elsewhere it has a closed form: below 2^-10 it is x/2 rounded to bf16 (the
// next term, x^2 / sqrt(2 pi), moves x/2 by less than 0.8 |x| of itself, which is under half
// a bf16 unit); from 16 up it is x (1 - Phi(16) < 2^-190); from -16 down it is -0 (below the
// smallest bf16 magnitude); +Inf gives +Inf, -Inf and NaN give NaN (0x7FC0).
constexpr uint32_t kGeluLo = 0x3A80u;                 // bf16 magnitude bits of 2^-10
constexpr uint32_t kGeluSpan = 14u * 128u;            // magnitudes 2^-10 ... 16 (exclusive)
constexpr uint32_t kGeluEntries = 2u * kGeluSpan;     // positive, then negative
constexpr uint32_t kGeluTableBytes = 2u * kGeluEntries;

// Entry i of the table: bf16 bits of GELU of the bf16 value with sign i / kGeluSpan and
// magnitude bits kGeluLo + i % kGeluSpan.  The fp64 GELU is rounded to 8 significant bits
// (to a multiple of 2^-133 below 2^-126, bf16's subnormal step) with rint, then read as
// bf16: one rounding.
__device__ __forceinline__ uint16_t gelu_table_value(uint32_t i)
{
    const uint32_t b = ((i / kGeluSpan) << 15) | (kGeluLo + i % kGeluSpan);
    const double x = static_cast<double>(__uint_as_float(b << 16));
    const double g = 0.5 * x * erfc(-x / sqrt(2.0));
    int e = 0;
    frexp(g, &e);  // |g| in [2^(e-1), 2^e)
    const double ulp = ldexp(1.0, max(e - 8, -133));
    const double r = rint(g / ulp) * ulp;
    return static_cast<uint16_t>(__float_as_uint(static_cast<float>(r)) >> 16);
}

// Threads tid, tid + nthreads, ... fill their entries of the shared-memory table.
__device__ __forceinline__ void gelu_table_fill(uint16_t* lut, uint32_t tid, uint32_t nthreads)
{
    for (uint32_t i = tid; i < kGeluEntries; i += nthreads) lut[i] = gelu_table_value(i);
}

// GELU of one bf16 value (bits b, low 16 bits) through the table.
__device__ __forceinline__ uint32_t gelu_bf16_bits(uint32_t b, const uint16_t* lut)
{
    const uint32_t m = b & 0x7FFFu;
    const uint32_t neg = b >> 15;
    const uint32_t idx = m - kGeluLo;
    const bool in = idx < kGeluSpan;
    const uint32_t t = lut[in ? neg * kGeluSpan + idx : 0u];
    const uint32_t half = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b << 16) * 0.5f));
    uint32_t big = neg ? 0x8000u : b;
    if (m >= 0x7F80u) big = (m == 0x7F80u && !neg) ? b : 0x7FC0u;
    return in ? t : (m < kGeluLo ? half : big);
}

// ---- activations in binary32 ------------------------------------------------------------
// Applied to the binary32 sum, so that the result is rounded to bf16 once; two values at a time
// on packed fp32 pairs.  The two sigmoid forms v / (1 + exp(-t)) keep their relative accuracy
// where v is far negative (1 + tanh would cancel there), and so does the erf form, which takes
// the tail's own function; where 1 + exp passes 2^126 (SiLU below v = -87.3) the quotient is 0, for
// a value below 2^-119.
__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

constexpr float kLog2E = 1.4426950408889634f;

// v / (1 + 2^e)
__device__ __forceinline__ float2 over_one_plus_exp2(float2 v, float2 e)
{
    const float2 d = __fadd2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), splat(1.0f));
    return make_float2(__fdividef(v.x, d.x), __fdividef(v.y, d.y));
}

template <int kAct>
__device__ __forceinline__ float2 act_f32x2(float2 v)
{
    if constexpr (kAct == MXQ_ACT_SILU) {
        return over_one_plus_exp2(v, __fmul2_rn(v, splat(-kLog2E)));
    } else if constexpr (kAct == MXQ_ACT_GELU_TANH) {
        // exp(-2 sqrt(2/pi) (v + 0.044715 v^3)) = 2^(v (c + 0.044715 c v^2))
        constexpr float c = -1.5957691216057308f * kLog2E;
        const float2 v2 = __fmul2_rn(v, v);
        return over_one_plus_exp2(v, __fmul2_rn(v, __ffma2_rn(splat(0.044715f * c), v2, splat(c))));
    } else if constexpr (kAct == MXQ_ACT_GELU) {
        // v Phi(v), with 1 - Phi(a) = exp(-a^2 / 2) q(t) for a = |v| >= 0, t = 1 / (1 + 0.24 a), q a
        // polynomial of degree 8 (fitted to Mills' ratio over [0, 40], relative error 4.3e-7; the
        // form is Hastings').  CUDA's erfcf in its place made the epilogue the GEMM's bound.
        const float2 d = __ffma2_rn(splat(0.24f), make_float2(fabsf(v.x), fabsf(v.y)), splat(1.0f));
        const float2 t = make_float2(__fdividef(1.0f, d.x), __fdividef(1.0f, d.y));
        float2 q = splat(-0.0529897924f);
        q = __ffma2_rn(q, t, splat(0.152786211f));
        q = __ffma2_rn(q, t, splat(-0.0656899739f));
        q = __ffma2_rn(q, t, splat(0.118377487f));
        q = __ffma2_rn(q, t, splat(0.0634029045f));
        q = __ffma2_rn(q, t, splat(0.0928372305f));
        q = __ffma2_rn(q, t, splat(0.0955223363f));
        q = __ffma2_rn(q, t, splat(0.0957537846f));
        const float2 e = __fmul2_rn(__fmul2_rn(v, v), splat(-0.5f * kLog2E));
        const float2 w = __fmul2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), __fmul2_rn(q, t));
        return __fmul2_rn(v, make_float2(v.x > 0.0f ? 1.0f - w.x : w.x, v.y > 0.0f ? 1.0f - w.y : w.y));
    }
    return v;
}

// f(integral constant of the activation): the choice is taken once, outside f's loops.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f)
{
    if (act == MXQ_ACT_SILU) f(std::integral_constant<int, MXQ_ACT_SILU>{});
    else if (act == MXQ_ACT_GELU_TANH) f(std::integral_constant<int, MXQ_ACT_GELU_TANH>{});
    else if (act == MXQ_ACT_GELU) f(std::integral_constant<int, MXQ_ACT_GELU>{});
    else f(std::integral_constant<int, MXQ_ACT_NONE>{});
}

// Two fp32 values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

}  // namespace mxq
