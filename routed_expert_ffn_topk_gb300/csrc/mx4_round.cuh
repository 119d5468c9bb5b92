// Divisions of the 4-bit quantiser by a corrected reciprocal, two values at a time,
// and the rounding to E2M1 codes. Included inside `namespace es { namespace { ... } }`.
#pragma once

// - x / d from nr = - 1 / d: a quotient, its exact remainder and one correction
// (Markstein 1990). For finite operands away from the ends of the exponent range.
// Two values an instruction, and negated throughout because a packed multiply-add
// takes no signs; a zero's sign comes out opposite to x's as well.
__device__ __forceinline__ float2 neg_quotient(float2 x, float2 d, float2 nr) {
    const float2 q = __fmul2_rn(x, nr);
    return __ffma2_rn(__ffma2_rn(q, d, x), nr, q);
}
// Eight values as E2M1 codes, the first in the lowest bits: nearest, ties to the
// even code, at most 6.
__device__ __forceinline__ uint32_t e2m1_codes(const float* v) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// v = - SiLU(v) * u in the written order g / (1 + exp(-g)) * u, each step rounded
// to fp32 (no contraction). The reciprocal is the hardware's, refined by one
// Newton step; one range check and branch for the values instead of the one
// that a general division carries for each. (For every finite fp32 g with
// 1 + exp(-g) < 1e30 the quotient is the division's: tests/rounding/rounding.cu
// goes through them all.)
template <int kN>
__device__ __forceinline__ void neg_silu_mul(float (&v)[kN], const float (&u)[kN]) {
    float y[kN];
    uint32_t top = 0;  // as bits: y >= 1, or a NaN, which is larger
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        y[j] = __fadd_rn(1.0f, expf(-v[j]));
        top = max(top, __float_as_uint(y[j]));
    }
    if (top < __float_as_uint(1e30f)) {
#pragma unroll
        for (int j = 0; j < kN; j += 2) {
            float2 r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-y[j]));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-y[j + 1]));
            const float2 d = make_float2(y[j], y[j + 1]);
            r = __ffma2_rn(__ffma2_rn(d, r, make_float2(1.0f, 1.0f)), r, r);
            const float2 h = __fmul2_rn(neg_quotient(make_float2(v[j], v[j + 1]), d, r), make_float2(u[j], u[j + 1]));
            v[j] = h.x;
            v[j + 1] = h.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] = -__fmul_rn(__fdiv_rn(v[j], y[j]), u[j]);
    }
}
