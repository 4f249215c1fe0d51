// q8.cuh -- the 8-bit state format: codes (int8 or e4m3) and one fp32 scale per key row.
//
// A state S [dk, dv] is kept as codes [dk, dv] and scales [dk]. With a = max_j |S_ij| over a
// key row i and M = 127 (int8) or 448 (e4m3, its largest finite value):
//   a infinite or NaN   scale = NaN, codes 0      the row reads back as NaN: a state that has
//                                                 blown up stays visible
//   a < 2^-100          scale = 0,   codes 0      (2^-100: 1 / a and a / M stay normal numbers)
//   otherwise           scale = fl(a / M), code_ij = RN(fl(S_ij fl(M / a)))
// and read back as S_ij = fl(code_ij scale). Every fl() is fp32 rounding to nearest. The two
// roundings before the code's own move it across a border between codes for about one value in
// 10^5, by 2^-23 of the row's largest magnitude; the code's own rounding is off by up to half a
// step: a / 254 (int8), or 2^-4 of the value and a / 458752 near zero (e4m3). One scale per
// key row because the decay acts on key rows: rows of one state differ in magnitude by their
// decays, a row's own values do not.
#pragma once

#include "internal.cuh"

namespace gdn2 {

constexpr float kQ8Tiny = 7.888609052210118e-31f;  // 2^-100

template <int kFmt> struct Q8;
template <> struct Q8<GDN2_Q8_INT8> { static constexpr float kTop = 127.f; };
template <> struct Q8<GDN2_Q8_E4M3> { static constexpr float kTop = 448.f; };

// Scale and inverse of a row from its largest magnitude; inv = 0 marks a row whose codes are 0.
//
// Both quotients are rounded to nearest by a fused multiply-add on the remainder of a first
// quotient (Markstein 1990): with y close to 1 / d, q = fl(n y) and the exact remainder
// r = n - q d, fl(q + r y) is the rounded quotient. For a / M, 1 / M is a rounded constant. For
// M / a, a's mantissa m in [1, 2) is divided by, with y from one Newton step on the hardware's
// approximate reciprocal, and the exponent subtracted after it, so nothing over- or underflows for any
// a from 2^-100 up. There are 2^23 mantissas: all of them were compared with __fdiv_rn (the test
// of the stored scales and codes covers them again).
template <int kFmt>
__device__ __forceinline__ void q8_scale(float amax, float& scale, float& inv) {
    constexpr float M = Q8<kFmt>::kTop, yM = 1.f / M;
    const uint32_t bits = __float_as_uint(amax);
    const float m = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(m));
    y = fmaf(y, fmaf(-m, y, 1.f), y);
    float q = __fmul_rn(M, y);
    q = fmaf(fmaf(-m, q, M), y, q);
    inv = __uint_as_float(__float_as_uint(q) - (bits & 0x7f800000u) + 0x3f800000u);
    const float s = __fmul_rn(amax, yM);
    scale = fmaf(fmaf(-M, s, amax), yM, s);
    const bool finite = bits < 0x7f800000u, keep = finite && amax >= kQ8Tiny;
    scale = keep ? scale : finite ? 0.f : __uint_as_float(0x7fc00000u);
    inv = keep ? inv : 0.f;
}

// Magnitudes are compared as integers: ordered like the values, and an infinity or a NaN wins.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Four values as e4m3 bytes and back (e4m3 is exact in fp16, and fp16 in fp32).
__device__ __forceinline__ uint32_t e4m3x4(float4 x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w));
    return r;
}
__device__ __forceinline__ float4 e4m3x4_values(uint32_t c) {
    float4 x;
    asm("{\n\t.reg .b16 l, h, a, b, c, d;\n\t.reg .b32 p, q;\n\tmov.b32 {l, h}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, l;\n\tcvt.rn.f16x2.e4m3x2 q, h;\n\tmov.b32 {a, b}, p;\n\tmov.b32 {c, d}, q;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\tcvt.f32.f16 %2, c;\n\tcvt.f32.f16 %3, d;\n\t}"
        : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
        : "r"(c));
    return x;
}

// Four codes of x * inv, packed in column order.
template <int kFmt>
__device__ __forceinline__ uint32_t q8_pack(float4 x, float inv) {
    x.x = __fmul_rn(x.x, inv); x.y = __fmul_rn(x.y, inv); x.z = __fmul_rn(x.z, inv); x.w = __fmul_rn(x.w, inv);
    uint32_t r;
    if (kFmt == GDN2_Q8_INT8) {
        // |x| <= 127.00002: adding 1.5 2^23 rounds to the nearest whole number, ties to even, and
        // leaves it as the low byte
        const float c = 12582912.f;
        const uint32_t a = __float_as_uint(__fadd_rn(x.x, c)), b = __float_as_uint(__fadd_rn(x.y, c));
        const uint32_t d = __float_as_uint(__fadd_rn(x.z, c)), e = __float_as_uint(__fadd_rn(x.w, c));
        r = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(d, e, 0x0040), 0x5410);
    } else {
        r = e4m3x4(x);
    }
    return inv == 0.f ? 0u : r;
}

// The values of four codes, before the scale.
template <int kFmt>
__device__ __forceinline__ float4 q8_unpack(uint32_t c) {
    if (kFmt == GDN2_Q8_INT8) {
        // code + 128 as the low byte of 2^23's mantissa, then 2^23 + 128 taken off: exact
        const uint32_t u = c ^ 0x80808080u;
        const float m = 8388736.f;
        return make_float4(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650)) - m,
                           __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7651)) - m,
                           __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7652)) - m,
                           __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7653)) - m);
    } else {
        return e4m3x4_values(c);
    }
}

// Two fp32 values in one 64-bit register, for packed arithmetic without moves between registers.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 d) {
    float2 x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(d));
    return x;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// q8_unpack for two rows at once, as pairs (row 0, row 1) per column; N columns in the low bytes of
// each row's word.
template <int kFmt, int N>
__device__ __forceinline__ void q8_unpack_pair(uint32_t w0, uint32_t w1, f32x2* x) {
    if (kFmt == GDN2_Q8_INT8) {
        const uint32_t u0 = w0 ^ 0x80808080u, u1 = w1 ^ 0x80808080u;
        const f32x2 m = pack2(-8388736.f, -8388736.f);
#pragma unroll
        for (int j = 0; j < N; ++j)
            x[j] = add2(pack2(__uint_as_float(__byte_perm(u0, 0x4b000000u, 0x7650 | j)),
                              __uint_as_float(__byte_perm(u1, 0x4b000000u, 0x7650 | j))), m);
    } else {
        const float4 a = q8_unpack<kFmt>(w0), b = q8_unpack<kFmt>(w1);
        x[0] = pack2(a.x, b.x);
        x[1] = pack2(a.y, b.y);
        if (N == 4) {
            x[2 % N] = pack2(a.z, b.z);
            x[3 % N] = pack2(a.w, b.w);
        }
    }
}

// Codes of two rows' values, inv = (row 0's, row 1's), without q8_pack's rule for inv = 0.
template <int kFmt, int N>
__device__ __forceinline__ void q8_pack_pair(const f32x2* x, f32x2 inv, uint32_t& w0, uint32_t& w1) {
    float2 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x2 z = j < N ? mul2(x[j % N], inv) : 0ull;
        if (kFmt == GDN2_Q8_INT8 && j < N) z = add2(z, pack2(12582912.f, 12582912.f));
        y[j] = unpack2(z);
    }
    if (kFmt == GDN2_Q8_INT8) {
        const auto pack = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040); };
        w0 = pack(y[0].x, y[1].x);
        w1 = pack(y[0].y, y[1].y);
        if (N == 4) {
            w0 = __byte_perm(w0, pack(y[2].x, y[3].x), 0x5410);
            w1 = __byte_perm(w1, pack(y[2].y, y[3].y), 0x5410);
        }
    } else {
        w0 = e4m3x4(make_float4(y[0].x, y[1].x, y[2].x, y[3].x));
        w1 = e4m3x4(make_float4(y[0].y, y[1].y, y[2].y, y[3].y));
    }
}

}  // namespace gdn2
