// rope.cuh -- the angle of a rotary position, shared by the rotation (rope.cu)
// and the append that quantises (append8.cu).
//
// In units of a whole turn the angle is P f_i / 2 pi, of which only the fraction
// matters; rope.cu's header has the derivation and the error bounds.
#pragma once

#include <cuda_runtime.h>

namespace attn {

// f / 2 pi modulo 1 as a 64-bit binary fraction, from the bits of f = +- m 2^e
// with m shifted to the top of 64 bits: m / 2 pi by 128 bits of 1 / 2 pi, as
// whole + part 2^-64, then shifted to units of 2^-64 turns.  Good to two units for
// |f| < 2^63 (beyond: 0).  Integers, because float64 is slow here: a product carried
// in two doubles cost every call 0.2 us.
__device__ __forceinline__ unsigned long long turn_fraction(unsigned long long m, int e, bool negative) {
    constexpr unsigned long long kHi = 0x28be60db9391054aULL, kLo = 0x7f09d5f47d4d3770ULL;
    const unsigned long long low = m * kHi, carry = __umul64hi(m, kLo), part = low + carry;
    const unsigned long long whole = __umul64hi(m, kHi) + (part < low ? 1ULL : 0ULL);
    const int s = 64 + e;
    const unsigned long long turns = s <= -64 ? 0ULL : s <= 0 ? whole >> -s : s < 64 ? whole << s | part >> (64 - s) : 0ULL;
    return negative ? 0ULL - turns : turns;
}
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(f);
    const int x = (int)(b >> 52) & 0x7ff;
    return turn_fraction(((b << 11) & 0x7fffffffffffffffULL) | (x ? 1ULL << 63 : 0ULL), (x ? x : 1) - 1086, (b >> 63) != 0);
}
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
    const unsigned b = __float_as_uint(f);
    const int x = (int)(b >> 23) & 0xff;
    return turn_fraction(((unsigned long long)(b << 8 & 0x7fffffffu) << 32) | (x ? 1ULL << 63 : 0ULL), (x ? x : 1) - 190, (b >> 31) != 0);
}

// Cosine and sine of position pos at the frequency whose turn_fraction is given:
// half turns as 24 bits exactly in fp32, and the 32 bits below them, in radians,
// as one more small rotation.
__device__ __forceinline__ void turned_cos_sin(unsigned long long fraction, int pos, float* c, float* s) {
    const unsigned long long phase = fraction * (unsigned long long)(long long)pos;
    const int top = (int)(phase >> 32) & ~0xff;
    const float e = (float)(unsigned)(phase >> 8) * 8.7196712450215807e-17f;  // 2^-55 pi
    float s0, c0;
    sincospif((float)top * 4.6566128730773926e-10f, &s0, &c0);  // 2^-31
    *c = fmaf(-e, s0, c0);
    *s = fmaf(e, c0, s0);
}

}  // namespace attn
