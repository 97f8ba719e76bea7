// Rows of 8-bit codes: q = 127 x / max|x| rounded to nearest, ties to even, and the scale
// max|x| / 127 that takes them back.
//
// The quotient is formed from p = 127 x, exact in fp32 for a 16-bit x (11 + 7 bits): the
// product with the hardware's reciprocal, then one Newton step on its residual.  That
// residual is exact (p and the product agree to a few units, and max|x| has 11 bits), so
// a quotient that fp32 holds comes out exactly, ties (n + 1/2) among them; any other
// quotient is at least 2^-19 of itself away from a tie, far more than its error.  So
// the codes of 16-bit rows are those of exact arithmetic.  32-bit rows take the same
// steps in 64 bits (24 + 7 bits).  The row is first scaled by the power of two that puts
// max|x| in [1, 2): nothing overflows, and what underflows has the code 0.
#pragma once
#include "device.hpp"

namespace moeffn {
namespace codes {

// What a row's codes are made with, from the bits of its largest |x|.
struct Row {
    float a, inv;                       // max|x| 2^-e in [1, 2) and its reciprocal (0: the codes are 0)
    int e;
    float scale;                        // max|x| / 127; NaN for a row with an infinity or NaN
};

// |x| as an integer that orders as |x| does, infinities above the numbers and NaN above those
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ Row row(uint32_t most)
{
    Row r{1.f, 0.f, 0, 0.f};
    if (most >= 0x7F800000u) {
        r.scale = __uint_as_float(0x7FC00000u);
    } else if (most != 0) {
        const float v = __uint_as_float(most);
        r.e = __builtin_amdgcn_frexp_expf(v) - 1;
        r.a = __builtin_amdgcn_ldexpf(v, -r.e);
        r.inv = __builtin_amdgcn_rcpf(r.a);
        r.scale = v / 127.f;
    }
    return r;
}

// Code of a 16-bit x, or of an fp32 one whose own last bits are not exact anyway
__device__ __forceinline__ int code(float x, const Row &r)
{
    const float p = __builtin_amdgcn_ldexpf(x, -r.e) * 127.f;
    const float c = p * r.inv;
    const float q = fmaf(fmaf(-c, r.a, p), r.inv, c);
    return r.inv != 0.f ? (int)__builtin_rintf(q) : 0;
}

// Code of an fp32 x
__device__ __forceinline__ int code64(float x, const Row &r)
{
    const double p = (double)__builtin_amdgcn_ldexpf(x, -r.e) * 127.0, a = r.a, i0 = r.inv;
    const double inv = fma(fma(-i0, a, 1.0), i0, i0);           // 46 bits
    const double c = p * inv;
    const double q = fma(fma(-c, a, p), inv, c);
    return r.inv != 0.f ? (int)__builtin_rint(q) : 0;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return (a & 0xFF) | (b & 0xFF) << 8 | (c & 0xFF) << 16 | (uint32_t)d << 24;
}

}  // namespace codes
}  // namespace moeffn
