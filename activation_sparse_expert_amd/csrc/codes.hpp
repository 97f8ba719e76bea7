// Rows of 8-bit codes: q = 127 x / max|x| rounded to nearest, ties to even, and the scale
// max|x| / 127 that takes them back.
//
// The quotient is formed from p = 127 x, exact in fp32 for a 16-bit x (11 + 7 bits): the
// product with the hardware's reciprocal, then one Newton step on its residual.  That
// residual is exact (p and the product agree to a few units, and max|x| has 11 bits), so
// a quotient that fp32 holds comes out exactly, ties (n + 1/2) among them; any other
// quotient is at least 2^-19 of itself away from a tie, far more than its error.  So
// the codes of 16-bit rows are those of exact arithmetic.  Both p and max|x| carry the power of
// two that puts max|x| in [1, 2) (that of 2^-100 for smaller ones): nothing overflows, and what
// underflows has the code 0.  The quotient is rounded by adding 1.5 2^23, whose last bits
// then are the code.
//
// 32-bit numbers: x (127 / max|x|) in 64 bits, with the factor to 2^-50 of itself, is off by at most
// 2^-43.  It is rounded to a multiple of 2^-38 first: ties are such multiples and come out
// exactly, and a quotient of 24-bit numbers that is no tie is at least 2^-33 away from one (2^-32
// of itself, which is 1/2 or more) and stays on its side.  Then it is rounded to an integer.
// Both roundings are those of additions, of 1.5 2^14 and of 1.5 2^52 less that.
#pragma once
#include "device.hpp"

namespace moeffn {
namespace codes {

// What a row's codes are made with, from the bits of its largest |x|.
struct Row {
    float k;                            // 127 2^-e
    float a, inv;                       // max|x| 2^-e and its reciprocal (a row of zeros: 1 and 0)
    float scale;                        // max|x| / 127; NaN for a row with an infinity or NaN
    bool ok;                            // no infinity or NaN: else the codes are 0
};

// |x| as an integer that orders as |x| does, infinities above the numbers and NaN above those
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ Row row(uint32_t most)
{
    Row r{0.f, 1.f, 0.f, 0.f, true};
    if (most >= 0x7F800000u) {
        r.scale = __uint_as_float(0x7FC00000u);
        r.ok = false;
    } else if (most != 0) {
        const float v = __uint_as_float(most);
        const int e = __builtin_amdgcn_frexp_expf(v) - 1, s = e < -100 ? 100 : -e;
        r.k = __builtin_amdgcn_ldexpf(127.f, s);
        r.a = __builtin_amdgcn_ldexpf(v, s);
        r.inv = __builtin_amdgcn_rcpf(r.a);
        r.scale = v / 127.f;
    }
    return r;
}

// A 16-bit x: bits whose last 8 are the code
__device__ __forceinline__ uint32_t code(float x, const Row &r)
{
    const float p = x * r.k, c = p * r.inv;
    return __float_as_uint(fmaf(fmaf(-c, r.a, p), r.inv, c) + 12582912.f);
}

// 127 / max|x|: two Newton steps take the reciprocal from 23 bits to 46 and to 64 bits' own
__device__ __forceinline__ double factor64(const Row &r)
{
    const double a = r.a, i0 = r.inv, i1 = fma(fma(-i0, a, 1.0), i0, i0);
    return (double)r.k * fma(fma(-i1, a, 1.0), i1, i1);
}

// An fp32 x; f: factor64 of its row
__device__ __forceinline__ uint32_t code64(float x, double f)
{
    constexpr double kGrid = 24576.0, kInt = 6755399441055744.0 - kGrid;
    double grid = kGrid;
    asm("" : "+s"(grid));               // (else it takes two registers of each lane, over a whole loop)
    return (uint32_t)__builtin_bit_cast(uint64_t, fma((double)x, f, grid) + kInt);
}

// The last bytes of four
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return lo | hi;
}

}  // namespace codes
}  // namespace moeffn
