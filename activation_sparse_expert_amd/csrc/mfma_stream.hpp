// Weight-streaming product for a few tokens (at most 16 per accumulator): one
// wave multiplies 16 weight rows by the tokens,
//   D[row][token] += sum_k W[row][k] X[token][k],
// with v_mfma_f32_16x16x32: weights as the A operand (lane l holds row l % 16,
// k 8 (l / 16) .. + 7), tokens as the B operand (lane l: token l % 16, the same
// k), so both are read straight from k-contiguous rows into the registers that
// feed the matrix core, 16 bytes per lane and without LDS.  Value r of lane l of
// D is row 4 (l / 16) + r, token l % 16.
//
// Such a product is bound by the weight stream: 16 rows x 32 k are 1 KB per 16
// matrix-core cycles, where a compute unit's share of HBM is about 10 bytes a
// cycle.  So nothing is shared between waves; each issues the loads of U steps
// (U KB of weights per matrix) together, and the other waves of the compute unit cover the wait.
#pragma once
#include "device.hpp"

namespace moeffn {
namespace st {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ floatx4 mma16(const uint4 &a, const uint4 &b, const floatx4 &c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// fp32 to the 16-bit type, round to nearest even, NaN kept
template <bool BF16>
__device__ __forceinline__ uint16_t to16(float v)
{
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <bool BF16>
__device__ __forceinline__ float from16(uint16_t v)
{
    if constexpr (BF16) return bf16_bits_to_float(v);
    else return half_bits_to_float(v);
}

// One element of an array of type dt (0 f16, 1 bf16, 2 f32)
__device__ __forceinline__ float load_el(const void *p, int dt, size_t i)
{
    if (dt == 2) return ((const float *)p)[i];
    const uint16_t v = ((const uint16_t *)p)[i];
    return dt == 1 ? from16<true>(v) : from16<false>(v);
}

__device__ __forceinline__ void store_el(void *p, int dt, size_t i, float v)
{
    if (dt == 2) ((float *)p)[i] = v;
    else ((uint16_t *)p)[i] = dt == 1 ? to16<true>(v) : to16<false>(v);
}

// Steps [s0, s1) of 32 k values each; K (a multiple of 8) ends inside the last.
//   w[m]: this lane's weight row of matrix m, at k = 8 (lane / 16)
//   x[j]: this lane's token row of B fragment j, likewise; a step advances it
//         by XS elements.  Fragment j adds into acc[m][j / HL]: HL = 2 sums two
//         16-bit parts of one value.
// Full batches read without a test; the last one clamps its reads to the row's
// last 8 values and zeroes what lies beyond K in both operands.
template <bool BF16, int NM, int NX, int HL, int U>
__device__ __forceinline__ void stream(floatx4 (&acc)[NM][NX / HL], const uint16_t *const (&w)[NM],
                                       const uint16_t *const (&x)[NX], int s0, int s1, int K, int kq)
{
    constexpr int XS = 32 * HL;
    const int full = K / 32;                        // steps that lie inside the rows
    int s = s0;
    for (; s + U <= s1 && s + U <= full; s += U) {
        uint4 av[NM][U], bv[NX][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < NM; ++m) av[m][u] = load_nt16(w[m] + (size_t)(s + u) * 32);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NX; ++j) bv[j][u] = *(const uint4 *)(x[j] + (size_t)(s + u) * XS);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NX; ++j)
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    acc[m][j / HL] = mma16<BF16>(av[m][u], bv[j][u], acc[m][j / HL]);
    }
    for (; s < s1; s += U) {
        uint4 av[NM][U], bv[NX][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // the last 8 values of the row, as an offset from this lane's pointers
            const int su = min(s + u, s1 - 1);
            const bool in = 32 * su + kq < K;
            const int ow = in ? 32 * su : K - 8 - kq;
            const int ox = in ? XS * su : HL * (K - 8 - kq);
#pragma unroll
            for (int m = 0; m < NM; ++m) av[m][u] = load_nt16(w[m] + ow);
#pragma unroll
            for (int j = 0; j < NX; ++j) bv[j][u] = *(const uint4 *)(x[j] + ox);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u < s1 && 32 * (s + u) + kq < K;
#pragma unroll
            for (int m = 0; m < NM; ++m) av[m][u] = in ? av[m][u] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const uint4 b = in ? bv[j][u] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int m = 0; m < NM; ++m) acc[m][j / HL] = mma16<BF16>(av[m][u], b, acc[m][j / HL]);
            }
        }
    }
}

}  // namespace st
}  // namespace moeffn
