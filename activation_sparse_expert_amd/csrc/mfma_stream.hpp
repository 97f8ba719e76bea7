// Weight-streaming product for a few tokens: one wave multiplies 16 NM weight
// rows by XR tokens over a run of k,
//   D[row][token] += sum_k W[row][k] X[token][k],
// with v_mfma_f32_16x16x32: weights as the A operand (lane l holds row l % 16,
// k 8 (l / 16) .. + 7), tokens as the B operand (lane l: token l % 16, the same
// k).  Value r of lane l of D is row 4 (l / 16) + r, token l % 16.
//
// Such a product is bound by the weight stream: 16 rows x 32 k are 1 KB per 16
// matrix-core cycles, where a compute unit's share of HBM is about 10 bytes a
// cycle.  So each wave keeps a ring of its own in LDS, D blocks of 64 k, that
// DMA copies fill (1 KB an instruction: 8 rows x 128 bytes, whole cache lines)
// while the wave waits for nothing but its oldest block: no barrier, and no
// register holds data in flight.  Measured on a 28672 x 4096 matrix, one token:
// 37 us (6.3 TB/s) this way, 41 us with fragments loaded straight into
// registers; at 16 tokens, whose 64-byte pieces then also have to be loaded,
// 39 us against 63.  Weights are copied with the nontemporal policy (38 us
// against 45 without), tokens without it.
#pragma once
#include "device.hpp"

namespace moeffn {
namespace st {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx4 __attribute__((ext_vector_type(4)));

// What an operand's 16-bit units hold: an fp16 number, a bf16 number or two 8-bit codes.
// Products of codes are summed in 32-bit integers; everything else about a unit, its place
// in a fragment included, is the same (a code of lane l's 16 bytes meets the code at the
// same place of the other operand).
enum Unit { kF16 = 0, kBF16 = 1, kI8 = 2 };

template <int U>
struct Sum {
    typedef floatx4 x4;
    typedef float floatx16 __attribute__((ext_vector_type(16)));
    typedef floatx16 x16;
};
template <>
struct Sum<kI8> {
    typedef intx4 x4;
    typedef int intx16 __attribute__((ext_vector_type(16)));
    typedef intx16 x16;
};

template <int U>
__device__ __forceinline__ typename Sum<U>::x4 mma16(const uint4 &a, const uint4 &b, const typename Sum<U>::x4 &c)
{
    if constexpr (U == kI8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, a), __builtin_bit_cast(intx4, b), c, 0, 0, 0);
    else if constexpr (U == kBF16)
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

// Read in place of k values past the end of the rows
__device__ __align__(16) const uint16_t zeros16[8] = {0, 0, 0, 0, 0, 0, 0, 0};

template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// XR: token rows of a block (1, 2, 4 or a multiple of 8), or 0 for one row that is in LDS already
template <int NM, int XR, int U = kF16>
struct Ring {
    static constexpr int kTok = (XR + 7) / 8;           // copy instructions of tokens
    static constexpr int kCopies = 2 * NM + kTok;       // instructions per block
    static constexpr int kBlock = 2048 * NM + 128 * XR; // bytes
    static constexpr int kFrag = XR ? (XR + 15) / 16 : 1;      // groups of 16 tokens
    typedef typename Sum<U>::x4 Acc[NM][kFrag];
    typedef const uint16_t *Src[kCopies];
};

// Row r0 = lane / 8 of the 8 rows that a copy instruction fills, and the k
// offset of the 16 bytes that this lane copies: a row's 8 chunks are stored
// XOR-permuted by r0, so that the rows a fragment read serves together fall in distinct banks.
__device__ __forceinline__ int copy_row(int lane) { return lane >> 3; }
__device__ __forceinline__ int copy_k(int lane) { return 8 * ((lane & 7) ^ (lane >> 3)); }

// nb >= 1 blocks of 64 k, of which the last holds kl (a multiple of 8) values.
//   src[i]: this lane's source of copy i at the first block (copy_row, copy_k):
//           2 NM of weights (rows 8 i ..), then those of the XR token rows
//   ring:   D blocks of LDS of this wave (wave-uniform)
//   row:    XR 0: the token's part of the first block in LDS, 128 bytes a block
//   ready:  called once the first blocks are on their way (all D - 1 of them, or fewer): what
//           the row needs before it is read
// Columns of D past the XR rows repeat some of them; rows and tokens that do not
// exist may be given as copies of others: their part of D means nothing.
struct Nothing {
    __device__ __forceinline__ void operator()(bool) const {}
};
template <int U, int NM, int XR, int D, class F = Nothing>
__device__ __forceinline__ void stream(typename Ring<NM, XR, U>::Acc &acc, unsigned char *ring,
                                       typename Ring<NM, XR, U>::Src &src, int nb, int kl, int lane,
                                       const unsigned char *row = nullptr, F ready = F())
{
    using R = Ring<NM, XR, U>;
    static_assert(XR == 1 || XR == 2 || XR == 4 || XR % 8 == 0, "token rows");
    const int li = lane & 15, q = lane >> 4;
    const int kc = copy_k(lane);
    int put = 0, get = 0, issued = 0;
    auto issue = [&]() {
        unsigned char *d = ring + put * R::kBlock;
        put = put + 1 == D ? 0 : put + 1;
        const bool tail = ++issued == nb && kl < 64;
#pragma unroll
        for (int i = 0; i < R::kCopies; ++i) {
            const uint16_t *p = tail && kc >= kl ? zeros16 : src[i];
            if (i < 2 * NM) copy16_to_lds<true>(p, d + 1024 * i);
            else if (XR >= 8 || lane < 8 * XR) copy16_to_lds(p, d + 1024 * i);
            src[i] += 64;
        }
    };
    auto use = [&]() {
        const unsigned char *d = ring + get * R::kBlock;
        get = get + 1 == D ? 0 : get + 1;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = 4 * s + q, at = li * 128 + 16 * (c ^ (li & 7));
            uint4 w[NM], x[R::kFrag];
#pragma unroll
            for (int m = 0; m < NM; ++m) w[m] = *(const uint4 *)(d + 2048 * m + at);
#pragma unroll
            for (int j = 0; j < R::kFrag; ++j) {
                if constexpr (XR == 0) {
                    x[j] = *(const uint4 *)(row + 16 * c);
                    continue;
                }
                int xt = at;
                if (XR == 1) xt = 16 * c;
                else if (XR < 8) xt = (li & (XR - 1)) * 128 + 16 * (c ^ (li & (XR - 1)));
                else if (16 * j + 8 == XR) xt = at & 1023;
                x[j] = *(const uint4 *)(d + 2048 * (NM + j) + xt);
            }
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int j = 0; j < R::kFrag; ++j) acc[m][j] = mma16<U>(w[m], x[j], acc[m][j]);
        }
        if (XR == 0) row += 128;
        // the block's reads are done before a copy may fill its place
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (i < nb) issue();
    ready(nb >= D - 1);
    int b = 0;
    for (; b + D - 1 < nb; ++b) {
        wait_copies<R::kCopies * (D - 2)>();            // block b has landed
        use();
        issue();                                        // into block b - 1's place
    }
    wait_copies<0>();
    for (; b < nb; ++b) use();
}

}  // namespace st
}  // namespace moeffn
