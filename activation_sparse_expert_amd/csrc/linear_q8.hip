// Linear layer on 8-bit codes: the 16-bit layer's kernels with two codes in each 16-bit unit
// (mfma_stream.hpp), so that K, strides and blocks count pairs of codes here.
// A block of 128 bytes takes the matrix core as long as one of 16-bit numbers (35 cycles a
// 32x32x32 instruction) and holds twice the k, so that what a block costs beside its MFMAs
// weighs twice as much: 64 x 128 and 128 x 128 tiles by 8 waves, two on a SIMD, which the
// 16-bit layer does without.  Measured: 300 x 4096 x 4096 17.5 us (64 x 64 by 4 waves 18.4,
// 128 x 256 in four parts of K 21.4), 1024 x 4096 x 4096 26.7 (128 x 128 by 4 waves 36, 128 x 64
// 32.7), 4096 x 4096 x (2 x 14336) 457-461, 2.1 POP/s, where the matrix cores alone reach 3.4
// on such codes (power) and 4.4 on zeros.
#include "linear_stream.hpp"
#include "linear_tile.hpp"

namespace moeffn {

namespace {

constexpr Tile kList[] = {{64, 64, 0.36, 0.50, 3.5}, {64, 128, 0.44, 0.84, 3.5}, {128, 128, 0.70, 0.0, 4.5},
                          {128, 256, 1.08, 0.0, 6.0}, {256, 256, 2.0, 0.0, 8.0}};
constexpr Tiles kTiles{kList, 5, 3.0, 8e-6 / 5.0};

hipError_t launch_t(const LinearQ8Args &a, const Plan &p, hipStream_t s)
{
    constexpr int U = st::kI8;
    switch (p.tile) {
    case 0:
        return a.wg ? launch_tile<U, 64, 64, 2, 1, true, 4>(a, p.c, s) : launch_tile<U, 64, 64, 2, 2, false, 4>(a, p.c, s);
    case 1:
        return a.wg ? launch_tile<U, 64, 128, 2, 2, true, 3>(a, p.c, s)
                    : launch_tile<U, 64, 128, 2, 4, false, 3>(a, p.c, s);
    case 2:
        return a.wg ? launch_tile<U, 128, 128, 4, 2, true, 3>(a, p.c, s)
                    : launch_tile<U, 128, 128, 4, 2, false, 3>(a, p.c, s);
    case 3:
        return a.wg ? launch_big<U, true, 128, 3>(a, p.c, s) : launch_big<U, false, 128, 3>(a, p.c, s);
    }
    return a.wg ? launch_big<U, true, 256, 2>(a, p.c, s) : launch_big<U, false, 256, 2>(a, p.c, s);
}

// Whether a call streams its weights past the tokens instead: up to 32 tokens, and small
// products, whose token tiles of 32 and groups of 16 outputs give each compute unit one
// workgroup (64 x 4096 x 2048 7.2 us against 9.6 in tiles, 64 x 8192 x 2048 10.3 against 12.2, but
// 40 x 14336 x 2048 17.3 against 14.6) or, over a short k, two (128 x 2048 x 1408 7.2 against
// 8.5, but 64 x 4096 x 4096 12.3 against 11.9).
bool q8_streams(int T, int K, int N)
{
    const long long wgs = (long long)((T + 31) / 32) * ((N + 15) / 16);
    return T <= 32 || (K <= 5120 && wgs <= kUnits) || (K <= 1280 && wgs <= 2 * kUnits);
}

}  // namespace

int linear_q8_parts(int T, int K, int N, bool gated, int *bm, int *bn)
{
    K /= 2;
    if (q8_streams(T, K, N)) return 0;
    const Plan p = plan(kTiles, T, K, N, gated);
    *bm = kList[p.tile].bm;
    *bn = kList[p.tile].bn;
    return p.c.split;
}

size_t linear_q8_split_bytes(int T, int K, int N)
{
    K /= 2;
    if (q8_streams(T, K, N)) return 0;
    const Plan p = plan(kTiles, T, K, N, false), g = plan(kTiles, T, K, N, true);
    const size_t np = p.c.split > 1 ? p.c.split : 0, ng = g.c.split > 1 ? 2 * g.c.split : 0;
    return (np > ng ? np : ng) * (size_t)T * N * 4;
}

// One token whose numbers and codes leave most of LDS to the weights: a launch less (1 x 4096 x 28672
// 21.6 us against 23.8 with the codes made first)
bool linear_q8_own_codes(int T, int K, int xdt)
{
    return T == 1 && xdt != 3 && own_raw_bytes(K, xdt) + (K + 127) / 128 * 128 <= 64 * 1024;
}

hipError_t launch_linear_q8(const LinearQ8Args &given, hipStream_t s)
{
    LinearQ8Args a = given;
    if (a.T < 1 || a.K < 16 || a.K % 16 != 0 || a.N < 1) return hipErrorInvalidValue;
    a.K /= 2;
    a.xs /= 2;
    if (a.xdt != 3) {
        if (!linear_q8_own_codes(a.T, given.K, a.xdt)) return hipErrorInvalidValue;
        return a.xdt == 2 ? launch_own<2>(a, s) : a.xdt == 1 ? launch_own<1>(a, s) : launch_own<0>(a, s);
    }
    // (the offsets of a tile's rows have 32 bits)
    if (q8_streams(a.T, a.K, a.N) || a.xs > kTileStride) return launch_stream<st::kI8>(a, s);
    return launch_plan<st::kI8>(a, plan(kTiles, a.T, a.K, a.N, a.wg != nullptr), launch_t, s);
}

}  // namespace moeffn
