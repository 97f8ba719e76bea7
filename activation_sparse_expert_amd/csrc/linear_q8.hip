// Linear layer on 8-bit codes: the 16-bit layer's kernels with two codes in each 16-bit unit
// (mfma_stream.hpp), so that K, strides and blocks count pairs of codes here.
#include "linear_stream.hpp"
#include "linear_tile.hpp"

namespace moeffn {

namespace {

bool q8_streams(int T, int K, int N)
{
    return T <= 32 || (K <= 8192 && (long long)((T + 31) / 32) * ((N + 15) / 16) <= kUnits);
}

}  // namespace

int linear_q8_parts(int T, int K, int N, bool gated, int *bm, int *bn)
{
    K /= 2;
    if (q8_streams(T, K, N)) return 0;
    const Plan p = plan(T, K, N, gated);
    *bm = kTiles[p.tile].bm;
    *bn = kTiles[p.tile].bn;
    return p.c.split;
}

size_t linear_q8_split_bytes(int T, int K, int N)
{
    K /= 2;
    if (q8_streams(T, K, N)) return 0;
    const Plan p = plan(T, K, N, false), g = plan(T, K, N, true);
    const size_t np = p.c.split > 1 ? p.c.split : 0, ng = g.c.split > 1 ? 2 * g.c.split : 0;
    return (np > ng ? np : ng) * (size_t)T * N * 4;
}

hipError_t launch_linear_q8(const LinearQ8Args &given, hipStream_t s)
{
    LinearQ8Args a = given;
    if (a.T < 1 || a.K < 16 || a.K % 16 != 0 || a.N < 1) return hipErrorInvalidValue;
    a.K /= 2;
    a.xs /= 2;
    // (the offsets of a tile's rows have 32 bits)
    if (q8_streams(a.T, a.K, a.N) || a.xs > kTileStride) return launch_stream<st::kI8>(a, s);
    return launch_plan<st::kI8>(a, plan(a.T, a.K, a.N, a.wg != nullptr), s);
}

}  // namespace moeffn
