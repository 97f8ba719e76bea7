// Linear layer on 16-bit types in tiles, and the choice between tiles and streams.
#include "linear_tile.hpp"

namespace moeffn {

namespace {

// Whether a call streams its weights past the tokens (linear_stream.hip) instead:
// up to 32 tokens, whose tiles would be half empty, and small products whose
// token tiles of 32 and groups of 16 outputs give each compute unit one workgroup
// at most (4096 x 1024 at 128 tokens: 8.8 us against 12.0 in tiles; with 267
// workgroups at 2056 x 1411 and 77 tokens 11.6 against 10.6).
bool streams(int T, int K, int N)
{
    return T <= 32 || (K <= 8192 && (long long)((T + 31) / 32) * ((N + 15) / 16) <= kUnits);
}

}  // namespace

int linear_parts(int T, int K, int N, bool gated, int *bm, int *bn)
{
    if (streams(T, K, N)) return 0;
    const Plan p = plan(T, K, N, gated);
    *bm = kTiles[p.tile].bm;
    *bn = kTiles[p.tile].bn;
    return p.c.split;
}

size_t linear_ws_bytes(int T, int K, int N)
{
    if (streams(T, K, N)) return 0;
    const Plan p = plan(T, K, N, false), g = plan(T, K, N, true);
    const size_t np = p.c.split > 1 ? p.c.split : 0, ng = g.c.split > 1 ? 2 * g.c.split : 0;
    return (np > ng ? np : ng) * (size_t)T * N * 4;
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t s)
{
    if (a.T < 1 || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    // (the offsets of a tile's rows have 32 bits)
    if (streams(a.T, a.K, a.N) || a.xs > kTileStride) return launch_linear_stream(a, s);
    const Plan p = plan(a.T, a.K, a.N, a.wg != nullptr);
    return a.bf16 ? launch_plan<st::kBF16>(a, p, s) : launch_plan<st::kF16>(a, p, s);
}

}  // namespace moeffn
