// Linear layer on 16-bit types in tiles, and the choice between tiles and streams.
#include "linear_tile.hpp"

namespace moeffn {

namespace {

// (128 x 256 costs 0.88 on a few units and 1.02 with all of them at work; products at 4 TB/s)
constexpr Tile kList[] = {{64, 64, 0.40, 0.55, 0.0}, {128, 64, 0.50, 0.75, 0.0}, {128, 128, 1.05, 1.25, 0.0},
                          {128, 256, 1.0, 0.0, 0.0}, {256, 256, 1.75, 0.0, 0.0}};
constexpr Tiles kTiles{kList, 5, 4.0, 8e-6 / 4.0};

template <int U>
hipError_t launch_t(const le::Args<U> &a, const Plan &p, hipStream_t s)
{
    switch (p.tile) {
    case 0:
        return a.wg ? launch_tile<U, 64, 64, 2, 1, true, 4>(a, p.c, s)
                    : launch_tile<U, 64, 64, 2, 2, false, 4>(a, p.c, s);
    case 1:
        return a.wg ? launch_tile<U, 128, 64, 4, 1, true, 3>(a, p.c, s)
                    : launch_tile<U, 128, 64, 2, 2, false, 3>(a, p.c, s);
    case 2:
        return a.wg ? launch_tile<U, 128, 128, 2, 2, true, 2>(a, p.c, s)
                    : launch_tile<U, 128, 128, 2, 2, false, 2>(a, p.c, s);
    case 3:
        return a.wg ? launch_big<U, true, 128, 3>(a, p.c, s) : launch_big<U, false, 128, 3>(a, p.c, s);
    }
    return a.wg ? launch_big<U, true, 256, 2>(a, p.c, s) : launch_big<U, false, 256, 2>(a, p.c, s);
}

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
    const Plan p = plan(kTiles, T, K, N, gated);
    *bm = kList[p.tile].bm;
    *bn = kList[p.tile].bn;
    return p.c.split;
}

size_t linear_ws_bytes(int T, int K, int N)
{
    if (streams(T, K, N)) return 0;
    const Plan p = plan(kTiles, T, K, N, false), g = plan(kTiles, T, K, N, true);
    const size_t np = p.c.split > 1 ? p.c.split : 0, ng = g.c.split > 1 ? 2 * g.c.split : 0;
    return (np > ng ? np : ng) * (size_t)T * N * 4;
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t s)
{
    if (a.T < 1 || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    // (the offsets of a tile's rows have 32 bits)
    if (streams(a.T, a.K, a.N) || a.xs > kTileStride) return launch_linear_stream(a, s);
    const Plan p = plan(kTiles, a.T, a.K, a.N, a.wg != nullptr);
    return a.bf16 ? launch_plan<st::kBF16>(a, p, launch_t<st::kBF16>, s) : launch_plan<st::kF16>(a, p, launch_t<st::kF16>, s);
}

}  // namespace moeffn
