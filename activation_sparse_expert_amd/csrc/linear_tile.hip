// Linear layer for more than 32 tokens: C = X W^T on MFMA, both operands
// k-contiguous, in tiles of BM tokens x BN weight rows staged through LDS (a
// gated tile holds BN / 2 rows of W and the same outputs' rows of Wg, so that a
// wave ends with both products of its outputs in registers).  Blocks of 64 k
// (128-byte rows) are copied global -> LDS by DMA into one stage while the other
// is multiplied; the 16-byte chunks of a row are XOR-swizzled so that the rows a
// fragment read serves together fall in distinct banks.
//
// With few tiles K is split over workgroups, whose fp32 products a second kernel
// adds in a fixed order before the epilogue.
#include "linear_epilogue.hpp"

namespace moeffn {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kKB = 64;                             // k values per block: 128-byte rows

template <bool BF16>
__device__ __forceinline__ floatx16 mma32(const uint4 &a, const uint4 &b, const floatx16 &c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(st::bf16x8_t, a),
                                                       __builtin_bit_cast(st::bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(st::f16x8_t, a),
                                                      __builtin_bit_cast(st::f16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }
__device__ __forceinline__ int lds_at(int row, int c) { return row * 128 + 16 * (c ^ swizzle(row)); }

// How a call is cut: tiles of outputs, and K in `split` runs of `blocks` blocks.
struct Cut {
    int tm, tn, split, blocks;
};

template <bool BF16, int BM, int BN, int WM, int WN, bool GATED>
__global__ void __launch_bounds__(64 * WM * WN)
linear_tile_kernel(LinearArgs a, Cut c)
{
    constexpr int W = WM * WN, ON = GATED ? BN / 2 : BN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32, HN = GATED ? TN / 2 : TN;
    constexpr int kStage = (BM + BN) * 128, NI = (BM + BN) / 8 / W;
    static_assert((BM + BN) % (8 * W) == 0 && (!GATED || TN % 2 == 0), "tile");
    extern __shared__ __align__(16) unsigned char smem[];   // [2][kStage]

    // Workgroup b runs on XCD b % 8: each XCD takes a contiguous run of the tile
    // order, in which groups of 4 token tiles pass over the outputs together, so
    // that the tiles resident on an XCD share operands in its L2.
    const int tiles = c.tm * c.tn * c.split, q8 = (tiles + 7) / 8;
    const int idx = (blockIdx.x & 7) * q8 + (blockIdx.x >> 3);
    if (idx >= tiles) return;
    const int ks = idx / (c.tm * c.tn), id = idx - ks * c.tm * c.tn;
    constexpr int GM = 4;
    const int grp = id / (GM * c.tn), gm = min(GM, c.tm - grp * GM);
    const int in = id - grp * GM * c.tn;
    const int t0 = (grp * GM + in % gm) * BM, n0 = in / gm * ON;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % WM, wn = wave / WM;
    const int kb0 = ks * c.blocks, kb1 = min(kb0 + c.blocks, (a.K + kKB - 1) / kKB);

    // copy sources: instruction q of this wave fills 8 rows of the stage, lane l
    // row l / 8, chunk l % 8 as stored; rows past the last token or output repeat it
    const uint16_t *src[NI];
    int ch[NI];
#pragma unroll
    for (int q = 0; q < NI; ++q) {
        const int row = 8 * (wave + W * q) + (lane >> 3);
        ch[q] = 8 * ((lane & 7) ^ swizzle(row));
        if (row < BM) {
            src[q] = a.x + (size_t)min(t0 + row, a.T - 1) * a.xs + ch[q];
        } else {
            const int br = row - BM;
            const bool gate = GATED && br >= BN / 2;
            const int n = min(n0 + (gate ? br - BN / 2 : br), a.N - 1);
            src[q] = (gate ? a.wg : a.w) + (size_t)n * a.K + ch[q];
        }
    }
    auto issue = [&](int kb, int stage) {
        unsigned char *base = smem + stage * kStage;
        if ((kb + 1) * kKB <= a.K) {
#pragma unroll
            for (int q = 0; q < NI; ++q)
                copy16_to_lds(src[q] + (size_t)kb * kKB, base + 1024 * (wave + W * q));
        } else {
#pragma unroll
            for (int q = 0; q < NI; ++q)
                copy16_to_lds(kb * kKB + ch[q] < a.K ? src[q] + (size_t)kb * kKB : st::zeros16,
                              base + 1024 * (wave + W * q));
        }
    };

    floatx16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const int li = lane & 31, hk = lane >> 5;
    int arow[TM], brow[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) arow[i] = BM / WM * wm + 32 * i + li;
#pragma unroll
    for (int j = 0; j < TN; ++j)
        brow[j] = BM + (j < HN ? 32 * HN * wn + 32 * j : BN / 2 + 32 * HN * wn + 32 * (j - HN)) + li;

    issue(kb0, 0);
    for (int kb = kb0; kb < kb1; ++kb) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();                            // block kb has landed; the other stage is free
        if (kb + 1 < kb1) issue(kb + 1, (kb + 1 - kb0) & 1);
        const unsigned char *stg = smem + ((kb - kb0) & 1) * kStage;
#pragma unroll
        for (int s = 0; s < kKB / 16; ++s) {
            uint4 av[TM], bv[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) av[i] = *(const uint4 *)(stg + lds_at(arow[i], 2 * s + hk));
#pragma unroll
            for (int j = 0; j < TN; ++j) bv[j] = *(const uint4 *)(stg + lds_at(brow[j], 2 * s + hk));
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma32<BF16>(av[i], bv[j], acc[i][j]);
        }
    }

    // value r of lane l of a subtile: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
    const size_t plane = (size_t)a.T * a.N;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < HN; ++j) {
            const int n = n0 + 32 * HN * wn + 32 * j + li;
            if (n >= a.N) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = t0 + BM / WM * wm + 32 * i + 8 * (r >> 2) + 4 * hk + (r & 3);
                if (t >= a.T) continue;
                const float g = GATED ? acc[i][GATED ? j + HN : j][r] : 0.f;
                if (c.split > 1) {
                    float *p = a.part + (size_t)ks * (GATED ? 2 : 1) * plane + (size_t)t * a.N + n;
                    p[0] = acc[i][j][r];
                    if (GATED) p[plane] = g;
                } else {
                    le::finish(a, t, n, acc[i][j][r], g);
                }
            }
        }
}

// Sum of the split's products, in order, and the epilogue.
__global__ void __launch_bounds__(256)
linear_join_kernel(LinearArgs a, int split)
{
    const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (n >= a.N) return;
    const size_t plane = (size_t)a.T * a.N;
    const int nm = a.wg ? 2 : 1;
    const float *p = a.part + (size_t)t * a.N + n;
    float v[2] = {0.f, 0.f};
    for (int s = 0; s < split; ++s)
        for (int m = 0; m < nm; ++m) v[m] += p[(size_t)(s * nm + m) * plane];
    le::finish(a, t, n, v[0], v[1]);
}

// Tile sizes by the number of tiles they give: 128 tokens x 128 weight rows, or
// 64 x 64 outputs while those leave compute units idle.
struct Plan {
    int bm;                                         // 128 or 64
    Cut c;
};

constexpr int kMaxSplit = 8;

Plan plan(int T, int K, int N, bool gated)
{
    const int nkb = (K + kKB - 1) / kKB;
    Plan p;
    const long long big = (long long)((T + 127) / 128) * ((N + (gated ? 63 : 127)) / (gated ? 64 : 128));
    p.bm = big >= 256 ? 128 : 64;
    const int on = p.bm == 128 && !gated ? 128 : 64;
    p.c.tm = (T + p.bm - 1) / p.bm;
    p.c.tn = (N + on - 1) / on;
    int split = 1;
    while (split < kMaxSplit && (long long)p.c.tm * p.c.tn * split < 256 && nkb >= 16 * split) split *= 2;
    p.c.blocks = (nkb + split - 1) / split;
    p.c.split = (nkb + p.c.blocks - 1) / p.c.blocks;
    return p;
}

template <bool BF16, int BM, int BN, int WM, int WN, bool GATED>
hipError_t launch_one(const LinearArgs &a, const Cut &c, hipStream_t s)
{
    constexpr int lds = 2 * (BM + BN) * 128;
    const void *k = (const void *)linear_tile_kernel<BF16, BM, BN, WM, WN, GATED>;
    hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)((c.tm * c.tn * c.split + 7) / 8 * 8);
    hipLaunchKernelGGL((linear_tile_kernel<BF16, BM, BN, WM, WN, GATED>), dim3(grid), dim3(64 * WM * WN), lds, s, a, c);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_t(const LinearArgs &a, const Plan &p, hipStream_t s)
{
    if (p.bm == 128)
        return a.wg ? launch_one<BF16, 128, 128, 2, 2, true>(a, p.c, s)
                    : launch_one<BF16, 128, 128, 2, 2, false>(a, p.c, s);
    return a.wg ? launch_one<BF16, 64, 128, 2, 2, true>(a, p.c, s) : launch_one<BF16, 64, 64, 2, 2, false>(a, p.c, s);
}

}  // namespace

size_t linear_tile_ws_bytes(int T, int K, int N)
{
    const Plan p = plan(T, K, N, false), g = plan(T, K, N, true);
    const size_t np = p.c.split > 1 ? p.c.split : 0, ng = g.c.split > 1 ? 2 * g.c.split : 0;
    return (np > ng ? np : ng) * (size_t)T * N * 4;
}

hipError_t launch_linear_tile(const LinearArgs &a, hipStream_t s)
{
    if (a.T < 1 || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    const Plan p = plan(a.T, a.K, a.N, a.wg != nullptr);
    const hipError_t e = a.bf16 ? launch_t<true>(a, p, s) : launch_t<false>(a, p, s);
    if (e != hipSuccess || p.c.split == 1) return e;
    hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.T), dim3(256), 0, s, a,
                       p.c.split);
    return hipGetLastError();
}

}  // namespace moeffn
