// Linear layer for more than 32 tokens: C = X W^T on MFMA, both operands
// k-contiguous, in tiles of BM tokens x BN weight rows staged through LDS (a
// gated tile holds BN / 2 rows of W and the same outputs' rows of Wg, so that a
// wave ends with both products of its outputs in registers).  Blocks of 64 k
// (128-byte rows) are copied global -> LDS by DMA while others are multiplied;
// the 16-byte chunks of a row are XOR-swizzled so that the rows a fragment read
// serves together fall in distinct banks.  The weights are the matrix
// instruction's A operand, so that a lane ends with four consecutive outputs of
// a token and stores them together.
//
// Two kernels.  Large products take 256 x 256 or 128 x 256 tiles and 8 waves in two
// groups a phase apart (linear_big_kernel), the others smaller tiles
// (linear_tile_kernel); where those are few, K is split over workgroups, whose
// fp32 products a second kernel adds in a fixed order before the epilogue.
// plan() chooses by what each was measured to cost.
// 4096 x 4096 x (2 x 14336), gated: 780-850 us, 1130-1230 TFLOP/s (MFMA busy 62%
// of the cycles at the 1.75 GHz that the power limit leaves).  300 x 4096 x 4096:
// 22 us in 128 x 256 tiles and 4 parts of K, and 5.6 us for their sum: 16 blocks of
// 0.88 us, of which the MFMAs are 0.43, and the start and end of the tile.
#include "linear_epilogue.hpp"

namespace moeffn {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kLgkm0 = 0xC07F;                      // s_waitcnt lgkmcnt(0)
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

// How a call is cut: tiles of outputs, K in `split` runs of `blocks` blocks, and
// whether the epilogue goes by fours.
struct Cut {
    int tm, tn, split, blocks, quads;
};

// The tile of workgroup b, which runs on XCD b % 8: each XCD takes a contiguous
// run of the tile order, in which groups of 4 token tiles pass over the outputs
// together, so that the tiles resident on an XCD share operands in its L2.
struct Place {
    int t, n, ks;                                   // tile of tokens and of outputs, run of K
    bool none;
};
__device__ __forceinline__ Place place(const Cut &c)
{
    constexpr int GM = 4;
    const int tiles = c.tm * c.tn * c.split, q8 = (tiles + 7) / 8;
    const int idx = (blockIdx.x & 7) * q8 + (blockIdx.x >> 3);
    Place p{};
    p.none = (int)(blockIdx.x >> 3) >= q8 || idx >= tiles;
    p.ks = idx / (c.tm * c.tn);
    const int id = idx - p.ks * c.tm * c.tn;
    const int grp = id / (GM * c.tn), gm = min(GM, c.tm - grp * GM), in = id - grp * GM * c.tn;
    p.t = grp * GM + in % gm;
    p.n = in / gm;
    return p;
}

// copy16_to_lds with the source as a scalar base and a 32-bit byte offset per
// lane, so that a block costs no vector arithmetic.
__device__ __forceinline__ void copy16_to_lds_at(const void *base, uint32_t off, void *lds_base)
{
    typedef __attribute__((address_space(3))) void lvoid;
    const uint32_t m = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lvoid *)lds_base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(m)
                 : "m0", "memory");
}

// Epilogue of a wave's subtiles (value r of lane l of a subtile is output
// 8 (r / 4) + 4 (l / 32) + r % 4, token l % 32): 32 tokens at a time through LDS
// of the wave's own, so that it stores whole runs of a token's outputs.
constexpr int kPadRow(int tn) { return 32 * tn + 4; }
constexpr int kWaveLds(int tn) { return 32 * kPadRow(tn) * 4; }

template <int TM, int TN, bool GATED>
__device__ __forceinline__ void store_tile(const LinearArgs &a, const Cut &c, int ks, int t0, int n0, int lane,
                                           float *lds, const floatx16 (&acc)[TM][TN])
{
    constexpr int HN = GATED ? TN / 2 : TN, LD = kPadRow(TN);
    const size_t plane = (size_t)a.T * a.N;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(float4 *)&lds[(lane & 31) * LD + 32 * j + 8 * q + 4 * (lane >> 5)] =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // written by other lanes of this wave
#pragma unroll 1
        for (int e = lane; e < 32 * 8 * HN; e += 64) {
            const int t = e / (8 * HN), col = 4 * (e % (8 * HN)), n = n0 + col;
            const float4 v4 = *(const float4 *)&lds[t * LD + col];
            const float4 g4 = *(const float4 *)&lds[t * LD + col + (GATED ? 32 * HN : 0)];
            float v[4] = {v4.x, v4.y, v4.z, v4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w};
            const int tok = t0 + 32 * i + t;
            if (tok >= a.T || n >= a.N) continue;
            if (c.split > 1) {
                float *p = a.part + (size_t)ks * (GATED ? 2 : 1) * plane + (size_t)tok * a.N + n;
                if (c.quads) {
                    *(float4 *)p = v4;
                    if (GATED) *(float4 *)(p + plane) = g4;
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (n + x < a.N) {
                            p[x] = v[x];
                            if (GATED) p[plane + x] = g[x];
                        }
                }
            } else if (c.quads) {
                le::finish4(a, tok, n, v, g);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (n + x < a.N) le::finish(a, tok, n + x, v[x], g[x]);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read before the next 32 tokens are written
    }
}

// S stages.  While block kb is multiplied the fragments of block kb + 1 are read
// from LDS and blocks kb + 2 .. kb + S are in flight; a barrier a block.
template <bool BF16, int BM, int BN, int WM, int WN, bool GATED, int S>
__global__ void __launch_bounds__(64 * WM * WN, 2)
linear_tile_kernel(LinearArgs a, Cut c)
{
    constexpr int W = WM * WN, ON = GATED ? BN / 2 : BN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32, HN = GATED ? TN / 2 : TN;
    constexpr int kStage = (BM + BN) * 128, NI = (BM + BN) / 8 / W, KS = kKB / 16;
    constexpr int NX = BM / 8 / W;                  // copies of token rows; then weight rows
    static_assert(S >= 2, "stages");
    static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0 && (!GATED || (TN % 2 == 0 && ON % (8 * W) == 0)), "tile");
    extern __shared__ __align__(16) unsigned char smem[];   // [S][kStage]
    const Place at = place(c);
    if (at.none) return;
    const int t0 = at.t * BM, n0 = at.n * ON;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int nkb = (a.K + kKB - 1) / kKB, kb0 = at.ks * c.blocks, kb1 = min(kb0 + c.blocks, nkb);

    // copy q of this wave fills rows 8 (wave + W q) .. of the stage; sources as byte
    // offsets from the tile's first token and weight rows
    const uint16_t *xb = a.x + (size_t)t0 * a.xs;
    const uint16_t *wb[2] = {a.w + (size_t)n0 * a.K, (GATED ? a.wg : a.w) + (size_t)n0 * a.K};
    uint32_t off[NI];
#pragma unroll
    for (int q = 0; q < NI; ++q) {
        const int row = 8 * (wave + W * q) + (lane >> 3), k = 8 * ((lane & 7) ^ swizzle(row));
        if (q < NX) off[q] = 2u * (uint32_t)(min(row, a.T - 1 - t0) * a.xs + k);
        else off[q] = 2u * (uint32_t)(min((row - BM) % ON, a.N - 1 - n0) * a.K + k);
    }
    // In a last block that K does not fill, lanes past K copy the row's last 8
    // values; once landed, zeros take their place.
    const int left = a.K - (nkb - 1) * kKB;         // k values of the last block
    auto past = [&](int q) { return 8 * ((lane & 7) ^ swizzle(8 * (wave + W * q) + (lane >> 3))) - (left - 8); };
    int next = kb0, put = 0;                        // the block that is copied next, and its stage
    auto issue = [&]() {
        unsigned char *base = smem + put * kStage + 1024 * wave;
        const bool tail = next == nkb - 1 && left < kKB;
#pragma unroll
        for (int q = 0; q < NI; ++q) {
            uint32_t o = off[q];
            if (tail) o -= 2u * (uint32_t)max(past(q), 0);
            const uint16_t *b = q < NX ? xb : wb[GATED && 8 * W * (q - NX) >= ON];
            copy16_to_lds_at(b + (size_t)next * kKB, o, base + 1024 * W * q);
        }
        put = put + 1 == S ? 0 : put + 1;
        ++next;
    };
    // this wave's copies of block kb have landed, `stage` being its stage
    auto landed = [&](int kb, int stage) {
        if (next - kb >= S - 1) st::wait_copies<NI * (S - 2)>();    // the S - 2 blocks after it may not have
        else st::wait_copies<0>();
        if (kb == nkb - 1 && left < kKB) {
            unsigned char *base = smem + stage * kStage + 1024 * wave + 16 * lane;
#pragma unroll
            for (int q = 0; q < NI; ++q)
                if (past(q) > 0) *(uint4 *)(base + 1024 * W * q) = make_uint4(0, 0, 0, 0);
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
        brow[j] = BM + (j < HN ? 32 * HN * wn + 32 * j : ON + 32 * HN * wn + 32 * (j - HN)) + li;
    struct Frags {
        uint4 a[TM][KS], b[TN][KS];
    };
    auto read = [&](Frags &f, int stage, int s) {   // 16 of a block's 64 k
        const unsigned char *stg = smem + stage * kStage;
#pragma unroll
        for (int i = 0; i < TM; ++i) f.a[i][s] = *(const uint4 *)(stg + lds_at(arow[i], 2 * s + hk));
#pragma unroll
        for (int j = 0; j < TN; ++j) f.b[j][s] = *(const uint4 *)(stg + lds_at(brow[j], 2 * s + hk));
    };
    int get = 0;                                    // stage of the block that is read next
    // the block in f, while the next one goes into g
    auto step = [&](int kb, Frags &f, Frags &g) {
        const bool more = kb + 1 < kb1;
        if (more) landed(kb + 1, get);
        // every wave has read block kb, whose stage is filled next, and can read block kb + 1
        // (a builtin, so that the compiler knows that f has arrived and does not wait
        // for g as well before it multiplies f)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kLgkm0);
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (more) read(g, get, s);
            if (s == 0 && next < kb1) issue();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma32<BF16>(f.b[j][s], f.a[i][s], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        get = get + 1 == S ? 0 : get + 1;
    };

#pragma unroll
    for (int s = 0; s < S; ++s)
        if (next < kb1) issue();
    Frags f0, f1;
    landed(kb0, 0);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < KS; ++s) read(f0, 0, s);
    get = 1;
    for (int kb = kb0; kb < kb1; kb += 2) {
        step(kb, f0, f1);
        if (kb + 1 < kb1) step(kb + 1, f1, f0);
    }
    __syncthreads();                                // the stages are done with
    static_assert(W * kWaveLds(TN) <= S * kStage, "the epilogue fits the stages");
    store_tile<TM, TN, GATED>(a, c, at.ks, t0 + BM / WM * wm, n0 + 32 * HN * wn, lane,
                              (float *)(smem + wave * kWaveLds(TN)), acc);
}

// Tiles of BM (256 or 128) tokens x 256 weight rows, 8 waves of BM / 2 tokens x 64 weight
// rows each (TM x 2 subtiles).  A block of 64 k takes a wave two phases, a barrier
// of the workgroup after each: it reads its fragments, then multiplies them
// (32 or 16 MFMAs).  Waves 4-7 run one phase behind waves 0-3 and every SIMD holds
// one of each, so that while one group multiplies the other reads LDS: in the 256
// x 256 tile 192 KB a block, with 64 KB written, which is all that LDS moves in
// the time of the MFMAs and would bound the tile by itself if the two did not
// overlap.  (There four phases of 16 MFMAs, whose barriers and first reads each cost
// about 270 cycles, took 3100 cycles a block.)
// S stages: the copies of block kb + S - 1 are issued when both groups have read
// block kb - 1, two phases (S 2) or four before they are needed.
template <bool BF16, bool GATED, int BM, int S>
__global__ void __launch_bounds__(512, 2)
linear_big_kernel(LinearArgs a, Cut c)
{
    constexpr int ON = GATED ? 128 : 256, HN = GATED ? 1 : 2, TM = BM / 64;
    constexpr int kStage = (BM + 256) * 128, NX = BM / 64, NI = NX + 4;
    extern __shared__ __align__(16) unsigned char smem[];   // [S][BM token rows, 256 weight rows][128 B]
    const Place at = place(c);
    if (at.none) return;
    const int t0 = at.t * BM, n0 = at.n * ON;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int nkb = (a.K + kKB - 1) / kKB, kb0 = at.ks * c.blocks, kb1 = min(kb0 + c.blocks, nkb);

    // copies 0 .. NX - 1 of this wave fill token rows 8 (wave + 8 q) .., the others
    // weight rows; sources as byte offsets from the tile's first row (launch_linear
    // sees to it that they fit)
    const uint16_t *xb = a.x + (size_t)t0 * a.xs;
    const uint16_t *wb[2] = {a.w + (size_t)n0 * a.K, (GATED ? a.wg : a.w) + (size_t)n0 * a.K};
    auto row_of = [&](int q) { return 8 * (wave + 8 * (q < NX ? q : q - NX)) + (lane >> 3); };
    uint32_t off[NI];
#pragma unroll
    for (int q = 0; q < NI; ++q) {
        const int row = row_of(q), k = 8 * ((lane & 7) ^ swizzle(row));
        if (q < NX) off[q] = 2u * (uint32_t)(min(row, a.T - 1 - t0) * a.xs + k);
        else off[q] = 2u * (uint32_t)(min(GATED ? row & 127 : row, a.N - 1 - n0) * a.K + k);
    }
    // In a last block that K does not fill, lanes past K copy the row's last 8
    // values; once landed, zero_tail puts zeros in their place.
    const int left = a.K - (nkb - 1) * kKB;         // k values of the last block
    auto past = [&](int q) { return 8 * ((lane & 7) ^ swizzle(row_of(q))) - (left - 8); };
    int put = 0, get = 0;                           // stages of the block copied next and of the one read next
    auto copy_block = [&](int kb) {
        unsigned char *st = smem + put * kStage + 1024 * wave;
        put = put + 1 == S ? 0 : put + 1;
        const bool tail = kb == nkb - 1 && left < kKB;
#pragma unroll
        for (int q = 0; q < NI; ++q) {
            const uint16_t *b = q < NX ? xb : wb[GATED && q >= NX + 2 ? 1 : 0];
            uint32_t o = off[q];
            if (tail) o -= 2u * (uint32_t)max(past(q), 0);
            copy16_to_lds_at(b + (size_t)kb * kKB, o, st + 8192 * q);
        }
    };
    // this wave's copies of block kb, in stage `get`, have landed
    auto landed = [&](int kb) {
        if (kb + S - 2 < kb1) st::wait_copies<NI * (S - 2)>();      // all S - 2 blocks after it are in flight
        else st::wait_copies<0>();
        if (kb != nkb - 1 || left == kKB) return;
        unsigned char *st = smem + get * kStage + 1024 * wave + 16 * lane;
#pragma unroll
        for (int q = 0; q < NI; ++q)
            if (past(q) > 0) *(uint4 *)(st + 8192 * q) = make_uint4(0, 0, 0, 0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };

    floatx16 acc[TM][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int li = lane & 31, hk = lane >> 5;
    int brow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) brow[j] = BM + (GATED ? 128 * j + 32 * wn : 64 * wn + 32 * j) + li;

    uint4 av[TM][4], bv[2][4];
    auto read_block = [&]() {
        const unsigned char *st = smem + get * kStage;
        get = get + 1 == S ? 0 : get + 1;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) bv[j][s] = *(const uint4 *)(st + lds_at(brow[j], 2 * s + hk));
#pragma unroll
            for (int i = 0; i < TM; ++i)
                av[i][s] = *(const uint4 *)(st + lds_at(32 * TM * wm + 32 * i + li, 2 * s + hk));
        }
    };
    auto multiply = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mma32<BF16>(bv[j][s], av[i][s], acc[i][j]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (kb0 + i < kb1) copy_block(kb0 + i);
    landed(kb0);
    asm volatile("s_barrier" ::: "memory");
    // phase p of the workgroup: waves 0-3 read block kb0 + p / 2 or multiply it, waves
    // 4-7 do what those did in phase p - 1; both copy in even phases and have
    // waited by the end of the odd ones for what is read next
    if (wm == 0) {
        for (int kb = kb0; kb < kb1; ++kb) {
            read_block();
            if (kb + S - 1 < kb1) copy_block(kb + S - 1);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            multiply();
            if (kb + 1 < kb1) landed(kb + 1);
            asm volatile("s_barrier" ::: "memory");
        }
        asm volatile("s_barrier" ::: "memory");
    } else {
        if (kb0 + S - 1 < kb1) copy_block(kb0 + S - 1);
        asm volatile("s_barrier" ::: "memory");
        for (int kb = kb0; kb < kb1; ++kb) {
            read_block();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (kb + 1 < kb1) landed(kb + 1);
            asm volatile("s_barrier" ::: "memory");
            if (kb + S < kb1) copy_block(kb + S);
            multiply();
            asm volatile("s_barrier" ::: "memory");
        }
    }
    __syncthreads();
    static_assert(8 * kWaveLds(2) <= S * kStage, "the epilogue fits the stages");
    store_tile<TM, 2, GATED>(a, c, at.ks, t0 + 32 * TM * wm, n0 + 32 * HN * wn, lane, (float *)(smem + wave * kWaveLds(2)),
                             acc);
}

constexpr int kMaxSplit = 8;

// Sum of the split's products, in order, and the epilogue: a thread takes four outputs
// of a token where they can be read and written together (Q 4), else one, and
// loads all their products before it uses the first (4096 outputs of 300 tokens
// in four parts: 5.6 us, against 8.4 by single outputs and loads).
template <int Q>
__global__ void __launch_bounds__(256)
linear_join_kernel(LinearArgs a, int split)
{
    const int n = Q * (blockIdx.x * 256 + threadIdx.x), nm = a.wg ? 2 : 1;
    const size_t plane = (size_t)a.T * a.N;
    if (n >= a.N) return;
    for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
        float v[2][Q] = {};
        for (int m = 0; m < nm; ++m) {
            const float *p = a.part + m * plane + (size_t)t * a.N + n;
            float q[kMaxSplit][Q];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)
                if (s < split) {
                    const float *ps = p + (size_t)s * nm * plane;
                    if constexpr (Q == 4) *(float4 *)q[s] = *(const float4 *)ps;
                    else q[s][0] = *ps;
                }
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)
                if (s < split)
#pragma unroll
                    for (int x = 0; x < Q; ++x) v[m][x] += q[s][x];
        }
        if constexpr (Q == 4) le::finish4(a, t, n, v[0], v[1]);
        else le::finish(a, t, n, v[0][0], v[1][0]);
    }
}

// The tiles that a call can take, and what a block of 64 k costs a compute unit, in
// microseconds as measured: one workgroup alone on it, and two together where
// two fit.  (Alone, a small tile waits: for its barrier, LDS and a chain of MFMAs.
// 128 x 256 costs 0.88 on a few units and 1.02 with all of them at work.)
struct Tile {
    int bm, bn;                                     // tokens x weight rows
    double one, two;                                // two: 0 where one workgroup's LDS fills the unit
};
constexpr Tile kTiles[] = {{64, 64, 0.40, 0.55}, {128, 64, 0.50, 0.75}, {128, 128, 1.05, 1.25}, {128, 256, 1.0, 0.0},
                           {256, 256, 1.75, 0.0}};
constexpr int kUnits = 256;                         // compute units

struct Plan {
    int tile;                                       // of kTiles
    Cut c;
};

constexpr long long kTileStride = 1 << 21;          // elements: 256 rows within 1 GB

// The tile and split of K with the least expected time: rounds of workgroups over the
// compute units, and for a split the second kernel (4 us) and the products written
// and read at 4 TB/s.
Plan plan(int T, int K, int N, bool gated)
{
    const int nkb = (K + kKB - 1) / kKB, g = gated ? 2 : 1;
    Plan best{};
    double least = 1e30;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const Tile &t = kTiles[i];
        Cut c{};
        c.tm = (T + t.bm - 1) / t.bm;
        c.tn = (N + t.bn / g - 1) / (t.bn / g);
        for (int want = 1; want <= (t.bm == 256 ? 1 : kMaxSplit); want *= 2) {
            if (want > 1 && nkb < 4 * want) break;
            c.blocks = (nkb + want - 1) / want;
            c.split = (nkb + c.blocks - 1) / c.blocks;
            const long long wgs = (long long)c.tm * c.tn * c.split;
            const int per = t.two > 0.0 ? 2 * kUnits : kUnits;
            const long long rest = wgs % per;
            double us = (double)(wgs / per) * (t.two > 0.0 ? t.two : t.one);
            if (rest > kUnits) us += t.two;
            else if (rest > 0) us += t.one;
            us *= c.blocks;
            if (c.split > 1) us += 4.0 + 8e-6 * c.split * g * (double)T * N / 4.0;
            if (us < least) {
                least = us;
                best = Plan{i, c};
            }
        }
    }
    return best;
}

hipError_t launch_cut(const void *k, const LinearArgs &a, const Cut &c, int threads, int lds, hipStream_t s)
{
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    void *args[] = {(void *)&a, (void *)&c};
    const unsigned grid = (unsigned)((c.tm * c.tn * c.split + 7) / 8 * 8);
    const hipError_t e = hipLaunchKernel(k, dim3(grid), dim3(threads), args, lds, s);
    return e != hipSuccess ? e : hipGetLastError();
}

template <bool BF16, int BM, int BN, int WM, int WN, bool GATED, int S>
hipError_t launch_tile(const LinearArgs &a, const Cut &c, hipStream_t s)
{
    return launch_cut((const void *)linear_tile_kernel<BF16, BM, BN, WM, WN, GATED, S>, a, c, 64 * WM * WN,
                      S * (BM + BN) * 128, s);
}

template <bool BF16, bool GATED, int BM, int S>
hipError_t launch_big(const LinearArgs &a, const Cut &c, hipStream_t s)
{
    return launch_cut((const void *)linear_big_kernel<BF16, GATED, BM, S>, a, c, 512, S * (BM + 256) * 128, s);
}

template <bool BF16>
hipError_t launch_t(const LinearArgs &a, const Plan &p, hipStream_t s)
{
    switch (p.tile) {
    case 0:
        return a.wg ? launch_tile<BF16, 64, 64, 2, 1, true, 4>(a, p.c, s)
                    : launch_tile<BF16, 64, 64, 2, 2, false, 4>(a, p.c, s);
    case 1:
        return a.wg ? launch_tile<BF16, 128, 64, 4, 1, true, 3>(a, p.c, s)
                    : launch_tile<BF16, 128, 64, 2, 2, false, 3>(a, p.c, s);
    case 2:
        return a.wg ? launch_tile<BF16, 128, 128, 2, 2, true, 2>(a, p.c, s)
                    : launch_tile<BF16, 128, 128, 2, 2, false, 2>(a, p.c, s);
    case 3:
        return a.wg ? launch_big<BF16, true, 128, 3>(a, p.c, s) : launch_big<BF16, false, 128, 3>(a, p.c, s);
    }
    return a.wg ? launch_big<BF16, true, 256, 2>(a, p.c, s) : launch_big<BF16, false, 256, 2>(a, p.c, s);
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
    Plan p = plan(a.T, a.K, a.N, a.wg != nullptr);
    p.c.quads = p.c.split > 1 ? a.N % 4 == 0 : le::quads(a);
    const hipError_t e = a.bf16 ? launch_t<true>(a, p, s) : launch_t<false>(a, p, s);
    if (e != hipSuccess || p.c.split == 1) return e;
    const bool four = le::quads(a);
    const int wide = four ? 1024 : 256;             // outputs of a workgroup
    hipLaunchKernelGGL(four ? linear_join_kernel<4> : linear_join_kernel<1>,
                       dim3((unsigned)((a.N + wide - 1) / wide), (unsigned)(a.T < 65535 ? a.T : 65535)), dim3(256), 0, s,
                       a, p.c.split);
    return hipGetLastError();
}

}  // namespace moeffn
