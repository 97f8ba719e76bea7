// Linear layer for at most 32 tokens, or a few times that in small layers: the
// weights are streamed past 32 tokens at a time (mfma_stream.hpp).  A wave takes 16 NM
// weight rows (of both matrices when gated) and a slice of K; the P waves of a
// workgroup that share the rows add their slices through LDS in a fixed order
// and apply the epilogue.  Workgroups are small (4 waves), so that several share a
// compute unit and one streams while another starts or ends.
// Bound by HBM: 1 x 4096 x 28672 (gated) 38 us, 6.2 TB/s; 16 x 14336 x 4096 24 us, 4.8 TB/s.
#include "linear_epilogue.hpp"

#include <algorithm>

namespace moeffn {

namespace {

using st::floatx4;

// NM: groups of 16 weight rows per wave, the second half of Wg when GATED;
// XR: token rows; D: blocks in the ring.
template <bool BF16, bool GATED, int NM, int XR, int D>
__global__ void __launch_bounds__(1024)
linear_stream_kernel(LinearArgs a, int P, int slice)
{
    using R = st::Ring<NM, XR>;
    constexpr int NB = R::kFrag, NO = GATED ? NM / 2 : NM;      // NO: groups of 16 outputs
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)(blockDim.x >> 6) / P;       // output groups in this workgroup
    const int g = wave / P, p = wave - g * P;
    const int units = (a.N + 16 * NO - 1) / (16 * NO);
    // Workgroup b runs on XCD b % 8.  The token tiles of one set of rows follow
    // each other on one XCD, where all but the first find the weights in L2.
    const int tiles = (a.T + XR - 1) / XR, q = blockIdx.x >> 3;
    const int u0 = (q / tiles * 8 + (blockIdx.x & 7)) * G, t0 = q % tiles * XR;

    floatx4 acc[NM][NB];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int blocks = (a.K + 63) / 64, b0 = p * slice, b1 = min(b0 + slice, blocks);
    if (u0 + g < units && b0 < b1) {
        const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
        const uint16_t *src[R::kCopies];
#pragma unroll
        for (int i = 0; i < 2 * NM; ++i) {
            const bool gate = GATED && i >= NM;
            const int n = min(16 * NO * (u0 + g) + 8 * (gate ? i - NM : i) + r, a.N - 1);
            src[i] = (gate ? a.wg : a.w) + (size_t)n * a.K + k;
        }
#pragma unroll
        for (int i = 0; i < R::kTok; ++i) src[2 * NM + i] = a.x + (size_t)min(t0 + 8 * i + r, a.T - 1) * a.xs + k;
        st::stream<BF16, NM, XR, D>(acc, smem + wave * D * R::kBlock, src, b1 - b0,
                                    b1 == blocks ? a.K - 64 * (blocks - 1) : 64, lane);
    }
    __syncthreads();                                // the rings are done with
    float *red = (float *)smem;                     // [waves][NM][NB][64 lanes][4]
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(floatx4 *)&red[((wave * NM + m) * NB + j) * 256 + 4 * lane] = acc[m][j];
    __syncthreads();
    for (int i = tid; i < G * NO * NB * 256; i += blockDim.x) {
        const int gg = i / (NO * NB * 256), e = i - gg * NO * NB * 256;
        const int t = e / (16 * NO), o = e - t * 16 * NO;       // token, output of the group
        const int n = 16 * NO * (u0 + gg) + o;
        if (t >= XR || t0 + t >= a.T || n >= a.N) continue;
        const int r = o & 15;
        const int at = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        float v = 0.f, g2 = 0.f;
        for (int q = 0; q < P; ++q) {
            const float *pr = red + ((gg * P + q) * NM + (o >> 4)) * NB * 256 + at;
            v += pr[0];
            if (GATED) g2 += pr[NO * NB * 256];
        }
        le::finish(a, t0 + t, n, v, g2);
    }
}

template <bool BF16, bool GATED, int NM, int XR, int D>
hipError_t launch_one(const LinearArgs &a, hipStream_t s)
{
    using R = st::Ring<NM, XR>;
    constexpr int NO = GATED ? NM / 2 : NM;
    const int units = (a.N + 16 * NO - 1) / (16 * NO), blocks = (a.K + 63) / 64;
    constexpr int ring = D * R::kBlock, red = NM * R::kFrag * 1024, per = ring > red ? ring : red;
    static_assert(4 * per <= 160 * 1024, "four waves' rings fit a compute unit");
    // slices of K: 4; 8 while the waves are too few to fill the chip, a slice
    // keeps 4 blocks and the rings fit; fewer when K is short
    int P = 4;
    if (8 * per <= 160 * 1024 && (long long)units * P < 2048 && blocks >= 8 * P) P = 8;
    while (P > 1 && blocks < P) P /= 2;
    const int G = P < 4 ? 4 / P : 1, slice = (blocks + P - 1) / P;
    const int lds = G * P * per;
    const void *k = (const void *)linear_stream_kernel<BF16, GATED, NM, XR, D>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const unsigned sets = (unsigned)((units + G - 1) / G + 7) / 8, tiles = (unsigned)((a.T + XR - 1) / XR);
    hipLaunchKernelGGL((linear_stream_kernel<BF16, GATED, NM, XR, D>), dim3(8 * sets * tiles),
                       dim3(64 * G * P), lds, s, a, P, slice);
    return hipGetLastError();
}

// Rows per wave: 16 (and 16 of Wg).  From 17 tokens a block of tokens is larger
// than that of 16 rows, so wide layers take 32 + 32 or 64.
template <bool BF16, int XR>
hipError_t launch_xr(const LinearArgs &a, hipStream_t s)
{
    if constexpr (XR > 16)
        if (a.N >= 16384)
            return a.wg ? launch_one<BF16, true, 4, XR, 3>(a, s) : launch_one<BF16, false, 4, XR, 3>(a, s);
    constexpr int D = XR <= 16 ? 4 : 3;
    return a.wg ? launch_one<BF16, true, 2, XR, 3>(a, s) : launch_one<BF16, false, 1, XR, D>(a, s);
}

template <bool BF16>
hipError_t launch_t(const LinearArgs &a, hipStream_t s)
{
    if (a.T == 1) return launch_xr<BF16, 1>(a, s);
    if (a.T <= 8) return launch_xr<BF16, 8>(a, s);
    if (a.T <= 16) return launch_xr<BF16, 16>(a, s);
    if (a.T <= 24) return launch_xr<BF16, 24>(a, s);
    return launch_xr<BF16, 32>(a, s);
}

}  // namespace

hipError_t launch_linear_stream(const LinearArgs &a, hipStream_t s)
{
    if (a.T < 1 || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    // A launch may have at most 2^32 - 1 threads, here 512 a workgroup and one workgroup
    // for 16 outputs of 32 tokens at the most: more tokens go in runs.
    const long long sets = ((long long)a.N + 127) / 128 * 8;
    const int run = 32 * (int)std::max(1ll, (1ll << 22) / sets);
    const size_t ye = a.ydt == 2 ? 4 : 2;
    LinearArgs b = a;
    for (int t = 0; t < a.T; t += run) {
        b.T = std::min(run, a.T - t);
        b.x = a.x + (size_t)t * a.xs;
        b.y = (char *)a.y + ye * t * a.ys;
        if (a.r) b.r = (const char *)a.r + ye * t * a.rs;
        const hipError_t e = a.bf16 ? launch_t<true>(b, s) : launch_t<false>(b, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moeffn
