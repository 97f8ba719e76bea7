// Linear layer for at most 32 tokens, or a few times that in small layers: the
// weights are streamed past 32 tokens at a time (mfma_stream.hpp).  A wave takes 16 NM
// weight rows (of both matrices when gated) and a slice of K; the P waves of a
// workgroup that share the rows add their slices through LDS in a fixed order
// and apply the epilogue.  Workgroups are small (4 waves), so that several share a
// compute unit and one streams while another starts or ends.
// Bound by HBM, 16-bit weights: 1 x 4096 x 28672 (gated) 38 us, 6.2 TB/s; 16 x 14336 x 4096 24 us,
// 4.8 TB/s.  8-bit codes, two to a 16-bit unit, are half the bytes: 20 us and 12.7 us; one token that is
// no codes yet is made some in LDS by each workgroup (OwnCodes).  17 to 32 tokens over a long k are
// bound by the copies into LDS, two thirds of which are tokens that each wave copies for
// itself: 32 x 14336 x 4096 17.3 us of codes.
#pragma once
#include "linear_epilogue.hpp"
#include "row_io.hpp"

#include <algorithm>

namespace moeffn {

namespace {

// LDS of a token of k numbers, in whole copies
__host__ __device__ constexpr int own_raw_bytes(int k, int xdt) { return (k * (xdt == 2 ? 4 : 2) + 1023) / 1024 * 1024; }

// One token of type XDT (0 f16, 1 bf16, 2 f32) that the workgroup makes codes of for itself: copied
// into LDS before the first weights, which are on their way meanwhile.
template <int XDT>
struct OwnCodes {
    unsigned char *raw, *codes;                     // LDS: the token, its codes (zeros up to whole blocks)
    int k, pad;                                     // codes, and those of whole blocks
    uint32_t *slots;                                // LDS [16]
    codes::Row row;

    __device__ __forceinline__ void copy(const void *x, int wave, int lane) const
    {
        const int bytes = k * (XDT == 2 ? 4 : 2);
        for (int c = 1024 * wave; c < bytes; c += 16 * blockDim.x)
            if (c + 16 * lane < bytes) copy16_to_lds((const unsigned char *)x + c + 16 * lane, raw + c);
    }
    // (the token's own copies have landed)
    __device__ __forceinline__ void make()
    {
        __syncthreads();
        uint32_t most = 0;
        for (int i = 8 * threadIdx.x; i < k; i += 8 * blockDim.x)
            most = rio::umax(most, rio::most<XDT == 2>(rio::load<XDT == 2, true>(raw, XDT, i, 8, 0), XDT));
        most = rio::seg_max<64>(most);
        if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = most;
        __syncthreads();
        for (int i = 0; i < (int)(blockDim.x >> 6); ++i) most = rio::umax(most, slots[i]);
        row = codes::row(most);
        const double f = XDT == 2 ? codes::factor64(row) : 0.0;
        for (int i = 8 * threadIdx.x; i < pad; i += 8 * blockDim.x) {
            float v[8];
            uint32_t q[8];
            rio::floats<XDT == 2>(rio::load<XDT == 2, true>(raw, XDT, i < k ? i : 0, 8, 0), XDT, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = XDT == 2 ? codes::code64(v[j], f) : codes::code(v[j], row);
            rio::store_codes<true>((int8_t *)codes, i, 8, 0, q, row.ok && i < k);
        }
        __syncthreads();
    }
};
template <>
struct OwnCodes<-1> {};

// NM: groups of 16 weight rows per wave, the second half of Wg when GATED;
// XR: token rows; D: blocks in the ring.  XDT: one token that is no codes yet (XR 0), or -1.
template <int U, bool GATED, int NM, int XR, int D, int XDT = -1>
__global__ void __launch_bounds__(1024)
linear_stream_kernel(le::Args<U> a, int P, int slice)
{
    static_assert((XDT >= 0) == (XR == 0) && (XDT < 0 || U == st::kI8), "a token of its own");
    using R = st::Ring<NM, XR, U>;
    constexpr int NB = R::kFrag, NO = GATED ? NM / 2 : NM;      // NO: groups of 16 outputs
    constexpr int XT = XR ? XR : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t slots[16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)(blockDim.x >> 6) / P;       // output groups in this workgroup
    const int g = wave / P, p = wave - g * P;
    const int units = (a.N + 16 * NO - 1) / (16 * NO);
    // Workgroup b runs on XCD b % 8.  The token tiles of one set of rows follow
    // each other on one XCD, where all but the first find the weights in L2.
    const int tiles = (a.T + XT - 1) / XT, q = blockIdx.x >> 3;
    const int u0 = (q / tiles * 8 + (blockIdx.x & 7)) * G, t0 = q % tiles * XT;

    typename R::Acc acc;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = typename st::Sum<U>::x4{0, 0, 0, 0};
    const int blocks = (a.K + 63) / 64, b0 = p * slice, b1 = min(b0 + slice, blocks);
    unsigned char *rings = smem;
    OwnCodes<XDT> own;
    if constexpr (XDT >= 0) {
        own.k = 2 * a.K;
        own.pad = 128 * blocks;
        own.raw = smem;
        own.codes = smem + own_raw_bytes(own.k, XDT);
        own.slots = slots;
        rings = own.codes + own.pad;
        own.copy(a.x, wave, lane);
    }
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
        const int kl = b1 == blocks ? a.K - 64 * (blocks - 1) : 64;
        if constexpr (XDT >= 0)
            st::stream<U, NM, XR, D>(acc, rings + wave * D * R::kBlock, src, b1 - b0, kl, lane, own.codes + 128 * b0,
                                     [&](bool all) {
                                         if (all) st::wait_copies<(D - 1) * R::kCopies>();
                                         else st::wait_copies<0>();
                                         own.make();
                                     });
        else
            st::stream<U, NM, XR, D>(acc, rings + wave * D * R::kBlock, src, b1 - b0, kl, lane);
    } else if constexpr (XDT >= 0) {
        st::wait_copies<0>();
        own.make();
    }
    __syncthreads();                                // the rings are done with
    typedef decltype(acc[0][0][0] + 0) sum_t;
    sum_t *red = (sum_t *)smem;                     // [waves][NM][NB][64 lanes][4]
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(typename st::Sum<U>::x4 *)&red[((wave * NM + m) * NB + j) * 256 + 4 * lane] = acc[m][j];
    __syncthreads();
    for (int i = tid; i < G * NO * NB * 256; i += blockDim.x) {
        const int gg = i / (NO * NB * 256), e = i - gg * NO * NB * 256;
        const int t = e / (16 * NO), o = e - t * 16 * NO;       // token, output of the group
        const int n = 16 * NO * (u0 + gg) + o;
        if (t >= XT || t0 + t >= a.T || n >= a.N) continue;
        const int r = o & 15;
        const int at = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        sum_t v = 0, g2 = 0;
        for (int q = 0; q < P; ++q) {
            const sum_t *pr = red + ((gg * P + q) * NM + (o >> 4)) * NB * 256 + at;
            v += pr[0];
            if (GATED) g2 += pr[NO * NB * 256];
        }
        if constexpr (XDT >= 0)
            le::finish(a, 0, n, (float)v * a.sw[n] * own.row.scale, GATED ? (float)g2 * a.sg[n] * own.row.scale : 0.f);
        else
            le::finish_sum<U>(a, t0 + t, n, v, g2);
    }
}

constexpr int kLds = 160 * 1024, kStreamUnits = 256;        // of a compute unit; compute units

// Whether `waves` keep HBM busy: 6 to a compute unit, or most of those whose rings fit
bool plenty(long long waves, int ring)
{
    return waves >= 6 * kStreamUnits || 8 * waves >= 7ll * kStreamUnits * (kLds / ring);
}

template <int U, bool GATED, int NM, int XR, int D, int XDT = -1>
hipError_t launch_one(const le::Args<U> &a, hipStream_t s)
{
    constexpr int XT = XR ? XR : 1;
    using R = st::Ring<NM, XR>;
    constexpr int NO = GATED ? NM / 2 : NM;
    const int units = (a.N + 16 * NO - 1) / (16 * NO), blocks = (a.K + 63) / 64;
    constexpr int ring = D * R::kBlock, red = NM * R::kFrag * 1024, per = ring > red ? ring : red;
    static_assert(4 * per <= kLds, "four waves' rings fit a compute unit");
    // slices of K: 4; 8 while the waves are too few to fill the chip, a slice
    // keeps 4 blocks and the rings fit; fewer when K is short
    int P = 4;
    const int own = XDT >= 0 ? own_raw_bytes(2 * a.K, XDT) + 128 * blocks : 0;
    constexpr int kSlots = XDT >= 0 ? 64 : 0;               // the kernel's static LDS
    if (8 * per + own + kSlots <= kLds && (long long)units * P < 2048 && blocks >= 8 * P) P = 8;
    // 2 where those are enough, codes only: their sums do not depend on it (1 x 4096 x 28672
    // 20.3 us against 21.4, 16 tokens 21.1 against 22.3)
    if (U == st::kI8 && plenty(2ll * units, per)) P = 2;
    while (P > 1 && blocks < P) P /= 2;
    const int G = P < 4 ? 4 / P : 1, slice = (blocks + P - 1) / P;
    const int lds = G * P * per + own;
    const void *k = (const void *)linear_stream_kernel<U, GATED, NM, XR, D, XDT>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const unsigned sets = (unsigned)((units + G - 1) / G + 7) / 8, tiles = (unsigned)((a.T + XT - 1) / XT);
    hipLaunchKernelGGL((linear_stream_kernel<U, GATED, NM, XR, D, XDT>), dim3(8 * sets * tiles),
                       dim3(64 * G * P), lds, s, a, P, slice);
    return hipGetLastError();
}

// Rows per wave: 16 (and 16 of Wg).  From 17 tokens a block of tokens is larger
// than that of 16 rows, so wide layers take 32 + 32 or 64.
template <int U, int XR>
hipError_t launch_xr(const le::Args<U> &a, hipStream_t s)
{
    if constexpr (XR > 16) {
        // (codes, 32 x 4096 x 28672: 24.8 us by 32 + 32 rows, 27.7 by 16 + 16)
        const int outputs = a.wg ? 32 : 64;
        const bool wide = U == st::kI8 ? plenty(2ll * (a.N / outputs), 3 * st::Ring<4, XR>::kBlock) : a.N >= 16384;
        if (wide)
            return a.wg ? launch_one<U, true, 4, XR, 3>(a, s) : launch_one<U, false, 4, XR, 3>(a, s);
    }
    constexpr int D = XR <= 16 ? 4 : 3;
    return a.wg ? launch_one<U, true, 2, XR, 3>(a, s) : launch_one<U, false, 1, XR, D>(a, s);
}

template <int U>
hipError_t launch_by_tokens(const le::Args<U> &a, hipStream_t s)
{
    if (a.T == 1) return launch_xr<U, 1>(a, s);
    if (a.T <= 8) return launch_xr<U, 8>(a, s);
    if (a.T <= 16) return launch_xr<U, 16>(a, s);
    if (a.T <= 24) return launch_xr<U, 24>(a, s);
    return launch_xr<U, 32>(a, s);
}

// One token that is no codes yet (launch_stream for the others)
template <int XDT>
hipError_t launch_own(const LinearQ8Args &a, hipStream_t s)
{
    return a.wg ? launch_one<st::kI8, true, 2, 0, 3, XDT>(a, s) : launch_one<st::kI8, false, 1, 0, 4, XDT>(a, s);
}

template <int U>
hipError_t launch_stream(const le::Args<U> &a, hipStream_t s)
{
    if (a.T < 1 || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    // A launch may have at most 2^32 - 1 threads, here 512 a workgroup and one workgroup
    // for 16 outputs of 32 tokens at the most: more tokens go in runs.
    const long long sets = ((long long)a.N + 127) / 128 * 8;
    const int run = 32 * (int)std::max(1ll, (1ll << 22) / sets);
    const size_t ye = a.ydt == 2 ? 4 : 2;
    le::Args<U> b = a;
    for (int t = 0; t < a.T; t += run) {
        b.T = std::min(run, a.T - t);
        b.x = a.x + (size_t)t * a.xs;
        if constexpr (U == st::kI8) b.sx = a.sx + t;
        b.y = (char *)a.y + ye * t * a.ys;
        if (a.r) b.r = (const char *)a.r + ye * t * a.rs;
        const hipError_t e = launch_by_tokens<U>(b, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace
}  // namespace moeffn
