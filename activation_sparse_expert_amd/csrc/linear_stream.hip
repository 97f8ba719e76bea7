// Linear layer for at most 32 tokens: the weights are read once, from HBM into
// the matrix core's operand registers (mfma_stream.hpp).  A wave takes 16
// outputs (of both matrices when gated) and a slice of K; the P waves of a
// workgroup that share the outputs add their slices through LDS in a fixed
// order and apply the epilogue.
#include "linear_epilogue.hpp"

namespace moeffn {

namespace {

using st::floatx4;

// NM: matrices (2 gated); NB: groups of 16 tokens; U: steps of 32 k in flight.
template <bool BF16, int NM, int NB, int U>
__global__ void __launch_bounds__(1024)
linear_stream_kernel(LinearArgs a, int P, int slice)
{
    extern __shared__ __align__(16) float red[];    // [waves][NM][NB][64 lanes][4]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int G = (int)(blockDim.x >> 6) / P;       // groups of 16 outputs in this workgroup
    const int g = wave / P, p = wave - g * P;
    const int units = (a.N + 15) / 16;
    const int u0 = blockIdx.x * G;
    const int li = lane & 15, kq = 8 * (lane >> 4);

    floatx4 acc[NM][NB];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int s0 = p * slice, s1 = min(s0 + slice, (a.K + 31) / 32);
    if (u0 + g < units && s0 < s1) {
        // outputs past N and tokens past T repeat the last one; they are not stored
        const int row = min(16 * (u0 + g) + li, a.N - 1);
        const uint16_t *w[NM], *x[NB];
        w[0] = a.w + (size_t)row * a.K + kq;
        if constexpr (NM == 2) w[1] = a.wg + (size_t)row * a.K + kq;
#pragma unroll
        for (int j = 0; j < NB; ++j) x[j] = a.x + (size_t)min(16 * j + li, a.T - 1) * a.xs + kq;
        st::stream<BF16, NM, NB, 1, U>(acc, w, x, s0, s1, a.K, kq);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(floatx4 *)&red[((wave * NM + m) * NB + j) * 256 + 4 * lane] = acc[m][j];
    __syncthreads();
    for (int i = tid; i < G * NB * 256; i += blockDim.x) {
        const int gg = i / (NB * 256), e = i - gg * NB * 256;
        const int t = e >> 4, r = e & 15;           // token, output of the group
        const int n = 16 * (u0 + gg) + r;
        if (t >= a.T || n >= a.N) continue;
        const int at = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        float v[2] = {0.f, 0.f};
        for (int q = 0; q < P; ++q)
#pragma unroll
            for (int m = 0; m < NM; ++m) v[m] += red[((gg * P + q) * NM + m) * NB * 256 + at];
        le::finish(a, t, n, v[0], v[1]);
    }
}

template <bool BF16, int NM, int NB>
hipError_t launch_nb(const LinearArgs &a, hipStream_t s)
{
    constexpr int U = NM * NB == 4 ? 4 : 8;
    const int units = (a.N + 15) / 16, steps = (a.K + 31) / 32;
    // slices of K: until there are about 4096 waves (16 per compute unit), while
    // a slice keeps a full batch of steps
    int P = 1;
    while (P < 16 && (long long)units * P < 4096 && steps >= 2 * U * P) P *= 2;
    int G = 1;
    while (G * P < 4) G *= 2;                       // at least 4 waves per workgroup
    const int slice = (steps + P - 1) / P;
    const unsigned grid = (unsigned)((units + G - 1) / G);
    const size_t lds = (size_t)G * P * NM * NB * 1024;
    hipLaunchKernelGGL((linear_stream_kernel<BF16, NM, NB, U>), dim3(grid), dim3(64 * G * P), lds, s, a, P, slice);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_t(const LinearArgs &a, hipStream_t s)
{
    if (a.T <= 16) return a.wg ? launch_nb<BF16, 2, 1>(a, s) : launch_nb<BF16, 1, 1>(a, s);
    return a.wg ? launch_nb<BF16, 2, 2>(a, s) : launch_nb<BF16, 1, 2>(a, s);
}

}  // namespace

hipError_t launch_linear_stream(const LinearArgs &a, hipStream_t s)
{
    if (a.T < 1 || a.T > kStreamTokens || a.K < 8 || a.K % 8 != 0 || a.N < 1) return hipErrorInvalidValue;
    return a.bf16 ? launch_t<true>(a, s) : launch_t<false>(a, s);
}

}  // namespace moeffn
