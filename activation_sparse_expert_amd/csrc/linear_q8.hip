// Linear layer on 8-bit codes: each wave multiplies 16 weight rows by 16 tokens over all of
// k with v_mfma_i32_16x16x64_i8 (lane l holds row l % 16, 16 codes at k 16 (l / 16); value r
// of lane l of the result is row 4 (l / 16) + r, token l % 16).
#include "linear_epilogue.hpp"
#include "rows.hpp"

namespace moeffn {

namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

__global__ void __launch_bounds__(256)
linear_q8_kernel(LinearQ8Args a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = 16 * (blockIdx.x * 4 + wave), t0 = 16 * blockIdx.y;
    if (n0 >= a.N) return;
    const int li = lane & 15, k0 = 16 * (lane >> 4);
    const int n = min(n0 + li, a.N - 1), t = min(t0 + li, a.T - 1);
    const int8_t *x = (const int8_t *)a.x + (size_t)t * a.xs;
    const int8_t *w = (const int8_t *)a.w + (size_t)n * a.K, *wg = (const int8_t *)(a.wg ? a.wg : a.w) + (size_t)n * a.K;
    intx4 acc = {0, 0, 0, 0}, gate = {0, 0, 0, 0};
    for (int k = k0; k - k0 < a.K; k += 64) {
        const intx4 none = {0, 0, 0, 0};
        const bool in = k < a.K;
        const intx4 xv = in ? *(const intx4 *)(x + k) : none;
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(in ? *(const intx4 *)(w + k) : none, xv, acc, 0, 0, 0);
        if (a.wg) gate = __builtin_amdgcn_mfma_i32_16x16x64_i8(in ? *(const intx4 *)(wg + k) : none, xv, gate, 0, 0, 0);
    }
    if (t0 + li >= a.T) return;
    for (int r = 0; r < 4; ++r) {
        const int j = n0 + 4 * (lane >> 4) + r;
        if (j >= a.N) break;
        const float sx = a.sx[t0 + li];
        le::finish(a, t0 + li, j, (float)acc[r] * a.sw[j] * sx, a.wg ? (float)gate[r] * a.sg[j] * sx : 0.f);
    }
}

}  // namespace

hipError_t launch_linear_q8(const LinearQ8Args &a, hipStream_t s)
{
    // (at most 65536 tokens: 4096 rows of the grid)
    hipLaunchKernelGGL(linear_q8_kernel, dim3((unsigned)((a.N + 63) / 64), (unsigned)((a.T + 15) / 16)), dim3(256), 0, s, a);
    return hipGetLastError();
}

size_t linear_q8_split_bytes(int, int, int) { return 0; }

}  // namespace moeffn
