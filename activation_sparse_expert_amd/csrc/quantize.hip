// Rows to 8-bit codes and back (codes.hpp has the arithmetic).
#include "codes.hpp"
#include "mfma_stream.hpp"
#include "rows.hpp"

namespace moeffn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *lds)
{
    for (int s = 32; s > 0; s >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, s));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int i = 0; i < kThreads / 64; ++i) v = max(v, lds[i]);
    return v;
}

__global__ void __launch_bounds__(kThreads)
quantize_kernel(QuantizeArgs a)
{
    __shared__ uint32_t lds[kThreads / 64];
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t at = (size_t)t * a.xs;
        uint32_t most = 0;
        for (int i = threadIdx.x; i < a.k; i += kThreads) most = max(most, codes::magnitude(st::load_el(a.x, a.xdt, at + i)));
        const codes::Row r = codes::row(block_max(most, lds));
        for (int i = threadIdx.x; i < a.k; i += kThreads) {
            const float v = st::load_el(a.x, a.xdt, at + i);
            a.q[(size_t)t * a.qs + i] = (int8_t)(a.xdt == 2 ? codes::code64(v, r) : codes::code(v, r));
        }
        if (threadIdx.x == 0) a.scale[t] = r.scale;
    }
}

__global__ void __launch_bounds__(kThreads)
dequantize_kernel(DequantizeArgs a)
{
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float s = a.scale[t];
        for (int i = threadIdx.x; i < a.k; i += kThreads)
            st::store_el(a.y, a.ydt, (size_t)t * a.ys + i, (float)a.q[(size_t)t * a.qs + i] * s);
    }
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(quantize_kernel, dim3((unsigned)(a.T < 65536 ? a.T : 65536)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dequantize_rows(const DequantizeArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(dequantize_kernel, dim3((unsigned)(a.T < 65536 ? a.T : 65536)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moeffn
